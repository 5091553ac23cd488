// Row-parallel products with 4-bit weights and group scales at decode-sized m.
#include "coc_kv.cuh"

namespace coc {
namespace {

// Thread: one output column and up to 4 rows, the whole contraction of all
// ranks.  A word holds the codes of 8 weights along k.
constexpr int kRows = 4;

template <bool BF16>
__global__ void __launch_bounds__(128) w4_kernel(const __grid_constant__ W4Args a) {
    const int j = blockIdx.x * 128 + threadIdx.x, m0 = blockIdx.y * kRows;
    if (j >= a.n) return;
    const int rows = min(kRows, a.m - m0);
    float acc[kRows] = {};
    for (int r = 0; r < a.R; ++r) {
        for (int g = 0; g < a.k / a.group; ++g) {
            const long long at = static_cast<long long>(g) * a.n + j;
            const float s = to_float16bit<BF16>(a.scale[r][at]);
            const int z = a.zero[r] != nullptr ? a.zero[r][at] : 8;
            float part[kRows] = {};
            for (int t = g * a.group; t < (g + 1) * a.group; t += 8) {
                const uint32_t w = a.w[r][static_cast<long long>(t / 8) * a.n + j];
                for (int i = 0; i < 8; ++i) {
                    const float c = static_cast<float>(static_cast<int>((w >> (4 * i)) & 15u) - z);
                    for (int y = 0; y < rows; ++y)
                        part[y] += c * to_float16bit<BF16>(a.x[r][static_cast<long long>(m0 + y) * a.k + t + i]);
                }
            }
            for (int y = 0; y < rows; ++y) acc[y] += s * part[y];
        }
    }
    for (int y = 0; y < rows; ++y)
        for (int r = 0; r < a.R; ++r) a.out[r][static_cast<long long>(m0 + y) * a.n + j] = from_float16bit<BF16>(acc[y]);
}

}  // namespace

cudaError_t launch_w4(const W4Args& a, bool bf16, cudaStream_t stream) {
    const dim3 g(static_cast<unsigned>((a.n + 127) / 128), static_cast<unsigned>((a.m + kRows - 1) / kRows));
    if (bf16) w4_kernel<true><<<g, 128, 0, stream>>>(a);
    else w4_kernel<false><<<g, 128, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace coc
