// Attention over the paged 8-bit key/value cache.
#include "coc_kv.cuh"

namespace coc {
namespace {

// Block (token, query head, rank): one query row, 128 keys at a time; thread
// i takes key i's product, then values d = i, i + 128 of the output.
constexpr int kKeys = 128;

template <bool BF16>
__global__ void __launch_bounds__(kKeys) kv_attention_kernel(const __grid_constant__ KvAttnArgs a) {
    __shared__ float q[256];
    __shared__ float w[kKeys];
    __shared__ int pg[kKeys];
    __shared__ float red[kKeys / 32];
    const int t = blockIdx.x, hq = blockIdx.y, r = blockIdx.z, i = threadIdx.x;
    const int h = hq / (a.q_heads / a.heads);
    int lo = 0, hi = a.seqs, b, e;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        seq_tokens(a.cu, mid, a.tokens, b, e);
        if (b <= t) lo = mid;
        else hi = mid;
    }
    const int s = lo;
    seq_tokens(a.cu, s, a.tokens, b, e);
    // keys [0, sinks) and [from, until)
    const int until = (t >= b && t < e) ? __ldg(a.lens + s) - (e - 1 - t) : 0;
    const int from = a.window > 0 ? max(0, until - a.window) : 0;
    const int sinks = min(from, a.sinks);
    const uint16_t* x = a.q[r] + t * a.q_token + hq * a.q_head;
    for (int j = i; j < a.d; j += kKeys) q[j] = to_float16bit<BF16>(x[j]) * a.scale;
    float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
    for (int j0 = 0; j0 < until; j0 = (j0 + kKeys >= sinks && j0 + kKeys < from) ? max(j0 + kKeys, from / kKeys * kKeys) : j0 + kKeys) {
        const int j = j0 + i;
        __syncthreads();
        float z = -INFINITY;
        pg[i] = -1;
        if (j < until && (j < sinks || j >= from)) {
            const int p = j / a.page;
            const int id = p < a.table_width ? __ldg(a.table + static_cast<long long>(s) * a.table_width + p) : -1;
            if (id < 0 || id >= a.pages) {
                atomicOr(a.status, DEV_ERR_BAD_PAGE);
            } else {
                pg[i] = id;
                const long long base = static_cast<long long>(id) * a.heads + h;
                const uint8_t* k = a.ck[r] + (base * a.page + j % a.page) * a.d;
                float acc = 0.f;
                for (int c = 0; c < a.d; ++c) acc += q[c] * __half2float(__half(__nv_cvt_fp8_to_halfraw(k[c], __NV_E4M3)));
                z = acc * a.sk[r][base];
            }
        }
        float top = z;
        for (int x2 = 16; x2 > 0; x2 >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x2));
        if ((i & 31) == 0) red[i >> 5] = top;
        __syncthreads();
        top = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
        const float ref = top == -INFINITY ? 0.f : top;
        w[i] = expf(z - ref);
        const float c = expf(m - ref);
        m = top;
        o0 *= c;
        o1 *= c;
        l *= c;
        __syncthreads();
        for (int n = 0; n < kKeys; ++n) {
            if (pg[n] < 0) continue;
            const float p = w[n];
            l += p;
            const long long base = static_cast<long long>(pg[n]) * a.heads + h;
            const uint8_t* v = a.cv[r] + (base * a.page + (j0 + n) % a.page) * a.d;
            const float ps = p * a.sv[r][base];
            if (i < a.d) o0 += ps * __half2float(__half(__nv_cvt_fp8_to_halfraw(v[i], __NV_E4M3)));
            if (i + kKeys < a.d) o1 += ps * __half2float(__half(__nv_cvt_fp8_to_halfraw(v[i + kKeys], __NV_E4M3)));
        }
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // a row that sees nothing is zero, NaN stays
    uint16_t* o = a.out[r] + (static_cast<long long>(t) * a.q_heads + hq) * a.d;
    if (i < a.d) o[i] = from_float16bit<BF16>(o0 * inv);
    if (i + kKeys < a.d) o[i + kKeys] = from_float16bit<BF16>(o1 * inv);
}

}  // namespace

cudaError_t launch_kv_attention(const KvAttnArgs& a, bool bf16, cudaStream_t stream) {
    const dim3 g(static_cast<unsigned>(a.tokens), static_cast<unsigned>(a.q_heads), static_cast<unsigned>(a.R));
    if (bf16) kv_attention_kernel<true><<<g, kKeys, 0, stream>>>(a);
    else kv_attention_kernel<false><<<g, kKeys, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace coc
