// Rows of 16-bit values to e4m3 codes with a power-of-two scale for every 128
// columns, as they are or behind the residual's addition and a
// root-mean-square norm.
//
// Mathematics.  s = x + residual; y = s / sqrt(mean(s^2) + eps) * weight; for
// each row and 128 columns S = the least power of two with max|y| <= 448 S and
// code = e4m3(y / S).  All in fp32, each result rounded once.
//
// What bounds it.  Every value is read and written once: 7 bytes a value with
// residual and sum, 3 without.  A row stays in registers between the sum of
// squares and the scaling, so HBM is the bound: 8 x 1024 rows of 8192 with
// residual take 69.3 us, 6.8 TB/s (a copy: 6.8); quantised alone, 2 x 4095 rows of
// 3584 15.0 us, 5.9 TB/s (instructions: 100 for 24 bytes a lane); one row 2.8 us,
// the launch and one chain of load, sum and store.  Rows that do not fill whole
// waves of blocks wait for the last (2 x 777 of 5008, fp16, 7.4 us, 3.2 TB/s). Rows
// beyond 16384 have one block on an SM (4096 of 32768 178 us, 5.3 TB/s), beyond 32768 also
// more than 128 registers a thread (560 bytes spilled; 2048 of 65536 338 us, 2.8 TB/s).
//
// Layout.  16 lanes hold a block of 128 (8 values, 16 bytes each), so its
// largest magnitude is four shuffles away and codes go out 8 bytes a lane.
#include "coc_f8.cuh"

namespace coc {
namespace {

constexpr float kDown = 8.271806125530277e-25f;     // 2^-80

template <bool BF16>
__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = to_float16bit<BF16>(static_cast<uint16_t>(w[i] & 0xFFFFu));
        f[2 * i + 1] = to_float16bit<BF16>(static_cast<uint16_t>(w[i] >> 16));
    }
}

// N blocks of the 16 lanes: their scale bytes, and this lane's 8 codes of each.
// Infinities do not count, but are seldom there to be taken out: one test for
// all blocks, so that their shuffles go side by side.
template <int N>
__device__ __forceinline__ void block_codes(const float (&y)[N][8], uint32_t (&byte)[N], uint2 (&codes)[N]) {
    float top[N], most = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        top[i] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) top[i] = fmaxf(top[i], fabsf(y[i][j]));
        most = fmaxf(most, top[i]);
    }
    if (__any_sync(0xffffffffu, most > kF8Largest)) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            top[i] = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) top[i] = fmaxf(top[i], f8_magnitude(y[i][j]));
        }
    }
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], d));
#pragma unroll
    for (int i = 0; i < N; ++i) {
        byte[i] = f8_scale_byte(top[i]);
        const float f = f8_inverse(byte[i]);
        codes[i] = make_uint2(f8_codes4(y[i][0], y[i][1], y[i][2], y[i][3], f), f8_codes4(y[i][4], y[i][5], y[i][6], y[i][7], f));
    }
}

// Half a warp a block of 128, kBlocksEach blocks of it in flight.
constexpr int kQuantThreads = 256;
constexpr int kBlocksEach = 2;

template <bool BF16>
__global__ void __launch_bounds__(kQuantThreads) f8_quantize_kernel(const __grid_constant__ F8RowsArgs a) {
    grid_dependency_wait();
    grid_dependents_launch();
    const int r = blockIdx.y;
    const uint32_t blocks = (a.hidden + 127) / 128, all = a.rows * blocks;      // at most 2^31
    const int lane16 = threadIdx.x & 15;
    const uint32_t first = blockIdx.x * (kQuantThreads / 16 * kBlocksEach) + (threadIdx.x >> 4);
    uint4 v[kBlocksEach];
    long long at[kBlocksEach];      // the lane's values in the matrix; -1: none
#pragma unroll
    for (int i = 0; i < kBlocksEach; ++i) {
        const uint32_t b = first + i * (kQuantThreads / 16);
        const uint32_t row = b / blocks;
        const int col = static_cast<int>(b - row * blocks) * 128 + lane16 * 8;
        at[i] = b < all && col < a.hidden ? static_cast<long long>(row) * a.hidden + col : -1;
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (at[i] >= 0) v[i] = load_uint4(a.x[r] + at[i]);
    }
    float y[kBlocksEach][8];
    uint32_t byte[kBlocksEach];
    uint2 codes[kBlocksEach];
#pragma unroll
    for (int i = 0; i < kBlocksEach; ++i) unpack8<BF16>(v[i], y[i]);
    block_codes(y, byte, codes);
#pragma unroll
    for (int i = 0; i < kBlocksEach; ++i)
        if (at[i] >= 0) {
            *reinterpret_cast<uint2*>(a.codes[r] + at[i]) = codes[i];
            if (lane16 == 0) a.scale[r][first + i * (kQuantThreads / 16)] = static_cast<uint8_t>(byte[i]);
        }
}

// blockDim.x threads a row (a multiple of 32), blockDim.y rows a block; VPT
// pieces of 8 values a thread.
constexpr int norm_threads(int vpt) { return vpt <= 2 ? 1024 : 512; }

// (VPT 4, two blocks of 512 on an SM: 8 x 1024 rows of 8192 75.7 to 70.2 us, 4096 of 16384 103 to 73.8)
template <bool BF16, int VPT>
__global__ void __launch_bounds__(norm_threads(VPT), VPT == 4 ? 2 : 1) f8_norm_kernel(const __grid_constant__ F8RowsArgs a) {
    __shared__ float sums[32];
    grid_dependency_wait();
    grid_dependents_launch();
    const int r = blockIdx.y, T = blockDim.x, t = threadIdx.x;
    const long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = row < a.rows;
    const int pieces = a.hidden / 8;
    const long long base = row * a.hidden;

    // all loads first; the weights' wait in registers where these are not many
    constexpr bool kAhead = VPT <= 4;
    float s[VPT][8];
    uint4 wv[kAhead ? VPT : 1];
    {
        uint4 xv[VPT], rv[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int p = t + i * T;
            xv[i] = rv[i] = make_uint4(0u, 0u, 0u, 0u);
            if (live && p < pieces) {
                xv[i] = load_uint4(a.x[r] + base + 8 * p);
                if (a.residual[r] != nullptr) rv[i] = load_uint4(a.residual[r] + base + 8 * p);
            }
        }
        if constexpr (kAhead) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int p = t + i * T;
                wv[i] = p < pieces ? load_uint4(a.weight + 8 * p) : make_uint4(0u, 0u, 0u, 0u);
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float f[8];
            unpack8<BF16>(xv[i], s[i]);
            if (a.residual[r] != nullptr) {
                unpack8<BF16>(rv[i], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[i][j] += f[j];
                const int p = t + i * T;
                if (live && p < pieces) {
                    uint4 o;
                    o.x = pack2<BF16>(__float_as_uint(s[i][0]), __float_as_uint(s[i][1]));
                    o.y = pack2<BF16>(__float_as_uint(s[i][2]), __float_as_uint(s[i][3]));
                    o.z = pack2<BF16>(__float_as_uint(s[i][4]), __float_as_uint(s[i][5]));
                    o.w = pack2<BF16>(__float_as_uint(s[i][6]), __float_as_uint(s[i][7]));
                    *reinterpret_cast<uint4*>(a.sum[r] + base + 8 * p) = o;
                }
            }
        }
    }

    // the row's sum of (s f)^2, in the same order every time
    const int warp = (threadIdx.y * T + t) >> 5, warps = T >> 5;
    auto total = [&](float f) {
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = s[i][j] * f;
                q = fmaf(v, v, q);
            }
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) q += __shfl_xor_sync(0xffffffffu, q, d);
        if (warps > 1) {
            if ((t & 31) == 0) sums[warp] = q;
            __syncthreads();
            q = 0.f;
            for (int w = 0; w < warps; ++w) q += sums[threadIdx.y * warps + w];
        }
        return q;
    };
    float f = 1.f, q = total(1.f);
    // Squares of values from 2^64 on overflow; the row is then taken 2^-80 times
    // (what underflows is nothing beside them).  All threads of a block go in or none
    // (a block of one row agrees by itself): the barriers are the block's.
    bool over = !(q <= kF8Largest);
    const bool mine = over;
    if (blockDim.y > 1 && warps > 1) over = __syncthreads_or(over);
    if (over) {
        if (warps > 1) __syncthreads();     // the sums have been read
        const float scaled = total(kDown);
        if (mine) {
            f = kDown;
            q = scaled;
        }
    }
    const float eps = f == 1.f ? a.eps : a.eps * kDown * kDown;
    const float inv = rsqrtf(q / static_cast<float>(a.hidden) + eps);

    // (piece after piece: two or four side by side cost registers, 8 x 1024 rows of 8192 70.7 and 71.8 us instead of 70.2)
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int p = t + i * T;
        const bool in = live && p < pieces;
        float w[8], y[1][8];
        if constexpr (kAhead) unpack8<BF16>(wv[i], w);
        else unpack8<BF16>(in ? load_uint4(a.weight + 8 * p) : make_uint4(0u, 0u, 0u, 0u), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[0][j] = in ? s[i][j] * f * inv * w[j] : 0.f;
        uint32_t byte[1];
        uint2 codes[1];
        block_codes(y, byte, codes);
        if (in) {
            *reinterpret_cast<uint2*>(a.codes[r] + base + 8 * p) = codes[0];
            if ((t & 15) == 0) a.scale[r][row * ((pieces + 15) / 16) + p / 16] = static_cast<uint8_t>(byte[0]);
        }
    }
}

cudaError_t launch_rows(const void* kern, const F8RowsArgs& a, dim3 grid, dim3 block, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = stream;
    cfg.attrs = attr;
    if (pdl_launch()) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 1;
    }
    void* args[] = {const_cast<F8RowsArgs*>(&a)};
    return cudaLaunchKernelExC(&cfg, kern, args);
}

template <bool BF16>
const void* norm_kernel(int vpt) {
    switch (vpt) {
        case 1: return reinterpret_cast<const void*>(f8_norm_kernel<BF16, 1>);
        case 2: return reinterpret_cast<const void*>(f8_norm_kernel<BF16, 2>);
        case 4: return reinterpret_cast<const void*>(f8_norm_kernel<BF16, 4>);
        case 8: return reinterpret_cast<const void*>(f8_norm_kernel<BF16, 8>);
        default: return reinterpret_cast<const void*>(f8_norm_kernel<BF16, 16>);
    }
}

}  // namespace

cudaError_t launch_f8_quantize(const F8RowsArgs& a, bool bf16, cudaStream_t stream) {
    const long long all = static_cast<long long>(a.rows) * ((a.hidden + 127) / 128);
    const int each = kQuantThreads / 16 * kBlocksEach;
    const dim3 grid(static_cast<unsigned>((all + each - 1) / each), static_cast<unsigned>(a.R));
    return launch_rows(bf16 ? reinterpret_cast<const void*>(f8_quantize_kernel<true>) : reinterpret_cast<const void*>(f8_quantize_kernel<false>), a,
                       grid, dim3(kQuantThreads), stream);
}

cudaError_t launch_f8_norm(const F8RowsArgs& a, bool bf16, int sm_count, cudaStream_t stream) {
    const int pieces = a.hidden / 8;
    // 4 pieces a thread, more only for long rows; fewer where rows are short, and
    // where there are fewer rows than SMs (one row of 4096: 2.8 us with 1, 4.1 with 4)
    const auto fits = [&](int v) { return (pieces + v - 1) / v <= norm_threads(v); };
    int vpt = 4;
    while (vpt < 16 && !fits(vpt)) vpt *= 2;
    while (vpt > 1 && fits(vpt / 2) && (static_cast<long long>(a.rows) * a.R <= sm_count || pieces <= 32 * (vpt / 2))) vpt /= 2;
    const int T = ((pieces + vpt - 1) / vpt + 31) / 32 * 32;
    const int rows = T >= 128 ? 1 : 128 / T;
    const dim3 grid(static_cast<unsigned>((static_cast<long long>(a.rows) + rows - 1) / rows), static_cast<unsigned>(a.R));
    return launch_rows(bf16 ? norm_kernel<true>(vpt) : norm_kernel<false>(vpt), a, grid, dim3(T, rows), stream);
}

}  // namespace coc
