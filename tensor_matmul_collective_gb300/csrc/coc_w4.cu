// Row-parallel products with 4-bit weights and group scales at decode-sized m,
// summed over the ranks.
//
// Mathematics.  out = sum over the groups G of the contraction (all ranks, one
// after another) of s_G(j) * sum_{t in G} x_t (code(t, j) - z_G(j)).  code - z
// is a small integer, exact in fp16 and bf16, and so is x: the inner sum runs
// on the tensor cores with fp32 accumulation, the scale is applied to it once
// per group in fp32, and the weight itself is never rounded.
//
// What bounds it.  k n / 2 bytes of weights, read once: the operations per
// byte (4 m) are few, but taking codes out of words costs instructions, about
// 1.2 per weight pair, near half of what the SMs issue at full bandwidth.
// W^T is the A operand of mma.sync (16 weight columns x 16 of k) and x^T the B
// operand (8 tokens).  A word holds 8 codes along k of one column; a mask
// takes two codes four apart into the halves of a register, so the pairs
// (k, k + 4) are the operand's neighbours, and x is permuted to match, once
// for the 64 columns of a warp.  or-ing the codes into the mantissa of 1024
// (bf16: 128) makes them floating-point numbers, and one addition takes off
// 1024 + z.
//
// A lane reads whole 16-byte pieces (4 columns) of the rows as they lie in
// memory, and the asynchronous copies land in a slot that the same lane reads
// back: no barrier, no bank conflict.
//
// Split.  A warp takes 64 columns and a contiguous range of the contraction;
// the ranges of a block's warps and of a cluster's blocks are added through
// shared memory in their order.
#include <algorithm>
#include <atomic>
#include <cstdlib>
#include <type_traits>

#include "coc_kv.cuh"
#include "coc_ptx.cuh"

namespace coc {
namespace {

constexpr int kWarps = 8;
constexpr int kCols = 64;               // columns of a warp
constexpr int kStep = 32;               // contraction of one step: 4 word rows
#ifndef T_WST
#define T_WST 4
#endif
#ifndef T_WOC
#define T_WOC 3
#endif
constexpr int kStages = T_WST;

template <int NT>
constexpr int stage_bytes() { return 32 * (2 * 16 + NT * 16 + 16 + 8); }   // words, x, scales, zero points
template <int NT>
constexpr int sum_floats() { return NT * 8 * kCols; }                      // one warp's sums
template <int NT>
constexpr int w4_smem() {
    const int ring = kWarps * kStages * stage_bytes<NT>();
    const int sums = kWarps * sum_floats<NT>() * 4;
    return ring > sums ? ring : sums;
}

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool in) {
    const int n = in ? BYTES : 0;
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "n"(BYTES), "r"(n)
                     : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (x & mask) | bits in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(mask), "r"(bits));
    return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t add2(uint32_t x, uint32_t y) {
    uint32_t r;
    if constexpr (BF16) asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    else asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}
__device__ __forceinline__ uint32_t fma2_half(uint32_t x, uint32_t y, uint32_t z) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(y), "r"(z));
    return r;
}

// (d0, d1) += (x0, x1) * s
__device__ __forceinline__ void fma2(float& d0, float& d1, float x0, float x1, float s) {
    asm("{\n\t.reg .b64 d, x, s;\n\tmov.b64 d, {%0, %1};\n\tmov.b64 x, {%2, %3};\n\tmov.b64 s, {%4, %4};\n\t"
        "fma.rn.f32x2 d, x, s, d;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "+f"(d0), "+f"(d1)
        : "f"(x0), "f"(x1), "f"(s));
}

// code - z of four of a word's 8 codes: the pairs (k, k + 4) for k = 2 H and
// 2 H + 1.  off: -(1024 + z) twice (fp16) or -(128 + z) (bf16); off16: -(64 + z)
// (fp16: a code four bits up is 16 times itself, and its product with 1/16
// costs the addition nothing).
template <bool BF16, int H>
__device__ __forceinline__ void codes(uint32_t w, uint32_t off, uint32_t off16, uint32_t& p0, uint32_t& p1) {
    if constexpr (BF16) {
        p0 = add2<true>(and_or(w >> (8 * H), 0x000F000Fu, 0x43004300u), off);
        p1 = add2<true>(and_or(w >> (8 * H + 4), 0x000F000Fu, 0x43004300u), off);
    } else {
        const uint32_t v = w >> (8 * H);
        p0 = add2<false>(and_or(v, 0x000F000Fu, 0x64006400u), off);
        p1 = fma2_half(and_or(v, 0x00F000F0u, 0x64006400u), 0x2C002C00u, off16);
    }
}

// f in both halves, rounded to the 16-bit type (exact for the offsets).
template <bool BF16>
__device__ __forceinline__ uint32_t pair(float f) {
    return pack2<BF16>(__float_as_uint(f), __float_as_uint(f));
}

// Block: WO x 64 columns, 8 / WO ranges of the contraction; cluster: blocks
// with the same columns and further ranges.  blockIdx.y: 8 NT rows of x.
template <bool BF16, int NT, bool ZERO, int WO>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 && !ZERO ? T_WOC : 2) w4_kernel(const __grid_constant__ W4Args a) {
    constexpr int WK = kWarps / WO;
    constexpr int SB = stage_bytes<NT>();
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int wo = warp % WO, wk = warp / WO;
    const int split = static_cast<int>(cluster_rank()), splits = a.splits;
    const int slab = blockIdx.x / splits;
    const int col0 = (slab * WO + wo) * kCols, row0 = blockIdx.y * 8 * NT;

    grid_dependency_wait();
    grid_dependents_launch();

    // this warp's steps, all ranks' shards one after another
    const int per_rank = a.k / kStep, per_group = a.group / kStep;
    const long long steps = static_cast<long long>(per_rank) * a.R, ways = static_cast<long long>(splits) * WK, way = split * WK + wk;
    const int s0 = static_cast<int>(steps * way / ways), s1 = static_cast<int>(steps * (way + 1) / ways);

    float acc[NT][4][4], part[NT][4][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[t][i][q] = part[t][i][q] = 0.f;

    if (col0 < a.n && s0 < s1) {
        // ---- producer: the next step to be copied.  All addresses run on by
        // constants inside a rank's shard.
        const bool in0 = col0 + 4 * g < a.n, in1 = col0 + 32 + 4 * g < a.n;
        const uint32_t ring = smem_u32(smem) + warp * kStages * SB;
        const uint8_t* ring_p = smem + warp * kStages * SB;
        int pr = s0 / per_rank, todo = s1 - s0;
        int in_rank, in_group;              // steps to the end of the rank's shard and of the group
        const uint32_t* wp;
        const uint16_t* xp[NT];
        const uint16_t* sp;
        const int8_t* zp = nullptr;
        bool new_group = true;
        auto enter = [&](int at) {          // step `at` of rank pr
            in_rank = per_rank - at;
            in_group = per_group - at % per_group;
            wp = a.w[pr] + (static_cast<long long>(at) * 4 + c) * a.n + col0 + 4 * g;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int row = row0 + 8 * t + g;
                xp[t] = a.x[pr] + static_cast<long long>(row < a.m ? row : 0) * a.k + at * kStep + 8 * c;
            }
            const long long so = static_cast<long long>(at / per_group) * a.n + col0 + 4 * g;
            sp = a.scale[pr] + so;
            if constexpr (ZERO) zp = a.zero[pr] + so;
        };
        enter(s0 - pr * per_rank);
        auto load = [&](int stage) {
            if (todo > 0) {
                const uint32_t so = ring + stage * SB;
                cp_async<16>(so + lane * 16, wp, in0);
                cp_async<16>(so + 512 + lane * 16, wp + 32, in1);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    cp_async<16>(so + 1024 + t * 512 + lane * 16, xp[t], row0 + 8 * t + g < a.m);
                    xp[t] += kStep;
                }
                wp += 4LL * a.n;
                if (new_group) {
                    new_group = false;
                    cp_async<8>(so + 1024 + NT * 512 + lane * 16, sp, in0);
                    cp_async<8>(so + 1024 + NT * 512 + lane * 16 + 8, sp + 32, in1);
                    sp += a.n;
                    if constexpr (ZERO) {
                        cp_async<4>(so + 1536 + NT * 512 + lane * 8, zp, in0);
                        cp_async<4>(so + 1536 + NT * 512 + lane * 8 + 4, zp + 32, in1);
                        zp += a.n;
                    }
                }
                --todo;
                if (--in_group == 0) {
                    in_group = per_group;
                    new_group = true;
                    if ((in_rank -= per_group) <= 0 && todo > 0) {      // groups do not cross shards
                        ++pr;
                        enter(0);
                    }
                }
            }
            cp_commit();
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) load(i);

        int left = per_group - s0 % per_group;      // steps to the end of the group (shards are whole groups)
        bool fresh = true;
        float sc[8];
        uint32_t off[ZERO ? 8 : 1], off16[ZERO ? 8 : 1];
        if constexpr (!ZERO) {
            off[0] = pair<BF16>(BF16 ? -136.f : -1032.f);
            off16[0] = BF16 ? 0u : pair<false>(-72.f);
        }
        for (int sb = s0; sb < s1; sb += kStages) {
#pragma unroll
            for (int st = 0; st < kStages; ++st) {
                if (sb + st >= s1) break;
                load((st + kStages - 1) % kStages);
                cp_wait<kStages - 1>();
                const uint8_t* slot = ring_p + st * SB;
                if (fresh) {
                    fresh = false;
                    const uint4 s4 = *reinterpret_cast<const uint4*>(slot + 1024 + NT * 512 + lane * 16);
                    const uint32_t sv[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) sc[i] = to_float16bit<BF16>(static_cast<uint16_t>(sv[i / 2] >> (16 * (i & 1))));
                    if constexpr (ZERO) {
                        const uint2 z2 = *reinterpret_cast<const uint2*>(slot + 1536 + NT * 512 + lane * 8);
                        const uint32_t zv[2] = {z2.x ^ 0x80808080u, z2.y ^ 0x80808080u};      // z + 128
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            // 2^23 + (z + 128) is exact, and so is what is taken off
                            const float z = __uint_as_float(__byte_perm(zv[i / 4], 0x4B000000u, 0x7650 + (i & 3)));
                            off[i] = pair<BF16>((BF16 ? 8388608.f : 8388608.f - 896.f) - z);
                            if constexpr (!BF16) off16[i] = add2<false>(off[i], 0x63806380u);           // + 960
                        }
                    }
                }
                const uint4 w0 = *reinterpret_cast<const uint4*>(slot + lane * 16);
                const uint4 w1 = *reinterpret_cast<const uint4*>(slot + 512 + lane * 16);
                uint32_t b[NT][4];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint4 x = *reinterpret_cast<const uint4*>(slot + 1024 + t * 512 + lane * 16);
                    b[t][0] = __byte_perm(x.x, x.z, 0x5410);    // (x0, x4)
                    b[t][1] = __byte_perm(x.x, x.z, 0x7632);    // (x1, x5)
                    b[t][2] = __byte_perm(x.y, x.w, 0x5410);
                    b[t][3] = __byte_perm(x.y, x.w, 0x7632);
                }
                const uint32_t wv[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
                // all tiles once per half: products into one accumulator do not follow each other
                auto half = [&](auto hc) {
                    constexpr int H = decltype(hc)::value;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {       // columns 2 i and 2 i + 1 of the lane's: rows g and g + 8 of the tile
                        uint32_t a0, a1, a2, a3;
                        codes<BF16, H>(wv[2 * i], off[ZERO ? 2 * i : 0], off16[ZERO ? 2 * i : 0], a0, a2);
                        codes<BF16, H>(wv[2 * i + 1], off[ZERO ? 2 * i + 1 : 0], off16[ZERO ? 2 * i + 1 : 0], a1, a3);
#pragma unroll
                        for (int t = 0; t < NT; ++t) mma16816<BF16>(part[t][i], a0, a1, a2, a3, b[t][2 * H], b[t][2 * H + 1]);
                    }
                };
                half(std::integral_constant<int, 0>{});
                half(std::integral_constant<int, 1>{});
                if (--left == 0 || sb + st + 1 == s1) {
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int q = 0; q < 4; q += 2) {
                                fma2(acc[t][i][q], acc[t][i][q + 1], part[t][i][q], part[t][i][q + 1], sc[2 * i + (q >> 1)]);
                                part[t][i][q] = part[t][i][q + 1] = 0.f;
                            }
                    left = per_group;
                    fresh = true;
                }
            }
        }
        cp_wait<0>();
    }

    // ---- join the ranges: sums[warp][token][column]
    __syncthreads();
    float* sums = reinterpret_cast<float*>(smem);
    constexpr int SF = sum_floats<NT>();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                // columns 4 g + 2 (i & 1) and the next of half i / 2, token 2 c + q
                *reinterpret_cast<float2*>(sums + warp * SF + (8 * t + 2 * c + q) * kCols + 32 * (i >> 1) + 4 * g + 2 * (i & 1)) =
                    make_float2(acc[t][i][q], acc[t][i][q + 2]);
            }
    __syncthreads();
    if (splits > 1) cluster_sync();
    // block `split` of the cluster finishes every splits-th pair of columns
    constexpr int pairs = WO * NT * 8 * kCols / 2;
    for (int x = threadIdx.x + split * kWarps * 32; x < pairs; x += kWarps * 32 * splits) {
        const int cw = x / (SF / 2), in = x % (SF / 2) * 2;     // column group, place in its sums
        const int row = row0 + in / kCols, col = (slab * WO + cw) * kCols + in % kCols;
        if (row >= a.m || col >= a.n) continue;
        float2 y = make_float2(0.f, 0.f);
        for (int b = 0; b < splits; ++b)
#pragma unroll
            for (int k = 0; k < WK; ++k) {
                const uint32_t at = smem_u32(sums + (k * WO + cw) * SF + in);
                float2 v;
                if (splits > 1) {
                    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(map_to_rank(at, b)) : "memory");
                } else {
                    v = *reinterpret_cast<const float2*>(sums + (k * WO + cw) * SF + in);
                }
                y.x += v.x;
                y.y += v.y;
            }
        const uint32_t o = pack2<BF16>(__float_as_uint(y.x), __float_as_uint(y.y));
        for (int r = 0; r < a.R; ++r) *reinterpret_cast<uint32_t*>(a.out[r] + static_cast<long long>(row) * a.n + col) = o;
    }
    if (splits > 1) cluster_sync();     // no block leaves while its sums are read
}

template <bool BF16, int NT, bool ZERO, int WO>
cudaError_t launch_t(const W4Args& a, cudaStream_t stream) {
    auto kern = w4_kernel<BF16, NT, ZERO, WO>;
    static std::atomic<unsigned char> smem_set[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !smem_set[dev].load(std::memory_order_acquire)) {
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, w4_smem<NT>())) != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) smem_set[dev].store(1, std::memory_order_release);
    }
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.n + WO * kCols - 1) / (WO * kCols) * a.splits), static_cast<unsigned>((a.m + 8 * NT - 1) / (8 * NT)), 1);
    cfg.blockDim = dim3(kWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = w4_smem<NT>();
    cfg.stream = stream;
    cfg.attrs = attr;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(a.splits);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.numAttrs = 1;
    if (pdl_launch()) {
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <bool BF16, int NT, bool ZERO>
cudaError_t launch_w(const W4Args& a, int wo, cudaStream_t stream) {
    return wo == 4 ? launch_t<BF16, NT, ZERO, 4>(a, stream) : wo == 2 ? launch_t<BF16, NT, ZERO, 2>(a, stream) : launch_t<BF16, NT, ZERO, 1>(a, stream);
}
template <bool BF16>
cudaError_t launch_b(const W4Args& a, int wo, cudaStream_t stream) {
    const bool two = a.m > 8, zero = a.zero[0] != nullptr;
    if (two) return zero ? launch_w<BF16, 2, true>(a, wo, stream) : launch_w<BF16, 2, false>(a, wo, stream);
    return zero ? launch_w<BF16, 1, true>(a, wo, stream) : launch_w<BF16, 1, false>(a, wo, stream);
}

}  // namespace

cudaError_t launch_w4(const W4Args& args, bool bf16, int sm_count, cudaStream_t stream) {
    W4Args a = args;
    const long long steps = static_cast<long long>(a.k / kStep) * a.R;
    const long long resident = 2LL * sm_count, tiles = (a.m + (a.m > 8 ? 15 : 7)) / (a.m > 8 ? 16 : 8);
    double best = 1e300;
    int wo = 1;
    a.splits = 1;
    for (int w : {4, 2, 1})
        for (int k : {1, 2, 4, 8}) {
            const long long blocks = (a.n + w * kCols - 1) / (w * kCols) * k * tiles;
            const double per = std::max(1.0, static_cast<double>(steps) / (k * (kWarps / w)));
            const double t = static_cast<double>((blocks + resident - 1) / resident) * (per + 8.0);
            if (t < best) {
                best = t;
                wo = w;
                a.splits = k;
            }
        }
    if (const char* e = std::getenv("W4_WO")) wo = std::atoi(e);
    if (const char* e = std::getenv("W4_KS")) a.splits = std::atoi(e);
    return bf16 ? launch_b<true>(a, wo, stream) : launch_b<false>(a, wo, stream);
}

}  // namespace coc
