// Shared by the 8-bit floating-point kernels (coc_f8_rows.cu, coc_f8_slab.cu,
// coc_f8_tile.cu): quantisation of a block of 128 values, and the
// block-scaled tcgen05 products.
//
// Values are e4m3 codes with power-of-two scales (e8m0 bytes: exponent + 127)
// for 128 columns of a row (activations) or 128 x 128 (weights).  A power of
// two costs e4m3 no precision, and the tensor cores apply it inside the
// product (kind::mxf8f6f4), so accumulators stay in tensor memory over the
// whole contraction: nothing has to be read back, scaled and added per block.
#pragma once

#include <cuda_fp8.h>

#include "coc_kv.cuh"
#include "coc_ptx.cuh"

namespace coc {
namespace {

// The scale byte of a block whose largest finite magnitude is amax (scale_for's
// power of two), and the factor 1 / S, which is exact: S lies in [2^-100, 2^120].
__device__ __forceinline__ uint32_t f8_scale_byte(float amax) { return __float_as_uint(scale_for(amax)) >> 23; }
__device__ __forceinline__ float f8_inverse(uint32_t scale_byte) { return __uint_as_float((254u - scale_byte) << 23); }

constexpr float kF8Largest = 3.4028234663852886e38f;     // fp32's

// |v| where it is finite, else 0: what counts in a block's largest magnitude.
__device__ __forceinline__ float f8_magnitude(float v) {
    const float a = fabsf(v);
    return a <= kF8Largest ? a : 0.f;
}

// Four codes, e4m3(v * f), round-to-nearest-even; beyond 448 (infinities) +-448, NaN stays NaN.
__device__ __forceinline__ uint32_t f8_codes4(float a, float b, float c, float d, float f) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a * f, b * f), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c * f, d * f), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// silu(g) u = g u / (1 + e^-g), e^-g = 2^(-g log2 e).  From g = -87 on e^-g or
// its reciprocal leaves fp32's range, but g e^g u need not, u may be large. FAR: below
// -69 numerator and denominator are taken 2^-120 times (above, the same factor
// is 1, which changes no bit).  From g = -170 on the quotient is -0, where |h| is below
// 2^-110, half of the least code, whatever u; NaN comes through.
constexpr float kF8Far = -69.f;
template <bool FAR>
__device__ __forceinline__ float f8_gate(float g, float u) {
    const bool far = FAR && g < kF8Far;
    const float s = far ? 0x1p-120f : 1.f;
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(g, -1.4426950408889634f, far ? -120.f : 0.f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s + e));
    return g * r * (u * s);
}
// N values of every lane of a warp.  Gates that far out are seldom there: one
// vote for all.  What it costs, 2048 rows, f 9728: k 8192 nothing (186 us), k 1024, where
// the epilogue is the bound, 50 to 54 (without the vote 59; lows in 8 chains, or a sum of
// the exponentials instead, 54 and 56).
template <int N>
__device__ __forceinline__ void f8_gated(const uint32_t (&g)[N], const uint32_t (&u)[N], float* h) {
    float low = __uint_as_float(g[0]);
#pragma unroll
    for (int i = 1; i < N; ++i) low = fminf(low, __uint_as_float(g[i]));
    if (__any_sync(0xffffffffu, low < kF8Far)) {
#pragma unroll
        for (int i = 0; i < N; ++i) h[i] = f8_gate<true>(__uint_as_float(g[i]), __uint_as_float(u[i]));
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) h[i] = f8_gate<false>(__uint_as_float(g[i]), __uint_as_float(u[i]));
    }
}

// ---- block-scaled products ----
//
// What the sums keep.  Accumulators are fp32 in tensor memory. A product adds 32
// of k: its addends are aligned to 2^-25 of the largest (measured: 2^16 + 4 x 2^-9 -
// 2^16 gives all four, of 2^-10 none) and the sum is cut to 24 bits, towards zero (1 + 2
// x 0.75 x 2^-23 - 1 gives 0, with 1.0 in place of 0.75 both). That is the
// instruction's rounding, the 16-bit operators' too. Over 28672 of k, 896 steps, it comes to 2 to
// 4e-5 of the outputs' size; half a step of bf16 is 4e-3, of fp16 5e-4. Sums taken
// out every few thousand of k and added in registers would be nearer, for a read of
// the whole tile each time.

// Instruction descriptor, kind::mxf8f6f4 with e4m3 operands, both K-major, ue8m0
// scales (bit 23); N >> 3 at bit 17, M >> 4 at bit 24; which byte of the scale
// words is meant at bits 4 (B) and 29 (A).
__host__ __device__ constexpr uint32_t f8_idesc(int M, int N) {
    return (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t f8_idesc_byte(uint32_t idesc, uint32_t byte) { return idesc | (byte << 4) | (byte << 29); }

// Issued by a whole warp in step, of which one elected thread (the same one every
// time) carries them out.  With a branch around them instead the descriptors
// would be moved to uniform registers before every product: a k-block then took
// 870 cycles, 344 of them to issue four products and their commit, where the
// tensor cores need 512 (4096 x 4864 x 32768: 470 us; issued so: 374).
template <bool PAIR>
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t a_scale, uint32_t b_scale,
                                          uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %6, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %6, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(accumulate)
            : "memory");
}
// The barrier (PAIR: at this offset in both CTAs) arrives once the products issued so far are done.
template <bool PAIR>
__device__ __forceinline__ void tc_commit_f8(uint32_t bar) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
            "h"(static_cast<uint16_t>(3))
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
            "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
            : "memory");
}
// Copies of a whole warp in step likewise: `bytes` announced on `bar`, boxes of
// 2-D and 3-D maps (coordinates innermost first).
__device__ __forceinline__ void expect_tx_f8(uint32_t bar, uint32_t bytes) {
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void tma_load_2d_f8(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar, uint64_t policy) {
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d_f8(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar, uint64_t policy) {
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
        : "memory");
}
// The box into L2 only.
__device__ __forceinline__ void tma_prefetch_2d_f8(const CUtensorMap* map, int c0, int c1) {
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];\n\t}" ::"l"(reinterpret_cast<uint64_t>(map)),
        "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ void tma_prefetch_3d_f8(const CUtensorMap* map, int c0, int c1, int c2) {
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];\n\t}" ::"l"(reinterpret_cast<uint64_t>(map)),
        "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// Arrival at a barrier of the cluster that hands nothing over in memory: a
// release at the cluster's scope waits for all that the thread has stored (1600
// cycles of an epilogue).
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// warp_wait that costs a test and a vote where the phase is over already.
template <bool CLUSTER>
__device__ __forceinline__ bool warp_wait_soon(uint32_t bar, uint32_t parity, const Ctl& c, unsigned where) {
    if (__all_sync(0xffffffffu, try_wait_scoped<CLUSTER>(bar, parity))) return true;
    return warp_wait<CLUSTER>(bar, parity, c, where);
}

// Scale words of 128 rows, shared memory -> 4 columns of tensor memory (in all
// four lane quadrants): row i + 32 j's word, whose byte b is the scale of the
// row's k-block 4 g + b, lies at bytes 16 i + 4 j of the 512.
constexpr int kScaleBlock = 512;
__device__ __forceinline__ uint32_t scale_word_at(uint32_t row) { return (row & 31u) * 16u + (row >> 5) * 4u; }
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    // no swizzle; eight-row groups of 16 bytes follow each other at 128 bytes
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 32) | (1ull << 46);
}
template <bool PAIR>
__device__ __forceinline__ void tc_copy_scales(uint32_t taddr, uint64_t desc) {
    if constexpr (PAIR)
        asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
                     "l"(desc)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
                     "l"(desc)
                     : "memory");
}

// One byte that an earlier kernel on the stream may have written.
__device__ __forceinline__ uint32_t load_byte(const uint8_t* p) {
    uint32_t v;
    asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
// Scale words of N rows at once: word i holds bytes [kb, kb + 4) of the
// `blocks` scale bytes at p[i], zero past them and where on[i] is false (p[i] is
// then not read).  kb is a multiple of 4 below `blocks`.  All loads are in
// flight together; whole words where rows of scales are words.
template <int N>
__device__ __forceinline__ void load_scale_words(const uint8_t* const (&p)[N], const bool (&on)[N], int kb, int blocks, bool words,
                                                 uint32_t (&v)[N]) {
    if (words) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\tmov.u32 %0, 0;\n\t@q ld.global.u32 %0, [%1];\n\t}"
                         : "=r"(v[i]) : "l"(p[i] + kb), "r"(static_cast<int>(on[i])));
        return;
    }
    uint32_t byte[N][4];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int b = 0; b < 4; ++b)
            asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\tmov.u32 %0, 0;\n\t@q ld.global.u8 %0, [%1];\n\t}"
                         : "=r"(byte[i][b]) : "l"(p[i] + kb + b), "r"(static_cast<int>(on[i] && kb + b < blocks)));
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = byte[i][0] | byte[i][1] << 8 | byte[i][2] << 16 | byte[i][3] << 24;
}

// The k-blocks of all shards one after another, in runs that share a scale
// word: up to 4 blocks of one shard.
struct F8Run {
    int shard, kb, count;      // blocks kb .. kb + count - 1 of the shard
};
__device__ __forceinline__ F8Run f8_run(int i, int per_shard, int kblocks) {
    F8Run r;
    r.shard = i / per_shard;
    r.kb = 4 * (i - r.shard * per_shard);
    r.count = min(4, kblocks - r.kb);
    return r;
}

}  // namespace
}  // namespace coc
