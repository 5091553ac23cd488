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
// byte (4 m) are few, but taking codes out of words costs instructions: a
// shift, a mask and an addition per pair, 88 of the 139 that a warp issues for
// 2048 weights at up to 8 tokens (197 at 16 with zero points), and their dependent sequences are
// the bound: 3.4 TB/s of weights at n 8192, k 8 x 1024, m 8 (10.5 us), 3.4 at
// n 14336, k 8 x 7168, m 16 with zero points (127 us); where they took
// 11.0 and 130, copying nothing at all left 9.6 and 109.
// W^T is the A operand of mma.sync (16 weight columns x 16 of k) and x^T the B
// operand (8 tokens).  A word holds 8 codes along k of one column; a mask
// takes two codes four apart into the halves of a register, so the pairs
// (k, k + 4) are the operand's neighbours, and x is permuted to match, once
// for the 64 columns of a warp.  or-ing the codes into the mantissa of 1024
// (bf16: 128) makes them floating-point numbers, and one addition takes off
// 1024 + z.
//
// Words and x come through a ring in shared memory in which a lane reads back
// only what it copied itself (but for the scales): no barrier in the loop.
//
// Split.  A block takes 64 columns, its 8 warps contiguous ranges of the
// contraction; a cluster's blocks take further ranges.  All ranges are added
// through shared memory in their order.
//
// Tried: codes as the A operand of tcgen05.mma in tensor memory, roles in 16
// warps.  Writing operands, permuting x and waiting cost more instructions
// (444 per 2048 weights at 16 tokens) than the registers' way: 221 us at
// n 14336, when that took 150.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "coc_kv.cuh"
#include "coc_ptx.cuh"

namespace coc {
namespace {

constexpr int kWarps = 8;
constexpr int kCols = 64;               // columns of a block; its warps split the contraction
constexpr int kStep = 32;               // contraction of one step: 4 word rows
// Stages of a warp's ring: two blocks' rings fill an SM's shared memory.
template <int SS>
constexpr int stages() { return SS == 4 ? 2 : SS == 2 ? 3 : 5; }

// A stage: SS x (two 16-byte pieces of words a lane, NT of x), then scales
// (16 bytes) and zero points (8 bytes) of the lanes 4 g.
template <int NT, int SS>
constexpr int stage_bytes() { return SS * 512 * (2 + NT) + 8 * 24; }
template <int NT>
constexpr int sum_floats() { return NT * 8 * kCols; }                      // one warp's sums
template <int NT, int SS>
constexpr int w4_smem() {
    const int ring = kWarps * stages<SS>() * stage_bytes<NT, SS>();
    const int sums = kWarps * sum_floats<NT>() * 4;
    return ring > sums ? ring : sums;
}

// Where every block can have an SM of its own it asks for more than half of an
// SM's shared memory: else the next launch's blocks, which come while this
// one's still run, gather two by two on the SMs that are free, and so do those
// of the launch after it.  n 8192, k 8 x 1024, m 8 then took 17.7 us a call
// instead of 10.9 for as long as calls followed each other, or 10.9, by the
// order the first blocks came in.
constexpr int kAloneSmem = 116 * 1024;

// n of BYTES bytes, the rest zero.
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, int n) {
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

// The same onto nothing: no accumulator has to be cleared.
template <bool BF16>
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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
// 2 H + 1.  off: -(B + z) twice, B the number whose mantissa takes the code: 128
// (bf16), 1024, or 1152 where z is an argument (fp16; -(1152 + z) is then the
// byte z + 128 in -1024's mantissa); off16: -(64 + z) (fp16: a code four bits up
// is 16 times itself, and its product with 1/16 costs the addition nothing).
template <bool BF16, bool ZERO, int H>
__device__ __forceinline__ void codes(uint32_t w, uint32_t off, uint32_t off16, uint32_t& p0, uint32_t& p1) {
    if constexpr (BF16) {
        p0 = add2<true>(and_or(w >> (8 * H), 0x000F000Fu, 0x43004300u), off);
        p1 = add2<true>(and_or(w >> (8 * H + 4), 0x000F000Fu, 0x43004300u), off);
    } else {
        const uint32_t v = w >> (8 * H);
        p0 = add2<false>(and_or(v, 0x000F000Fu, ZERO ? 0x64806480u : 0x64006400u), off);
        p1 = fma2_half(and_or(v, 0x00F000F0u, 0x64006400u), 0x2C002C00u, off16);
    }
}

// f in both halves, rounded to the 16-bit type (exact for the offsets).
template <bool BF16>
__device__ __forceinline__ uint32_t pair(float f) {
    return pack2<BF16>(__float_as_uint(f), __float_as_uint(f));
}

// Where part i of `all` stages in `ways` nearly equal parts begins.
__device__ __forceinline__ int part_begin(int all, int i, int ways) {
    const int each = all / ways;
    return each * i + min(i, all - each * ways);
}

// Block: 64 columns, 8 NT rows of x (blockIdx.y), kWarps ranges of the
// contraction; cluster: blocks with the same columns and further ranges.  SS
// steps make a stage (groups are whole stages; ONE: a group is one stage, which
// spares the bookkeeping of groups: groups of 32 at n 14336, m 16 take 130 us
// with it and 179 without, of 128 in stages of 64 take 124).
template <bool BF16, int NT, bool ZERO, int SS, bool ONE>
__global__ void __launch_bounds__(kWarps * 32, 2) w4_kernel(const __grid_constant__ W4Args a) {
    constexpr int SB = stage_bytes<NT, SS>(), kStages = stages<SS>();
    constexpr int XO = SS * 1024, CO = SS * 512 * (2 + NT);      // x, scales in a stage
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int split = static_cast<int>(cluster_rank()), splits = a.splits;
    const int col0 = static_cast<int>(blockIdx.x / splits) * kCols, row0 = blockIdx.y * 8 * NT;

    grid_dependency_wait();
    grid_dependents_launch();

    // this warp's stages, all ranks' shards one after another
    const int per_rank = a.k / (kStep * SS), per_group = a.group / (kStep * SS);
    const int s0 = part_begin(per_rank * a.R, split * kWarps + warp, splits * kWarps);
    const int s1 = part_begin(per_rank * a.R, split * kWarps + warp + 1, splits * kWarps);

    float acc[NT][4][4], part[NT][4][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[t][i][q] = part[t][i][q] = 0.f;

    if (s0 < s1) {
        // ---- producer: the next stage to be copied.  All addresses run on by
        // constants inside a rank's shard.
        const int n0 = col0 + 4 * g < a.n ? 16 : 0, n1 = col0 + 32 + 4 * g < a.n ? 16 : 0;       // bytes copied: none past the columns
        const uint32_t ring = smem_u32(smem) + warp * kStages * SB;
        const uint8_t* ring_p = smem + warp * kStages * SB;
        const size_t rows_w = size_t(16) * a.n;                         // bytes of a step's word rows
        // The 8 pieces of a word row stay together in shared memory (a copy writes a row at a time; scattered by lane, the
        // copies' writes alone took 73 cycles per 2048 weights), permuted so that the lanes' reads meet no bank twice.
        const uint32_t wslot = c * 128 + ((g ^ (2 * c)) << 4);
        int pr = s0 / per_rank, todo = s1 - s0;
        int in_rank, in_group;              // stages to the end of the rank's shard and of the group
        const uint8_t* wp;
        const uint16_t* xp[NT];
        const uint16_t* sp;
        const int8_t* zp = nullptr;
        bool new_group = true;
        auto enter = [&](int at) {          // stage `at` of rank pr
            in_rank = per_rank - at;
            in_group = per_group - at % per_group;
            wp = reinterpret_cast<const uint8_t*>(a.w[pr] + (static_cast<long long>(at) * 4 * SS + c) * a.n + col0 + 4 * g);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int row = row0 + 8 * t + g;
                xp[t] = a.x[pr] + static_cast<long long>(row < a.m ? row : 0) * a.k + at * SS * kStep + 8 * c;
            }
            const long long so = static_cast<long long>(at / per_group) * a.n + col0 + 4 * g;
            sp = a.scale[pr] + so;
            if constexpr (ZERO) zp = a.zero[pr] + so;
        };
        enter(s0 - pr * per_rank);
        int nx[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) nx[t] = row0 + 8 * t + g < a.m ? 16 : 0;
        auto load = [&](int stage) {
            if (todo > 0) {
                const uint32_t so = ring + stage * SB;
#pragma unroll
                for (int u = 0; u < SS; ++u) {
                    cp_async<16>(so + u * 1024 + wslot, wp, n0);
                    cp_async<16>(so + u * 1024 + 512 + wslot, wp + 128, n1);
                    wp += rows_w;
#pragma unroll
                    for (int t = 0; t < NT; ++t) cp_async<16>(so + XO + (u * NT + t) * 512 + lane * 16, xp[t] + u * kStep, nx[t]);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) xp[t] += SS * kStep;
                if (new_group) {
                    new_group = false;
                    if (c == 0) {
                        cp_async<8>(so + CO + g * 16, sp, n0 / 2);
                        cp_async<8>(so + CO + g * 16 + 8, sp + 32, n1 / 2);
                        if constexpr (ZERO) {
                            cp_async<4>(so + CO + 128 + g * 8, zp, n0 / 4);
                            cp_async<4>(so + CO + 128 + g * 8 + 4, zp + 32, n1 / 4);
                        }
                    }
                    sp += a.n;
                    if constexpr (ZERO) zp += a.n;
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

        int left = per_group - s0 % per_group;      // stages to the end of the group (shards are whole groups)
        bool fresh = true;
        uint4 sc;                                   // scales of the lane's 8 columns
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
                const bool first = fresh;           // of its group
                if (ONE || fresh) {
                    fresh = false;
                    __syncwarp();                   // the lanes 4 g copied it for the others
                    sc = *reinterpret_cast<const uint4*>(slot + CO + g * 16);
                    if constexpr (ZERO) {
                        const uint2 z2 = *reinterpret_cast<const uint2*>(slot + CO + 128 + g * 8);
                        const uint32_t zv[2] = {z2.x ^ 0x80808080u, z2.y ^ 0x80808080u};      // z + 128
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if constexpr (BF16) {
                                // 2^23 + (z + 128) is exact, and so is what is taken off
                                off[i] = pair<true>(8388608.f - __uint_as_float(__byte_perm(zv[i / 4], 0x4B000000u, 0x7650 + (i & 3))));
                            } else {
                                off[i] = __byte_perm(zv[i / 4], 0xE4E4E4E4u, 0x4040 + 0x0101 * (i & 3));
                                off16[i] = add2<false>(off[i], 0x64406440u);        // + 1088
                            }
                        }
                    }
                    __syncwarp();                   // read before a later stage's copy lands in the slot
                }
#pragma unroll
                for (int u = 0; u < SS; ++u) {
                    const uint4 w0 = *reinterpret_cast<const uint4*>(slot + u * 1024 + wslot);
                    const uint4 w1 = *reinterpret_cast<const uint4*>(slot + u * 1024 + 512 + wslot);
                    uint32_t b[NT][4];
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const uint4 x = *reinterpret_cast<const uint4*>(slot + XO + (u * NT + t) * 512 + lane * 16);
                        b[t][0] = __byte_perm(x.x, x.z, 0x5410);    // (x0, x4)
                        b[t][1] = __byte_perm(x.x, x.z, 0x7632);    // (x1, x5)
                        b[t][2] = __byte_perm(x.y, x.w, 0x5410);
                        b[t][3] = __byte_perm(x.y, x.w, 0x7632);
                    }
                    const uint32_t wv[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
                    // all tiles once per half: products into one accumulator do not follow each other
                    auto half = [&](auto hc, auto onto_nothing) {
                        constexpr int H = decltype(hc)::value;
                        constexpr bool FIRST = decltype(onto_nothing)::value;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {       // columns 2 i and 2 i + 1 of the lane's: rows g and g + 8 of the tile
                            uint32_t a0, a1, a2, a3;
                            codes<BF16, ZERO, H>(wv[2 * i], off[ZERO ? 2 * i : 0], off16[ZERO ? 2 * i : 0], a0, a2);
                            codes<BF16, ZERO, H>(wv[2 * i + 1], off[ZERO ? 2 * i + 1 : 0], off16[ZERO ? 2 * i + 1 : 0], a1, a3);
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                if (FIRST) mma16816_first<BF16>(part[t][i], a0, a1, a2, a3, b[t][0], b[t][1]);
                                else mma16816<BF16>(part[t][i], a0, a1, a2, a3, b[t][2 * H], b[t][2 * H + 1]);
                            }
                        }
                    };
                    using zeroth = std::integral_constant<int, 0>;
                    if (u == 0 && (ONE || first)) half(zeroth{}, std::true_type{});
                    else half(zeroth{}, std::false_type{});
                    half(std::integral_constant<int, 1>{}, std::false_type{});
                }
                if (ONE || --left == 0 || sb + st + 1 == s1) {
                    const uint32_t sv[4] = {sc.x, sc.y, sc.z, sc.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int q = 0; q < 4; q += 2) {
                            const float f = to_float16bit<BF16>(static_cast<uint16_t>(q ? sv[i] >> 16 : sv[i]));
#pragma unroll
                            for (int t = 0; t < NT; ++t) fma2(acc[t][i][q], acc[t][i][q + 1], part[t][i][q], part[t][i][q + 1], f);
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
    // the blocks of a cluster share the pairs of columns
    for (int x = threadIdx.x + split * kWarps * 32; x < SF / 2; x += kWarps * 32 * splits) {
        const int row = row0 + 2 * x / kCols, col = col0 + 2 * x % kCols;
        if (row >= a.m || col >= a.n) continue;
        float2 y = make_float2(0.f, 0.f);
        for (int b = 0; b < splits; ++b) {
            const uint32_t at = splits > 1 ? map_to_rank(smem_u32(sums + 2 * x), b) : 0u;
            float2 v[kWarps];
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                if (splits > 1)
                    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v[k].x), "=f"(v[k].y) : "r"(at + k * SF * 4) : "memory");
                else
                    v[k] = *reinterpret_cast<const float2*>(sums + k * SF + 2 * x);
            }
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                y.x += v[k].x;
                y.y += v[k].y;
            }
        }
        const uint32_t o = pack2<BF16>(__float_as_uint(y.x), __float_as_uint(y.y));
        for (int r = 0; r < a.R; ++r) *reinterpret_cast<uint32_t*>(a.out[r] + static_cast<long long>(row) * a.n + col) = o;
    }
    if (splits > 1) cluster_sync();     // no block leaves while its sums are read
}

template <bool BF16, int NT, bool ZERO, int SS, bool ONE>
cudaError_t launch_t(const W4Args& a, bool alone, cudaStream_t stream) {
    constexpr int kAlone = std::max(w4_smem<NT, SS>(), kAloneSmem);
    auto kern = w4_kernel<BF16, NT, ZERO, SS, ONE>;
    static std::atomic<unsigned char> smem_set[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !smem_set[dev].load(std::memory_order_acquire)) {
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kAlone)) != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) smem_set[dev].store(1, std::memory_order_release);
    }
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.n + kCols - 1) / kCols * a.splits), static_cast<unsigned>((a.m + 8 * NT - 1) / (8 * NT)), 1);
    cfg.blockDim = dim3(kWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = alone ? kAlone : w4_smem<NT, SS>();
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
cudaError_t launch_s(const W4Args& a, bool alone, cudaStream_t stream) {
    auto with = [&](auto steps) {
        constexpr int SS = decltype(steps)::value;
        return a.group == SS * kStep ? launch_t<BF16, NT, ZERO, SS, true>(a, alone, stream) : launch_t<BF16, NT, ZERO, SS, false>(a, alone, stream);
    };
    if constexpr (NT == 1)
        if (a.group % (4 * kStep) == 0) return with(std::integral_constant<int, 4>{});
    return a.group % (2 * kStep) == 0 ? with(std::integral_constant<int, 2>{}) : with(std::integral_constant<int, 1>{});
}
template <bool BF16>
cudaError_t launch_b(const W4Args& a, bool alone, cudaStream_t stream) {
    const bool two = a.m > 8, zero = a.zero[0] != nullptr;
    if (two) return zero ? launch_s<BF16, 2, true>(a, alone, stream) : launch_s<BF16, 2, false>(a, alone, stream);
    return zero ? launch_s<BF16, 1, true>(a, alone, stream) : launch_s<BF16, 1, false>(a, alone, stream);
}

// Blocks that run at once in clusters of k, one on an SM: a cluster lies within
// a part of the GPU whose SMs need not be a multiple of k (152 SMs hold 76, 36
// and 15 clusters of 2, 4 and 8).
cudaError_t alone_blocks(int k, int* out) {
    static std::atomic<int> known[64][9];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64 && (*out = known[dev][k].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
    auto kern = w4_kernel<true, 1, false, 1, true>;     // any: the shared memory asked for decides
    constexpr int kSmem = std::max(w4_smem<1, 1>(), kAloneSmem);
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)) != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(k);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(k), 1, 1);
    cfg.blockDim = dim3(kWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = kSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if ((e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg)) != cudaSuccess) return e;
    *out = n * k;
    if (dev >= 0 && dev < 64) known[dev][k].store(*out, std::memory_order_relaxed);
    return cudaSuccess;
}

}  // namespace

// Blocks of a cluster (ranges of the contraction) by the steps of the busiest
// SM: 64-column slabs that do not divide evenly over the SMs are evened out by
// halves to eighths, as far as joining them costs less: about 3 steps a block,
// and for a further range 1 where every block has an SM of its own and 14 where
// clusters wait for SMs.  (Two blocks on an SM take 1.8 times as long as one.)
// Measured, ranges 1 / 2 / 4 / 8: n 4096, k 4096, m 1 6.2 / 5.5 / 5.6 us; k 8 x
// 1024, m 8 at n 2048 10.1 / 8.3 / 7.2, n 4096 10.2 / 8.4 / 9.4, n 8192 10.4 /
// 12.4 / 17.6, n 10240 17.3 / 18.1 / 21.7, n 22528 25.9 / 28.6 / 39.6; n 704, k
// 2 x 16256, m 6 35.1 / 20.7 / 12.6 / 9.5; n 1280, k 4 x 4672, m 12 29.7 / 19.0 /
// 13.1 / 17.0; n 14336, k 8 x 7168, m 16 154 / 126 / 148.
cudaError_t launch_w4(const W4Args& args, bool bf16, int sm_count, cudaStream_t stream) {
    W4Args a = args;
    const double steps = static_cast<double>(a.k / kStep) * a.R;
    const int rows = a.m > 8 ? 16 : 8;
    const long long tiles = static_cast<long long>((a.n + kCols - 1) / kCols) * ((a.m + rows - 1) / rows);
    double best = 1e300;
    bool alone = false;
    for (int k : {1, 2, 4, 8}) {
        int room = sm_count;
        if (k > 1) {
            const cudaError_t e = alone_blocks(k, &room);
            if (e != cudaSuccess) return e;
            if (room < k) continue;
        }
        const long long rounds = (tiles * k + room - 1) / room;
        const double t = static_cast<double>(rounds) * (steps / (k * kWarps) + 3.0) + (rounds == 1 ? 1.0 : 14.0) * (k - 1);
        if (t < best) {
            best = t;
            a.splits = k;
            alone = rounds == 1;
        }
    }
    return bf16 ? launch_b<true>(a, alone, stream) : launch_b<false>(a, alone, stream);
}

}  // namespace coc
