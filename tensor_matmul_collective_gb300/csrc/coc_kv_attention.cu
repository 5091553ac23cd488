// Attention over the paged 8-bit key/value cache.
//
// Mathematics.  A row is one query head of one new token; the rows of a
// (sequence, key head) are packed token by token, 8 to a tile.  With a code c
// of a page whose scale is s, k = c s_k and v = c s_v, so with z = scale q.k
// in log2 units
//     out = sum_j 2^z_j s_vj c_j / sum_j 2^z_j.
// The page scale of V goes into the weight, w_j = 2^(z_j + log2 s_vj - m): it
// then needs no multiplication of its own, and m, the running maximum, is
// taken over z + log2 s_v, so that the products w c of all pages stay in the
// range of a 16-bit type whatever the scales are.  The denominator adds w / s_v.
//
// What bounds it.  2 d bytes of codes per key and key head are read once for
// up to 8 rows: 16 to 32 operations a byte, far below the tensor cores' rate,
// so it is the cache's bandwidth.  What the SMs must not do is spend many
// instructions per byte.  Codes go from e4m3 to fp16 in pairs (exact), as the
// operand of mma.sync: S^T = K Q^T with the keys in the 16 rows of the tile
// and the query rows in its 8 columns, O^T = V^T P^T with the head's values in
// the rows.  Both operands are permuted along the contraction so that each
// lane takes whole 16-byte pieces of the cache as they lie in memory, and a
// piece is read by exactly one lane: the asynchronous copies land in a
// lane-private slot of shared memory, with no bank conflict and no barrier.
// Q is fp16 (exact for fp16; a bf16 row is scaled by a power of two to the top
// of fp16's range first, so that it keeps its 8 bits down to 2^-29 of the
// row's largest value).  Weights are rounded to fp16 (11 bits); with fp16
// outputs a second product adds what that rounding left.
//
// Split.  The tiles of 64 keys of all (sequence, head, row tile) items form
// one list, cut into equal contiguous runs, one per resident block: lengths
// may be as unlike as they are, no SM idles.  An item that spans blocks leaves
// unnormalised parts, which a second kernel adds in order.
#include <algorithm>
#include <mutex>

#include "coc_kv.cuh"
#include "coc_ptx.cuh"

namespace coc {
namespace {

constexpr int kWarps = 4;
constexpr int kChunk = 16;                 // keys of one warp's step
constexpr int kTile = kWarps * kChunk;     // keys of one block's step
constexpr int kRows = 8;                   // query rows of a tile
constexpr int kStages = 3;                 // chunks in flight per warp
constexpr float kNoMax = -3.0e38f;         // running maximum before any key
// Weights are 2^(z - m + kOffset), with m at most 2^kSlack behind the true
// maximum (it moves only when a key exceeds it by more): at most 2^15, and
// normal fp16 numbers down to 2^-23 of m.
constexpr float kOffset = 9.f;
constexpr float kSlack = 6.f;

// Bytes of one chunk's slots: d-padded K and V, and two scales per lane.
template <int D>
constexpr int chunk_bytes() { return 2 * kChunk * D + 256; }
template <int D>
constexpr int merge_stride() { return D + 4; }
template <int D>
constexpr int attn_smem() {
    const int ring = kWarps * kStages * chunk_bytes<D>();
    const int merge = kWarps * kRows * merge_stride<D>() * 4;
    return ring > merge ? ring : merge;
}

// Scratch: per block two parts (kRows x D sums, then kRows maxima and sums),
// and a record of the item that the block begins and does not end.
struct Record {
    int open;        // 1: there is one
    int seq, head, row_tile;
    int last_block;
    int pad[3];
};
template <int D>
constexpr long long part_floats() { return kRows * (D + 2); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
    const int n = in ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(n) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, bool in) {
    const int n = in ? BYTES : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "n"(BYTES), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Two e4m3 codes (the low or high half of a word) as two fp16 values.
__device__ __forceinline__ uint32_t half2_of(uint16_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
    return r;
}
__device__ __forceinline__ uint32_t lo2(uint32_t w) { return half2_of(static_cast<uint16_t>(w)); }
__device__ __forceinline__ uint32_t hi2(uint32_t w) { return half2_of(static_cast<uint16_t>(w >> 16)); }

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The transpose of an 8 x 8 tile of 16-bit values held two to a lane.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float log2_fast(float x) {
    float r;
    asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// ---- the list of work ----

// New tokens of a sequence and the units (64-key tiles) that each of its
// (head, row tile) items counts: an upper bound over the row tiles, at least
// one so that every row is written.
struct SeqWork {
    int begin, n, len;      // first new token, how many, tokens in the cache
    int row_tiles, tiles;
};
__device__ __forceinline__ SeqWork seq_work(const KvAttnArgs& a, int s) {
    SeqWork w;
    int end;
    seq_tokens(a.cu, s, a.tokens, w.begin, end);
    w.n = end - w.begin;
    w.len = max(0, __ldg(a.lens + s));
    const long long room = a.table_width * a.page;
    if (w.len > room && w.n > 0) atomicOr(a.status, DEV_ERR_BAD_PAGE);
    const int group = a.q_heads / a.heads;
    w.row_tiles = static_cast<int>((static_cast<long long>(w.n) * group + kRows - 1) / kRows);
    // positions past the table are left out, by the pages' lookup too
    const int keys = static_cast<int>(min(static_cast<long long>(w.len), room));
    const int full = (keys + kTile - 1) / kTile;
    w.tiles = full;
    if (a.window > 0) {
        const long long span = static_cast<long long>(a.window) + (kRows - 1) / group + 1;   // keys of a row tile's window
        const long long most = (static_cast<long long>(a.sinks) + kTile - 1) / kTile + (span + kTile - 2) / kTile + 1;
        if (most < full) w.tiles = static_cast<int>(most);
    }
    if (w.tiles < 1) w.tiles = 1;
    return w;
}

__device__ __forceinline__ long long seq_units(const KvAttnArgs& a, int s) {
    const SeqWork w = seq_work(a, s);
    return static_cast<long long>(w.row_tiles) * w.tiles;
}

// Per-row limits of a row tile.
struct Rows {
    int end_min, end_max, from_min, from_max;   // over the tile's rows
};

template <bool BF16, int D>
__global__ void __launch_bounds__(kWarps * 32, D == 256 ? 2 : 4) kv_attention_kernel(const __grid_constant__ KvAttnArgs a) {
    constexpr int KL = D / 64;              // 16-byte pieces of a key per lane
    constexpr int VB = D >= 128 ? 16 : 8;   // bytes of a value row in one piece
    constexpr int VL = D >= 128 ? D / 128 : 1;
    constexpr int MT = D / 16;              // value tiles of 16
    constexpr int CB = chunk_bytes<D>();
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long scan[kWarps];
    __shared__ long long found[3];
    __shared__ float wm[kWarps][kRows], wl[kWarps][kRows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const int group = a.q_heads / a.heads;
    const int RH = a.R * a.heads;
    const int page_shift = 31 - __clz(a.page);

    grid_dependency_wait();
    grid_dependents_launch();

    // ---- this block's run of units: each thread adds a contiguous range of
    // sequences; the scan of the threads' sums gives the total and the start
    const int per = (a.seqs + kWarps * 32 - 1) / (kWarps * 32);
    const int s_lo = min(a.seqs, static_cast<int>(threadIdx.x) * per), s_hi = min(a.seqs, s_lo + per);
    long long mine = 0;
    for (int s = s_lo; s < s_hi; ++s) mine += seq_units(a, s);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    long long before = incl - mine, total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        if (i < warp) before += scan[i];
        total += scan[i];
    }
    total *= RH;
    before *= RH;
    const long long quota = max(1LL, (total + gridDim.x - 1) / gridDim.x);
    const long long u0 = quota * blockIdx.x, u1 = min(total, u0 + quota);
    Record* rec = reinterpret_cast<Record*>(a.scratch) + blockIdx.x;
    float* parts = reinterpret_cast<float*>(reinterpret_cast<Record*>(a.scratch) + gridDim.x);
    if (u0 >= u1) {
        if (threadIdx.x == 0) rec->open = 0;
        return;
    }
    if (before <= u0 && u0 < before + mine * RH) {
        long long at = before;
        for (int s = s_lo; s < s_hi; ++s) {
            const long long n = seq_units(a, s) * RH;
            if (u0 < at + n) {
                found[0] = s;
                found[1] = at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    int s = static_cast<int>(found[0]);
    long long base = found[1];      // first unit of sequence s
    SeqWork sw = seq_work(a, s);
    bool left_open = false;

    const uint32_t ring = smem_u32(smem) + warp * kStages * CB + lane * 16;
    const uint32_t ring8 = smem_u32(smem) + warp * kStages * CB + lane * VB;
    const uint32_t ring4 = smem_u32(smem) + warp * kStages * CB + lane * 4;
    const uint8_t* ring_p = smem + warp * kStages * CB;

    for (long long u = u0; u < u1;) {
        while (u >= base + static_cast<long long>(sw.row_tiles) * sw.tiles * RH) {
            base += static_cast<long long>(sw.row_tiles) * sw.tiles * RH;
            sw = seq_work(a, ++s);
        }
        // item (rank and head, row tile), tiles [t0, t1) of it
        const long long off = u - base;
        const int item = static_cast<int>(off / sw.tiles);
        const int t0 = static_cast<int>(off - static_cast<long long>(item) * sw.tiles);
        const int t1 = static_cast<int>(min(static_cast<long long>(sw.tiles), t0 + (u1 - u)));
        const int rh = item / sw.row_tiles, rt = item - rh * sw.row_tiles;
        const int r = rh / a.heads, h = rh - r * a.heads;

        // ---- rows and their limits
        const int rows = static_cast<int>(min(static_cast<long long>(kRows), static_cast<long long>(sw.n) * group - rt * kRows));
        const int i0 = rt * kRows / group, i1 = (rt * kRows + rows - 1) / group;
        const int shift = sw.len - sw.n + 1;        // token i's keys end at shift + i
        const int room = static_cast<int>(min(static_cast<long long>(0x7fffffff), a.table_width << page_shift));
        auto end_of = [&](int i) { return max(0, min(room, shift + i)); };
        // the window counts from the true end, the table's end only cuts
        auto from_of = [&](int i) { return a.window > 0 ? max(0, shift + i - a.window) : 0; };
        const int end_min = end_of(i0), end_max = end_of(i1), from_min = min(end_max, from_of(i0)), from_max = from_of(i1);
        const int sinks = a.window > 0 ? a.sinks : 0;
        const int far = from_min / kTile;
        const int near = min(far, (min(sinks, end_max) + kTile - 1) / kTile);   // sink tiles ahead of the window's
        const int tiles = near + max(0, (end_max + kTile - 1) / kTile - far);
        auto tile_of = [&](int t) { return t < near ? t : far + t - near; };
        int row_end[2], row_from[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int rr = min(2 * c + x, rows - 1);
            const int i = (rt * kRows + rr) / group;
            row_end[x] = end_of(i);
            row_from[x] = from_of(i);
        }

        // ---- Q as the B operand: lane (g, c) holds row g, the 16 values of
        // each of its pieces (i * 4 + c), as the keys' lanes hold theirs
        uint32_t qf[KL * 8];
        float qscale = a.scale * 1.4426950408889634f;
        {
            const int rho = rt * kRows + g;
            const bool valid = g < rows;
            const int tok = sw.begin + rho / group;
            const uint16_t* qp = a.q[r] + (valid ? tok * a.q_token + (h * group + rho % group) * a.q_head : 0);
#pragma unroll
            for (int i = 0; i < KL; ++i) {
                const int e = (i * 4 + c) * 16;
                uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
                if (valid && e < a.d) {
                    v0 = *reinterpret_cast<const uint4*>(qp + e);
                    v1 = *reinterpret_cast<const uint4*>(qp + e + 8);
                }
                qf[8 * i + 0] = v0.x; qf[8 * i + 1] = v0.y; qf[8 * i + 2] = v0.z; qf[8 * i + 3] = v0.w;
                qf[8 * i + 4] = v1.x; qf[8 * i + 5] = v1.y; qf[8 * i + 6] = v1.z; qf[8 * i + 7] = v1.w;
            }
            if constexpr (BF16) {
                uint32_t top = 0;   // the largest magnitude's bits
#pragma unroll
                for (int i = 0; i < KL * 8; ++i) {
                    const uint32_t x = qf[i] & 0x7fff7fffu;
                    top = max(top, max(x & 0xffffu, x >> 16));
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int ex = static_cast<int>(top >> 7);                     // biased exponent; 255: not finite
                const int up = (ex == 255 || ex == 0) ? 0 : min(126, 127 + 14 - ex);   // largest value to 2^14
                const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
#pragma unroll
                for (int i = 0; i < KL * 8; ++i)
                    qf[i] = pack_half2(__uint_as_float(qf[i] << 16) * f, __uint_as_float(qf[i] & 0xffff0000u) * f);
                qscale *= __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
            }
        }
        // row factors of the columns 2c, 2c + 1 of S^T
        const float qs0 = __shfl_sync(0xffffffffu, qscale, 8 * c), qs1 = __shfl_sync(0xffffffffu, qscale, 8 * c + 4);

        float acc[MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
        float m0 = kNoMax, m1 = kNoMax, l0 = 0.f, l1 = 0.f;

        // ---- the chunks of this warp: tile t's keys j .. j + 15
        const int tn = min(t1, tiles);
        const int32_t* table = a.table + static_cast<long long>(s) * a.table_width;
        auto page_at = [&](int t) {     // page id of this warp's chunk of tile t, -1 if it has none
            if (t >= tn) return -1;
            const int j = tile_of(t) * kTile + warp * kChunk;
            if (j >= end_max) return -1;
            const int id = __ldg(table + (j >> page_shift));
            if (id < 0 || id >= a.pages) {
                // reported only where a row looks at the page
                if (lane == 0 && (j + kChunk > from_min || j < sinks)) atomicOr(a.status, DEV_ERR_BAD_PAGE);
                return -1;
            }
            return id;
        };
        auto seen = [&](int j) { return j < end_max && (j >= from_min || j < sinks); };   // by any row of the tile
        auto load = [&](int t, int id, int stage) {
            if (id >= 0) {
                const int j = tile_of(t) * kTile + warp * kChunk;
                const long long ph = static_cast<long long>(id) * a.heads + h;
                const uint8_t* kp = a.ck[r] + ((ph << page_shift) + (j & (a.page - 1))) * a.d;
                const uint8_t* vp = a.cv[r] + ((ph << page_shift) + (j & (a.page - 1))) * a.d;
                const uint32_t so = stage * CB;
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int i = 0; i < KL; ++i) {
                        const int e = (i * 4 + c) * 16;
                        cp_async16(ring + so + (x * KL + i) * 512, kp + (g + 8 * x) * a.d + e, e < a.d && seen(j + g + 8 * x));
                    }
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int tok = 2 * c + (y & 1) + 8 * (y >> 1);
                    const bool in = seen(j + tok);
#pragma unroll
                    for (int i = 0; i < VL; ++i) {
                        const int e = i * 128 + g * VB;
                        if constexpr (VB == 16)
                            cp_async16(ring + so + kChunk * D + (y * VL + i) * 512, vp + tok * a.d + e, in && e < a.d);
                        else
                            cp_async_small<8>(ring8 + so + kChunk * D + y * 256, vp + tok * a.d + e, in && e < a.d);
                    }
                }
                cp_async_small<4>(ring4 + so + 2 * kChunk * D, a.sk[r] + ph, true);
                cp_async_small<4>(ring4 + so + 2 * kChunk * D + 128, a.sv[r] + ph, true);
            }
            cp_commit();
        };
        int ids[kStages];       // page ids of the chunks in flight
        int next_id;            // of the chunk to be loaded next
        {
#pragma unroll
            for (int i = 0; i < kStages - 1; ++i) ids[i] = page_at(t0 + i);
            next_id = page_at(t0 + kStages - 1);
#pragma unroll
            for (int i = 0; i < kStages - 1; ++i) load(t0 + i, ids[i], i);
        }
        for (int tb = t0; tb < tn; tb += kStages) {
#pragma unroll
            for (int st = 0; st < kStages; ++st) {
                const int t = tb + st;
                if (t >= tn) break;
                constexpr int last = kStages - 1;
                const int into = (st + last) % kStages;
                ids[into] = next_id;
                load(t + last, next_id, into);
                next_id = page_at(t + kStages);
                cp_wait<last>();
                if (ids[st] < 0) continue;
                const int j = tile_of(t) * kTile + warp * kChunk;
                const uint8_t* slot = ring_p + st * CB;
                const float sk = *reinterpret_cast<const float*>(slot + 2 * kChunk * D + lane * 4);
                const float sv = fmaxf(*reinterpret_cast<const float*>(slot + 2 * kChunk * D + 128 + lane * 4), 1.2e-38f);
                // S^T = K Q^T
                float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < KL; ++i) {
                    const uint4 ka = *reinterpret_cast<const uint4*>(slot + i * 512 + lane * 16);
                    const uint4 kb = *reinterpret_cast<const uint4*>(slot + (KL + i) * 512 + lane * 16);
                    const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t af[4] = {lo2(wa[w]), lo2(wb[w]), hi2(wa[w]), hi2(wb[w])};
                        mma16816(sc, af, qf[8 * i + 2 * w], qf[8 * i + 2 * w + 1]);
                    }
                }
                const float ev = log2_fast(sv);
                const float f0 = qs0 * sk, f1 = qs1 * sk;
                float z[4] = {fmaf(sc[0], f0, ev), fmaf(sc[1], f1, ev), fmaf(sc[2], f0, ev), fmaf(sc[3], f1, ev)};
                const bool whole = j + kChunk <= end_min && (j >= from_max || j + kChunk <= sinks);
                uint32_t see = 0xf;     // bit x: z[x]'s row sees its key
                if (!whole) {
                    see = 0;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int key = j + g + 8 * (x >> 1);
                        const bool in = key < row_end[x & 1] && (key >= row_from[x & 1] || key < sinks);
                        see |= static_cast<uint32_t>(in) << x;
                        if (!in) z[x] = -INFINITY;
                    }
                }
                // the reference moves only when a key is well above it
                if (__any_sync(0xffffffffu, fmaxf(z[0], z[2]) > m0 + kSlack || fmaxf(z[1], z[3]) > m1 + kSlack)) {
                    float t0m = fmaxf(m0, fmaxf(z[0], z[2])), t1m = fmaxf(m1, fmaxf(z[1], z[3]));
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) {
                        t0m = fmaxf(t0m, __shfl_xor_sync(0xffffffffu, t0m, o));
                        t1m = fmaxf(t1m, __shfl_xor_sync(0xffffffffu, t1m, o));
                    }
                    const float c0 = exp2_fast(m0 - t0m), c1 = exp2_fast(m1 - t1m);
                    m0 = t0m;
                    m1 = t1m;
                    l0 *= c0;
                    l1 *= c1;
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        acc[i][0] *= c0;
                        acc[i][1] *= c1;
                        acc[i][2] *= c0;
                        acc[i][3] *= c1;
                    }
                }
                const float b0 = kOffset - m0, b1 = kOffset - m1;
                float w[4] = {exp2_fast(z[0] + b0), exp2_fast(z[1] + b1), exp2_fast(z[2] + b0), exp2_fast(z[3] + b1)};
                const float inv = __frcp_rn(sv);
                l0 = fmaf(w[0] + w[2], inv, l0);
                l1 = fmaf(w[1] + w[3], inv, l1);
                const uint32_t plo = pack_half2(w[0], w[1]), phi = pack_half2(w[2], w[3]);
                const uint32_t p0 = transposed(plo), p1 = transposed(phi);
                uint32_t e0 = 0, e1 = 0;
                if constexpr (!BF16) {
                    const float2 rl = __half22float2(*reinterpret_cast<const __half2*>(&plo));
                    const float2 rh2 = __half22float2(*reinterpret_cast<const __half2*>(&phi));
                    e0 = transposed(pack_half2(w[0] - rl.x, w[1] - rl.y));
                    e1 = transposed(pack_half2(w[2] - rh2.x, w[3] - rh2.y));
                }
                // O^T += V^T P^T
                uint32_t vw[4][VL * VB / 4];
#pragma unroll
                for (int y = 0; y < 4; ++y)
#pragma unroll
                    for (int i = 0; i < VL; ++i) {
                        if constexpr (VB == 16) {
                            const uint4 v = *reinterpret_cast<const uint4*>(slot + kChunk * D + (y * VL + i) * 512 + lane * 16);
                            vw[y][4 * i] = v.x; vw[y][4 * i + 1] = v.y; vw[y][4 * i + 2] = v.z; vw[y][4 * i + 3] = v.w;
                        } else {
                            const uint2 v = *reinterpret_cast<const uint2*>(slot + kChunk * D + y * 256 + lane * 8);
                            vw[y][0] = v.x; vw[y][1] = v.y;
                        }
                    }
                if (!whole) {
                    // a NaN of a key that only some rows see would reach the others as 0 x NaN: where the
                    // chunk has one, it is taken out of the product and put into the rows that see it
                    uint32_t nan = 0;
#pragma unroll
                    for (int y = 0; y < 4; ++y)
#pragma unroll
                        for (int i = 0; i < VL * VB / 4; ++i) nan |= ((vw[y][i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                    if (__any_sync(0xffffffffu, nan != 0)) {
                        const uint32_t i0b = transposed(pack_half2(see & 1 ? 1.f : 0.f, see & 2 ? 1.f : 0.f));
                        const uint32_t i1b = transposed(pack_half2(see & 4 ? 1.f : 0.f, see & 8 ? 1.f : 0.f));
#pragma unroll
                        for (int i = 0; i < MT / 2; ++i) {
                            uint32_t x[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const uint32_t bad = ((((vw[y][i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xffu;
                                x[y] = bad & 0x38383838u;       // e4m3 1.0 where NaN
                                vw[y][i] &= ~bad;
                            }
                            const uint32_t a01 = __byte_perm(x[0], x[1], 0x5140), a23 = __byte_perm(x[2], x[3], 0x5140);
                            const uint32_t b01 = __byte_perm(x[0], x[1], 0x7362), b23 = __byte_perm(x[2], x[3], 0x7362);
                            const uint32_t fa[4] = {lo2(a01), hi2(a01), lo2(a23), hi2(a23)}, fb[4] = {lo2(b01), hi2(b01), lo2(b23), hi2(b23)};
                            float ta[4] = {0.f, 0.f, 0.f, 0.f}, tb2[4] = {0.f, 0.f, 0.f, 0.f};
                            mma16816(ta, fa, i0b, i1b);
                            mma16816(tb2, fb, i0b, i1b);
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                if (ta[q] > 0.f) acc[2 * i][q] = __uint_as_float(0x7fc00000u);
                                if (tb2[q] > 0.f) acc[2 * i + 1][q] = __uint_as_float(0x7fc00000u);
                            }
                        }
                    }
                }
                // word i of the four keys: bytes 0, 1 make value tile 2i, bytes 2, 3 tile 2i + 1
#pragma unroll
                for (int i = 0; i < MT / 2; ++i) {
                    const uint32_t a01 = __byte_perm(vw[0][i], vw[1][i], 0x5140), a23 = __byte_perm(vw[2][i], vw[3][i], 0x5140);
                    const uint32_t b01 = __byte_perm(vw[0][i], vw[1][i], 0x7362), b23 = __byte_perm(vw[2][i], vw[3][i], 0x7362);
                    const uint32_t fa[4] = {lo2(a01), hi2(a01), lo2(a23), hi2(a23)}, fb[4] = {lo2(b01), hi2(b01), lo2(b23), hi2(b23)};
                    mma16816(acc[2 * i], fa, p0, p1);
                    mma16816(acc[2 * i + 1], fb, p0, p1);
                    if constexpr (!BF16) {
                        mma16816(acc[2 * i], fa, e0, e1);
                        mma16816(acc[2 * i + 1], fb, e0, e1);
                    }
                }
            }
        }
        cp_wait<0>();

        // ---- join the warps: maxima and sums, then the value sums in the
        // accumulators' order (value d = g VB + 2 i + b at 16 i + 2 g + b)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, o);
            l1 += __shfl_xor_sync(0xffffffffu, l1, o);
        }
        if (g == 0) {
            wm[warp][2 * c] = m0;
            wm[warp][2 * c + 1] = m1;
            wl[warp][2 * c] = l0;
            wl[warp][2 * c + 1] = l1;
        }
        __syncthreads();    // the ring is free too
        float M0 = wm[0][2 * c], M1 = wm[0][2 * c + 1];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) {
            M0 = fmaxf(M0, wm[i][2 * c]);
            M1 = fmaxf(M1, wm[i][2 * c + 1]);
        }
        const float k0 = exp2_fast(m0 - M0), k1 = exp2_fast(m1 - M1);
        constexpr int MS = merge_stride<D>();
        float* mine_s = reinterpret_cast<float*>(smem) + warp * kRows * MS;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            *reinterpret_cast<float2*>(mine_s + 2 * c * MS + 16 * i + 2 * g) = make_float2(acc[i][0] * k0, acc[i][2] * k0);
            *reinterpret_cast<float2*>(mine_s + (2 * c + 1) * MS + 16 * i + 2 * g) = make_float2(acc[i][1] * k1, acc[i][3] * k1);
        }
        __syncthreads();
        const bool begins = t0 == 0, ends = t1 == sw.tiles;
        float* part = parts + (2LL * blockIdx.x + (begins ? 1 : 0)) * part_floats<D>();
        for (int x = threadIdx.x; x < kRows * D / 2; x += kWarps * 32) {
            const int row = x / (D / 2), p = x % (D / 2) * 2;
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const float2 v = *reinterpret_cast<const float2*>(reinterpret_cast<const float*>(smem) + (i * kRows + row) * MS + p);
                sum.x += v.x;
                sum.y += v.y;
            }
            float M = wm[0][row];
#pragma unroll
            for (int i = 1; i < kWarps; ++i) M = fmaxf(M, wm[i][row]);
            float L = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) L += wl[i][row] * exp2_fast(wm[i][row] - M);
            if (begins && ends) {
                const int tile = p / 16, gg = (p % 16) / 2;
                const int e = VB == 16 ? tile / 8 * 128 + gg * 16 + tile % 8 * 2 : gg * 8 + tile * 2;
                if (row < rows && e < a.d) {
                    const int rho = rt * kRows + row;
                    const float inv = L == 0.f ? 0.f : 1.f / L;     // no key seen: zero
                    uint16_t* o = a.out[r] + (static_cast<long long>(sw.begin + rho / group) * a.q_heads + h * group + rho % group) * a.d + e;
                    *reinterpret_cast<uint32_t*>(o) = pack2<BF16>(__float_as_uint(sum.x * inv), __float_as_uint(sum.y * inv));
                }
            } else {
                *reinterpret_cast<float2*>(part + row * D + p) = sum;
                if (p == 0) {
                    part[kRows * D + row] = M;
                    part[kRows * D + kRows + row] = L;
                }
            }
        }
        if (begins && !ends) {
            left_open = true;
            if (threadIdx.x == 0) {
                rec->seq = s;
                rec->head = rh;
                rec->row_tile = rt;
                rec->last_block = static_cast<int>((u - t0 + sw.tiles - 1) / quota);
            }
        }
        __syncthreads();    // the merge area and wm are read before the next item
        u += t1 - t0;
    }
    if (threadIdx.x == 0) rec->open = left_open ? 1 : 0;
}

// Block (b, row): adds the parts of the item that block b began and others
// went on with, in their order.
template <bool BF16, int D>
__global__ void __launch_bounds__(D / 2) kv_attention_merge(const __grid_constant__ KvAttnArgs a) {
    constexpr int VB = D >= 128 ? 16 : 8;
    grid_dependency_wait();
    const Record* recs = reinterpret_cast<const Record*>(a.scratch);
    const Record rec = recs[blockIdx.x];
    if (!rec.open) return;
    const int group = a.q_heads / a.heads;
    int begin, end;
    seq_tokens(a.cu, rec.seq, a.tokens, begin, end);
    const int rho = rec.row_tile * kRows + blockIdx.y;
    if (rho >= (end - begin) * group) return;
    const float* parts = reinterpret_cast<const float*>(recs + gridDim.x);
    const int row = blockIdx.y, first = blockIdx.x, count = rec.last_block - first + 1, p = 2 * threadIdx.x;
    auto part = [&](int i) { return parts + (2LL * (first + i) + (i == 0 ? 1 : 0)) * part_floats<D>(); };
    float M = kNoMax;
    for (int i = 0; i < count; ++i) M = fmaxf(M, part(i)[kRows * D + row]);
    float L = 0.f;
    float2 sum = make_float2(0.f, 0.f);
    for (int i = 0; i < count; ++i) {
        const float* q = part(i);
        const float f = exp2_fast(q[kRows * D + row] - M);
        L = fmaf(q[kRows * D + kRows + row], f, L);
        const float2 v = *reinterpret_cast<const float2*>(q + row * D + p);
        sum.x = fmaf(v.x, f, sum.x);
        sum.y = fmaf(v.y, f, sum.y);
    }
    const int tile = p / 16, gg = (p % 16) / 2;
    const int e = VB == 16 ? tile / 8 * 128 + gg * 16 + tile % 8 * 2 : gg * 8 + tile * 2;
    if (e >= a.d) return;
    const int r = rec.head / a.heads, h = rec.head - r * a.heads;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    uint16_t* o = a.out[r] + (static_cast<long long>(begin + rho / group) * a.q_heads + h * group + rho % group) * a.d + e;
    *reinterpret_cast<uint32_t*>(o) = pack2<BF16>(__float_as_uint(sum.x * inv), __float_as_uint(sum.y * inv));
}

template <bool BF16, int D>
cudaError_t resident_blocks(int* out) {
    static std::mutex mu;
    static int cached[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lk(mu);
    if (dev >= 0 && dev < 64 && cached[dev] > 0) {
        *out = cached[dev];
        return cudaSuccess;
    }
    e = cudaFuncSetAttribute(kv_attention_kernel<BF16, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, attn_smem<D>());
    if (e != cudaSuccess) return e;
    int n = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kv_attention_kernel<BF16, D>, kWarps * 32, attn_smem<D>());
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    if (dev >= 0 && dev < 64) cached[dev] = n;
    *out = n;
    return cudaSuccess;
}

// Head sizes up to 64, 128 and 256 have instances of their own (shorter heads
// are padded with zero bytes that are never read).
int padded_d(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

template <bool BF16, int D>
cudaError_t launch_t(const KvAttnArgs& a, int grid, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(kWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = attn_smem<D>();
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_launch() ? 1 : 0;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kv_attention_kernel<BF16, D>, a);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(grid), kRows, 1);
    cfg.blockDim = dim3(D / 2, 1, 1);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, kv_attention_merge<BF16, D>, a);
}

}  // namespace

cudaError_t kv_attention_plan(const KvAttnArgs& a, bool bf16, int sm_count, int* grid, size_t* scratch) {
    const int D = padded_d(a.d);
    int n = 0;
    cudaError_t e;
    if (bf16) e = D == 64 ? resident_blocks<true, 64>(&n) : D == 128 ? resident_blocks<true, 128>(&n) : resident_blocks<true, 256>(&n);
    else e = D == 64 ? resident_blocks<false, 64>(&n) : D == 128 ? resident_blocks<false, 128>(&n) : resident_blocks<false, 256>(&n);
    if (e != cudaSuccess) return e;
    // never more blocks than there can be units
    const int group = a.q_heads / a.heads;
    const long long items = (static_cast<long long>(a.tokens) * group / kRows + a.seqs) * a.R * a.heads;
    const long long tiles = std::max<long long>(1, (a.table_width * a.page + kTile - 1) / kTile);
    const long long resident = static_cast<long long>(n) * sm_count;
    *grid = static_cast<int>(tiles >= resident ? resident : std::min(resident, items * tiles));
    *scratch = static_cast<size_t>(*grid) * (sizeof(Record) + 2 * kRows * (D + 2) * sizeof(float));
    return cudaSuccess;
}

cudaError_t launch_kv_attention(const KvAttnArgs& a, bool bf16, int grid, cudaStream_t stream) {
    const int D = padded_d(a.d);
    if (bf16) return D == 64 ? launch_t<true, 64>(a, grid, stream) : D == 128 ? launch_t<true, 128>(a, grid, stream) : launch_t<true, 256>(a, grid, stream);
    return D == 64 ? launch_t<false, 64>(a, grid, stream) : D == 128 ? launch_t<false, 128>(a, grid, stream) : launch_t<false, 256>(a, grid, stream);
}

}  // namespace coc
