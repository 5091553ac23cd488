// Attention over the paged 8-bit key/value cache.
//
// Mathematics.  A row is one query head of one new token; the rows of a
// (sequence, key head) are packed token by token, 8 or 16 to a tile.  With a code c
// of a page whose scale is s, k = c s_k and v = c s_v, so with z = scale q.k
// in log2 units
//     out = sum_j 2^z_j s_vj c_j / sum_j 2^z_j.
// The page scale of V goes into the weight, w_j = 2^(z_j + log2 s_vj - m): it
// then needs no multiplication of its own, and m, the running maximum, is
// taken over z + log2 s_v, so that the products w c of all pages stay in the
// range of a 16-bit type whatever the scales are.  The denominator adds w / s_v;
// where pages differ by more than 2^kFarScale that weight may be below fp32's
// range while the key still counts (its values do not): 2^(z_j - m) is taken
// instead.  A sum that moves to another maximum is scaled in two steps, by the
// square root of a factor that may be below that range itself.
//
// What bounds it.  2 d bytes of codes per key and key head are read once for
// up to 8 or 16 rows: 16 to 32 operations a byte, far below the tensor cores' rate,
// so it is the cache's bandwidth.  What the SMs must not do is spend many
// instructions per byte.  Codes go from e4m3 to fp16 in pairs (exact), as the
// operand of mma.sync: S^T = K Q^T with the keys in the 16 rows of the tile
// and the query rows in its 8 columns, O^T = V^T P^T with the head's values in
// the rows.  Both operands are permuted along the contraction so that each
// lane takes whole 16-byte pieces of the cache as they lie in memory, and a
// piece is read by exactly one lane, straight into registers: no shared
// memory, no barrier.  The next chunk is loaded while one is worked on.
// (The same pieces through asynchronous copies into lane-private slots of
// shared memory measured 118 against 106 us for two sequences of 131071 keys
// on 8 ranks: the copies and their reads fill the memory pipe twice.)
// Q is fp16 (exact for fp16; a bf16 row is scaled by a power of two to the top
// of fp16's range first, so that it keeps its 8 bits down to 2^-29 of the
// row's largest value).  A weight is two fp16 numbers, itself rounded to 11 bits
// and what that left, and V is multiplied by both: 22 bits.  (One product with
// 11 bits moved bf16 outputs by up to 2^-12 of sum p |v|, more than their own
// rounding where values cancel; with the second the same batch of 48 sequences
// takes 74.7 instead of 73.5 us, with 16 rows a tile 94 instead of 87.)
//
// Split.  The tiles of 64 keys of all (sequence, head, row tile) items form
// one list, in which every item also counts kItemCost tiles for its beginning
// and end, cut into equal contiguous runs, one per resident block: whatever the
// lengths, no SM idles in this kernel.  An item that spans blocks leaves
// unnormalised parts, which a second kernel adds in order.
//
// Measured: 48 sequences of 1 to 8192 keys, 8 ranks of one key head with 8
// query heads of 128: 73 to 79 us by their lengths, 5.1 to 5.4 TB/s; two of
// 131071: 93 us, 5.8 TB/s.  With 16 query heads (16 rows a tile) 48 sequences of
// 4096 keys take 94 us, 4.3 TB/s: the conversions and products of a byte, at
// two blocks an SM.  24 of 4096 keys with 8 query heads of 256: 80 us, 5.1 TB/s.
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "coc_kv.cuh"
#include "coc_ptx.cuh"

namespace coc {
namespace {

constexpr int kWarps = 4;
constexpr int kSub = 16;                   // keys of one matrix product
constexpr int kTile = kWarps * kSub;       // keys of one block's step
constexpr float kNoMax = -1.0e38f;         // running maximum before any key
// What beginning and ending an item costs, in tiles: an item counts as so many
// units more than it has tiles.
constexpr int kItemCost = 3;
// Weights are 2^(z - m + kOffset), with m at most 2^kSlack behind the true
// maximum (it moves only when a key exceeds it by more): at most 2^15, and
// normal fp16 numbers down to 2^-23 of m.
constexpr float kOffset = 9.f;
constexpr float kSlack = 6.f;
// Binary digits between a page's scale of V and the largest so far, up to which
// w / s_v may be added: a key whose w is below 2^-126 there has less than 2^-70
// of the weight of the key that the maximum stands for.
constexpr float kFarScale = 60.f;

// Shared memory: the warps' sums, joined at the end of an item.
template <int D>
constexpr int merge_stride() { return D + 4; }
template <int D, int ROWS>
constexpr int attn_smem() { return kWarps * ROWS * merge_stride<D>() * 4; }

// Scratch: per block two parts (ROWS x D sums, then ROWS maxima and sums),
// and a record of the item that the block begins and does not end.
struct __align__(32) Record {
    int rows;                   // 0: there is none
    int last_block;
    int head;                   // rank and key head
    int token, row;             // the sequence's first token, the tile's first row after it
    int pad[3];
};
template <int D, int ROWS>
constexpr long long part_floats() { return ROWS * (D + 2); }

// value of the head that the pair p of an accumulator row begins with
template <int D>
__device__ __forceinline__ int value_of(int p) {
    const int tile = p / 16, g = (p % 16) / 2;
    return D >= 128 ? tile / 8 * 128 + g * 16 + tile % 8 * 2 : g * 8 + tile * 2;
}

// Where the outputs of a token's query head lie.
__device__ __forceinline__ uint16_t* out_at(const KvAttnArgs& a, int rank, int token, int head) {
    return a.out[rank] + (static_cast<long long>(token) * a.q_heads + head) * a.d;
}

// Codes are read once by one lane: no place in L1.
__device__ __forceinline__ uint4 load16(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 load8(const uint8_t* p) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

__device__ __forceinline__ uint4 load16_if(const uint8_t* p, bool in) {
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"(static_cast<int>(in)));
    return v;
}
__device__ __forceinline__ uint2 load8_if(const uint8_t* p, bool in) {
    uint2 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %3, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
        "@p ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];\n\t}"
        : "=&r"(v.x), "=&r"(v.y)
        : "l"(p), "r"(static_cast<int>(in)));
    return v;
}

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
template <int ROWS>
__device__ __forceinline__ SeqWork seq_work(const KvAttnArgs& a, int s) {
    SeqWork w;
    int end;
    seq_tokens(a.cu, s, a.tokens, w.begin, end);
    w.n = end - w.begin;
    w.len = max(0, load_index(a.lens + s));
    const long long room = a.table_width * a.page;
    if (w.len > room && w.n > 0) atomicOr(a.status, DEV_ERR_BAD_PAGE);
    const int group = a.q_heads / a.heads;
    w.row_tiles = static_cast<int>((static_cast<long long>(w.n) * group + ROWS - 1) / ROWS);
    // positions past the table are left out, by the pages' lookup too
    const int keys = static_cast<int>(min(static_cast<long long>(w.len), room));
    const int full = (keys + kTile - 1) / kTile;
    w.tiles = full;
    if (a.window > 0) {
        const long long span = static_cast<long long>(a.window) + (ROWS - 1) / group + 1;   // keys of a row tile's window
        const long long most = (static_cast<long long>(a.sinks) + kTile - 1) / kTile + (span + kTile - 2) / kTile + 1;
        if (most < full) w.tiles = static_cast<int>(most);
    }
    if (w.tiles < 1) w.tiles = 1;
    return w;
}

template <int ROWS>
__device__ __forceinline__ long long seq_units(const KvAttnArgs& a, int s) {
    const SeqWork w = seq_work<ROWS>(a, s);
    return static_cast<long long>(w.row_tiles) * (w.tiles + kItemCost);
}

// The keys that the rows of a tile see: row x those from row_from[x] (and the
// sinks) up to row_end[x]; end and from are the last and the first of these.
template <int ROWS>
struct Limits {
    int end, from, sinks;
    int row_end[ROWS], row_from[ROWS];
};

// Resident blocks: what the registers allow.
template <int D, int ROWS>
constexpr int blocks_per_sm() { return D == 256 || (D == 128 && ROWS == 16) ? 2 : 3; }

// An item's end: each row's maximum and sum over the warps, one over the sum
// (0 if there is none: no key seen, zero), and its place in the output.
template <int ROWS>
struct Ending {
    float max[ROWS], sum[ROWS], inv[ROWS];
    uint16_t* out[ROWS];
};

// EXACT: the head has D values (every offset inside a chunk is a constant);
// otherwise fewer, and the pieces past them are zero.
template <bool BF16, int D, bool EXACT, int ROWS>
__global__ void __launch_bounds__(kWarps * 32, blocks_per_sm<D, ROWS>()) kv_attention_kernel(const __grid_constant__ KvAttnArgs a) {
    constexpr int NT = ROWS / 8;            // row tiles that a chunk's operands serve
    constexpr int BUF = D == 256 ? 1 : 2;   // chunks held: the next one is loaded while this one is worked on
    constexpr int KL = D / 64;              // 16-byte pieces of a key per lane
    constexpr int VB = D >= 128 ? 16 : 8;   // bytes of a value row in one piece
    constexpr int VL = D >= 128 ? D / 128 : 1;
    constexpr int MT = D / 16;              // value tiles of 16
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long scan[kWarps];
    __shared__ long long found[3];
    __shared__ float wm[kWarps][ROWS], wl[kWarps][ROWS];
    __shared__ Limits<ROWS> limits;
    __shared__ Ending<ROWS> ending;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const int group = a.q_heads / a.heads;
    const int RH = a.R * a.heads;
    const int page_shift = 31 - __clz(a.page);

    grid_dependency_wait();
    grid_dependents_launch();

    // ---- rows of the new tokens that no sequence has, ahead of the first offset and past the last: zero
    if (a.cu != nullptr) {
        int first, last, unused;
        seq_tokens(a.cu, 0, a.tokens, first, unused);
        seq_tokens(a.cu, a.seqs - 1, a.tokens, unused, last);
        const int spare = first + a.tokens - last;
        if (spare > 0) {
            const int pieces = a.d / 8;         // of 16 bytes, in a head
            const long long each = static_cast<long long>(spare) * a.q_heads * pieces;
            for (int r = 0; r < a.R; ++r)
                for (long long i = blockIdx.x * static_cast<long long>(kWarps * 32) + threadIdx.x; i < each; i += static_cast<long long>(gridDim.x) * (kWarps * 32)) {
                    const long long row = i / pieces, x = row / a.q_heads;
                    const int token = static_cast<int>(x < first ? x : x - first + last);
                    uint16_t* o = out_at(a, r, token, static_cast<int>(row - x * a.q_heads));
                    *reinterpret_cast<uint4*>(o + (i - row * pieces) * 8) = make_uint4(0, 0, 0, 0);
                }
        }
    }

    // ---- this block's run of units: each thread adds a contiguous range of
    // sequences; the scan of the threads' sums gives the total and the start
    const int per = (a.seqs + kWarps * 32 - 1) / (kWarps * 32);
    const int s_lo = min(a.seqs, static_cast<int>(threadIdx.x) * per), s_hi = min(a.seqs, s_lo + per);
    long long mine = 0;
    for (int s = s_lo; s < s_hi; ++s) mine += seq_units<ROWS>(a, s);
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
        if (threadIdx.x == 0) rec->rows = 0;
        return;
    }
    if (before <= u0 && u0 < before + mine * RH) {
        long long at = before;
        for (int s = s_lo; s < s_hi; ++s) {
            const long long n = seq_units<ROWS>(a, s) * RH;
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
    SeqWork sw = seq_work<ROWS>(a, s);
    bool left_open = false;

    const int d = EXACT ? D : a.d;
    const int head_bytes = d << page_shift;                            // one (page, head)
    const int page_bytes = a.heads * head_bytes;                       // at most 2^25
    const uint32_t pages = static_cast<uint32_t>(a.pages);

    // Items follow each other: row tiles, heads, ranks, sequences.  `unit` is
    // the first of the item's units; those ahead of its first tile go with that
    // tile.
    int rt, r, h;
    long long unit;
    {
        const int span = sw.tiles + kItemCost;
        const long long item = (u0 - base) / span;
        const int rh = static_cast<int>(item / sw.row_tiles);
        rt = static_cast<int>(item - static_cast<long long>(rh) * sw.row_tiles);
        r = rh / a.heads;
        h = rh - r * a.heads;
        unit = base + item * span;
    }
    for (;;) {
        const long long start = unit + kItemCost;       // unit of its first tile
        const int t0 = static_cast<int>(max(0LL, u0 - start));
        if (start + t0 >= u1) break;
        const int t1 = static_cast<int>(min(static_cast<long long>(sw.tiles), u1 - start));

        // ---- rows and their limits
        const int row0 = rt * ROWS, rows = static_cast<int>(min(static_cast<long long>(ROWS), static_cast<long long>(sw.n) * group - row0));
        const int i0 = row0 / group, i1 = (row0 + rows - 1) / group;
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

        float acc[NT][MT][4];
        // the columns' references, as what is added to log2 of a weight: kOffset - maximum
        float b0[NT], b1[NT], l0[NT], l1[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[n][i][0] = acc[n][i][1] = acc[n][i][2] = acc[n][i][3] = 0.f;
            b0[n] = b1[n] = kOffset - kNoMax;
            l0[n] = l1[n] = 0.f;
        }

        const volatile Limits<ROWS>& lim = limits;
        // ---- the chunks of this warp: 16 keys j .. j + 15 of every tile
        const int tn = min(t1, tiles);
        // a chunk between these is seen whole by every row
        const int clean_lo = from_max, clean_hi = end_min - kSub;
        const int32_t* table = a.table + static_cast<long long>(s) * a.table_width;
        struct Seen {           // by any row of the tile
            int end, from, sinks;
            __device__ bool operator()(int j) const { return j < end && (j >= from || j < sinks); }
        };
        auto any_row = [&]() { return Seen{lim.end, lim.from, lim.sinks}; };
        auto wanted = [&](int j) { return j < lim.end && (j + kSub > lim.from || j < lim.sinks); };
        // Place of the chunk whose table entry is read next, the tile it belongs to, and where the sinks' tiles end.
        int ahead = t0, place = (t0 < near ? t0 : far + t0 - near) * kTile + warp * kSub;
        const int skip_at = near * kTile + warp * kSub, skip = (far - near) * kTile;
        auto advance = [&]() {
            ++ahead;
            place += kTile;
            if (place == skip_at) place += skip;
        };
        // Nothing looks at an entry before the next step, so that the load's latency is not waited for.
        auto entry_here = [&]() { return ahead < tn && place < end_max ? load_index(table + (place >> page_shift)) : -1; };
        // Entries outside the cache are left out, and reported where a row sees a key of the chunk.
        auto checked = [&](int id, int j, bool in) {
            if (static_cast<uint32_t>(id) >= pages) {
                if (lane == 0 && in && wanted(j)) atomicOr(a.status, DEV_ERR_BAD_PAGE);
                id = -1;
            }
            return id;
        };
        // the lane's first piece of 16 keys, for page 0 and slot 0
        const uint8_t* k_lane = a.ck[r] + static_cast<long long>(h) * head_bytes + g * d + c * 16;
        const uint8_t* v_lane = a.cv[r] + static_cast<long long>(h) * head_bytes + 2 * c * d + g * VB;
        const float* sk_head = a.sk[r] + h;
        const float* sv_head = a.sv[r] + h;
        uint32_t kw[BUF][2][KL * 4], vw[BUF][4][VL * VB / 4];
        // A clean chunk is loaded without a look at any key's place; else the lanes whose key no row sees (or whose piece
        // lies past the head) hold zeros.
        auto load_k = [&](int j, int id, int buf) {
            const uint8_t* kp = k_lane + static_cast<long long>(id) * page_bytes + (j & (a.page - 1)) * d;
            auto go = [&](auto all) {
                constexpr bool ALL = decltype(all)::value;
                Seen seen{};
                if constexpr (!ALL) seen = any_row();
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int i = 0; i < KL; ++i) {
                        const uint8_t* p = kp + 8 * x * d + i * 64;
                        const uint4 v = ALL && EXACT ? load16(p) : load16_if(p, (ALL || seen(j + g + 8 * x)) && (EXACT || (i * 4 + c) * 16 < d));
                        kw[buf][x][4 * i] = v.x; kw[buf][x][4 * i + 1] = v.y; kw[buf][x][4 * i + 2] = v.z; kw[buf][x][4 * i + 3] = v.w;
                    }
            };
            if (j >= clean_lo && j <= clean_hi) go(std::true_type{});
            else go(std::false_type{});
        };
        auto load_v = [&](int j, int id, int buf) {
            const uint8_t* vp = v_lane + static_cast<long long>(id) * page_bytes + (j & (a.page - 1)) * d;
            auto go = [&](auto all) {
                constexpr bool ALL = decltype(all)::value;
                Seen seen{};
                if constexpr (!ALL) seen = any_row();
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int tok = (y & 1) + 8 * (y >> 1);     // after key 2 c
#pragma unroll
                    for (int i = 0; i < VL; ++i) {
                        const uint8_t* p = vp + tok * d + i * 128;
                        const bool have = (ALL || seen(j + 2 * c + tok)) && (EXACT || i * 128 + g * VB < d);
                        if constexpr (VB == 16) {
                            const uint4 v = ALL && EXACT ? load16(p) : load16_if(p, have);
                            vw[buf][y][4 * i] = v.x; vw[buf][y][4 * i + 1] = v.y; vw[buf][y][4 * i + 2] = v.z; vw[buf][y][4 * i + 3] = v.w;
                        } else {
                            const uint2 v = ALL && EXACT ? load8(p) : load8_if(p, have);
                            vw[buf][y][0] = v.x; vw[buf][y][1] = v.y;
                        }
                    }
                }
            };
            if (j >= clean_lo && j <= clean_hi) go(std::true_type{});
            else go(std::false_type{});
        };

        // First the loads that wait for nothing, then those behind them: table
        // entries and Q, then the first keys and values, while Q is converted.
        int j = place;                          // this chunk's place
        const int entry0 = entry_here();
        advance();
        int j1 = place, entry = entry_here();   // the next one's
        // ---- Q as the B operand: lane (g, c) holds row g, the 16 values of
        // each of its pieces (i * 4 + c), as the keys' lanes hold theirs
        uint32_t qf[NT][KL * 8];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int rho = row0 + 8 * n + g;
            const bool valid = 8 * n + g < rows;
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
                qf[n][8 * i + 0] = v0.x; qf[n][8 * i + 1] = v0.y; qf[n][8 * i + 2] = v0.z; qf[n][8 * i + 3] = v0.w;
                qf[n][8 * i + 4] = v1.x; qf[n][8 * i + 5] = v1.y; qf[n][8 * i + 6] = v1.z; qf[n][8 * i + 7] = v1.w;
            }
        }
        // What only chunks at the ends of a row's keys need is kept out of the registers.
        if (threadIdx.x < ROWS) {
            const int i = (rt * ROWS + min(static_cast<int>(threadIdx.x), rows - 1)) / group;
            limits.row_end[threadIdx.x] = end_of(i);
            limits.row_from[threadIdx.x] = from_of(i);
            if (threadIdx.x == 0) {
                limits.end = end_max;
                limits.from = from_min;
                limits.sinks = sinks;
            }
        }
        __syncthreads();

        int id = checked(entry0, j, t0 < tn);   // this chunk's page
        float sk = 0.f, sv = 0.f;
        if (id >= 0) {
            sk = load_float(sk_head + static_cast<long long>(id) * a.heads);
            sv = load_float(sv_head + static_cast<long long>(id) * a.heads);
            load_k(j, id, 0);
            load_v(j, id, 0);
        }
        float qs0[NT], qs1[NT];     // row factors of the columns 2c, 2c + 1 of S^T
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float qscale = a.scale * 1.4426950408889634f;
            if constexpr (BF16) {
                uint32_t top = 0;   // the largest magnitude's bits
#pragma unroll
                for (int i = 0; i < KL * 8; ++i) {
                    const uint32_t x = qf[n][i] & 0x7fff7fffu;
                    top = max(top, max(x & 0xffffu, x >> 16));
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int ex = static_cast<int>(top >> 7);                     // biased exponent; 255: not finite
                const int up = (ex == 255 || ex == 0) ? 0 : min(126, 127 + 14 - ex);   // largest value to 2^14
                const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
#pragma unroll
                for (int i = 0; i < KL * 8; ++i)
                    qf[n][i] = pack_half2(__uint_as_float(qf[n][i] << 16) * f, __uint_as_float(qf[n][i] & 0xffff0000u) * f);
                qscale *= __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
            }
            qs0[n] = __shfl_sync(0xffffffffu, qscale, 8 * c);
            qs1[n] = __shfl_sync(0xffffffffu, qscale, 8 * c + 4);
        }

        float ev_top = -INFINITY;   // log2 of the largest scale of V so far
        for (int tb = t0; tb < tn; tb += BUF) {
#pragma unroll
            for (int cur = 0; cur < BUF; ++cur) {
                const int t = tb + cur;
                if (t >= tn) break;
                const int nxt = BUF == 2 ? 1 - cur : 0;
                const int here = id, j0 = j;
                const float sk0 = sk, sv0 = sv;
                id = checked(entry, j1, t + 1 < tn);
                j = j1;
                advance();
                j1 = place;
                entry = entry_here();
                if (id >= 0) {
                    sk = load_float(sk_head + static_cast<long long>(id) * a.heads);
                    sv = load_float(sv_head + static_cast<long long>(id) * a.heads);
                    if (BUF == 2) {
                        load_k(j, id, nxt);
                        load_v(j, id, nxt);
                    }
                }
                if (here < 0) {
                    if (BUF == 1 && id >= 0) {
                        load_k(j, id, nxt);
                        load_v(j, id, nxt);
                    }
                    continue;
                }
                // S^T = K Q^T; one row tile in two accumulators: products into one wait for each other
                float sc[NT][4], sb[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) sc[n][x] = sb[n][x] = 0.f;
#pragma unroll
                for (int w = 0; w < KL * 4; ++w) {
                    const uint32_t af[4] = {lo2(kw[cur][0][w]), lo2(kw[cur][1][w]), hi2(kw[cur][0][w]), hi2(kw[cur][1][w])};
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma16816(NT == 1 && (w & 1) ? sb[n] : sc[n], af, qf[n][2 * w], qf[n][2 * w + 1]);
                }
                if (BUF == 1 && id >= 0) load_k(j, id, nxt);
                const float ev = log2_fast(fmaxf(sv0, 1.2e-38f));
                const float inv = exp2_fast(-ev);
                ev_top = fmaxf(ev_top, ev);
                const bool far = ev < ev_top - kFarScale;       // the same in all lanes
                const bool clean = j0 >= clean_lo && j0 <= clean_hi;
                uint32_t see[NT];                       // bit x: the row of sc[x] sees its key
                uint32_t p0[NT], p1[NT], e0[NT], e1[NT];    // weights, and what their rounding left
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (NT == 1) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) sc[n][x] += sb[n][x];
                    }
                    const float f0 = qs0[n] * sk0, f1 = qs1[n] * sk0;
                    see[n] = 0xf;
                    if (!clean) {
                        see[n] = 0;
                        const int row = 8 * n + 2 * c;
                        const Seen by[2] = {{lim.row_end[row], lim.row_from[row], lim.sinks}, {lim.row_end[row + 1], lim.row_from[row + 1], lim.sinks}};
#pragma unroll
                        for (int x = 0; x < 4; ++x) see[n] |= static_cast<uint32_t>(by[x & 1](j0 + g + 8 * (x >> 1))) << x;
                    }
                    float z[4];             // log2 of the weights
                    auto logs = [&](float a0, float a1) {
                        z[0] = fmaf(sc[n][0], f0, a0);
                        z[1] = fmaf(sc[n][1], f1, a1);
                        z[2] = fmaf(sc[n][2], f0, a0);
                        z[3] = fmaf(sc[n][3], f1, a1);
                        if (!clean) {
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                if (!(see[n] >> x & 1)) z[x] = -INFINITY;
                        }
                    };
                    logs(ev + b0[n], ev + b1[n]);
                    // a reference moves only when a key is well above it
                    if (__any_sync(0xffffffffu, fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])) > kOffset + kSlack)) {
                        logs(ev, ev);
                        float n0 = fmaxf(kOffset - b0[n], fmaxf(z[0], z[2])), n1 = fmaxf(kOffset - b1[n], fmaxf(z[1], z[3]));
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) {
                            n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, o));
                            n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, o));
                        }
                        n0 = kOffset - n0;
                        n1 = kOffset - n1;
                        const float h0 = exp2_fast(0.5f * (n0 - b0[n])), h1 = exp2_fast(0.5f * (n1 - b1[n]));
                        const float c0 = h0 * h0, c1 = h1 * h1;
                        b0[n] = n0;
                        b1[n] = n1;
                        l0[n] = l0[n] * h0 * h0;
                        l1[n] = l1[n] * h1 * h1;
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            acc[n][i][0] *= c0;
                            acc[n][i][1] *= c1;
                            acc[n][i][2] *= c0;
                            acc[n][i][3] *= c1;
                        }
                        logs(ev + b0[n], ev + b1[n]);
                    }
                    if (far) {
                        l0[n] += exp2_fast(z[0] - ev) + exp2_fast(z[2] - ev);
                        l1[n] += exp2_fast(z[1] - ev) + exp2_fast(z[3] - ev);
                    }
#pragma unroll
                    for (int x = 0; x < 4; ++x) z[x] = exp2_fast(z[x]);
                    if (!far) {
                        l0[n] = fmaf(z[0] + z[2], inv, l0[n]);
                        l1[n] = fmaf(z[1] + z[3], inv, l1[n]);
                    }
                    const uint32_t plo = pack_half2(z[0], z[1]), phi = pack_half2(z[2], z[3]);
                    p0[n] = transposed(plo);
                    p1[n] = transposed(phi);
                    const float2 rl = __half22float2(*reinterpret_cast<const __half2*>(&plo));
                    const float2 rh2 = __half22float2(*reinterpret_cast<const __half2*>(&phi));
                    e0[n] = transposed(pack_half2(z[0] - rl.x, z[1] - rl.y));
                    e1[n] = transposed(pack_half2(z[2] - rh2.x, z[3] - rh2.y));
                }
                // O^T += V^T P^T
                if (!clean) {
                    // a NaN of a key that only some rows see would reach the others as 0 x NaN: where the
                    // chunk has one, it is taken out of the product and put into the rows that see it
                    uint32_t nan = 0;
#pragma unroll
                    for (int y = 0; y < 4; ++y)
#pragma unroll
                        for (int i = 0; i < VL * VB / 4; ++i) nan |= ((vw[cur][y][i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                    if (__any_sync(0xffffffffu, nan != 0)) {
                        uint32_t i0b[NT], i1b[NT];
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            i0b[n] = transposed(pack_half2(see[n] & 1 ? 1.f : 0.f, see[n] & 2 ? 1.f : 0.f));
                            i1b[n] = transposed(pack_half2(see[n] & 4 ? 1.f : 0.f, see[n] & 8 ? 1.f : 0.f));
                        }
#pragma unroll
                        for (int i = 0; i < MT / 2; ++i) {
                            uint32_t x[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const uint32_t bad = ((((vw[cur][y][i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xffu;
                                x[y] = bad & 0x38383838u;       // e4m3 1.0 where NaN
                                vw[cur][y][i] &= ~bad;
                            }
                            const uint32_t a01 = __byte_perm(x[0], x[1], 0x5140), a23 = __byte_perm(x[2], x[3], 0x5140);
                            const uint32_t b01 = __byte_perm(x[0], x[1], 0x7362), b23 = __byte_perm(x[2], x[3], 0x7362);
                            const uint32_t fa[4] = {lo2(a01), hi2(a01), lo2(a23), hi2(a23)}, fb[4] = {lo2(b01), hi2(b01), lo2(b23), hi2(b23)};
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                float ta[4] = {0.f, 0.f, 0.f, 0.f}, tb2[4] = {0.f, 0.f, 0.f, 0.f};
                                mma16816(ta, fa, i0b[n], i1b[n]);
                                mma16816(tb2, fb, i0b[n], i1b[n]);
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    if (ta[q] > 0.f) acc[n][2 * i][q] = __uint_as_float(0x7fc00000u);
                                    if (tb2[q] > 0.f) acc[n][2 * i + 1][q] = __uint_as_float(0x7fc00000u);
                                }
                            }
                        }
                    }
                }
                // word i of the four keys: bytes 0, 1 make value tile 2i, bytes 2, 3 tile 2i + 1
#pragma unroll
                for (int i = 0; i < MT / 2; ++i) {
                    const uint32_t a01 = __byte_perm(vw[cur][0][i], vw[cur][1][i], 0x5140), a23 = __byte_perm(vw[cur][2][i], vw[cur][3][i], 0x5140);
                    const uint32_t b01 = __byte_perm(vw[cur][0][i], vw[cur][1][i], 0x7362), b23 = __byte_perm(vw[cur][2][i], vw[cur][3][i], 0x7362);
                    const uint32_t fa[4] = {lo2(a01), hi2(a01), lo2(a23), hi2(a23)}, fb[4] = {lo2(b01), hi2(b01), lo2(b23), hi2(b23)};
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma16816(acc[n][2 * i], fa, p0[n], p1[n]);
                        mma16816(acc[n][2 * i + 1], fb, p0[n], p1[n]);
                        mma16816(acc[n][2 * i], fa, e0[n], e1[n]);
                        mma16816(acc[n][2 * i + 1], fb, e0[n], e1[n]);
                    }
                }
                if (BUF == 1 && id >= 0) load_v(j, id, nxt);
            }
        }

        // ---- join the warps: maxima and sums, then the value sums in the
        // accumulators' order (value d = g VB + 2 i + b at 16 i + 2 g + b)
        constexpr int MS = merge_stride<D>();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                l0[n] += __shfl_xor_sync(0xffffffffu, l0[n], o);
                l1[n] += __shfl_xor_sync(0xffffffffu, l1[n], o);
            }
            if (g == 0) {
                wm[warp][8 * n + 2 * c] = kOffset - b0[n];
                wm[warp][8 * n + 2 * c + 1] = kOffset - b1[n];
                wl[warp][8 * n + 2 * c] = l0[n];
                wl[warp][8 * n + 2 * c + 1] = l1[n];
            }
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int x0 = 8 * n + 2 * c, x1 = x0 + 1;
            float M0 = wm[0][x0], M1 = wm[0][x1];
#pragma unroll
            for (int i = 1; i < kWarps; ++i) {
                M0 = fmaxf(M0, wm[i][x0]);
                M1 = fmaxf(M1, wm[i][x1]);
            }
            const float k0 = exp2_fast(kOffset - b0[n] - M0), k1 = exp2_fast(kOffset - b1[n] - M1);
            float* mine_s = reinterpret_cast<float*>(smem) + warp * ROWS * MS;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                *reinterpret_cast<float2*>(mine_s + x0 * MS + 16 * i + 2 * g) = make_float2(acc[n][i][0] * k0, acc[n][i][2] * k0);
                *reinterpret_cast<float2*>(mine_s + x1 * MS + 16 * i + 2 * g) = make_float2(acc[n][i][1] * k1, acc[n][i][3] * k1);
            }
        }
        if (threadIdx.x < ROWS) {
            const int row = threadIdx.x, rho = row0 + min(row, rows - 1);
            float M = wm[0][row], L = 0.f;
#pragma unroll
            for (int i = 1; i < kWarps; ++i) M = fmaxf(M, wm[i][row]);
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const float h = exp2_fast(0.5f * (wm[i][row] - M));
                L += wl[i][row] * h * h;
            }
            ending.max[row] = M;
            ending.sum[row] = L;
            ending.inv[row] = L == 0.f ? 0.f : 1.f / L;
            ending.out[row] = out_at(a, r, sw.begin + rho / group, h * group + rho % group);
        }
        __syncthreads();
        const bool begins = t0 == 0, ends = t1 == sw.tiles;
        float* part = parts + (2LL * blockIdx.x + (begins ? 1 : 0)) * part_floats<D, ROWS>();
        static_assert(kWarps * 32 % (D / 2) == 0 || D / 2 % (kWarps * 32) == 0);
#pragma unroll
        for (int x0 = 0; x0 < ROWS * D / 2; x0 += kWarps * 32) {
            const int x = x0 + threadIdx.x, row = x / (D / 2), p = x % (D / 2) * 2;
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const float2 v = *reinterpret_cast<const float2*>(reinterpret_cast<const float*>(smem) + (i * ROWS + row) * MS + p);
                sum.x += v.x;
                sum.y += v.y;
            }
            if (begins && ends) {
                const int e = value_of<D>(p);
                const float inv = ending.inv[row];
                if (row < rows && e < a.d)
                    *reinterpret_cast<uint32_t*>(ending.out[row] + e) = pack2<BF16>(__float_as_uint(sum.x * inv), __float_as_uint(sum.y * inv));
            } else {
                *reinterpret_cast<float2*>(part + row * D + p) = sum;
            }
        }
        if (!(begins && ends) && threadIdx.x < ROWS) {
            part[ROWS * D + threadIdx.x] = ending.max[threadIdx.x];
            part[ROWS * D + ROWS + threadIdx.x] = ending.sum[threadIdx.x];
        }
        if (begins && !ends) {
            left_open = true;
            if (threadIdx.x == 0) *rec = {rows, static_cast<int>((start + sw.tiles - 1) / quota), r * a.heads + h, sw.begin, row0, {0, 0, 0}};
        }
        if (!ends) break;       // the run ends inside the item
        unit = start + sw.tiles;
        if (++rt == sw.row_tiles) {
            rt = 0;
            if (++h == a.heads) {
                h = 0;
                if (++r == a.R) {
                    r = 0;
                    if (unit >= u1) break;
                    do sw = seq_work<ROWS>(a, ++s);
                    while (sw.row_tiles == 0);      // there is one: unit < total
                }
            }
        }
        __syncthreads();    // the merge area, wm and the limits are read before the next item
    }
    if (threadIdx.x == 0 && !left_open) rec->rows = 0;
}

// Where the outputs of a row of a merged item lie.
__device__ __forceinline__ uint16_t* out_at(const KvAttnArgs& a, const Record& rec, int row) {
    const int group = a.q_heads / a.heads, r = rec.head / a.heads, h = rec.head - r * a.heads, rho = rec.row + row;
    return out_at(a, r, rec.token + rho / group, h * group + rho % group);
}

// Merging the parts of the item that block b began and others went on with.
// Its time is latency, the record's and then the parts': the first values are
// asked for together with the maxima, before their weights are known.
constexpr int kAtOnce = 8;          // parts whose values a thread has in flight

// Block (x, row): the records from x kMergeSpan on, few of which are of an item
// (a block for each would be four times the blocks, most of them for nothing:
// 94.5 instead of 92.6 us for two sequences of 131071).  Group y of the threads
// adds the parts y, y + kMergeGroups, ... in order, then the groups are added
// in order.
constexpr int kMergeGroups = 4;
constexpr int kMergeSpan = 4;
constexpr int kMaxGrid = 2048;      // blocks of the attention kernel

template <bool BF16, int D, int ROWS>
__global__ void __launch_bounds__(kMergeGroups * D / 2) kv_attention_merge(const __grid_constant__ KvAttnArgs a) {
    constexpr int T = kMergeGroups * D / 2;
    __shared__ float weight[kMaxGrid];
    __shared__ float red[2][T / 32];
    __shared__ float2 sums[kMergeGroups][D / 2];
    grid_dependency_wait();
    const Record* recs = reinterpret_cast<const Record*>(a.scratch);
    const int row = blockIdx.y, y = threadIdx.x / (D / 2), x = threadIdx.x % (D / 2), p = 2 * x;
    const int lane = threadIdx.x & 31, at = blockIdx.x * kMergeSpan + lane;
    const float* parts = reinterpret_cast<const float*>(recs + a.grid);
    uint32_t open = __ballot_sync(0xffffffffu, lane < kMergeSpan && at < a.grid && recs[at].rows > row);
    for (; open != 0; open &= open - 1) {
        const int first = blockIdx.x * kMergeSpan + __ffs(open) - 1;
        const Record rec = recs[first];
        const int count = rec.last_block - first + 1;
        auto part = [&](int i) { return parts + (2LL * (first + i) + (i == 0 ? 1 : 0)) * part_floats<D, ROWS>(); };
        float2 v[kAtOnce];
        auto fetch = [&](int i0) {
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int i = i0 + k * kMergeGroups;
                v[k] = i < count ? *reinterpret_cast<const float2*>(part(i) + row * D + p) : make_float2(0.f, 0.f);
            }
        };
        fetch(y);
        float M = kNoMax, l = 0.f;      // l: of part threadIdx.x
        for (int i = threadIdx.x; i < count; i += T) {
            M = fmaxf(M, weight[i] = part(i)[ROWS * D + row]);
            if (i == threadIdx.x) l = part(i)[ROWS * D + ROWS + row];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        if ((threadIdx.x & 31) == 0) red[0][threadIdx.x >> 5] = M;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < T / 32; ++i) M = fmaxf(M, red[0][i]);
        float L = 0.f;
        for (int i = threadIdx.x; i < count; i += T) {
            const float h = exp2_fast(0.5f * (weight[i] - M));
            weight[i] = h * h;
            L = fmaf((i == threadIdx.x ? l : part(i)[ROWS * D + ROWS + row]) * h, h, L);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        if ((threadIdx.x & 31) == 0) red[1][threadIdx.x >> 5] = L;
        __syncthreads();
        float2 sum = make_float2(0.f, 0.f);
        for (int i0 = y; i0 < count; i0 += kAtOnce * kMergeGroups) {
            if (i0 != y) fetch(i0);
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int i = i0 + k * kMergeGroups;
                if (i < count) {
                    sum.x = fmaf(v[k].x, weight[i], sum.x);
                    sum.y = fmaf(v[k].y, weight[i], sum.y);
                }
            }
        }
        sums[y][x] = sum;
        __syncthreads();
        if (y == 0) {
#pragma unroll
            for (int i = 1; i < kMergeGroups; ++i) {
                sum.x += sums[i][x].x;
                sum.y += sums[i][x].y;
            }
            L = 0.f;
#pragma unroll
            for (int i = 0; i < T / 32; ++i) L += red[1][i];
            const int e = value_of<D>(p);
            const float inv = L == 0.f ? 0.f : 1.f / L;
            if (e < a.d) *reinterpret_cast<uint32_t*>(out_at(a, rec, row) + e) = pack2<BF16>(__float_as_uint(sum.x * inv), __float_as_uint(sum.y * inv));
        }
        __syncthreads();    // the sums are read before the next item's
    }
}

// The same with a warp a row and the parts one after another: block b, warp =
// row; an eighth of the blocks and no barrier.  It is taken where the blocks
// share few parts an item, fewer than kFewParts if every sequence has a row
// tile: the whole call takes 75.7 instead of 82.7 us for 48 sequences of up to
// 8192 keys on 8 ranks (1.2 blocks an item), but 95.6 instead of 93.5 for two
// of 131071 (28 blocks an item), 51 instead of 22 for one on one rank.  The rule
// knows the sizes, not the lengths: of 128 sequences on one rank one of 131072
// keys beside 127 of 16 takes 45 us, a warp a row adding its hundreds of parts,
// where that one alone takes 21.
constexpr int kFewParts = 4;

template <bool BF16, int D, int ROWS>
__global__ void __launch_bounds__(ROWS * 32) kv_attention_merge_rows(const __grid_constant__ KvAttnArgs a) {
    constexpr int P = D / 64;       // pairs of values of a lane: 2 lane + 64 i
    constexpr int AT_ONCE = 4;
    grid_dependency_wait();
    const Record* recs = reinterpret_cast<const Record*>(a.scratch);
    const Record rec = recs[blockIdx.x];
    const int row = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (row >= rec.rows) return;
    const float* parts = reinterpret_cast<const float*>(recs + gridDim.x);
    const int first = blockIdx.x, count = rec.last_block - first + 1;
    auto part = [&](int i) { return parts + (2LL * (first + i) + (i == 0 ? 1 : 0)) * part_floats<D, ROWS>(); };
    float2 v[AT_ONCE][P];
    auto fetch = [&](int i0) {
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i)
#pragma unroll
            for (int k = 0; k < P; ++k)
                v[i][k] = i0 + i < count ? *reinterpret_cast<const float2*>(part(i0 + i) + row * D + 2 * lane + 64 * k) : make_float2(0.f, 0.f);
    };
    fetch(0);
    float m = kNoMax, l = 0.f;      // of part `lane`
    if (lane < count) {
        m = part(lane)[ROWS * D + row];
        l = part(lane)[ROWS * D + ROWS + row];
    }
    float M = m;
    for (int i = lane + 32; i < count; i += 32) M = fmaxf(M, part(i)[ROWS * D + row]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f, f = 0.f;
    float2 sum[P];
#pragma unroll
    for (int k = 0; k < P; ++k) sum[k] = make_float2(0.f, 0.f);
    for (int i0 = 0; i0 < count; i0 += AT_ONCE) {
        if (i0 != 0) fetch(i0);
        if (i0 % 32 == 0) {
            if (i0 != 0 && i0 + lane < count) {
                m = part(i0 + lane)[ROWS * D + row];
                l = part(i0 + lane)[ROWS * D + ROWS + row];
            }
            const float h = i0 + lane < count ? exp2_fast(0.5f * (m - M)) : 0.f;
            f = h * h;
            L = fmaf(l * h, h, L);
        }
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            const float w = __shfl_sync(0xffffffffu, f, (i0 + i) % 32);
            if (i0 + i < count) {
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    sum[k].x = fmaf(v[i][k].x, w, sum[k].x);
                    sum[k].y = fmaf(v[i][k].y, w, sum[k].y);
                }
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    const float inv = L == 0.f ? 0.f : 1.f / L;
    uint16_t* o = out_at(a, rec, row);
#pragma unroll
    for (int k = 0; k < P; ++k) {
        const int e = value_of<D>(2 * lane + 64 * k);
        if (e < a.d) *reinterpret_cast<uint32_t*>(o + e) = pack2<BF16>(__float_as_uint(sum[k].x * inv), __float_as_uint(sum[k].y * inv));
    }
}

template <bool BF16, int D, bool EXACT, int ROWS>
struct Launcher {
    // Blocks that one SM holds; sets the kernel up on the current device.
    static cudaError_t resident(int* out) {
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
        auto kern = kv_attention_kernel<BF16, D, EXACT, ROWS>;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, attn_smem<D, ROWS>());
        if (e != cudaSuccess) return e;
        int n = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kWarps * 32, attn_smem<D, ROWS>());
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorInvalidConfiguration;
        if (dev >= 0 && dev < 64) cached[dev] = n;
        *out = n;
        return cudaSuccess;
    }
    static cudaError_t launch(const KvAttnArgs& args, int grid, cudaStream_t stream) {
        KvAttnArgs a = args;
        a.grid = grid;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
        cfg.blockDim = dim3(kWarps * 32, 1, 1);
        cfg.dynamicSmemBytes = attn_smem<D, ROWS>();
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = pdl_launch() ? 1 : 0;
        cudaError_t e = cudaLaunchKernelEx(&cfg, kv_attention_kernel<BF16, D, EXACT, ROWS>, a);
        if (e != cudaSuccess) return e;
        // no item spans blocks where none has more than one tile
        if (a.table_width * a.page <= kTile) return cudaSuccess;
        cfg.dynamicSmemBytes = 0;
        if (grid < static_cast<long long>(kFewParts) * a.seqs * a.R * a.heads) {
            cfg.blockDim = dim3(ROWS * 32, 1, 1);
            return cudaLaunchKernelEx(&cfg, kv_attention_merge_rows<BF16, D, ROWS>, a);
        }
        cfg.gridDim = dim3(static_cast<unsigned>((grid + kMergeSpan - 1) / kMergeSpan), ROWS, 1);
        cfg.blockDim = dim3(kMergeGroups * D / 2, 1, 1);
        return cudaLaunchKernelEx(&cfg, kv_attention_merge<BF16, D, ROWS>, a);
    }
};

// Query rows of a tile.  16 rows share one conversion of the codes, at two
// blocks an SM instead of three for heads of 128: worth it where the keys, not
// the items' beginnings and ends, take the time, and tiles of 8 would read them
// for a quarter of the items again.  How many tokens each sequence has is known
// on the device only: as many as the others where they divide evenly, else so
// much on average that a quarter has more than 8 rows (and the rest half empty
// tiles: it takes more keys to pay).  8 ranks of one key head of 128, 8 against
// 16 rows: 48 sequences of 4096 keys with 16 query heads 138 and 94 us, with 8
// heads and 1 to 8 tokens 330 and 243, with 6 heads and 1 or 2 tokens 111 and
// 94, with 8 heads and one token 75 and 93; 32 sequences of up to 512 keys (2048
// tiles) with 16 heads 18.0 and 18.1, of up to 1024 23.6 and 22.1; 64 of up to
// 1024 keys (8192 tiles) with 8 heads and 1 or 2 tokens 33.3 and 36.4, of up to
// 2048 51.3 and 51.5.  Heads of 256 have no registers for more than 8 rows (with
// Q in shared memory 300 and 300), and 32 rows leave no second buffer (heads of
// 128: 224 and 272 with 1 to 8 tokens).
constexpr long long kManyTiles = 2048, kManyRaggedTiles = 12288;

long long table_tiles(const KvAttnArgs& a) { return std::max<long long>(1, (a.table_width * a.page + kTile - 1) / kTile); }

int tile_rows(const KvAttnArgs& a) {
    const int group = a.q_heads / a.heads;
    const long long tokens = a.tokens, seqs = a.seqs, tiles = table_tiles(a);
    const bool even = tokens % seqs == 0;
    const bool many_rows = even ? tokens / seqs * group > 8 : 2 * tokens * group >= 15 * seqs && 4 * tokens >= 5 * seqs;
    const long long many = even ? kManyTiles : kManyRaggedTiles;
    return a.d <= 128 && many_rows && (tiles >= many || tiles * seqs * a.R * a.heads >= many) ? 16 : 8;
}

// Head sizes 64, 128 and 256 have instances of their own; the others take the
// next of them with the rest of the head zero.
int padded_d(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

template <bool BF16, typename F>
cudaError_t with_rows(int d, int rows, F f) {
    const bool exact = padded_d(d) == d;
#define COC_ATTN(D, ROWS) return exact ? f(Launcher<BF16, D, true, ROWS>()) : f(Launcher<BF16, D, false, ROWS>())
    if (padded_d(d) == 256) COC_ATTN(256, 8);
    if (rows == 16) {
        if (padded_d(d) == 64) COC_ATTN(64, 16);
        COC_ATTN(128, 16);
    }
    if (padded_d(d) == 64) COC_ATTN(64, 8);
    COC_ATTN(128, 8);
#undef COC_ATTN
}

template <typename F>
cudaError_t with_instance(const KvAttnArgs& a, bool bf16, F f) {
    return bf16 ? with_rows<true>(a.d, tile_rows(a), f) : with_rows<false>(a.d, tile_rows(a), f);
}

}  // namespace

cudaError_t kv_attention_plan(const KvAttnArgs& a, bool bf16, int sm_count, int* grid, size_t* scratch) {
    int n = 0;
    const cudaError_t e = with_instance(a, bf16, [&](auto l) { return l.resident(&n); });
    if (e != cudaSuccess) return e;
    // never more blocks than there can be units
    const int group = a.q_heads / a.heads, rows = tile_rows(a);
    const long long items = (static_cast<long long>(a.tokens) * group / rows + a.seqs) * a.R * a.heads;
    const long long tiles = table_tiles(a);
    long long resident = static_cast<long long>(n) * sm_count;
    resident = std::min<long long>(resident, kMaxGrid);
    *grid = static_cast<int>(tiles >= resident ? resident : std::min(resident, items * (tiles + kItemCost)));
    *scratch = static_cast<size_t>(*grid) * (sizeof(Record) + 2 * rows * (padded_d(a.d) + 2) * sizeof(float));
    return cudaSuccess;
}

cudaError_t launch_kv_attention(const KvAttnArgs& a, bool bf16, int grid, cudaStream_t stream) {
    return with_instance(a, bf16, [&](auto l) { return l.launch(a, grid, stream); });
}

}  // namespace coc
