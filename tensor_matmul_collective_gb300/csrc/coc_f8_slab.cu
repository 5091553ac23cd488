// Products of 8-bit activations and weights for few rows: the weights' rows are
// the M side of the tensor core tile, the activations' rows its N side.
//
// Mathematics.  Y(i, j) = sum over the shards' k-blocks b of
// 2^(sx(i, b) + sw(j / 128, b)) sum_{t in b} x(i, t) w(j, t), accumulated in
// fp32 in tensor memory; the gated form takes two weight tiles (gate, up) over
// the same activations, h = silu(g) u, and quantises h per row and 128 columns,
// which is one tile.
//
// What bounds it.  n k bytes of weights, read once: n 8192, k 8 x 3584, 64 rows
// on 8 ranks take 38 us, 6.4 TB/s with the outputs; gated 8 x 3584, k 8192, 64 rows
// 74 to 79 us, 6.0 to 6.4 TB/s; gated 11008, k 4096, one row 16.9 to 17.8 us, 5.2 TB/s; n
// 4096, k 4096, one row 5.5 us, of which the weights' bytes are 2.5.  A tile is 128
// weight rows by NT activation rows, so few rows cost the tensor cores little (a
// product of 32 of k takes 40 cycles with 16 rows, 65 with 128).
//
// Stages.  A k-block is 128 of k, one 128-byte swizzled row; two of them come
// in one box where the ring has room (a block's SM took 600 cycles a k-block
// before, 470 then), and the loads start before the rest is set up.
//
// Split.  Where the tiles do not fill the GPU, the blocks of a cluster take
// contiguous ranges of the k-blocks.  Each finishes a part of the rows: the
// others' sums of them come as bulk copies between shared memories and are added
// in the ranges' order.
//
// Roles: warp 0 copies tiles (TMA), warp 1 issues products and owns tensor
// memory, warps 2 and 3 gather scale words, alternating; then all eight warps
// read the accumulators.
#include <algorithm>
#include <cstdlib>

#include "coc_f8.cuh"
#include "coc_f8_plan.h"

namespace coc {
namespace {

constexpr int kWTile = 128 * 128;       // bytes of 128 weight rows' k-block
constexpr int kSlabThreads = 256;
constexpr int kMaxStages = 8;
// Weights that all blocks together ask L2 for ahead of their turn, where there
// are 40 MiB of them and one row tile: calls that follow each other, n 8192, k 8 x
// 3584, m 64 39.0 to 37.7 us, gated 8 x 3584, k 8192, m 64 78.6 to 74.9, 11008, k 4096,
// m 1 18.2 to 17.1 (16 MiB: 37.8, 77.5, 17.2; 64: 39.5, 75.8, 18.5); with less, n
// 8192, k 4096, m 16 8.2 to 8.9.
constexpr long long kAheadBytes = 32LL << 20;
constexpr int kSfStages = 4;            // scale words: runs of up to 4 k-blocks in flight, in shared and in tensor memory
constexpr int kSfCols = 16;             // columns of a run's scale words in tensor memory

template <int NT, bool GATED>
struct SlabCfg {
    static constexpr int WT = GATED ? 2 : 1;
    static constexpr int BLOCK = WT * kWTile + NT * 128;        // a k-block's tiles
    static constexpr int KPS = !GATED && NT <= 64 ? 2 : 1;      // k-blocks of a stage
    static constexpr int STAGE = KPS * BLOCK;
    static constexpr int SF_BYTES = kSfStages * (WT + 1) * kScaleBlock;
    static constexpr int REST = 1024 + SF_BYTES + 512;          // alignment, scale words, barriers
    static constexpr int SUMS = WT * NT * 128 * 4;
    static constexpr int COLS = WT * NT + kSfStages * kSfCols;
    static constexpr int TMEM = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
    // stages of a ring that has an SM to itself, and of one that shares it with another block's
    static constexpr int ALONE = (224 * 1024 - REST) / STAGE;
    static constexpr int SHARED = (112 * 1024 - REST) / STAGE;
    static constexpr int PARTS = WT * (NT + 7) * 512;           // the cluster's sums of a block's rows, rounded up for each block
    static_assert(ALONE >= 2 && ALONE <= kMaxStages && SUMS + PARTS <= ALONE * STAGE && ALONE * STAGE + REST <= kSlabSmemCap, "shared memory");
    static_assert(SHARED >= 2 && TMEM <= 256 && SUMS <= SHARED * STAGE, "shared memory, tensor memory (blocks that share an SM)");
    // Blocks of a cluster share an SM only where a stage has two k-blocks (launch_t).
    static_assert(KPS == 1 || SUMS + PARTS <= SHARED * STAGE, "shared memory (blocks of a cluster that share an SM)");
    static_assert(KPS == 1 || !GATED, "a gated stage has one k-block: its boxes are 2-D");
};

// 32 lanes x 16 consecutive columns: thread t receives lane (base + t).
__device__ __forceinline__ void tmem_ld_16cols(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
          "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ float4 load_part(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }

template <int NT, bool GATED, bool BF16>
__global__ void __launch_bounds__(kSlabThreads) f8_slab_kernel(const __grid_constant__ F8Args p) {
    using C = SlabCfg<NT, GATED>;
    constexpr int WT = C::WT, KPS = C::KPS;
    const uint32_t S = p.stages;
    constexpr int kXAt = KPS * WT * kWTile;     // a stage: W tiles of its k-blocks, second W tiles (gated), X tiles
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sf = smem + S * C::STAGE;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sf + C::SF_BYTES);
    uint64_t* full = bars;                  // [S] tiles landed
    uint64_t* empty = full + kMaxStages;    // [S] tiles read by the products
    uint64_t* sf_full = empty + kMaxStages; // [kSfStages] a run's scale words written
    uint64_t* sf_empty = sf_full + kSfStages;   // [kSfStages] the run's products are done
    uint64_t* done = sf_empty + kSfStages;  // all products are done
    uint64_t* idle = done + 1;              // the products of all the cluster's blocks are done: their rings are free
    uint64_t* parts = idle + 1;             // the other blocks' sums of this block's rows are here
    uint64_t* never = parts + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(never + 1);
    uint32_t* abort_word = tmem_slot + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Ctl ctl{abort_word, p.status};
    const int splits = p.splits, split = splits > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int tile = static_cast<int>(blockIdx.x) / splits;
    const int mt = tile % p.m_tiles, col_tile = tile / p.m_tiles;
    const int nt = col_tile % p.n_tiles, r = col_tile / p.n_tiles;      // r: the AllGather's rank
    const int row0 = mt * NT;
    const int per_shard = (p.kblocks + 3) / 4, total = p.shards * per_shard;     // runs of k-blocks
    const int b0 = static_cast<int>(static_cast<long long>(total) * split / splits);
    const int b1 = static_cast<int>(static_cast<long long>(total) * (split + 1) / splits);
    const bool ag = p.op == OP_AG;
    // the cluster's blocks finish own_rows of the tile's rows each
    const int rows = min(NT, p.m - row0), own_rows = (rows + splits - 1) / splits;
    const int own = max(0, min(own_rows, rows - split * own_rows));

    // The producer needs the barriers alone, and nobody but warp 1 tensor memory
    // before the end: loads are on their way while the rest is set up.
    if (warp == 0) {
        // a lane a barrier (one lane for all took 700 cycles): they lie one after another
        constexpr int kBars = 2 * kMaxStages + 2 * kSfStages + 4;
        static_assert(kBars <= 32, "a lane a barrier");
        if (lane < kBars) mbar_init(smem_u32(&bars[lane]), &bars[lane] == idle ? splits : 1);
        if (lane == 0) *abort_word = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (splits > 1 && lane == 0) mbar_expect_tx(smem_u32(parts), (splits - 1) * WT * own * 512);
        if (total > 0 && lane < p.shards) {
            prefetch_tmap(&p.tm_w[ag ? r : lane]);
            prefetch_tmap(&p.tm_x[ag ? 0 : lane]);
        }
        __syncwarp();
        named_arrive(1, kSlabThreads);
    } else {
        named_sync(1, kSlabThreads);
    }
    if (splits > 1) cluster_arrive_relaxed();       // the cluster's barriers are there (waited for before they are used)
    if (warp == 4) {
        // Weights on their way into L2 while the kernel before this one ends.  L2 is
        // where all writes meet: should that kernel write them, the loads behind the
        // wait find what it wrote.
        int left = p.ahead;
        for (int i = b0; i < b1 && left > 0; ++i) {
            const F8Run run = f8_run(i, per_shard, p.kblocks);
            const CUtensorMap* wm = &p.tm_w[ag ? r : run.shard];
            for (int j = 0; j < run.count && left > 0; j += KPS, left -= KPS) {
                if (KPS == 2 && p.maps_3d) {
                    tma_prefetch_3d_f8(wm, 0, nt * 128, run.kb + j);
                } else {
#pragma unroll
                    for (int q = 0; q < KPS; ++q) {
                        if (j + q >= run.count) break;
                        tma_prefetch_2d_f8(wm, (run.kb + j + q) * 128, nt * 128);
                        if constexpr (GATED) tma_prefetch_2d_f8(wm, (run.kb + j + q) * 128, p.n + nt * 128);
                    }
                }
            }
        }
    }
    grid_dependency_wait();
    // Tensor memory is asked for behind the wait, so that no kernel before this
    // one finds it taken by a block that waits for that kernel; and later kernels
    // may come only when this block has its own.
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), C::TMEM);
        tmem_relinquish();
        tc_fence_before();
        __syncwarp();
        tc_fence_after();
        grid_dependents_launch();
    }
    bool ok = true;
    if (p.inject_timeout) ok = warp_wait(smem_u32(never), 0, ctl, 0x700u);

    if (warp == 0) {
        uint32_t stage = 0, phase = 0, filled = 0, parity = 0;
        const uint64_t pol_w = make_l2_policy(p.m_tiles > 1 ? 0 : 1), pol_x = make_l2_policy(2);
        const uint32_t ring = smem_u32(smem);
        for (int i = b0; ok && i < b1; ++i) {
            const F8Run run = f8_run(i, per_shard, p.kblocks);
            const CUtensorMap *wm = &p.tm_w[ag ? r : run.shard], *xm = &p.tm_x[ag ? 0 : run.shard];
            for (int j = 0; j < run.count; j += KPS) {
                ok = warp_wait_soon<false>(smem_u32(&empty[stage]), phase ^ 1u, ctl, 0x710u + stage);
                if (!ok) break;
                const uint32_t fb = smem_u32(&full[stage]), dst = ring + stage * C::STAGE;
                const int kb = run.kb + j;
                if (KPS == 2 && p.maps_3d) {
                    // both k-blocks in one box (a last odd one: zeros behind it)
                    expect_tx_f8(fb, C::STAGE);
                    tma_load_3d_f8(dst, wm, 0, nt * 128, kb, fb, pol_w);
                    tma_load_3d_f8(dst + kXAt, xm, 0, row0, kb, fb, pol_x);
                } else {
                    const int count = min(KPS, run.count - j);
                    expect_tx_f8(fb, count * C::BLOCK);
#pragma unroll
                    for (int q = 0; q < KPS; ++q) {
                        if (q == count) break;
                        tma_load_2d_f8(dst + q * kWTile, wm, (kb + q) * 128, nt * 128, fb, pol_w);
                        if constexpr (GATED) tma_load_2d_f8(dst + (KPS + q) * kWTile, wm, (kb + q) * 128, p.n + nt * 128, fb, pol_w);
                        tma_load_2d_f8(dst + kXAt + q * NT * 128, xm, (kb + q) * 128, row0, fb, pol_x);
                    }
                }
                filled |= 1u << stage;
                parity = (parity & ~(1u << stage)) | (phase << stage);
                if (++stage == S) { stage = 0; phase ^= 1u; }
            }
        }
        if (!ok && lane == 0)       // no copy stays in flight into shared memory
            for (uint32_t s = 0; s < S; ++s)
                if (filled & (1u << s)) drain_wait(smem_u32(&full[s]), (parity >> s) & 1u, kDrainNs);
        __syncwarp();
    } else if (warp == 1) {
        const uint32_t tmem = *tmem_slot;
        const uint64_t tiles = make_sdesc(smem_u32(smem), 16, 1024);
        uint32_t stage = 0, phase = 0, onto = 0;
        int run_i = 0;
        for (int i = b0; ok && i < b1; ++i, ++run_i) {
            const F8Run run = f8_run(i, per_shard, p.kblocks);
            const uint32_t ss = run_i % kSfStages, sph = (run_i / kSfStages) & 1u;
            ok = warp_wait_soon<false>(smem_u32(&sf_full[ss]), sph, ctl, 0x720u + ss);
            if (!ok) break;
            tc_fence_after();
            // (the columns' words of four runs ago have been used: their bytes in shared memory would not have been replaced else)
            const uint32_t sc = tmem + WT * NT + ss * kSfCols;
            const uint64_t src = scale_desc(smem_u32(sf)) + ss * ((WT + 1) * kScaleBlock / 16);
#pragma unroll
            for (int w = 0; w < WT + 1; ++w) tc_copy_scales<false>(sc + 4 * w, src + w * (kScaleBlock / 16));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j >= run.count) break;
                if (j % KPS == 0) {
                    ok = warp_wait_soon<false>(smem_u32(&full[stage]), phase, ctl, 0x740u + stage);
                    if (!ok) break;
                    tc_fence_after();
                }
                const uint64_t wd = tiles + stage * (C::STAGE / 16) + (j % KPS) * (kWTile / 16);
                const uint64_t xd = tiles + stage * (C::STAGE / 16) + (kXAt + (j % KPS) * NT * 128) / 16;
#pragma unroll
                for (int w = 0; w < WT; ++w)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)      // 32 of k: 32 bytes of the swizzled row
                        tc_mma_f8<false>(tmem + w * NT, wd + w * KPS * (kWTile / 16) + 2 * kk, xd + 2 * kk, f8_idesc_byte(f8_idesc(128, NT), j),
                                         sc + 4 * w, sc + 4 * WT, kk > 0 ? 1u : onto);
                onto = 1;
                if (j % KPS == KPS - 1 || j == run.count - 1) {
                    tc_commit_f8<false>(smem_u32(&empty[stage]));
                    if (++stage == S) { stage = 0; phase ^= 1u; }
                }
            }
            if (ok) tc_commit_f8<false>(smem_u32(&sf_empty[ss]));
        }
        tc_commit_f8<false>(smem_u32(done));
        if (!ok || !warp_wait(smem_u32(done), 0, ctl, 0x760u)) drain_wait(smem_u32(done), 0, kDrainNs);
        tc_fence_before();
        __syncwarp();
    } else if (warp < 4) {
        // scale words: the weights' are one for all of a tile's rows, the activations' one a row
        constexpr int XW = NT > 32 ? NT / 32 : 1;
        int run_i = 0;
        for (int i = b0; ok && i < b1; ++i, ++run_i) {
            if ((run_i & 1) != warp - 2) continue;
            const F8Run run = f8_run(i, per_shard, p.kblocks);
            const uint8_t* ws = p.w_scale[ag ? r : run.shard];
            const uint8_t* xs = p.x_scale[ag ? 0 : run.shard];
            const uint8_t* at_row[WT + XW];
            bool on[WT + XW];
            uint32_t v[WT + XW];
#pragma unroll
            for (int w = 0; w < WT; ++w) {
                at_row[w] = ws + static_cast<long long>(nt + w * p.n_tiles) * p.kblocks;
                on[w] = true;
            }
#pragma unroll
            for (int i = 0; i < XW; ++i) {
                const int row = row0 + lane + 32 * i;
                on[WT + i] = row < p.m && lane + 32 * i < NT;
                at_row[WT + i] = xs + static_cast<long long>(row) * p.kblocks;
            }
            load_scale_words(at_row, on, run.kb, p.kblocks, p.scale_words != 0, v);
            const uint32_t ss = run_i % kSfStages, sph = (run_i / kSfStages) & 1u;
            ok = warp_wait(smem_u32(&sf_empty[ss]), sph ^ 1u, ctl, 0x750u + ss);
            if (!ok) break;
            uint8_t* dst = sf + ss * (WT + 1) * kScaleBlock;
#pragma unroll
            for (int w = 0; w < WT; ++w)
                *reinterpret_cast<uint4*>(dst + w * kScaleBlock + lane * 16) = make_uint4(v[w], v[w], v[w], v[w]);
#pragma unroll
            for (int i = 0; i < XW; ++i) *reinterpret_cast<uint32_t*>(dst + WT * kScaleBlock + scale_word_at(lane + 32 * i)) = v[WT + i];
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sf_full[ss]));
        }
    }

    // ---- accumulators to shared memory: sums[weight tile][activation row][weight row].  All products are done and the
    // ring is idle (after an abort too: warp 1 waited for them, warp 0 for its copies).
    __syncthreads();
    tc_fence_after();
    if (splits > 1) {
        cluster_wait();
        if (warp == 0 && lane < splits) mbar_arrive_cluster_relaxed(map_to_rank(smem_u32(idle), lane));
    }
    const uint32_t tmem = *tmem_slot;
    float* sums = reinterpret_cast<float*>(smem);
    const uint32_t sums_at = smem_u32(sums), parts_at = sums_at + C::SUMS;
    // two warps a quadrant of lanes, pieces of 16 columns in turns, two on their way at a time
    for (int c = 16 * (warp >> 2); c < WT * NT; c += 64) {
        uint32_t v[2][16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (c + 32 * h >= WT * NT || (c + 32 * h) % NT >= rows) continue;
            if (b1 > b0) {
                tmem_ld_16cols(tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + c + 32 * h, v[h]);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) v[h][i] = 0u;
            }
        }
        tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (c + 32 * h >= WT * NT || (c + 32 * h) % NT >= rows) continue;
#pragma unroll
            for (int i = 0; i < 16; ++i) sums[(c + 32 * h + i) * 128 + 32 * (warp & 3) + lane] = __uint_as_float(v[h][i]);
        }
    }
    tc_fence_before();
    if (splits > 1) fence_proxy_async_smem();
    __syncthreads();
    if (splits > 1) {
        // every block's rows of this block's sums go to it in one piece a weight tile, behind its own sums in its idle ring:
        // parts[block][weight tile][own row][weight row].  (Read row by row from the others' shared memory between two
        // cluster barriers they took longer: n 4096, k 4096, m 64 8.9 us, with nothing exchanged 5.5.)
        // (a warp a block: one warp's lanes took 100 cycles a copy)
        if (warp < splits && warp != split) {
            const bool go = warp_wait<true>(smem_u32(idle), 0, ctl, 0x770u);
            const int theirs = min(own_rows, rows - warp * own_rows);
            if (go && lane == 0 && theirs > 0) {
                const uint32_t bar = map_to_rank(smem_u32(parts), warp);
#pragma unroll
                for (int w = 0; w < WT; ++w)
                    bulk_copy_s2s_signal(map_to_rank(parts_at + (split * WT + w) * own_rows * 512, warp), sums_at + (w * NT + warp * own_rows) * 512,
                                         theirs * 512, bar);
            }
            __syncwarp();
        }
        if (own > 0) warp_wait<true>(smem_u32(parts), 0, ctl, 0x780u);
        __syncwarp();
        cluster_arrive_relaxed();       // this block's part is over; waited for before it leaves
    }

    // ---- 16 threads an activation row, 8 columns each
    for (int x = threadIdx.x; x < ((own * 16 + 31) & ~31); x += kSlabThreads) {
        const int o = x >> 4, i = split * own_rows + o, row = row0 + i, c8 = (x & 15) * 8, col = nt * 128 + c8;
        float y[WT][8];
#pragma unroll
        for (int w = 0; w < WT; ++w) {
            for (int b = 0; b < splits; ++b) {      // in the ranges' order
                const uint32_t at = b == split ? sums_at + ((w * NT + i) * 128 + c8) * 4 : parts_at + (((b * WT + w) * own_rows + o) * 128 + c8) * 4;
                const float4 lo = load_part(at), hi = load_part(at + 16);
                const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) y[w][j] = b == 0 ? v[j] : y[w][j] + v[j];
            }
        }
        const bool in = o < own && col < p.n;
        if constexpr (GATED) {
            // (all eight at once, whatever comes of them: with the test in front they took turns, 110 cycles each)
            float top = 0.f, h[8];
            uint32_t g[8], u[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                g[j] = __float_as_uint(y[0][j]);
                u[j] = __float_as_uint(y[1][j]);
            }
            f8_gated(g, u, h);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                y[0][j] = in ? h[j] : 0.f;
                top = fmaxf(top, f8_magnitude(y[0][j]));
            }
#pragma unroll
            for (int d = 8; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const uint32_t byte = f8_scale_byte(top);
            const float f = f8_inverse(byte);
            if (in) {
                uint8_t* out = static_cast<uint8_t*>(p.out[r]);
                *reinterpret_cast<uint2*>(out + static_cast<long long>(row) * p.n + col) =
                    make_uint2(f8_codes4(y[0][0], y[0][1], y[0][2], y[0][3], f), f8_codes4(y[0][4], y[0][5], y[0][6], y[0][7], f));
                if (c8 == 0) p.out_scale[r][static_cast<long long>(row) * p.n_tiles + nt] = static_cast<uint8_t>(byte);
            }
        } else if (in) {
            uint4 o;
            o.x = pack2<BF16>(__float_as_uint(y[0][0]), __float_as_uint(y[0][1]));
            o.y = pack2<BF16>(__float_as_uint(y[0][2]), __float_as_uint(y[0][3]));
            o.z = pack2<BF16>(__float_as_uint(y[0][4]), __float_as_uint(y[0][5]));
            o.w = pack2<BF16>(__float_as_uint(y[0][6]), __float_as_uint(y[0][7]));
            if (p.op == OP_AR) {
                for (int q = 0; q < p.R; ++q) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out[q]) + static_cast<long long>(row) * p.n + col) = o;
            } else {
                const int q = ag ? r : row / p.rows_per_rank;
                const long long at = ag ? row : row - q * p.rows_per_rank;
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out[q]) + at * p.n + col) = o;
            }
        }
    }
    if (splits > 1) {
        cluster_wait();     // every block has its parts: none leaves while its sums are copied
        if (*reinterpret_cast<volatile uint32_t*>(abort_word) != 0u) {      // copies to this block that it did not wait for
            const uint64_t t0 = globaltimer();
            while (globaltimer() - t0 < 200000ull) {
            }
        }
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM);
    }
}

template <int NT, bool GATED, bool BF16>
cudaError_t launch_t(F8Args a, int sm_count, cudaStream_t stream) {
    using C = SlabCfg<NT, GATED>;
    auto kern = f8_slab_kernel<NT, GATED, BF16>;
    static KnownCount known[64][9];         // clusters of k that run at once, a block on an SM each
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kSlabThreads, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.numAttrs = 1;
    // k == 1 raises the kernel's shared memory limit, once a device
    auto clusters = [&](int k, int* n) -> cudaError_t {
        if (dev >= 0 && dev < 64 && known[dev][k].get(n)) return cudaSuccess;
        cfg.dynamicSmemBytes = C::REST + C::ALONE * C::STAGE;
        cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(cfg.dynamicSmemBytes));
        if (err != cudaSuccess) return err;
        *n = sm_count;
        if (k > 1) {
            cfg.gridDim = dim3(static_cast<unsigned>(k), 1, 1);
            attr[0].val.clusterDim.x = static_cast<unsigned>(k);
            if ((err = cudaOccupancyMaxActiveClusters(n, kern, &cfg)) != cudaSuccess) return err;
        }
        if (dev >= 0 && dev < 64) known[dev][k].set(*n);
        return cudaSuccess;
    };
    const long long tiles = static_cast<long long>(a.m_tiles) * a.n_tiles * (a.op == OP_AG ? a.R : 1);
    const int total = a.shards * ((a.kblocks + 3) / 4);
    int room = 0;
    if ((e = clusters(1, &room)) != cudaSuccess) return e;
    if ((e = f8_ranges(tiles, total, sm_count, clusters, &a.splits)) != cudaSuccess) return e;
    // (room is every SM, and clusters have an SM for every block: with one k-block a stage a split tile is always alone)
    const bool alone = tiles <= room && (C::KPS == 1 || (total + a.splits - 1) / a.splits > 2);
    a.stages = alone ? C::ALONE : C::SHARED;
    const long long blocks = static_cast<long long>(a.n_tiles) * (a.op == OP_AG ? a.R : 1) * a.shards * a.kblocks;      // of weights
    const long long ahead = kAheadBytes / (C::WT * kWTile);
    a.ahead = pdl_launch() && a.m_tiles == 1 && 4 * blocks >= 5 * ahead ? static_cast<int>(ahead / (tiles * a.splits)) : 0;
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * a.splits), 1, 1);
    cfg.dynamicSmemBytes = C::REST + a.stages * C::STAGE;
    attr[0].val.clusterDim.x = static_cast<unsigned>(a.splits);
    if (pdl_launch()) {
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <bool GATED, bool BF16>
cudaError_t launch_n(const F8Args& a, int nt, int sm_count, cudaStream_t stream) {
    switch (nt) {
        case 16: return launch_t<16, GATED, BF16>(a, sm_count, stream);
        case 32: return launch_t<32, GATED, BF16>(a, sm_count, stream);
        case 64: return launch_t<64, GATED, BF16>(a, sm_count, stream);
        default:
            if constexpr (!GATED) return launch_t<128, GATED, BF16>(a, sm_count, stream);
            else return cudaErrorInvalidValue;
    }
}

}  // namespace

bool f8_use_tiles(int op, bool gated, int R, int64_t m, int64_t n, int64_t k, int sm_count) {
    if (const char* e = std::getenv("COC_F8_TILE")) return std::atoi(e) != 0;
    return f8_tiles_sooner(op == OP_AG, gated, R, m, n, k, sm_count);
}

// (gated slabs have two weight tiles: 128 rows of both would leave no ring)
int f8_slab_rows(int64_t m, bool gated) { return m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 || gated ? 64 : 128; }

template <int NT>
static int kps_of(bool gated) { return gated ? SlabCfg<NT, true>::KPS : SlabCfg<NT, false>::KPS; }
int f8_slab_kblocks(int64_t m, bool gated) {
    switch (f8_slab_rows(m, gated)) {
        case 16: return kps_of<16>(gated);
        case 32: return kps_of<32>(gated);
        case 64: return kps_of<64>(gated);
        default: return SlabCfg<128, false>::KPS;
    }
}

// Where the tiles leave SMs free, a tile's contraction is cut into as
// many ranges (2 to 8) as clusters of that size find an SM for every block: a
// block alone on an SM has all its shared memory for the ring.  More tiles
// than SMs go unsplit, two blocks on an SM, which overlaps one's beginning and end
// with the other's middle.  So do blocks of up to 8 k-blocks: the next launch's
// set themselves up beside them.  Measured, ranges 1 / 2 / 4 / 8 (us, graphs of calls
// in a row), alone on an SM and two to an SM:
//   n 4096, k 4096, m 1          9.6 / 6.9 / 6.0 / 11.6    9.6 / 6.8 / 5.5 (taken) / 7.5
//   n 4096, k 4096, m 64         10.3 / 8.2 / 7.3 / 16.4   10.8 / 8.4 / 7.0 (taken) / 8.9
//   n 8192, k 8 x 3584, m 64     51 / 37.6 (taken) / 42 / 60   71 / 45 / 38.4 / 43
//   n 14336, k 8 x 7168, m 16    117 (taken) / 125 / 131 / 144   147 / 121 / 126 / 136
//   n 1024, k 2 x 8192, m 16     29 / 16.5 / 10.9 / 8.2 (taken)   38 / 22 / 13.0 / 9.1
//   gated, 8 x 3584, k 8192, m 64   77 / 81   75 to 77 (taken), not split
cudaError_t launch_f8_slab(const F8Args& args, bool gated, bool bf16, int sm_count, cudaStream_t stream) {
    F8Args a = args;
    const int nt = f8_slab_rows(a.m, gated);
    a.m_tiles = (a.m + nt - 1) / nt;
    if (gated) return launch_n<true, true>(a, nt, sm_count, stream);
    return bf16 ? launch_n<false, true>(a, nt, sm_count, stream) : launch_n<false, false>(a, nt, sm_count, stream);
}

// ---- the shards' activations one after another (AllGather of shards that lie apart)
namespace {
__global__ void __launch_bounds__(256) f8_stack_kernel(const __grid_constant__ F8StackArgs a) {
    grid_dependency_wait();
    grid_dependents_launch();
    const int r = blockIdx.y;
    const long long step = static_cast<long long>(gridDim.x) * blockDim.x, first = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    uint4* dst = reinterpret_cast<uint4*>(a.x_dst) + r * a.vecs;
    for (long long i = first; i < a.vecs; i += step) dst[i] = load_uint4(reinterpret_cast<const uint16_t*>(a.x[r]) + 8 * i);
    for (long long i = first; i < a.scale_bytes; i += step) a.scale_dst[r * a.scale_bytes + i] = static_cast<uint8_t>(load_byte(a.scale[r] + i));
}
}  // namespace

cudaError_t launch_f8_stack(const F8StackArgs& a, int sm_count, cudaStream_t stream) {
    const long long work = std::max(a.vecs, a.scale_bytes);
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>((work + 255) / 256, 4LL * sm_count)), static_cast<unsigned>(a.R), 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    if (pdl_launch()) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, f8_stack_kernel, a);
}

}  // namespace coc
