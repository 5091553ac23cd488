// Products of 8-bit activations and weights for many rows: CTA pairs compute
// 256 x 256 tiles (256 activation rows by 256 weight rows; gated: by 128 rows
// of the gate and the same 128 of the up projection), persistent over the tiles.
//
// Mathematics as in coc_f8_slab.cu.
//
// What bounds it.  The tensor cores: a k-block of a pair is four products of
// 256 x 256 x 32, 512 cycles, and 32 KiB of copies a CTA, 64 bytes a cycle.  Gated, 8
// x 3584, k 8192, 4096 rows: 1054 to 1069 us for a short while (3.6 PFLOP/s; tensor
// pipes 82% active under the profiler at 1.69 GHz, 13.9 TB/s out of L2), 1190 to
// 1250 in a long loop, where the GPU's power holds the clock at 1.4 GHz; n 8192, k 8
// x 3584, 4096 rows scattered: 548 and 620 to 643 us.  With a quarter of the copies
// left out (wrong results) the loops take 1179 and 563 us: what moves between L2
// and the SMs costs both time and power.
//
// Tensor memory.  Two accumulators of 256 columns would fill it, and the scale
// words need 24 columns: the accumulators lie at columns 0 and 224 and share
// 32.  A tile's epilogue reads those first; then the next tile's products may
// start, and the rest is read beside them.  Between a tile's last product and the
// next tile's first some 1500 cycles remain.
//
// Order.  Row tiles in groups whose activations stay in L2, the row tiles of a
// column tile adjacent, so that pairs that run together share both operands.
//
// Roles: warp 0 copies tiles (TMA), warp 1 issues the pair's products (leader),
// warps 2-5 are the epilogue, warps 6 and 7 gather scale words, alternating.
#include <algorithm>
#include <atomic>

#include "coc_f8.cuh"

namespace coc {
namespace {

constexpr int kStages = 6;
constexpr int kTileBytes = 128 * 128;           // 128 rows' k-block: X and W each, per CTA
constexpr int kSfStages = 4;
constexpr int kSfBytes = 3 * kScaleBlock;       // X rows; two sets of W rows
constexpr int kAcc1 = 224;                      // the second accumulator's first column
constexpr int kSfCol = 480;                     // two sets of 16 columns
constexpr int kTileThreads = 256;
constexpr int kTileSmem = 1024 + kStages * 2 * kTileBytes + kSfStages * kSfBytes + 4 * EPI_BUF_BYTES + 512;
static_assert(kTileSmem <= kSlabSmemCap, "shared memory");

template <bool GATED, bool BF16>
__global__ void __launch_bounds__(kTileThreads, 1) f8_tile_kernel(const __grid_constant__ F8Args p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* epi = smem + kStages * 2 * kTileBytes;
    uint8_t* sf = epi + 4 * EPI_BUF_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sf + kSfStages * kSfBytes);
    uint64_t* full = bars;                      // [kStages] both CTAs' tiles landed (leader)
    uint64_t* empty = full + kStages;           // [kStages] read by the products
    uint64_t* sf_full = empty + kStages;        // [kSfStages] both CTAs' scale words written (leader)
    uint64_t* sf_empty = sf_full + kSfStages;   // [kSfStages] the run's products are done
    uint64_t* acc_full = sf_empty + kSfStages;  // a tile's products are done
    uint64_t* acc_early = acc_full + 1;         // its shared columns have been read by both CTAs (leader)
    uint64_t* never = acc_early + 1;
    uint64_t* drain = never + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    uint32_t* abort_word = tmem_slot + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Ctl ctl{abort_word, p.status};
    const uint32_t rank = cluster_rank();       // 0: leader
    const int first = static_cast<int>(cluster_id()), step = static_cast<int>(cluster_count());
    const bool ag = p.op == OP_AG;
    const int cols = GATED ? p.n_tiles : (p.n_tiles + 1) / 2;      // column tiles of a rank
    const int all_cols = cols * (ag ? p.R : 1);
    const int units = all_cols * p.m_tiles;
    const int total = p.shards * p.kblocks;
    // Units go by groups of group_mt row tiles, whose activations stay in L2
    // while the columns stream past; inside a group the row tiles of a column are adjacent.
    auto decode = [&](int u, int& r, int& mt, int& nt) {
        const int per = p.group_mt * all_cols, g = u / per;
        const int rows = min(p.group_mt, p.m_tiles - g * p.group_mt);
        u -= g * per;
        int c = u / rows;
        mt = g * p.group_mt + u - c * rows;
        if (g & 1) c = all_cols - 1 - c;
        r = c / cols;
        nt = c - r * cols;
    };

    if (warp == 0 && lane < p.R && total > 0) {
        if (lane < (ag ? 1 : p.R)) prefetch_tmap(&p.tm_x[lane]);
        prefetch_tmap(&p.tm_w[lane]);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int s = 0; s < kSfStages; ++s) {
            mbar_init(smem_u32(&sf_full[s]), 2);
            mbar_init(smem_u32(&sf_empty[s]), 1);
        }
        mbar_init(smem_u32(acc_full), 1);
        mbar_init(smem_u32(acc_early), 2 * NUM_EPI_WARPS);
        mbar_init(smem_u32(never), 1);
        mbar_init(smem_u32(drain), 1);
        *abort_word = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async_smem();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();     // both CTAs' barriers exist before any traffic between them
    tc_fence_after();
    grid_dependency_wait();
    grid_dependents_launch();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;

    if (warp == 0) {
        uint32_t stage = 0, phase = 0, filled = 0, parity = 0;
        const uint64_t pol_x = make_l2_policy(2), pol_w = make_l2_policy(0);
        for (int u = first; ok && u < units; u += step) {
            int r, mt, nt;
            decode(u, r, mt, nt);
            const int x_row = mt * 256 + static_cast<int>(rank) * 128;
            const int w_row = GATED ? nt * 128 + static_cast<int>(rank) * p.n : nt * 256 + static_cast<int>(rank) * 128;
            for (int shard = 0; ok && shard < p.shards; ++shard) {
                const CUtensorMap *xm = &p.tm_x[shard], *wm = &p.tm_w[ag ? r : shard];
                for (int kb = 0; kb < p.kblocks; ++kb) {
                    ok = warp_wait(smem_u32(&empty[stage]), phase ^ 1u, ctl, 0x810u + stage);
                    if (!ok) break;
                    if (lane == 0) {
                        const uint32_t here = smem_u32(&full[stage]), fb = map_to_rank(here, 0);
                        const uint32_t dst = smem_u32(smem) + stage * 2 * kTileBytes;
                        if (rank == 0) mbar_expect_tx(here, 4 * kTileBytes);
                        tma_load_2d_pair(dst, xm, kb * 128, x_row, fb, pol_x);
                        tma_load_2d_pair(dst + kTileBytes, wm, kb * 128, w_row, fb, pol_w);
                        filled |= 1u << stage;
                        parity = (parity & ~(1u << stage)) | (phase << stage);
                    }
                    __syncwarp();
                    if (++stage == kStages) { stage = 0; phase ^= 1u; }
                }
            }
        }
        if (!ok && lane == 0) {     // no copy stays in flight into shared memory
            if (rank == 0) {
                for (int s = 0; s < kStages; ++s)
                    if (filled & (1u << s)) drain_wait(smem_u32(&full[s]), (parity >> s) & 1u, kDrainNs);
            } else {
                const uint64_t t0 = globaltimer();
                while (globaltimer() - t0 < 200000ull) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            const uint64_t tiles = make_sdesc(smem_u32(smem), 16, 1024);
            uint32_t stage = 0, phase = 0;
            int run_i = 0, tile_i = 0;
            for (int u = first; ok && u < units; u += step, ++tile_i) {
                bool shared_free = tile_i == 0;     // the columns this accumulator shares with the one before
                const uint32_t d = tmem + (tile_i & 1) * kAcc1;
                uint32_t onto = 0;
                for (int shard = 0; ok && shard < p.shards; ++shard)
                    for (int kb = 0; kb < p.kblocks; kb += 4, ++run_i) {
                        const uint32_t ss = run_i % kSfStages;
                        ok = warp_wait_soon<true>(smem_u32(&sf_full[ss]), (run_i / kSfStages) & 1u, ctl, 0x830u + ss);
                        // the words two runs ago, in the same columns, have been used
                        if (ok && run_i >= 2) {
                            const int was = run_i - 2;
                            ok = warp_wait_soon<true>(smem_u32(&sf_empty[was % kSfStages]), (was / kSfStages) & 1u, ctl, 0x840u);
                        }
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t sc = tmem + kSfCol + (run_i & 1) * 16;
                        const uint64_t src = scale_desc(smem_u32(sf)) + ss * (kSfBytes / 16);
#pragma unroll
                        for (int w = 0; w < 3; ++w) tc_copy_scales<true>(sc + 4 * w, src + w * (kScaleBlock / 16));
                        const int count = min(4, p.kblocks - kb);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (j == count) break;
                            ok = warp_wait_soon<true>(smem_u32(&full[stage]), phase, ctl, 0x850u + stage);
                            if (!shared_free && ok) {
                                ok = warp_wait_soon<true>(smem_u32(acc_early), (tile_i - 1) & 1, ctl, 0x820u);
                                shared_free = true;
                            }
                            if (!ok) break;
                            tc_fence_after();
                            const uint64_t xd = tiles + stage * (2 * kTileBytes / 16), wd = xd + kTileBytes / 16;
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                tc_mma_f8<true>(d, xd + 2 * kk, wd + 2 * kk, f8_idesc_byte(f8_idesc(256, 256), j), sc, sc + 4, onto);
                                onto = 1;
                            }
                            tc_commit_f8<true>(smem_u32(&empty[stage]));
                            if (++stage == kStages) { stage = 0; phase ^= 1u; }
                        }
                        if (!ok) break;
                        tc_commit_f8<true>(smem_u32(&sf_empty[ss]));
                    }
                if (ok && !shared_free) ok = warp_wait_soon<true>(smem_u32(acc_early), (tile_i - 1) & 1, ctl, 0x820u);   // (no k at all)
                if (!ok) break;
                tc_commit_f8<true>(smem_u32(acc_full));
            }
            tc_commit_f8<true>(smem_u32(drain));    // every product is done before tensor memory is given back
            drain_wait(smem_u32(drain), 0, kDrainNs);
            __syncwarp();
        }
    } else if (warp < 6) {
        const int q = warp & 3;                 // the lanes this warp may read
        uint8_t* stage_buf = epi + (warp - 2) * EPI_BUF_BYTES;
        const uint32_t early = map_to_rank(smem_u32(acc_early), 0);
        int tile_i = 0;
        if (p.inject_timeout) ok = warp_wait(smem_u32(never), 0, ctl, 0x800u);
        for (int u = first; ok && u < units; u += step, ++tile_i) {
            int r, mt, nt;
            decode(u, r, mt, nt);
            ok = warp_wait<true>(smem_u32(acc_full), tile_i & 1, ctl, 0x860u);
            if (!ok) break;
            tc_fence_after();
            const int buf = tile_i & 1;
            const int row0 = mt * 256 + static_cast<int>(rank) * 128 + 32 * q;
            const uint32_t acc = tmem + (static_cast<uint32_t>(32 * q) << 16) + buf * kAcc1;
            // the shared columns are in registers (their loads are complete): the next tile may begin
            auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(early);
            };
            auto load = [&](uint32_t at, uint32_t (&v)[32]) {
                if (total > 0) {
                    tmem_ld_32cols(at, v);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0u;
                }
            };
            // lane l: 16-byte piece l % 8 of rows l / 8 + 4 i of the staged 32 x 128 bytes
            const int piece = lane & 7;
            if constexpr (GATED) {
                // quarters of the gate's and the up projection's columns, the shared ones first
                float h[128];
                const int col0 = nt * 128;
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int j = buf ? s : 3 - s;
                    uint32_t g[32], up[32];
                    load(acc + 32 * j, g);
                    load(acc + 128 + 32 * j, up);
                    tmem_wait_ld();
                    if (s == 0) release();
                    f8_gated(g, up, h + 32 * s);
#pragma unroll
                    for (int i = 0; i < 32; ++i) h[32 * s + i] = col0 + 32 * j + i < p.n ? h[32 * s + i] : 0.f;
                }
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < 128; ++i) top = fmaxf(top, f8_magnitude(h[i]));
                const uint32_t byte = f8_scale_byte(top);
                const float f = f8_inverse(byte);
                if (row0 + lane < p.m) p.out_scale[r][static_cast<long long>(row0 + lane) * p.n_tiles + nt] = static_cast<uint8_t>(byte);
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int j = buf ? s : 3 - s;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float* v = h + 32 * s + 16 * c;
                        const uint4 w = make_uint4(f8_codes4(v[0], v[1], v[2], v[3], f), f8_codes4(v[4], v[5], v[6], v[7], f),
                                                   f8_codes4(v[8], v[9], v[10], v[11], f), f8_codes4(v[12], v[13], v[14], v[15], f));
                        *reinterpret_cast<uint4*>(stage_buf + lane * 128 + (((2 * j + c) ^ (lane & 7)) << 4)) = w;
                    }
                }
                __syncwarp();
                uint8_t* out = static_cast<uint8_t*>(p.out[r]) + col0 + piece * 16;
                const bool in = col0 + piece * 16 < p.n;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int rr = (lane >> 3) + 4 * i;
                    const uint4 v = *reinterpret_cast<const uint4*>(stage_buf + rr * 128 + ((piece ^ (rr & 7)) << 4));
                    if (in && row0 + rr < p.m) *reinterpret_cast<uint4*>(out + static_cast<long long>(row0 + rr) * p.n) = v;
                }
                __syncwarp();
            } else {
                // where this lane's 8 rows lie in their rank's output (AllReduce: in rank 0's), once for the tile
                uint16_t* at[8];
                const int col0 = nt * 256 + piece * 8;
                if (p.op == OP_RS) {
                    int o = min(row0, p.m - 1) / p.rows_per_rank, begin = o * p.rows_per_rank;      // a rank and its first row
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int row = row0 + (lane >> 3) + 4 * i;
                        while (row < p.m && row - begin >= p.rows_per_rank) {
                            begin += p.rows_per_rank;
                            ++o;
                        }
                        at[i] = row < p.m ? static_cast<uint16_t*>(p.out[o]) + static_cast<long long>(row - begin) * p.n + col0 : nullptr;
                    }
                } else {
                    uint16_t* out = static_cast<uint16_t*>(p.out[ag ? r : 0]) + col0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int row = row0 + (lane >> 3) + 4 * i;
                        at[i] = row < p.m ? out + static_cast<long long>(row) * p.n : nullptr;
                    }
                }
                const int copies = p.op == OP_AR ? p.R : 1;
                for (int s = 0; s < 4; ++s) {
                    const int sub = buf ? s : 3 - s;
                    uint32_t va[32], vb[32];
                    load(acc + 64 * sub, va);
                    load(acc + 64 * sub + 32, vb);
                    tmem_wait_ld();
                    if (s == 0) release();
                    if (row0 >= p.m || nt * 256 + 64 * sub >= p.n) continue;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t* v = j < 4 ? va + 8 * j : vb + 8 * (j - 4);
                        const uint4 w = make_uint4(pack2<BF16>(v[0], v[1]), pack2<BF16>(v[2], v[3]), pack2<BF16>(v[4], v[5]), pack2<BF16>(v[6], v[7]));
                        *reinterpret_cast<uint4*>(stage_buf + lane * 128 + ((j ^ (lane & 7)) << 4)) = w;
                    }
                    __syncwarp();
                    uint4 v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int rr = (lane >> 3) + 4 * i;
                        v[i] = *reinterpret_cast<const uint4*>(stage_buf + rr * 128 + ((piece ^ (rr & 7)) << 4));
                    }
                    if (col0 + 64 * sub < p.n) {
                        for (int c = 0; c < copies; ++c) {
                            const long long to = reinterpret_cast<intptr_t>(p.out[c]) - reinterpret_cast<intptr_t>(p.out[0]);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (at[i] != nullptr)
                                    *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(at[i] + 64 * sub) + (copies > 1 ? to : 0)) = v[i];
                        }
                    }
                    __syncwarp();
                }
            }
        }
    } else {
        // scale words: this CTA's 128 activation rows, and all 256 weight rows (two words)
        const int per_shard = (p.kblocks + 3) / 4;
        int run_i = 0;
        for (int u = first; ok && u < units; u += step) {
            int r, mt, nt;
            decode(u, r, mt, nt);
            const int row0 = mt * 256 + static_cast<int>(rank) * 128;
            const int w0 = GATED ? nt : 2 * nt, w1 = GATED ? p.n_tiles + nt : 2 * nt + 1;
            for (int i = 0; i < p.shards * per_shard; ++i, ++run_i) {
                if ((run_i & 1) != warp - 6) continue;
                const F8Run run = f8_run(i, per_shard, p.kblocks);
                const uint8_t *xs = p.x_scale[run.shard], *ws = p.w_scale[ag ? r : run.shard];
                const uint8_t* at_row[6];
                bool on[6];
                uint32_t v[6];      // four activation rows', two weight tiles'
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = row0 + lane + 32 * i;
                    on[i] = row < p.m;
                    at_row[i] = xs + static_cast<long long>(row) * p.kblocks;
                }
                at_row[4] = ws + static_cast<long long>(w0) * p.kblocks;
                at_row[5] = ws + static_cast<long long>(w1) * p.kblocks;
                on[4] = true;
                on[5] = GATED || w1 < p.n_tiles;
                load_scale_words(at_row, on, run.kb, p.kblocks, p.scale_words != 0, v);
                const uint32_t ss = run_i % kSfStages;
                ok = warp_wait<true>(smem_u32(&sf_empty[ss]), ((run_i / kSfStages) & 1u) ^ 1u, ctl, 0x870u + ss);
                if (!ok) break;
                uint8_t* dst = sf + ss * kSfBytes;
                // rows lane, lane + 32, lane + 64, lane + 96 are 16 bytes
                *reinterpret_cast<uint4*>(dst + lane * 16) = make_uint4(v[0], v[1], v[2], v[3]);
#pragma unroll
                for (int w = 0; w < 2; ++w)
                    *reinterpret_cast<uint4*>(dst + (w + 1) * kScaleBlock + lane * 16) = make_uint4(v[4 + w], v[4 + w], v[4 + w], v[4 + w]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_u32(&sf_full[ss]), 0));
            }
        }
    }

    tc_fence_before();
    if (*reinterpret_cast<volatile uint32_t*>(abort_word) != 0u) {
        // the peer may still have copies in flight towards the leader
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 200000ull) {
        }
    }
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

template <bool GATED, bool BF16>
cudaError_t launch_t(const F8Args& args, cudaStream_t stream) {
    F8Args a = args;
    auto kern = f8_tile_kernel<GATED, BF16>;
    static std::atomic<int> known[64];          // pairs that run at once; 0: not asked yet
    int dev = 0, pairs = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(kTileThreads, 1, 1);
    cfg.dynamicSmemBytes = kTileSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.numAttrs = 1;
    if (dev >= 0 && dev < 64) pairs = known[dev].load(std::memory_order_acquire);
    if (pairs == 0) {
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileSmem)) != cudaSuccess) return e;
        if ((e = cudaOccupancyMaxActiveClusters(&pairs, kern, &cfg)) != cudaSuccess) return e;
        if (pairs < 1) return cudaErrorLaunchOutOfResources;
        if (dev >= 0 && dev < 64) known[dev].store(pairs, std::memory_order_release);
    }
    a.m_tiles = (a.m + 255) / 256;
    const long long units = static_cast<long long>(GATED ? a.n_tiles : (a.n_tiles + 1) / 2) * (a.op == OP_AG ? a.R : 1) * a.m_tiles;
    // row tiles whose activations take a quarter of L2 (half: 8192 x 8192 x 8192 391 us instead of 366)
    const long long x_tile = 256LL * 128 * a.kblocks * a.shards;
    a.group_mt = static_cast<int>(std::min<long long>(a.m_tiles, std::max<long long>(8, (32LL << 20) / std::max<long long>(1, x_tile))));
    cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<long long>(units, pairs)), 1, 1);
    if (pdl_launch()) {
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_f8_tile(const F8Args& a, bool gated, bool bf16, cudaStream_t stream) {
    if (gated) return launch_t<true, true>(a, stream);
    return bf16 ? launch_t<false, true>(a, stream) : launch_t<false, false>(a, stream);
}

}  // namespace coc
