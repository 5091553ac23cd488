// Append to the paged 8-bit key/value cache: rotation of q and k by position,
// quantisation of k and v to e4m3 with one scale per (page, head).
//
// Mathematics.  A pair (x, y) of a head becomes (x c - y s, y c + x s), every
// product and sum rounded to fp32 on its own (no fused multiply-add), so that
// a result does not depend on how a compiler contracts it.  A page's scale is
// the least power of two that brings its largest value to e4m3's 448; where a
// page already holds tokens it only grows, and the older codes are multiplied
// by the quotient, exact but for e4m3's underflow.
//
// What bounds it.  Bytes: q is read and written, k and v are read and their
// codes written.  With few tokens it is the launch and the chain of dependent
// loads (length, page id, values), so everything is one kernel.
//
// Split.  A unit is one page of one (sequence, key head, rank, k or v): its
// largest value has to be known before a code is written.  TPU threads take a
// unit: a warp where sequences bring a token or a few, a block where they bring
// pages.  Behind the units' blocks come those of q, a thread taking the same 16
// values of four heads, whose cosines it loads once.
//
// Measured (8 ranks, 8 query heads and one key head of 128 each): 128 tokens,
// one a sequence, 4.0 us; 7686 tokens of 7 prompts 59 us, 5.1 TB/s
// (two blocks an SM instead of three: 73; two heads a thread: 61 to 69).
#include "coc_kv.cuh"
#include "coc_ptx.cuh"

namespace coc {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;       // heads of q that a thread takes
constexpr int kKeep = 2;        // tasks whose values a thread keeps between the two passes of a unit

// Value e of a head rotated: the general form, for rotations whose halves do
// not lie on 16-byte boundaries.
template <bool BF16>
__device__ __noinline__ float rotated(const KvAppendArgs& a, const uint16_t* x, int e, int pos) {
    const float v = to_float16bit<BF16>(x[e]);
    if (e >= a.rot) return v;
    const int half = a.rot / 2;
    const int j = a.interleaved ? e / 2 : (e < half ? e : e - half);
    const bool first = a.interleaved ? (e & 1) == 0 : e < half;
    const int pe = a.interleaved ? (e ^ 1) : (first ? e + half : e - half);
    const float w = to_float16bit<BF16>(x[pe]);
    const float c = load_float(a.cos + static_cast<long long>(pos) * half + j);
    const float s = load_float(a.sin + static_cast<long long>(pos) * half + j);
    return first ? __fsub_rn(__fmul_rn(v, c), __fmul_rn(w, s)) : __fadd_rn(__fmul_rn(v, c), __fmul_rn(w, s));
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = to_float16bit<BF16>(static_cast<uint16_t>(w[i]));
        f[2 * i + 1] = to_float16bit<BF16>(static_cast<uint16_t>(w[i] >> 16));
    }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack2<BF16>(__float_as_uint(f[2 * i]), __float_as_uint(f[2 * i + 1]));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Task t of a head (d / 16 of them): two pieces of 8 values, at e0 and e1, and
// what happens to them.
enum Turn : int { kCopy = 0, kPair = 1, kFirst = 2, kBoth = 3, kGeneral = 4 };
struct Task {
    int e0, e1, turn;
};
__device__ __forceinline__ Task task_of(const KvAppendArgs& a, int t, bool rot) {
    Task k{16 * t, 16 * t + 8, kCopy};
    if (!rot) return k;
    if (a.interleaved) {
        if (a.rot % 8 != 0) k.turn = kGeneral;
        else k.turn = k.e1 < a.rot ? kBoth : k.e0 < a.rot ? kFirst : kCopy;      // adjacent pairs inside each piece
    } else if (a.rot % 16 != 0) {
        k.turn = kGeneral;
    } else if (t < a.rot / 16) {
        k = {8 * t, 8 * t + a.rot / 2, kPair};                                    // pairs across the pieces
    }
    return k;
}

// Cosines and sines of a task: 8 of each (kPair: the pairs j = e0 .. e0 + 7;
// interleaved: 4 of each piece).
struct Angles {
    float c[8], s[8];
};
__device__ __forceinline__ void load4(const float* p, float* f, bool vec) {
    if (vec) {
        const float4 v = load_float4(p);
        f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = load_float(p + i);
    }
}
__device__ __forceinline__ void angles_of(const KvAppendArgs& a, const Task& k, int pos, Angles& g) {
    if (k.turn == kCopy || k.turn == kGeneral) return;
    const long long row = static_cast<long long>(pos) * (a.rot / 2);
    const int j0 = k.turn == kPair ? k.e0 : k.e0 / 2, j1 = k.turn == kPair ? k.e0 + 4 : k.e1 / 2;
    load4(a.cos + row + j0, g.c, a.vec_angles);
    load4(a.sin + row + j0, g.s, a.vec_angles);
    if (k.turn != kFirst) {
        load4(a.cos + row + j1, g.c + 4, a.vec_angles);
        load4(a.sin + row + j1, g.s + 4, a.vec_angles);
    }
}

// The task's 16 values in fp32, from raw pieces p0, p1 (head x for kGeneral).
template <bool BF16>
__device__ __forceinline__ void turned(const KvAppendArgs& a, const uint16_t* x, const uint4& p0, const uint4& p1, const Task& k,
                                       const Angles& g, int pos, float (&v)[16]) {
    unpack8<BF16>(p0, v);
    unpack8<BF16>(p1, v + 8);
    if (k.turn == kPair) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p = v[i], q = v[8 + i];
            v[i] = __fsub_rn(__fmul_rn(p, g.c[i]), __fmul_rn(q, g.s[i]));
            v[8 + i] = __fadd_rn(__fmul_rn(q, g.c[i]), __fmul_rn(p, g.s[i]));
        }
    } else if (k.turn == kBoth || k.turn == kFirst) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= 4 && k.turn == kFirst) continue;
            const float p = v[2 * i], q = v[2 * i + 1];
            v[2 * i] = __fsub_rn(__fmul_rn(p, g.c[i]), __fmul_rn(q, g.s[i]));
            v[2 * i + 1] = __fadd_rn(__fmul_rn(q, g.c[i]), __fmul_rn(p, g.s[i]));
        }
    } else if (k.turn == kGeneral) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = rotated<BF16>(a, x, k.e0 + i, pos);
    }
}

__device__ __forceinline__ uint2 codes8(const float* v, float inv) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(v[4 * i], inv), __fmul_rn(v[4 * i + 1], inv)), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(v[4 * i + 2], inv), __fmul_rn(v[4 * i + 3], inv)), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    return make_uint2(w[0], w[1]);
}
// Four codes times f.
__device__ __forceinline__ uint32_t rescaled4(uint32_t w, float f) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * i)), __NV_E4M3);
        const float2 x = __half22float2(__half2(h));
        r |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(x.x, f), __fmul_rn(x.y, f)), __NV_SATFINITE, __NV_E4M3)) << (16 * i);
    }
    return r;
}

// One unit by TPU threads, `tid` of them.  Every thread of the unit takes the
// same way through the barriers.
template <bool BF16, int TPU>
__device__ __forceinline__ void append_unit(const KvAppendArgs& a, int item, int tid, float* red) {
    const int which = item & 1, r = (item >> 1) % a.R, rest = (item >> 1) / a.R;
    const int h = rest % a.heads, unit = rest / a.heads;
    AppendUnit u;
    if (!append_unit_of(a.cu, a.lens, a.seqs, a.tokens, a.page, unit, u)) return;
    int page_id = -1;
    if (u.page < a.table_width) page_id = load_index(a.table + static_cast<long long>(u.s) * a.table_width + u.page);
    const int start = u.start, first = u.first, last = u.last;
    if (a.cos != nullptr && last > a.positions) {
        if (tid == 0) atomicOr(a.status, DEV_ERR_BAD_PAGE);
        return;
    }
    const bool rot = which == 0 && a.cos != nullptr;
    const uint16_t* src = (which ? a.v[r] : a.k[r]) + (u.token + first) * (which ? a.v_token : a.k_token) + h * (which ? a.v_head : a.k_head);
    const long long stride = which ? a.v_token : a.k_token;
    const int per_row = a.d / 16, tasks = (last - first) * per_row;

    auto values = [&](int i, float (&v)[16], Task& k, int& row) {
        row = i / per_row;
        k = task_of(a, i - row * per_row, rot);
        const uint16_t* x = src + row * stride;
        const uint4 p0v = load_uint4(x + k.e0), p1v = load_uint4(x + k.e1);
        Angles g;
        angles_of(a, k, first + row, g);
        turned<BF16>(a, x, p0v, p1v, k, g, first + row, v);
    };
    auto largest = [](const float (&v)[16], float top) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float x = fabsf(v[i]);
            if (x <= 3.4028235e38f) top = fmaxf(top, x);    // NaN and infinities take no part
        }
        return top;
    };
    float kept[kKeep][16];
    float amax = 0.f;
    const bool keep = tasks <= kKeep * TPU;
    if (keep) {
#pragma unroll
        for (int q = 0; q < kKeep; ++q) {
            const int i = tid + q * TPU;
            if (i < tasks) {
                Task k;
                int row;
                values(i, kept[q], k, row);
                amax = largest(kept[q], amax);
            }
        }
    } else {
        for (int i = tid; i < tasks; i += TPU) {
            float v[16];
            Task k;
            int row;
            values(i, v, k, row);
            amax = largest(v, amax);
        }
    }
    // nothing so far has waited for the page's number
    if (page_id < 0 || page_id >= a.pages) {
        if (tid == 0) atomicOr(a.status, DEV_ERR_BAD_PAGE);
        return;
    }
    uint8_t* codes = (which ? a.cv[r] : a.ck[r]) + (static_cast<long long>(page_id) * a.heads + h) * a.page * a.d;
    float* scale = (which ? a.sv[r] : a.sk[r]) + static_cast<long long>(page_id) * a.heads + h;
    const float old = first > start ? *scale : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if constexpr (TPU > 32) {
        if ((tid & 31) == 0) red[tid >> 5] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TPU / 32; ++i) amax = fmaxf(amax, red[i]);
    } else {
        __syncwarp();       // the shuffles order no memory
    }
    const float now = fmaxf(scale_for(amax), old);      // behind the barrier: every thread has read the old scale
    if (tid == 0) *scale = now;
    const float inv = __frcp_rn(now);
    if (first > start && now != old) {
        const float f = __fmul_rn(old, inv);
        uint4* c = reinterpret_cast<uint4*>(codes);
        for (int i = tid; i < (first - start) * per_row; i += TPU) {
            uint4 w = c[i];
            w.x = rescaled4(w.x, f);
            w.y = rescaled4(w.y, f);
            w.z = rescaled4(w.z, f);
            w.w = rescaled4(w.w, f);
            c[i] = w;
        }
    }
    uint8_t* dst = codes + static_cast<long long>(first - start) * a.d;
    auto store = [&](const float (&v)[16], const Task& k, int row) {
        *reinterpret_cast<uint2*>(dst + row * a.d + k.e0) = codes8(v, inv);
        *reinterpret_cast<uint2*>(dst + row * a.d + k.e1) = codes8(v + 8, inv);
    };
    if (keep) {
#pragma unroll
        for (int q = 0; q < kKeep; ++q) {
            const int i = tid + q * TPU;
            if (i < tasks) store(kept[q], task_of(a, i % per_row, rot), i / per_row);
        }
    } else {
        for (int i = tid; i < tasks; i += TPU) {
            float v[16];
            Task k;
            int row;
            values(i, v, k, row);
            store(v, k, row);
        }
    }
}

template <bool BF16, int TPU>
__global__ void __launch_bounds__(kThreads, 3) kv_append_kernel(const __grid_constant__ KvAppendArgs a, int items, int unit_blocks, uint32_t q_tasks) {
    __shared__ float red[kThreads / 32];
    grid_dependency_wait();
    grid_dependents_launch();
    if (static_cast<int>(blockIdx.x) < unit_blocks) {
        const int item = blockIdx.x * (kThreads / TPU) + threadIdx.x / TPU;
        if (item < items) append_unit<BF16, TPU>(a, item, threadIdx.x % TPU, red);
        return;
    }
    // ---- q: task, group of heads, rank, token
    const uint32_t per_row = a.d / 16, groups = (a.q_heads + kHeads - 1) / kHeads;
    const uint32_t i = (blockIdx.x - static_cast<uint32_t>(unit_blocks)) * kThreads + threadIdx.x;
    if (i >= q_tasks) return;
    uint32_t rest = i / per_row;
    const int task = static_cast<int>(i - rest * per_row);
    const uint32_t above = rest / groups;
    const int g0 = static_cast<int>(rest - above * groups) * kHeads;
    const int t = static_cast<int>(above / a.R), r = static_cast<int>(above - t * a.R);
    const int heads = min(kHeads, a.q_heads - g0);
    const uint16_t* x = a.q[r] + t * a.q_token + g0 * a.q_head;
    uint16_t* o = a.q_out[r] + (static_cast<long long>(t) * a.q_heads + g0) * a.d;
    // the values first: they wait for nothing
    Task k = task_of(a, task, a.cos != nullptr);
    uint4 p0[kHeads], p1[kHeads];
#pragma unroll
    for (int h = 0; h < kHeads; ++h)
        if (h < heads) {
            p0[h] = load_uint4(x + h * a.q_head + k.e0);
            p1[h] = load_uint4(x + h * a.q_head + k.e1);
        }
    int s = t, pos = 0;
    bool rot = a.cos != nullptr;
    if (rot) {
        int b, e;
        if (a.cu != nullptr) {
            int lo = 0, hi = a.seqs;
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                seq_tokens(a.cu, mid, a.tokens, b, e);
                if (b <= t) lo = mid;
                else hi = mid;
            }
            s = lo;
        }
        seq_tokens(a.cu, s, a.tokens, b, e);
        pos = load_index(a.lens + s) - (e - t);
        const bool owned = t >= b && t < e;     // else the token is no sequence's and has no position
        rot = owned && pos >= 0 && pos < a.positions;
        if (owned && pos >= a.positions) atomicOr(a.status, DEV_ERR_BAD_PAGE);
    }
    if (!rot) k.turn = kCopy;       // the same pieces as they are
    Angles g;
    angles_of(a, k, pos, g);
#pragma unroll
    for (int h = 0; h < kHeads; ++h)
        if (h < heads) {
            if (k.turn != kCopy) {
                float v[16];
                turned<BF16>(a, x + h * a.q_head, p0[h], p1[h], k, g, pos, v);
                p0[h] = pack8<BF16>(v);
                p1[h] = pack8<BF16>(v + 8);
            }
            *reinterpret_cast<uint4*>(o + h * a.d + k.e0) = p0[h];
            *reinterpret_cast<uint4*>(o + h * a.d + k.e1) = p1[h];
        }
}

template <bool BF16, int TPU>
cudaError_t launch_t(const KvAppendArgs& a, cudaStream_t stream) {
    const long long units = a.cu != nullptr ? a.tokens / a.page + 2LL * a.seqs : a.seqs;
    const long long items = units * a.heads * a.R * 2, per = kThreads / TPU;
    const long long unit_blocks = (items + per - 1) / per;
    const long long q_tasks = static_cast<long long>(a.tokens) * a.R * ((a.q_heads + kHeads - 1) / kHeads) * (a.d / 16);
    const long long blocks = unit_blocks + (q_tasks + kThreads - 1) / kThreads;
    if (items > 0x7fffffffLL || q_tasks > 0xffffff00LL || blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;    // the caller checks
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_launch() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kv_append_kernel<BF16, TPU>, a, static_cast<int>(items), static_cast<int>(unit_blocks),
                              static_cast<uint32_t>(q_tasks));
}

}  // namespace

// A warp a unit while sequences bring a few tokens on average, else a block.
cudaError_t launch_kv_append(const KvAppendArgs& args, bool bf16, cudaStream_t stream) {
    KvAppendArgs a = args;
    a.vec_angles = a.rot % 8 == 0 && ((reinterpret_cast<uintptr_t>(a.cos) | reinterpret_cast<uintptr_t>(a.sin)) & 15u) == 0;
    const bool warp = a.tokens <= 4LL * a.seqs;
    if (bf16) return warp ? launch_t<true, 32>(a, stream) : launch_t<true, kThreads>(a, stream);
    return warp ? launch_t<false, 32>(a, stream) : launch_t<false, kThreads>(a, stream);
}

}  // namespace coc
