// Append to the paged 8-bit key/value cache: rotation of q and k by position,
// quantisation of k and v to e4m3 with one scale per (page, head).
#include "coc_kv.cuh"

namespace coc {
namespace {

// Value e of a head of `x` (d values) rotated by the token's row of the
// tables: every product and sum rounded on its own (no fused multiply-add),
// so that a result does not depend on how a compiler contracts it.
template <bool BF16>
__device__ __forceinline__ float rotated(const KvAppendArgs& a, const uint16_t* x, int e, int pos) {
    const float v = to_float16bit<BF16>(x[e]);
    if (e >= a.rot) return v;
    const int half = a.rot / 2;
    const int j = a.interleaved ? e / 2 : (e < half ? e : e - half);
    const bool first = a.interleaved ? (e & 1) == 0 : e < half;
    const int pe = a.interleaved ? (e ^ 1) : (first ? e + half : e - half);
    const float w = to_float16bit<BF16>(x[pe]);
    const float c = __ldg(a.cos + static_cast<long long>(pos) * half + j);
    const float s = __ldg(a.sin + static_cast<long long>(pos) * half + j);
    return first ? __fsub_rn(__fmul_rn(v, c), __fmul_rn(w, s)) : __fadd_rn(__fmul_rn(v, c), __fmul_rn(w, s));
}

// Block (unit, head, 2 x rank + {0: k, 1: v}).  Sequence s owns the units
// [cu[s] / page + 2 s, cu[s + 1] / page + 2 (s + 1)), at least as many as the
// pages its new tokens touch; unit i of it is the i-th such page.
template <bool BF16>
__global__ void __launch_bounds__(128) kv_append_kernel(const __grid_constant__ KvAppendArgs a) {
    __shared__ float red[4];
    const int unit = blockIdx.x, h = blockIdx.y, r = blockIdx.z >> 1, which = blockIdx.z & 1;
    int lo = 0, hi = a.seqs;   // the last s whose first unit is <= unit
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        int b, e;
        seq_tokens(a.cu, mid, a.tokens, b, e);
        if (b / a.page + 2 * mid <= unit) lo = mid;
        else hi = mid;
    }
    const int s = lo;
    int begin, end;
    seq_tokens(a.cu, s, a.tokens, begin, end);
    const int n = end - begin;
    const int len = __ldg(a.lens + s);
    const int past = len - n;
    const int p0 = max(past, 0) / a.page + (unit - (begin / a.page + 2 * s));   // this unit's page of the sequence
    if (n <= 0 || len <= 0 || p0 > (len - 1) / a.page) return;
    int page_id = -1;
    if (p0 < a.table_width) page_id = __ldg(a.table + static_cast<long long>(s) * a.table_width + p0);
    if (page_id < 0 || page_id >= a.pages) {
        if (threadIdx.x == 0) atomicOr(a.status, DEV_ERR_BAD_PAGE);
        return;
    }
    const int start = p0 * a.page;
    const int first = max(past, start), last = min(len, start + a.page);   // new positions in this page
    const bool rot = which == 0 && a.cos != nullptr;
    if (rot && last > a.positions) {
        if (threadIdx.x == 0) atomicOr(a.status, DEV_ERR_BAD_PAGE);
        return;
    }
    const uint16_t* src = which ? a.v[r] : a.k[r];
    const long long ts = which ? a.v_token : a.k_token, hs = which ? a.v_head : a.k_head;
    uint8_t* codes = (which ? a.cv[r] : a.ck[r]) + (static_cast<long long>(page_id) * a.heads + h) * a.page * a.d;
    float* scale = (which ? a.sv[r] : a.sk[r]) + static_cast<long long>(page_id) * a.heads + h;

    float amax = 0.f;
    for (int i = threadIdx.x; i < (last - first) * a.d; i += blockDim.x) {
        const int p = first + i / a.d, e = i % a.d;
        const uint16_t* x = src + (begin + p - past) * ts + h * hs;
        const float v = fabsf(rot ? rotated<BF16>(a, x, e, p) : to_float16bit<BF16>(x[e]));
        if (v <= 3.4028235e38f) amax = fmaxf(amax, v);   // NaN and infinities take no part
    }
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
    __syncthreads();
    amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float old = first > start ? *scale : 0.f;
    const float now = fmaxf(scale_for(amax), old);
    __syncthreads();
    if (threadIdx.x == 0) *scale = now;
    const float inv = __frcp_rn(now);
    if (first > start && now != old) {
        const float f = __fmul_rn(old, inv);
        for (int i = threadIdx.x; i < (first - start) * a.d; i += blockDim.x) {
            const __half_raw hr = __nv_cvt_fp8_to_halfraw(codes[i], __NV_E4M3);
            codes[i] = __nv_cvt_float_to_fp8(__fmul_rn(__half2float(__half(hr)), f), __NV_SATFINITE, __NV_E4M3);
        }
    }
    for (int i = threadIdx.x; i < (last - first) * a.d; i += blockDim.x) {
        const int p = first + i / a.d, e = i % a.d;
        const uint16_t* x = src + (begin + p - past) * ts + h * hs;
        const float v = rot ? rotated<BF16>(a, x, e, p) : to_float16bit<BF16>(x[e]);
        codes[(p - start) * a.d + e] = __nv_cvt_float_to_fp8(__fmul_rn(v, inv), __NV_SATFINITE, __NV_E4M3);
    }
}

// Block (token, head, rank): q rotated into q_out.
template <bool BF16>
__global__ void __launch_bounds__(64) q_rotate_kernel(const __grid_constant__ KvAppendArgs a) {
    const int t = blockIdx.x, h = blockIdx.y, r = blockIdx.z;
    int lo = 0, hi = a.seqs, b, e;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        seq_tokens(a.cu, mid, a.tokens, b, e);
        if (b <= t) lo = mid;
        else hi = mid;
    }
    seq_tokens(a.cu, lo, a.tokens, b, e);
    const int pos = __ldg(a.lens + lo) - (e - t);
    const bool in = t >= b && t < e && pos >= 0 && (a.cos == nullptr || pos < a.positions);
    if (!in && pos >= 0 && threadIdx.x == 0) atomicOr(a.status, DEV_ERR_BAD_PAGE);
    const uint16_t* x = a.q[r] + t * a.q_token + h * a.q_head;
    uint16_t* o = a.q_out[r] + (static_cast<long long>(t) * a.q_heads + h) * a.d;
    for (int i = threadIdx.x; i < a.d; i += blockDim.x) o[i] = in && a.cos != nullptr ? from_float16bit<BF16>(rotated<BF16>(a, x, i, pos)) : x[i];
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, bool bf16, cudaStream_t stream) {
    const unsigned units = static_cast<unsigned>(a.tokens / a.page + 2 * a.seqs);
    const dim3 g(units, static_cast<unsigned>(a.heads), static_cast<unsigned>(2 * a.R));
    if (bf16) kv_append_kernel<true><<<g, 128, 0, stream>>>(a);
    else kv_append_kernel<false><<<g, 128, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || a.q_heads == 0) return e;
    const dim3 gq(static_cast<unsigned>(a.tokens), static_cast<unsigned>(a.q_heads), static_cast<unsigned>(a.R));
    if (bf16) q_rotate_kernel<true><<<gq, 64, 0, stream>>>(a);
    else q_rotate_kernel<false><<<gq, 64, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace coc
