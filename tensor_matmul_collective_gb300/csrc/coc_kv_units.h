// Which new tokens a sequence has, and which page of which sequence a unit of
// the append is: index arithmetic alone, the same on the device and on the host
// (where it is tested over offsets and lengths of every kind).
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define COC_HD __host__ __device__ __forceinline__
#else
#define COC_HD inline
#endif

namespace coc {
namespace {

// (On the device not by __ldg: these kernels begin while the one that writes the
// array may still run, and a load from memory that is said to be read-only need
// not stay behind the wait for it.)
COC_HD int load_index(const int32_t* p) {
#ifdef __CUDA_ARCH__
    int v;
    asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
#else
    return *p;
#endif
}

// First and one-past-last new token of sequence s (cu NULL: one token each).
// Offsets outside [0, tokens] or descending are clamped, so that no lookup
// leaves the caller's buffers whatever the device array holds.
COC_HD void seq_tokens(const int32_t* cu, int s, int tokens, int& begin, int& end) {
    if (cu == nullptr) {
        begin = s;
        end = s + 1;
        return;
    }
    begin = load_index(cu + s);
    begin = begin < 0 ? 0 : begin > tokens ? tokens : begin;
    end = load_index(cu + s + 1);
    end = end < begin ? begin : end > tokens ? tokens : end;
}

// A page that receives new tokens: the new positions [first, last) of sequence
// s, whose token at position p is the new token p + token.
struct AppendUnit {
    int s, page;            // sequence, and the page's place in it
    int start;              // the page's first position
    int first, last;
    int token;
};

// Unit `unit` of tokens / page + 2 seqs (cu NULL: of seqs), false where there
// is none.  Sequence s has the units from cu[s] / page + 2 s on: n tokens touch
// at most n / page + 2 pages, so that no two sequences share one.  Units ahead of
// the first sequence's belong to nobody: there are some where cu[0] >= page.
COC_HD bool append_unit_of(const int32_t* cu, const int32_t* lens, int seqs, int tokens, int page, int unit, AppendUnit& u) {
    u.s = unit;
    if (cu != nullptr) {        // the last s whose first unit is <= unit (0 if none is)
        int lo = 0, hi = seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            int b, e;
            seq_tokens(cu, mid, tokens, b, e);
            if (b / page + 2 * mid <= unit) lo = mid;
            else hi = mid;
        }
        u.s = lo;
    }
    int begin, end;
    seq_tokens(cu, u.s, tokens, begin, end);
    const int n = end - begin, len = load_index(lens + u.s);
    const int after = cu != nullptr ? unit - (begin / page + 2 * u.s) : 0;      // pages after the sequence's first touched
    if (n <= 0 || len <= 0 || after < 0) return false;
    const int past = len - n;
    u.page = (past > 0 ? past : 0) / page + after;
    if (u.page > (len - 1) / page) return false;
    u.start = u.page * page;
    u.first = past > u.start ? past : u.start;
    u.last = len - u.start > page ? u.start + page : len;
    u.token = begin - past;
    return true;
}

}  // namespace
}  // namespace coc
