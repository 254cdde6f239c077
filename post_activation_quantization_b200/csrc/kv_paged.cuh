// kv_paged.cuh -- the paged packed K/V cache as its kernels see it.
//
// A position p of sequence b lives in page table[b][p / P], slot p % P (P a power of two); a pool is
// [n_pages, H, P, D*BITS/8] bytes, so the P rows of one (page, head) are contiguous.  A ragged batch of
// token rows belongs to the sequences by start[0..B]: rows start[b] .. start[b + 1] - 1 are the newest
// positions of sequence b, whose length lens[b] counts them.
#pragma once

#include "common.cuh"

namespace rptq {

struct Paged {
    const int32_t *start, *lens, *table;
    int B, max_pages, shift;  // P = 1 << shift
    int64_t n_pages, T;
    int max_q, max_len;
    int *err;
};

// Rows [s0, s0 + n) and length L of sequence b.  False (the sequence is left out) where the device
// tables contradict the call's sizes.
__device__ __forceinline__ bool paged_sequence(const Paged &p, int b, int &s0, int &n, int &L)
{
    s0 = p.start[b];
    const int s1 = p.start[b + 1];
    L = p.lens[b];
    const bool ok = s0 >= 0 && s1 >= s0 && s1 <= p.T && L >= 0 && L <= p.max_len && s1 - s0 <= p.max_q;
    n = s1 - s0;
    if (!ok) raise_error(p.err, RPTQ_DEVERR_RANGE);
    return ok;
}

// The sequence that holds row t: the largest b with start[b] <= t (rows of empty sequences belong to
// none).  -1 for a row before the first sequence, or behind the last.  The tables are not trusted: the
// caller checks the row against the sequence it gets.
__device__ __forceinline__ int paged_row_sequence(const Paged &p, int64_t t)
{
    int lo = 0, hi = p.B;  // start[lo] <= t < start[hi] once found
    if (t < p.start[0] || t >= p.start[p.B]) return -1;
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (p.start[m] <= t)
            lo = m;
        else
            hi = m;
    }
    return t >= p.start[lo] && t < p.start[lo + 1] ? lo : -1;
}

// Page id of page number pg of sequence b; -1 (reported) outside the pool.
__device__ __forceinline__ int paged_page(const Paged &p, int b, int pg)
{
    const int id = p.table[(int64_t)b * p.max_pages + pg];
    if (id >= 0 && id < p.n_pages) return id;
    raise_error(p.err, RPTQ_DEVERR_PAGE);
    return -1;
}

// First row of (page, head) in units of rows.
__device__ __forceinline__ int64_t paged_row(int page, int H, int h, int shift)
{
    return ((int64_t)page * H + h) << shift;
}

}  // namespace rptq
