/* rc_paged_bounds.h -- whether what a paged call reads from device memory is within what the host was told: plain
   integer checks, the same in the kernels and on the host. */
#ifndef RC_PAGED_BOUNDS_H
#define RC_PAGED_BOUNDS_H
#include <stdint.h>

#ifdef __CUDACC__
#define RC_BOTH __host__ __device__ __forceinline__
#else
#define RC_BOTH static inline
#endif

/* kv cached tokens, query rows [q0, end) of `tokens`, at most max_new of them and max_kv cached tokens. */
RC_BOTH bool paged_seq_ok(int kv, int q0, int end, int tokens, int max_new, int max_kv) {
    /* (end - q0 cannot overflow once 0 <= q0 <= end) */
    return kv >= 0 && kv <= max_kv && q0 >= 0 && end >= q0 && end <= tokens && end - q0 <= max_new;
}

RC_BOTH bool paged_len_ok(int kv, int max_kv) { return kv >= 0 && kv <= max_kv; }

RC_BOTH bool paged_page_ok(int page, int pages) { return page >= 0 && page < pages; }

/* Whether a byte lies in a row of each of two sets of rows (host): na rows of wa bytes, sa bytes apart, from address a;
   nb rows of wb bytes, sb apart, from b.  Counts and widths >= 1, sa >= wa, sb >= wb. */
static inline int paged_rows_meet(uint64_t a, int64_t sa, int64_t na, int64_t wa, uint64_t b, int64_t sb, int64_t nb,
                                  int64_t wb) {
    const __int128 d = (__int128)b - (__int128)a;
    if (d >= (__int128)(na - 1) * sa + wa || -d >= (__int128)(nb - 1) * sb + wb) return 0;
    if (na == 1 || nb == 1 || sa == sb) {
        /* row j of the second begins d + (j - i) s behind row i of the first, and must begin less than wa behind it:
           the largest j - i for which it does */
        const __int128 s = na == 1 ? sb : sa, top = wa - 1 - d;
        __int128 k = top >= 0 ? top / s : -((-top + s - 1) / s);
        if (k > nb - 1) k = nb - 1;
        return k >= -(__int128)(na - 1) && d + k * s + wb > 0;
    }
    for (int64_t i = 0; i < na; ++i) {
        const __int128 at = (__int128)i * sa - d; /* row i of the first, counted from b */
        if (at + wa <= 0) continue;
        __int128 j = (at + wa - 1) / sb;
        if (j > nb - 1) j = nb - 1;
        if (j * sb + wb > at) return 1;
    }
    return 0;
}

#endif
