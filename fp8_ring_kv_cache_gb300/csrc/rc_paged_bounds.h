/* rc_paged_bounds.h -- whether what a paged call reads from device memory is within what the host was told: plain
   integer checks, the same in the kernels and on the host. */
#ifndef RC_PAGED_BOUNDS_H
#define RC_PAGED_BOUNDS_H

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

#endif
