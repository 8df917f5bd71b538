// The paged cache's parameter blocks and address arithmetic, shared by the
// insertion, eviction and attention kernels.
#pragma once

#include "rotary.cuh"

namespace tc {

struct CacheParams {
    void *k, *v;
    float *mass;
    int32_t *pos;
    const int32_t *table;
    int64_t *len, *clock;
    float *A;
    const float *lam, *eta;
    int B, H, page, n_pages, max_pages;
    int *status;
    uint64_t page_mul;  // ceil(2^40 / page): slot / page = slot * page_mul >> 40 for slots below 2^24

    __host__ __device__ int64_t capacity() const { return (int64_t)max_pages * page; }
    __device__ __forceinline__ int page_of(int slot) const { return (int)(((uint64_t)slot * page_mul) >> 40); }
};

// Room for a row's pairs: the capacity in whole words of a bit each.
__host__ __device__ inline int pairs_room(int64_t capacity) { return (int)((capacity + 31) / 32 * 32); }

// Row (of d elements) of slot s, head h, in the pools: page pg is valid.
__device__ __forceinline__ int64_t pool_row(const CacheParams &c, int pg, int h, int in_page) {
    return ((int64_t)pg * c.H + h) * c.page + in_page;
}
__device__ __forceinline__ bool page_ok(const CacheParams &c, int pg) { return pg >= 0 && pg < c.n_pages; }

// Block-wide: whether every table entry for the slots first .. last of row b
// (last < capacity) names a page of the pool.
__device__ __forceinline__ bool block_pages_ok(const CacheParams &c, int b, int64_t first, int64_t last) {
    int bad = 0;
    if (last >= first)
        for (int64_t i = first / c.page + threadIdx.x; i <= last / c.page; i += blockDim.x)
            bad |= !page_ok(c, c.table[(int64_t)b * c.max_pages + i]);
    return __syncthreads_or(bad) == 0;
}

struct AppendParams {
    CacheParams c;
    const void *q, *k, *v;
    void *q_out;
    const int64_t *counts;
    const float *mass_in;
    int64_t T;
    int Hq, d;
    int64_t qs[3], ks[3], vs[3];
    RotaryTable table;
};
cudaError_t launch_cache_append(const AppendParams &p, tc_dtype dtype, cudaStream_t s);

struct EvictParams {
    CacheParams c;
    int64_t budget, recent;
    int64_t *row_len;        // [B] -1: skipped; a step: what the row holds afterwards;
                             // an eviction: what it held before
    unsigned char *sort_ws;  // rows that do not fit shared memory; else null
    // tc_cache_step: the new token (one per row) and the queries
    const void *q, *k_new, *v_new;
    int64_t qs[2], ks[2], vs[2];  // strides of b, h
    void *q_rot;             // [B,Hq,d] rotated queries
    float *memo;             // [B,H,slices,G,d] q A by slices of A's rows; null: no read
    int Hq;
    RotaryTable table;
};
// Blocks a head's A is cut over in a step's first kernel (and p.memo's slices).
int evict_slices(int64_t BH, int d, int num_sms);
size_t evict_sort_bytes(int64_t BH, int d, int64_t capacity, int num_sms);
// The new token enters, at most one pair leaves, the queries read A; lengths and
// clocks are left to the attention's join.
cudaError_t launch_cache_step_insert(const EvictParams &p, tc_dtype dtype, int d, int slices, cudaStream_t s);
cudaError_t launch_cache_evict(const EvictParams &p, tc_dtype dtype, int d, int num_sms, cudaStream_t s);

struct AttendParams {
    CacheParams c;
    const void *q;
    void *y;
    const float *g;          // null: no memory read
    const int64_t *row_len;  // pairs to attend to, per row (c.len, or a step's own)
    const float *memo;       // q A already formed, in `slices` parts; null: the join forms it
    int slices;
    bool step;               // the join also stores row_len to c.len and advances c.clock
    int Hq, G, d;
    int heads;               // query heads one work item covers
    int items;               // work items a row and key/value head has
    int *prefix;             // [B+1] tiles before each row
    float *part;             // partial results, one per (block, item) met
    float *z;                // scaled scores [n_pages,H,page,G]; null: weights are not kept
    unsigned long long wait_ns;
};
int attend_heads_per_item(int G, tc_dtype dtype);
int attend_grid(int num_sms);
size_t attend_part_bytes(int64_t BH, int G, int d, tc_dtype dtype, int num_sms);
bool attend_supported(int d);
// Units of work (tiles) at most, for the limit of 31 bits.
double attend_units(double items, int64_t capacity);
cudaError_t launch_cache_attend(const AttendParams &p, tc_dtype dtype, int num_sms, cudaStream_t s);

// Lets a kernel use this much dynamic shared memory.  Below 16 KB it needs no
// leave: with the static arrays (at most 32 KB) it stays within the 48 KB every
// kernel may use.
template <typename K>
inline cudaError_t allow_smem(K kernel, size_t bytes) {
    return bytes < 16 * 1024 ? cudaSuccess
                              : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

}  // namespace tc
