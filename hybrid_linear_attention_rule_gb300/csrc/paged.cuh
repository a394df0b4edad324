// paged.cuh -- the paged key/value cache as the kernels see it (layout: include/k3kda.h).
#pragma once

#include <cuda_fp16.h>

#include "rope.cuh"

namespace k3kda {

constexpr int kStrip = 16;                                     // tokens of a strip
constexpr int kPlaneI4 = 576, kPlaneBf16 = 2048;               // bytes of a plane (16 tokens x 64 channels)

struct Paged {
    char *pool;
    const int32_t *table, *kv_len;
    int num_pages, page_size, max_pages, N, heads, dqk, dv;
    int planes;                                                // (dqk + dv) / 64
    int strip_bytes;
    int64_t block_bytes, page_bytes;                           // of a (page, head), of a page
};

inline Paged make_paged(const k3mla_paged_cache *c) {
    Paged p;
    p.pool = static_cast<char *>(c->pool);
    p.table = c->block_table; p.kv_len = c->kv_len;
    p.num_pages = c->num_pages; p.page_size = c->page_size; p.max_pages = c->max_pages;
    p.N = c->N; p.heads = c->heads; p.dqk = c->dqk; p.dv = c->dv;
    p.planes = (c->dqk + c->dv) / 64;
    p.strip_bytes = p.planes * (c->format == K3MLA_CACHE_I4 ? kPlaneI4 : kPlaneBf16);
    p.block_bytes = (int64_t)p.strip_bytes * (c->page_size / kStrip);
    p.page_bytes = p.block_bytes * c->heads;
    return p;
}

// Length of sequence n, or -1 when it lies outside the table's reach.
__device__ __forceinline__ int paged_len(const Paged &P, int n) {
    const int len = P.kv_len[n];
    return len >= 0 && len <= (int64_t)P.max_pages * P.page_size ? len : -1;
}

// Page number of position pos of sequence n, or -1 when it is outside the pool.
__device__ __forceinline__ int paged_page(const Paged &P, int n, int pos) {
    const int p = P.table[(int64_t)n * P.max_pages + pos / P.page_size];
    return p >= 0 && p < P.num_pages ? p : -1;
}

}  // namespace k3kda
