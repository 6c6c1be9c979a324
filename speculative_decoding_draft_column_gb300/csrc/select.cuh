// Pieces of the selection in a column that the group-maxima kernel and the verify of trees share:
// bounds from maxima, elements of a vector, list entries, and clusters of CTAs.
#pragma once

#include "common.cuh"

namespace gm {

__device__ __forceinline__ uint32_t key_of(uint32_t m2) { return order_key(hmax_splat(m2) & 0xFFFFu); }

// The largest T such that at least kk of the 64 values {v0, v1 of every
// lane} reach T (the kk-th largest; 1 <= kk <= 64): a bisection between the
// smallest and the largest value, in every lane of the warp (the values
// cluster: a few steps).
__device__ __forceinline__ uint32_t kth_of_64(uint32_t v0, uint32_t v1, int kk)
{
    uint32_t lo = __reduce_min_sync(kFull, v0 < v1 ? v0 : v1);   // all 64 reach it
    uint32_t hi = __reduce_max_sync(kFull, v0 > v1 ? v0 : v1);
    if (kk == 1) return hi;
    while (lo < hi) {
        const uint32_t mid = (lo + hi + 1) >> 1;
        const int n = __popc(__ballot_sync(kFull, v0 >= mid)) + __popc(__ballot_sync(kFull, v1 >= mid));
        if (n >= kk) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The kk-th largest of the n values v[0 .. n) (n a multiple of 32, at most
// 512), in every lane of the warp: a bisection between the smallest and the
// largest.  For kk above 8, where 64 section maxima bound too loosely.
__device__ __forceinline__ uint32_t kth_of_smem(const uint32_t *v, int n, int kk, int lane)
{
    uint32_t x[16];
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        x[i] = i * 32 < n ? v[i * 32 + lane] : 0u;
        if (i * 32 < n) {
            lo = x[i] < lo ? x[i] : lo;
            hi = x[i] > hi ? x[i] : hi;
        }
    }
    lo = __reduce_min_sync(kFull, lo);   // all n values reach it
    hi = __reduce_max_sync(kFull, hi);
    while (lo < hi) {
        const uint32_t mid = (lo + hi + 1) >> 1;
        uint32_t cnt = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) cnt += (i * 32 < n && x[i] >= mid) ? 1u : 0u;
        if ((int)__reduce_add_sync(kFull, cnt) >= kk) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// What phase 2's rare paths need of a run, passed by value (a GmRun passed
// by reference would have to live in local memory).
struct RunView {
    const uint16_t *buf;
    const uint4 *vb;
    const int32_t *id_map;
    int64_t jlo, jhi;
    int mis, kk;
};

// Vector j restricted to column [cb, ce): elements outside it (or outside
// the buffer) as NaN.
__device__ __forceinline__ uint4 load_col_vec(const RunView &v, int64_t j, int64_t cb, int64_t ce)
{
    const int64_t g0 = 8 * j - v.mis;
    if (j >= v.jlo && j < v.jhi && g0 >= cb && g0 + 8 <= ce) return __ldg(v.vb + j);
    return load_edge(v.buf, j, v.mis, cb, ce);
}

__device__ __forceinline__ uint32_t half_of(const uint4 &q, int e)
{
    const uint32_t w = (e & 4) ? ((e & 2) ? q.w : q.z) : ((e & 2) ? q.y : q.x);
    return (e & 1) ? (w >> 16) : (w & 0xFFFFu);
}

// Vector u of a thread's registers, u not known at compile time (selects:
// a short, branch-free sequence instead of a copy of the caller's code per
// vector).
template <int L>
__device__ __forceinline__ uint4 pick(const uint4 (&q)[L], int u)
{
    uint4 v = q[0];
#pragma unroll
    for (int i = 1; i < L; ++i)
        if (i == u) v = q[i];
    return v;
}

__device__ __forceinline__ unsigned long long make_entry(uint32_t key, uint32_t id, uint32_t raw)
{
    return ((unsigned long long)key << 48) | ((unsigned long long)(~id) << 16) | raw;
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// the address of this CTA's shared variable p in the CTA of the given rank
__device__ __forceinline__ uint32_t cluster_map(const void *p, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, unsigned long long v)
{
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

}  // namespace gm
