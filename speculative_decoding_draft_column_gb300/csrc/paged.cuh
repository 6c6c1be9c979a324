// The paged key/value cache's bookkeeping: the plan of a step (block tables,
// positions and slots from the lanes' lengths) and the store of new keys and
// values into their slots.
#pragma once

#include "common.cuh"

namespace paged {

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;

inline size_t plan_smem(int64_t lanes) { return (size_t)(2 * (lanes + 1) * 8 + 3 * lanes * 4); }

struct PlanArgs {
    spec_paged_batch b;
    const int32_t *free_pages;
    int64_t num_free;
    const int32_t *cursor;
};

// What a lane needs: its new tokens and the pages it wants beyond those held.
struct LaneNeed {
    int64_t ctx, n, need;   // need: pages for ctx + n tokens, of any number
    int64_t held, want;     // want: pages to add, within the table row
};

__device__ __forceinline__ LaneNeed lane_need(const spec_paged_batch &b, int lane)
{
    LaneNeed r;
    const int32_t c = __ldg(b.context_lens + lane), n = __ldg(b.new_lens + lane), h = __ldg(b.held + lane);
    r.ctx = c > 0 ? c : 0;
    r.n = n > 0 ? n : 0;
    r.need = udiv(r.ctx + r.n + b.page_size - 1, b.page_size);
    r.held = h < 0 ? 0 : h > b.max_pages ? b.max_pages : h;
    const int64_t most = r.need < b.max_pages ? r.need : b.max_pages;
    r.want = most > r.held ? most - r.held : 0;
    return r;
}

__device__ __forceinline__ int64_t warp_inclusive_sum64(int64_t v, int lane)
{
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, v, d);
        if (lane >= d) v += y;
    }
    return v;
}

// Every CTA scans all lanes' lengths (a few KB, from L2) into shared memory and
// then writes its share of the lanes' and the tokens' outputs: one launch, no
// exchange between CTAs.  The step is bound by that chain of dependent reads
// (lengths, scan, table), not by its bytes: 2.8 us for 8 lanes of 8 tokens, 7.1 us for
// 1,024 lanes with 262,144 new tokens (3.4 MB).
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    // [lanes + 1] new tokens, then [lanes + 1] wanted pages, before each lane;
    // [lanes] each: cached tokens, pages held before, pages held after
    extern __shared__ int64_t sums[];
    __shared__ int64_t warp_n[kPlanWarps], warp_w[kPlanWarps];
    __shared__ int over_lanes;
    const spec_paged_batch &b = a.b;
    const int lanes = (int)b.lanes, tid = threadIdx.x, wl = tid & 31, wid = tid >> 5;
    int64_t *cu = sums, *cw = sums + lanes + 1;
    int32_t *ctx = reinterpret_cast<int32_t *>(cw + lanes + 1), *had = ctx + lanes, *has = had + lanes;
    if (tid == 0) over_lanes = 0;
    __syncthreads();

    const int per = (lanes + kPlanThreads - 1) / kPlanThreads;
    const int l0 = tid * per < lanes ? tid * per : lanes, l1 = l0 + per < lanes ? l0 + per : lanes;
    int64_t sn = 0, sw = 0;
    int over = 0;
    for (int l = l0; l < l1; ++l) {
        const LaneNeed r = lane_need(b, l);
        cu[l] = sn;
        cw[l] = sw;
        ctx[l] = (int32_t)r.ctx;
        had[l] = (int32_t)r.held;
        has[l] = (int32_t)r.want;       // until the free pages are shared out
        sn += r.n;
        sw += r.want;
        over += r.need > b.max_pages;
    }
    const int64_t in = warp_inclusive_sum64(sn, wl), iw = warp_inclusive_sum64(sw, wl);
    if (wl == 31) { warp_n[wid] = in; warp_w[wid] = iw; }
    if (over) atomicAdd(&over_lanes, over);
    __syncthreads();
    int64_t bn = in - sn, bw = iw - sw;
    for (int w = 0; w < wid; ++w) { bn += warp_n[w]; bw += warp_w[w]; }
    for (int l = l0; l < l1; ++l) {
        cu[l] += bn;
        cw[l] += bw;
    }
    if (tid == kPlanThreads - 1) {
        cu[lanes] = bn + sn;
        cw[lanes] = bw + sw;
    }
    __syncthreads();
    const int64_t total = cu[lanes], wanted = cw[lanes];
    int64_t cursor = a.cursor ? __ldg(a.cursor) : 0;
    cursor = cursor < 0 ? 0 : cursor > a.num_free ? a.num_free : cursor;
    const int64_t avail = a.num_free - cursor;
    for (int l = tid; l < lanes; l += kPlanThreads) {
        const int64_t left = avail - cw[l], want = has[l];
        has[l] = had[l] + (int32_t)(left < 0 ? 0 : left < want ? left : want);
    }
    __syncthreads();

    // lanes: one warp each, in turn
    for (int l = blockIdx.x * kPlanWarps + wid; l < lanes; l += gridDim.x * kPlanWarps) {
        const int held = had[l], got = has[l] - held;
        int32_t *row = b.block_table + (int64_t)l * b.max_pages + held;
        const int32_t *src = a.free_pages + cursor + cw[l];
        for (int i = wl; i < got; i += 32) row[i] = __ldg(src + i);
        if (wl == 0) {
            b.cu_new[l] = (int32_t)cu[l];
            b.seq_lens[l] = (int32_t)(ctx[l] + (cu[l + 1] - cu[l]));
            b.held_out[l] = held + got;
        }
    }
    if (blockIdx.x == 0 && tid == 0) {
        b.cu_new[lanes] = (int32_t)total;
        b.info[0] = (int32_t)total;
        b.info[1] = (int32_t)(cursor + (wanted < avail ? wanted : avail));
        b.info[2] = (int32_t)(wanted > avail ? wanted - avail : 0);
        b.info[3] = over_lanes;
    }

    // tokens: the lane by bisection, the page from the table or, if the step
    // adds it, from the free list (another CTA may be writing the table entry);
    // kAhead tokens of a thread on their way together
    constexpr int kAhead = 4;
    const int64_t stride = (int64_t)gridDim.x * kPlanThreads;
    for (int64_t t0 = (int64_t)blockIdx.x * kPlanThreads + tid; t0 < b.tokens; t0 += kAhead * stride) {
        int32_t pos[kAhead], in[kAhead], id[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t t = t0 + u * stride;
            pos[u] = in[u] = 0;
            id[u] = -1;
            if (t >= total || t >= b.tokens) continue;
            int lo = 0, hi = lanes - 1;   // the last lane with cu <= t
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (cu[mid] <= t) lo = mid; else hi = mid - 1;
            }
            const int64_t p = ctx[lo] + (t - cu[lo]), page = udiv(p, b.page_size);
            pos[u] = (int32_t)p;
            in[u] = (int32_t)(p - page * b.page_size);
            if (page < had[lo]) id[u] = b.block_table[(int64_t)lo * b.max_pages + page];
            else if (page < has[lo]) id[u] = __ldg(a.free_pages + cursor + cw[lo] + (page - had[lo]));
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t t = t0 + u * stride;
            if (t >= b.tokens) continue;
            b.positions[t] = pos[u];
            b.slots[t] = id[u] < 0 ? -1 : (int64_t)id[u] * b.page_size + in[u];
        }
    }
}

struct StoreArgs {
    const uint16_t *k, *v;
    int64_t tokens, ks_t, ks_h, vs_t, vs_h;
    const int64_t *slots;
    spec_paged_cache c;
};

constexpr int kStoreThreads = 256;

// A copy bound by its bytes: 16-byte vectors, consecutive threads on
// consecutive vectors of a token's heads.  16,384 tokens of 8 heads of 128: 19.1 us, 0.97
// of a measured copy.
__global__ void __launch_bounds__(kStoreThreads) store_kernel(const __grid_constant__ StoreArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int vh = a.c.head_dim / 8, vt = vh * a.c.heads;   // vectors of a head, of a token
    const int64_t nv = a.tokens * vt, limit = a.c.pages * a.c.page_size;
    for (int64_t i = (int64_t)blockIdx.x * kStoreThreads + threadIdx.x; i < nv; i += (int64_t)gridDim.x * kStoreThreads) {
        const int64_t t = udiv(i, vt);
        const int r = (int)(i - t * vt), h = r / vh, e = (r - h * vh) * 8;
        const int64_t slot = __ldg(a.slots + t);
        if (slot < 0 || slot >= limit) continue;
        const int64_t page = udiv(slot, a.c.page_size), in = slot - page * a.c.page_size;
        const uint4 kv = __ldg(reinterpret_cast<const uint4 *>(a.k + t * a.ks_t + h * a.ks_h + e));
        const uint4 vv = __ldg(reinterpret_cast<const uint4 *>(a.v + t * a.vs_t + h * a.vs_h + e));
        uint16_t *kd = static_cast<uint16_t *>(a.c.k) + page * a.c.k_strides[0] + in * a.c.k_strides[1] +
                       h * a.c.k_strides[2] + e;
        uint16_t *vd = static_cast<uint16_t *>(a.c.v) + page * a.c.v_strides[0] + in * a.c.v_strides[1] +
                       h * a.c.v_strides[2] + e;
        *reinterpret_cast<uint4 *>(kd) = kv;
        *reinterpret_cast<uint4 *>(vd) = vv;
    }
}

}  // namespace paged
