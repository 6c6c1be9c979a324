// Verify of trees of drafts: a walk from the anchor along the drafts that the target
// agrees with, one column of target logits a step.
//
// A lane reads the columns of its path, a + 1 of them, and no others: of 64 nodes of a
// tree some 4.  A column is shared by the CTAs of a thread-block cluster: each holds its
// part in registers, selects the part's k best (k = 1: the argmax), and stores them
// into the shared memory of every CTA of the cluster, so that behind one cluster barrier
// each merges the lists and takes the same decision by itself: nothing has to be sent back before
// the next column's loads begin.  The lists lie in two inboxes in turn: a CTA writes the
// next-but-one only past a barrier that all pass after they have read this one.
//
// Where there are so few nodes that all their columns are on the GPU at once, a cluster takes a
// column of its own instead (kWide), leaves its list in scratch, and the lane's last cluster
// walks over the lists: one column's time whatever the depth.
//
// The bound of a part's selection: the k-th largest of 64 maxima, each over the elements of 8 threads
// (of 512, a thread each, for k above 32); k elements reach it, and few more do.
// Should many (ties), a bisection over values and then places finds exactly the k best.
//
// What bounds it is the chain of a column, not its bytes: 13,000 cycles, of which the load takes 2,100, bound and
// candidates 3,300, their ranks 1,100, the exchange 1,500, the merge 1,600, matching and decision 3,500.  8 trees of
// 64 nodes over 248,046 tokens 31.7 us, 64 of 8 to 32 nodes 58 (78 MB: 11.5 at the copy's rate), 16 nodes
// greedy, all columns at once, 10.2.  (One thread an entry: the merge 4,900 cycles, lists on the same
// banks; decisions left to FP64 within 5e-4 instead of 5e-5 of a border: 5,000.)
#pragma once

#include "select.cuh"
#include "tree.cuh"

namespace tree {

constexpr int kThreads = 512;
constexpr int kLoads = 8;                        // 16-byte vectors of a thread
constexpr int kPart = kThreads * kLoads;         // vectors of a part at a time
constexpr int kMostCtas = 8;                     // of a cluster
constexpr int kCand = 1024;                      // candidates of a part
constexpr int kInbox = SPEC_MAX_K + 1;           // (the lists' entries of one place on different banks)

struct VerifyArgs {
    const uint16_t *logits;
    const int32_t *drafts, *parents, *cu;
    int64_t tokens, lanes, V;
    int32_t depth, k;
    double temperature, top_p;
    float inv_temperature, top_p_single;         // (no FP64 division on the walk)
    const double *uniforms;                      // null: greedy
    int32_t *accept, *commit, *path;
    unsigned long long *lists;                   // kWide: [tokens][k]
    unsigned int *tickets;                       // kWide: [lanes], zero between calls
};

struct VerifySmem {
    unsigned long long cand[kCand + SPEC_MAX_K];
    unsigned long long inbox[2][kMostCtas][kInbox];
    unsigned long long list[SPEC_MAX_K];         // a part's list, then the column's
    double2 uniform[kNodes];
    int32_t parent[kNodes], token[kNodes];
    uint32_t hits[kNodes / 32];                  // children of the walk's node whose tokens are in its list,
    int32_t place[kNodes];                       // and where
    uint32_t top[kThreads];                      // the threads' maxima
    uint32_t sec[64];                            // of 8 threads each
    uint32_t ncand, first, count;
    int32_t next, chosen;                        // the decision: the accepted child (-1: none) and the token
    int32_t lane, n;
    int64_t row0;
};

// ---- a column's k best ----------------------------------------------------------

// A piece of a column: vectors [jb, j1), at most kPart of them (vector j: elements [8j - mis, 8j - mis + 8) of the
// logits), of which those outside [cb, ce) are not the column's.
struct Piece {
    const uint16_t *logits;
    const uint4 *vb;
    int mis;
    int64_t jb, j1, cb, ce;
};

// f(key, place, raw) for each element of the piece that is this thread's, read again (from L2).
template <typename F>
__device__ __forceinline__ void each_element(const Piece &p, F f)
{
    const gm::RunView v = {p.logits, p.vb, nullptr, (p.cb + p.mis + 7) >> 3, (p.ce + p.mis) >> 3, p.mis, 0};
#pragma unroll 1
    for (int64_t j = p.jb + threadIdx.x; j < p.j1 && j < p.jb + kPart; j += kThreads) {
        const uint4 q = gm::load_col_vec(v, j, p.cb, p.ce);
#pragma unroll 1
        for (int e = 0; e < 8; ++e) {
            const uint32_t raw = gm::half_of(q, e), key = order_key(raw);
            if (key) f(key, (uint32_t)(8 * (j - p.jb) + e), raw);
        }
    }
}

// The number of the piece's elements up to (key0, place0) in the order of the list (larger
// keys first, then smaller places).
__device__ __forceinline__ uint32_t count_upto(const Piece &p, uint32_t key0, uint32_t place0, VerifySmem &s)
{
    uint32_t n = 0;
    each_element(p, [&](uint32_t key, uint32_t place, uint32_t) { n += key > key0 || (key == key0 && place <= place0); });
    n = __reduce_add_sync(kFull, n);
    if (threadIdx.x == 0) s.count = 0u;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) atomicAdd(&s.count, n);
    __syncthreads();
    n = s.count;
    __syncthreads();
    return n;
}

// More candidates than the buffer holds (ties): the k-th best by bisection, over the keys
// and then over the places of those at the k-th key; then exactly k are candidates.  T: a key that k
// elements reach.
__device__ __noinline__ void exact_candidates(const Piece p, int k, uint32_t T, uint32_t id0, VerifySmem &s)
{
    uint32_t lo = T, hi = 0xFFFFu;
    while (lo < hi) {
        const uint32_t mid = (lo + hi + 1) >> 1;
        if (count_upto(p, mid, 0xFFFFFFFFu, s) >= (uint32_t)k) lo = mid;
        else hi = mid - 1;
    }
    uint32_t a = 0, b = 8 * kPart - 1;           // the smallest place up to which k are counted
    while (a < b) {
        const uint32_t mid = (a + b) >> 1;
        if (count_upto(p, lo, mid, s) >= (uint32_t)k) b = mid;
        else a = mid + 1;
    }
    if (threadIdx.x == 0) s.ncand = 0u;
    __syncthreads();
    each_element(p, [&](uint32_t key, uint32_t place, uint32_t raw) {
        if (key > lo || (key == lo && place <= a)) s.cand[atomicAdd(&s.ncand, 1u)] = gm::make_entry(key, id0 + place, raw);
    });
    __syncthreads();
}

// The sum over eight neighbouring threads.
__device__ __forceinline__ int sum_of_8(int x)
{
    x += __shfl_xor_sync(kFull, x, 1);
    x += __shfl_xor_sync(kFull, x, 2);
    return x + __shfl_xor_sync(kFull, x, 4);
}

// The k best elements of vectors [j0, j1) of column [cb, ce) of the logits (vector j: elements
// [8j - mis, 8j - mis + 8) of the whole), sorted into s.list (zeros behind them where the part has fewer).  A part of more than kPart vectors is taken in pieces, each with the
// list of those before among its candidates.  All threads of the CTA call it.
__device__ __forceinline__ void part_best(const VerifyArgs &a, int64_t j0, int64_t j1, int64_t cb, int64_t ce, VerifySmem &s)
{
    const int t = threadIdx.x, lane = t & 31, w = t >> 5, k = a.k;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.logits);
    const int mis = (int)((a0 >> 1) & 7);
    const uint4 *vb = reinterpret_cast<const uint4 *>(a0 - 2 * (uintptr_t)mis);
    const int64_t whole0 = (cb + mis + 7) >> 3, whole1 = (ce + mis) >> 3;   // vectors that lie in the column
    int have = 0;
    for (int64_t jb = j0; jb < j1; jb += kPart) {
        uint4 q[kLoads];
        uint32_t mt = 0;
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const int64_t j = jb + u * kThreads + t;
            q[u] = j < j1 && j >= whole0 && j < whole1 ? __ldcg(vb + j) : make_uint4(kNaN2, kNaN2, kNaN2, kNaN2);
        }
        // the column's first and last vector, where it shares them with its neighbours
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            const int64_t j = i ? whole1 : whole0 - 1;
            if (j < jb || j >= j1 || j >= jb + kPart || ((j - jb) & (kThreads - 1)) != t || 8 * j - mis >= ce ||
                8 * j - mis + 8 <= cb || (j >= whole0 && j < whole1))
                continue;
            const uint4 v = load_edge(a.logits, j, mis, cb, ce);
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const bool here = u == (int)((j - jb) / kThreads);
                q[u].x = here ? v.x : q[u].x;
                q[u].y = here ? v.y : q[u].y;
                q[u].z = here ? v.z : q[u].z;
                q[u].w = here ? v.w : q[u].w;
            }
        }
        const uint32_t id0 = (uint32_t)(8 * jb - mis - cb);   // id of place 0 (wraps back where the first vector starts before the column)
        uint32_t um = 0, vk[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            vk[u] = gm::key_of(vmax(q[u]));
            mt = vk[u] > mt ? vk[u] : mt;
        }
        uint32_t m8 = mt;
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) {
            const uint32_t o = __shfl_xor_sync(kFull, m8, d);
            m8 = o > m8 ? o : m8;
        }
        if ((lane & 7) == 0) s.sec[4 * w + (lane >> 3)] = m8;
        if (k > 32) s.top[t] = mt;
        if (t == 0) {
            s.ncand = 0u;
            s.first = 0xFFFFFFFFu;
        }
        __syncthreads();
        // (0 where fewer than k of the maxima are of any element: then every element is a candidate)
        uint32_t T = k <= 32 ? gm::kth_of_64(s.sec[lane], s.sec[lane + 32], k) : gm::kth_of_smem(s.top, kThreads, k, lane);
        if (T == 0u) T = 1u;
#pragma unroll
        for (int u = 0; u < kLoads; ++u) um |= vk[u] >= T ? 1u << u : 0u;
        int n;
        if (k == 1) {
            // the largest: of the elements that have it the first place
            if (um) {
                const int u = __ffs(um) - 1;
                const uint4 v = gm::pick(q, u);
                int e = 7;
#pragma unroll 1
                for (int i = 6; i >= 0; --i)
                    if (order_key(gm::half_of(v, i)) == T) e = i;
                atomicMin(&s.first, (uint32_t)(8 * (u * kThreads + t) + e));
            }
            __syncthreads();
            // (a piece's place comes after every one before: only a larger value takes over)
            if (t == 0 && s.first != 0xFFFFFFFFu && (have == 0 || T > entry_key(s.list[0]))) s.list[0] = gm::make_entry(T, id0 + s.first, key_to_raw(T));
            have = have || s.first != 0xFFFFFFFFu;
            __syncthreads();
            continue;
        }
#pragma unroll 1
        for (; um; um &= um - 1) {
            const int u = __ffs(um) - 1;
            const uint4 v = gm::pick(q, u);
            // (most vectors here hold one such element: the eight are compared at once, and those that reach T dealt with)
            uint32_t hits = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) hits |= order_key(gm::half_of(v, e)) >= T ? 1u << e : 0u;
#pragma unroll 1
            for (; hits; hits &= hits - 1) {
                const int e = __ffs(hits) - 1;
                const uint32_t raw = gm::half_of(v, e), at = atomicAdd(&s.ncand, 1u);
                if (at < (uint32_t)kCand) s.cand[at] = gm::make_entry(order_key(raw), id0 + (uint32_t)(8 * (u * kThreads + t) + e), raw);
            }
        }
        __syncthreads();
        n = (int)s.ncand;
        if (n > kCand) {
            exact_candidates(Piece{a.logits, vb, mis, jb, j1, cb, ce}, k, T, id0, s);
            n = (int)s.ncand;
        }
        if (t < have) s.cand[n + t] = s.list[t];
        __syncthreads();
        n += have;
        // a candidate's rank, by eight threads that compare it with an eighth of them each
        for (int base = 0; base < n; base += kThreads / 8) {
            const int i = base + (t >> 3);
            const unsigned long long e = i < n ? s.cand[i] : ~0ull;
            int rank = 0;
#pragma unroll 4
            for (int j = t & 7; j < n; j += 8) rank += s.cand[j] > e ? 1 : 0;
            rank = sum_of_8(rank);
            if ((t & 7) == 0 && i < n && rank < k) s.list[rank] = e;
        }
        have = n < k ? n : k;
        __syncthreads();
    }
    if (t < k && t >= have) s.list[t] = 0ull;
    __syncthreads();
}

// The lists of the cluster's CTAs, merged into s.list: an entry's rank is its place in its own list and,
// in each of the others, the number of larger ones, which eight threads (one a list) look for by bisection.
__device__ __forceinline__ void merge_parts(const unsigned long long (*in)[kInbox], int ctas, int k, VerifySmem &s)
{
    static_assert(kMostCtas == 8 && kThreads == 512, "eight entries of each of eight lists at a time");
    const int t = threadIdx.x, mine = (t >> 3) & 7, other = t & 7, top = 1 << (31 - __clz(k));
    if (t < k) s.list[t] = 0ull;                 // (fewer than k where the column has fewer)
    __syncthreads();
    // (the k best of all are among the first eight of each list, mostly: then one turn places them)
    for (int base = 0, placed = 0; base < k && placed < k; base += 8) {
        const int i = base + (t >> 6);
        const unsigned long long e = mine < ctas && i < k ? in[mine][i] : 0ull;
        int above = 0;                           // entries above e in the other list: [0, above)
        if (e && other < ctas && other != mine)
            for (int step = top; step; step >>= 1)
                if (above + step <= k && in[other][above + step - 1] > e) above += step;
        const int rank = i + sum_of_8(above);
        const bool in_list = other == 0 && e && rank < k;
        if (in_list) s.list[rank] = e;
        placed += __syncthreads_count(in_list);
    }
}

// ---- the decision at a node -------------------------------------------------------

// The children of node `cur` whose tokens are in its list, by `threads` threads (whole warps).
__device__ __forceinline__ void match_children(const VerifyArgs &a, VerifySmem &s, int cur, bool last_level, int t, int threads)
{
    for (int i = t; (i & ~31) < s.n; i += threads) {
        const int32_t x = i > 0 && i < s.n && !last_level && s.parent[i] == cur ? s.token[i] : -1;
        int place = -1;
        if (x >= 0)
#pragma unroll 4
            for (int e = 0; e < a.k; ++e)
                if ((int32_t)entry_id(s.list[e]) == x && s.list[e]) place = e;
        const uint32_t hits = __ballot_sync(kFull, place >= 0);
        if (place >= 0) s.place[i] = place;
        if ((i & 31) == 0) s.hits[i >> 5] = hits;
    }
}

__device__ __forceinline__ float warp_sum(float v) { return warp_sum_f(v); }
__device__ __forceinline__ double warp_sum(double v) { return warp_sum_d(v); }
__device__ __forceinline__ float warp_scan(float v, int lane) { return warp_scan_f(v, lane); }
__device__ __forceinline__ double warp_scan(double v, int lane) { return warp_scan_d(v, lane); }

// Sampled decision at node `cur` from its column's list, by one warp, in R.  Entry t of the list is in lane t,
// or t - 32, n entries.  In double the rounding of sums by trees is some 1e-16.  In float it is first
// tried whether every comparison is clear of its border (FP64 runs at a small fraction of the FP32 rate here), else
// false is returned and double decides.  With at most 32 terms e = exp(x), x = (v - v0) / T: x is off by
// 3 * 2^-24 |x| and exp by 2 units, so a term by 1.8e-7 |x| e + 2.4e-7 e, of which |x| e <= 0.37; the terms' sum S >= 1 by
// 2.1e-6 + 2.4e-7 S and five roundings; running sums of e / S by 6e-6 then, and those over a nucleus of
// weight C by 1.2e-5 / C, a uniform's product with what is left the same.
template <typename R>
__device__ __forceinline__ bool decide_sampled(const VerifyArgs &a, VerifySmem &s, int n, int cur, int lane, int32_t &next,
                                               int32_t &token)
{
    constexpr bool kSingle = sizeof(R) == 4;
    constexpr R kSureP = (R)2e-5, kSureQ = (R)5e-5;   // above 6e-6; above 2 * 1.2e-5, over C
    if (kSingle && n > 32) return false;
    auto near = [&](R x, R y, R sure) { return kSingle && !(x - y > sure || y - x > sure); };   // (a NaN is near)
    const bool ha = lane < n, hb = lane + 32 < n;
    const unsigned long long ea_ = ha ? s.list[lane] : 0ull, eb_ = hb ? s.list[lane + 32] : 0ull;
    const float v0 = bf16_as_float(entry_raw(s.list[0]));
    R ea, eb = 0;
    if (kSingle) {
        ea = ha ? (R)expf((bf16_as_float(entry_raw(ea_)) - v0) * a.inv_temperature) : (R)0;
    } else {
        const double z0 = (double)v0 / a.temperature;
        ea = ha ? (R)exp((double)bf16_as_float(entry_raw(ea_)) / a.temperature - z0) : (R)0;
        eb = hb ? (R)exp((double)bf16_as_float(entry_raw(eb_)) / a.temperature - z0) : (R)0;
    }
    const int32_t ida = ha ? (int32_t)entry_id(ea_) : -1, idb = hb ? (int32_t)entry_id(eb_) : -1;
    const R inv = (R)1 / warp_sum(ea + eb);
    const R pa = ea * inv, pb = eb * inv;
    // the nucleus: the shortest prefix whose running sum reaches top_p
    const R top_p = kSingle ? (R)a.top_p_single : (R)a.top_p;
    const R ca = warp_scan(pa, lane), cb = __shfl_sync(kFull, ca, 31) + (kSingle ? (R)0 : warp_scan(pb, lane));
    if (__any_sync(kFull, (ha && near(ca, top_p, kSureP)) || (hb && near(cb, top_p, kSureP)))) return false;
    const uint32_t ra = __ballot_sync(kFull, ha && ca >= top_p), rb = __ballot_sync(kFull, hb && cb >= top_p);
    const int last = ra ? __ffs(ra) - 1 : rb ? 31 + __ffs(rb) : n - 1;
    const R C = last < 32 ? __shfl_sync(kFull, ca, last & 31) : __shfl_sync(kFull, cb, last & 31);
    if (kSingle && !(C >= (R)0.25)) return false;
    const R invC = (R)1 / C, sure = kSureQ * invC;
    R qa = lane <= last ? pa * invC : (R)0, qb = lane + 32 <= last ? pb * invC : (R)0;   // of what is left
    R left = warp_sum(qa + qb);
    next = -1;
    for (int base = 0; base < s.n; base += 32) {
        for (uint32_t kids = s.hits[base >> 5]; kids; kids &= kids - 1) {
            const int c = base + __ffs(kids) - 1, at = s.place[c];
            if (at > last) continue;             // not in the nucleus
            const R xa = __shfl_sync(kFull, qa, at & 31), xb = __shfl_sync(kFull, qb, at & 31);
            const R q = at < 32 ? xa : xb, goal = (R)s.uniform[c].x * left;
            if (q == (R)0) continue;             // taken out before (or without weight)
            if (near(goal, q, sure)) return false;
            // taken out; with nothing left but rounding it is accepted: the uniform is below 1
            const R na = lane == at ? (R)0 : qa, nb = lane + 32 == at ? (R)0 : qb;
            const R rest = warp_sum(na + nb);
            if (goal < q || rest == (R)0) {
                next = c;
                token = s.token[c];
                return true;
            }
            qa = na;
            qb = nb;
            left = rest;
        }
    }
    // the draw from what is left
    const R goal = (R)s.uniform[cur].y * left;
    const R sa = warp_scan(qa, lane), sb = __shfl_sync(kFull, sa, 31) + (kSingle ? (R)0 : warp_scan(qb, lane));
    if (__any_sync(kFull, (ha && qa > (R)0 && near(sa, goal, sure)) || (hb && qb > (R)0 && near(sb, goal, sure)))) return false;
    const uint32_t xa = __ballot_sync(kFull, qa > (R)0 && sa > goal), xb = __ballot_sync(kFull, qb > (R)0 && sb > goal);
    if (kSingle && !xa) return false;
    // none exceeds it (rounding left the goal at the very end): the last that has weight
    const uint32_t la = __ballot_sync(kFull, qa > (R)0), lb = __ballot_sync(kFull, qb > (R)0);
    const int32_t from_a = __shfl_sync(kFull, ida, xa ? __ffs(xa) - 1 : la ? 31 - __clz((int)la) : 0);
    const int32_t from_b = __shfl_sync(kFull, idb, xb ? __ffs(xb) - 1 : lb ? 31 - __clz((int)lb) : 0);
    token = xa ? from_a : xb || lb ? from_b : from_a;
    return true;
}

// What the walk does at node `cur` from its column's list (a.k entries, zeros behind the last): s.next, s.chosen.  One warp.
__device__ __forceinline__ void decide(const VerifyArgs &a, VerifySmem &s, int cur, int lane)
{
    const int n = __popc(__ballot_sync(kFull, lane < a.k && s.list[lane])) + __popc(__ballot_sync(kFull, lane + 32 < a.k && s.list[lane + 32]));
    int32_t next = -1, token = -1;
    if (n == 0) {                                // (a column without a number is outside the contract)
    } else if (a.uniforms) {
        if (!decide_sampled<float>(a, s, n, cur, lane, next, token)) decide_sampled<double>(a, s, n, cur, lane, next, token);
    } else {
        token = (int32_t)entry_id(s.list[0]);
        for (int base = 0; base < s.n; base += 32)
            if (s.hits[base >> 5]) {
                next = base + __ffs(s.hits[base >> 5]) - 1;
                break;
            }
    }
    if (lane == 0) {
        s.next = next;
        s.chosen = token;
    }
}

// ---- the kernel ---------------------------------------------------------------------

// The nodes of lane l into shared memory (all threads).
__device__ __forceinline__ void load_lane(const VerifyArgs &a, int64_t l, VerifySmem &s)
{
    const LaneRows r = lane_rows(a.cu, l, a.tokens);
    const int n = r.n < kNodes ? (int)r.n : kNodes;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int32_t p = __ldg(a.parents + r.first + i);
        s.parent[i] = i > 0 && p >= 0 && p < i ? p : -1;
        s.token[i] = __ldg(a.drafts + r.first + i);
        if (a.uniforms) s.uniform[i] = make_double2(__ldg(a.uniforms + 2 * (r.first + i)), __ldg(a.uniforms + 2 * (r.first + i) + 1));
    }
    if (threadIdx.x == 0) {
        s.n = n;
        s.row0 = r.first;
    }
    __syncthreads();
}

// Thread `t` of the lane's writer: the outputs from level `level` on are -1.
__device__ __forceinline__ void end_lane(const VerifyArgs &a, int64_t l, int accepted, int committed, int t, int threads)
{
    if (t == 0) a.accept[l] = accepted;
    const int64_t at = l * (a.depth + 1);
    for (int i = t; i <= a.depth; i += threads) {
        if (i >= committed) a.commit[at + i] = -1;
        if (i > accepted || committed == 0) a.path[at + i] = -1;
    }
}

// CTA `rank` of `ctas`' share of column c: its best, into s.list.
__device__ __forceinline__ void column_part(const VerifyArgs &a, int64_t c, uint32_t rank, uint32_t ctas, VerifySmem &s)
{
    const int mis = (int)((reinterpret_cast<uintptr_t>(a.logits) >> 1) & 7);
    const int64_t cb = c * a.V, ce = cb + a.V;
    const int64_t jf = (cb + mis) >> 3, nv = ((ce - 1 + mis) >> 3) - jf + 1;
    const int64_t each = nv / ctas, more = nv - each * ctas;
    const int64_t j0 = jf + rank * each + (rank < more ? rank : more);
    part_best(a, j0, j0 + each + (rank < more ? 1 : 0), cb, ce, s);
}

// s.list into inbox `b` of every CTA of the cluster.
__device__ __forceinline__ void send_list(VerifySmem &s, int b, uint32_t rank, uint32_t ctas, int k)
{
    const int t = threadIdx.x, to = t / SPEC_MAX_K, i = t % SPEC_MAX_K;
    if (to < (int)ctas && i < k)
        gm::st_cluster_u64(gm::cluster_map(&s.inbox[b][rank][i], to), s.list[i]);
}

template <bool kWide>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const __grid_constant__ VerifyArgs a, const uint32_t ctas)
{
    extern __shared__ __align__(16) uint8_t raw[];
    VerifySmem &s = *reinterpret_cast<VerifySmem *>(raw);
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const uint32_t rank = ctas > 1 ? gm::cluster_rank() : 0u;
    if (ctas > 1) gm::cluster_arrive_relaxed();       // this CTA runs: others may write into it once all do
    pdl_launch_dependents();
    pdl_wait();
    const int64_t unit = blockIdx.x / ctas;

    if (!kWide) {
        const int64_t l = unit;
        load_lane(a, l, s);
        if (ctas > 1) gm::cluster_wait();
        int cur = 0, level = 0;
        const bool writer = rank == 0 && t == 0;
        if (s.n == 0) {
            if (rank == 0) end_lane(a, l, 0, 0, t, kThreads);
            return;                                   // (all CTAs of the cluster alike)
        }
        for (;; ++level) {
            column_part(a, s.row0 + cur, rank, ctas, s);
            if (ctas > 1) {
                send_list(s, level & 1, rank, ctas, a.k);
                gm::cluster_arrive();
                gm::cluster_wait();
                merge_parts(s.inbox[level & 1], (int)ctas, a.k, s);
            }
            match_children(a, s, cur, level == a.depth, t, kThreads);
            __syncthreads();
            if (w == 0) decide(a, s, cur, lane);
            __syncthreads();
            const int next = s.next;
            if (writer) {
                a.commit[l * (a.depth + 1) + level] = s.chosen;
                a.path[l * (a.depth + 1) + level] = cur;
            }
            if (next < 0) break;
            cur = next;
        }
        if (rank == 0) end_lane(a, l, level, level + 1, t, kThreads);
        return;
    }

    // a column a cluster; where it belongs
    const int64_t row = unit;
    if (t == 0) {
        s.lane = -1;
        s.count = 0u;
    }
    __syncthreads();
    for (int64_t l = t; l < a.lanes; l += kThreads) {
        const LaneRows r = lane_rows(a.cu, l, a.tokens);
        if (row >= r.first && row < r.first + r.n) s.lane = (int32_t)l;
        if (r.n == 0 && blockIdx.x == 0) end_lane(a, l, 0, 0, 0, 1);
        if (__ldg(a.cu + l) > __ldg(a.cu + l + 1)) s.count = 1u;
    }
    __syncthreads();
    if (ctas > 1) gm::cluster_wait();
    const int64_t l = s.lane;
    // (the cluster's CTAs alike.  Where cu decreases lanes may share rows, and a ticket would not come back to
    // zero: no lane is answered.)
    if (l < 0 || s.count) return;
    load_lane(a, l, s);
    if (row - s.row0 >= s.n) return;                  // past the nodes that a lane may have
    column_part(a, row, rank, ctas, s);
    if (ctas > 1) {
        send_list(s, 0, rank, ctas, a.k);
        gm::cluster_arrive();
        gm::cluster_wait();
        if (rank != 0) return;
        merge_parts(s.inbox[0], (int)ctas, a.k, s);
    }
    if (t < a.k) __stcg(a.lists + row * a.k + t, s.list[t]);
    __syncthreads();
    if (t == 0) {
        __threadfence();
        s.first = atom_add_acq_rel(a.tickets + l, 1u);
    }
    __syncthreads();
    if (s.first != (uint32_t)s.n - 1u) return;
    // the lane's last column: all lists are there
    if (t == 0) a.tickets[l] = 0u;                    // for the next call
    if (w != 0) return;
    int cur = 0, level = 0;
    for (;; ++level) {
        __syncwarp();
        for (int i = lane; i < a.k; i += 32) s.list[i] = __ldcg(a.lists + (s.row0 + cur) * a.k + i);
        __syncwarp();
        match_children(a, s, cur, level == a.depth, lane, 32);
        __syncwarp();
        decide(a, s, cur, lane);
        __syncwarp();
        const int next = s.next;
        if (lane == 0) {
            a.commit[l * (a.depth + 1) + level] = s.chosen;
            a.path[l * (a.depth + 1) + level] = cur;
        }
        if (next < 0) break;
        cur = next;
    }
    end_lane(a, l, level, level + 1, lane, 32);
}

}  // namespace tree
