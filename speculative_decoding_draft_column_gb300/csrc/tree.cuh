// Rounds whose drafts form a tree, and the 8-bit cache: the plan of a tree's masks and
// positions, the store that quantises, and the accepted path moved into place.
#pragma once

#include "common.cuh"

namespace tree {

constexpr int kNodes = SPEC_TREE_MAX_NODES;

// The lane's rows of the step, cut to [0, tokens).
struct LaneRows {
    int64_t first, n;
};
__device__ __forceinline__ LaneRows lane_rows(const int32_t *cu, int64_t l, int64_t tokens)
{
    int64_t c0 = __ldg(cu + l), c1 = __ldg(cu + l + 1);
    c0 = c0 < 0 ? 0 : c0 > tokens ? tokens : c0;
    c1 = c1 < c0 ? c0 : c1 > tokens ? tokens : c1;
    return {c0, c1 - c0};
}

// ---- masks and positions ------------------------------------------------------

struct PlanArgs {
    const int32_t *parents, *cu, *seq_lens;
    int64_t tokens, lanes;
    uint32_t *masks;
    int32_t words;
    int32_t *positions;
};

constexpr int kPlanThreads = 64;

// mask(i) = {i} + mask(parent(i)), by walking up the parents in shared memory: a thread a
// node, a CTA a lane.  Bound by its launch and two dependent reads (the lane's rows, then
// its parents): 3 us.  A walk takes as many steps as the node is deep; doubling the step
// would bound a chain of 256 nodes by 8 steps instead of 255, but costs trees of the
// usual depth barriers that they do not need.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanArgs a)
{
    __shared__ int32_t parent[kNodes];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x;
    for (int64_t l = blockIdx.x; l < a.lanes; l += gridDim.x) {
        const LaneRows r = lane_rows(a.cu, l, a.tokens);
        const int n = r.n < kNodes ? (int)r.n : kNodes;
        // (a lane cut by the buffer keeps its tokens' positions)
        const int32_t ctx = __ldg(a.seq_lens + l) - (__ldg(a.cu + l + 1) - __ldg(a.cu + l));
        __syncthreads();
        for (int i = tid; i < n; i += kPlanThreads) {
            const int32_t p = __ldg(a.parents + r.first + i);
            parent[i] = i > 0 && p >= 0 && p < i ? p : -1;
        }
        __syncthreads();
        for (int64_t i = tid; i < r.n; i += kPlanThreads) {
            uint32_t m[kNodes / 32];
#pragma unroll
            for (int w = 0; w < kNodes / 32; ++w) m[w] = 0u;
            int depth = -1;
            for (int j = i < kNodes ? (int)i : -1; j >= 0; j = parent[j]) {   // (parents come earlier: at most 256 steps)
#pragma unroll
                for (int w = 0; w < kNodes / 32; ++w) m[w] |= (j >> 5) == w ? 1u << (j & 31) : 0u;
                ++depth;
            }
            uint32_t *dst = a.masks + (r.first + i) * a.words;
#pragma unroll
            for (int w = 0; w < kNodes / 32; ++w)
                if (w < a.words) dst[w] = m[w];
            a.positions[r.first + i] = ctx + (depth > 0 ? depth : 0);
        }
    }
    // rows past the step's
    const LaneRows last = lane_rows(a.cu, a.lanes - 1, a.tokens);
    const int64_t end = last.first + last.n;
    for (int64_t t = end + (int64_t)blockIdx.x * kPlanThreads + tid; t < a.tokens; t += (int64_t)gridDim.x * kPlanThreads) {
        for (int w = 0; w < a.words; ++w) a.masks[t * a.words + w] = 0u;
        a.positions[t] = 0;
    }
}

// ---- the quantising store -----------------------------------------------------

struct StoreArgs {
    const uint16_t *k, *v;
    int64_t tokens, ks_t, ks_h, vs_t, vs_h;
    const int64_t *slots;
    spec_paged_cache8 c;
    int32_t group;         // threads of a vector, two pieces of 8 elements each: a power of two
    int32_t heads;         // of a token that a CTA deals with (blockIdx.y: which)
    int32_t per;           // tokens at a time: kStoreThreads / (group * heads)
    int32_t log_page;      // log2 of the page's size, -1 where it is no power of two
};

constexpr int kStoreThreads = 256, kStoreCtas = 5;   // of an SM

// The larger of each half of two pairs of 16-bit numbers, NaN where either is.
template <bool F16>
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b)
{
    uint32_t r;
    if (F16) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Two pieces of eight elements of a vector to codes; `group` threads hold a vector and agree on its scale.
// The exponent comes from the bits of the largest magnitude 1.f * 2^E: 1.f is at most 1.75 =
// 448 / 2^8 or not.  x * 2^-e is exact (what a 16-bit product would lose lies below half the least code),
// so each code is rounded once.
template <bool F16>
__device__ __forceinline__ void quantise(const uint4 (&q)[2], int group, uint2 (&codes)[2], uint32_t &scale)
{
    const uint32_t w[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
    uint32_t most = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max_pair<F16>(most, w[i] & 0x7FFF7FFFu);
    for (int d = 1; d < group; d <<= 1) most = max_pair<F16>(most, __shfl_xor_sync(kFull, most, d));
    most = max(most & 0x7FFFu, most >> 16 & 0x7FFFu);
    if (most >= (F16 ? 0x7C00u : 0x7F80u)) {          // an infinity or a NaN: no number throughout
        codes[0] = codes[1] = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
        scale = 255u;
        return;
    }
    constexpr int kBits = F16 ? 10 : 7, kBias = F16 ? 15 : 127, kLeast = F16 ? -14 : -120;
    // (a subnormal's exponent comes out too small, and is cut to the least anyway: fp16's below 2^-14, bf16's below 2^-126)
    int e = (int)(most >> kBits) - kBias - 8 + ((most & ((1u << kBits) - 1u)) > (3u << (kBits - 2)) ? 1 : 0);
    e = e < kLeast ? kLeast : e > 7 ? 7 : e;
    uint32_t c[8];
    if (F16) {
        const uint32_t f = (uint32_t)(15 - e) << 10, ff = f | f << 16;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint16_t two;
            asm("{\n\t.reg .b32 y;\n\tmul.rn.f16x2 y, %1, %2;\n\tcvt.rn.satfinite.e4m3x2.f16x2 %0, y;\n\t}" : "=h"(two) : "r"(w[i]), "r"(ff));
            c[i] = two;
        }
    } else {
        const float f = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint16_t two;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(__uint_as_float(w[i] & 0xFFFF0000u) * f), "f"(__uint_as_float(w[i] << 16) * f));
            c[i] = two;
        }
    }
    codes[0] = make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
    codes[1] = make_uint2(__byte_perm(c[4], c[5], 0x5410), __byte_perm(c[6], c[7], 0x5410));
    scale = (uint32_t)(e + 127);
}

// `group` threads take two pieces of 8 elements each of a token's key and value of a head, all four on their
// way together, and the slot of the next token (a CTA's rounds follow one another, and each
// waits for its slots and then for its vectors).  Bound by its bytes, with instructions close behind: 16,384 tokens
// of 8 heads of 128 (92 MB) 17.4 us, 5.4 TB/s; with a piece a thread, twice the shuffles and exponents, 23.5.
template <bool F16>
__global__ void __launch_bounds__(kStoreThreads, kStoreCtas) store_kernel(const __grid_constant__ StoreArgs a)
{
    pdl_launch_dependents();
    const int tid = threadIdx.x, each = a.group * a.heads, sub = tid / each, e0 = (tid & (a.group - 1)) * 8, e1 = e0 + a.group * 8;
    const int h = (int)blockIdx.y * a.heads + (tid - sub * each) / a.group;
    const bool in = e0 < a.c.head_dim && h < a.c.heads && sub < a.per, in1 = e1 < a.c.head_dim;
    const uint16_t *k = a.k + h * a.ks_h + e0, *v = a.v + h * a.vs_h + e0;
    uint8_t *kc = static_cast<uint8_t *>(a.c.k) + h * a.c.k_strides[2] + e0, *vc = static_cast<uint8_t *>(a.c.v) + h * a.c.v_strides[2] + e0;
    const int second = a.group * 8;
    const int64_t limit = a.c.pages * a.c.page_size, step = (int64_t)gridDim.x * a.per;
    int64_t first = (int64_t)blockIdx.x * a.per;
    pdl_wait();
    auto slot_of = [&](int64_t t) -> int64_t { return in && t < a.tokens ? __ldg(a.slots + t) : -1; };
    int64_t slot = slot_of(first + sub);
    for (; first < a.tokens; first += step) {           // (all threads of a warp stay for the shuffles)
        const int64_t t = first + sub, at = slot < limit ? slot : -1;
        uint4 x[2][2];
        x[0][0] = x[0][1] = x[1][0] = x[1][1] = make_uint4(0, 0, 0, 0);
        if (at >= 0) {
            const uint16_t *kt = k + t * a.ks_t, *vt = v + t * a.vs_t;
            x[0][0] = __ldg(reinterpret_cast<const uint4 *>(kt));
            x[1][0] = __ldg(reinterpret_cast<const uint4 *>(vt));
            if (in1) {
                x[0][1] = __ldg(reinterpret_cast<const uint4 *>(kt + second));
                x[1][1] = __ldg(reinterpret_cast<const uint4 *>(vt + second));
            }
        }
        slot = slot_of(t + step);
        uint2 code[2][2];
        uint32_t scale[2];
        quantise<F16>(x[0], a.group, code[0], scale[0]);
        quantise<F16>(x[1], a.group, code[1], scale[1]);
        if (at < 0) continue;
        const int64_t page = a.log_page >= 0 ? at >> a.log_page : udiv(at, a.c.page_size), row = at - page * a.c.page_size;
        uint8_t *ko = kc + page * a.c.k_strides[0] + row * a.c.k_strides[1], *vo = vc + page * a.c.v_strides[0] + row * a.c.v_strides[1];
        *reinterpret_cast<uint2 *>(ko) = code[0][0];
        *reinterpret_cast<uint2 *>(vo) = code[1][0];
        if (in1) {
            *reinterpret_cast<uint2 *>(ko + second) = code[0][1];
            *reinterpret_cast<uint2 *>(vo + second) = code[1][1];
        }
        if (e0 == 0) {
            const int64_t s = (page * a.c.heads + h) * a.c.page_size + row;
            a.c.k_scales[s] = (uint8_t)scale[0];
            a.c.v_scales[s] = (uint8_t)scale[1];
        }
    }
}

// ---- the accepted path ----------------------------------------------------------

struct CommitArgs {
    uint8_t *k, *v;                     // elements of `bytes` bytes
    uint8_t *k_scales, *v_scales;       // 8 bits only
    int64_t k_strides[3], v_strides[3];   // bytes
    int64_t pages, max_pages, lanes;
    int32_t page_size, heads, vector;   // vector: 16-byte pieces of a head's key
    int32_t depth;
    const int32_t *block_table, *cu, *seq_lens, *path, *accept;
    int32_t *context_out;
};

constexpr int kCommitThreads = 256;
constexpr int kAhead = 8;               // pieces of a thread on their way together

// A CTA a lane.  A thread moves one 16-byte piece of a token (or a byte of scales) along the
// whole path, in order: node path[i] >= i goes to i, so what a later step reads (path[j] >= j > i)
// no earlier one has written, and no threads meet.  The path's places are worked out once, a thread
// a step.  Bound by that chain (lengths, path, table, piece: four dependent reads), not by its bytes.
__global__ void __launch_bounds__(kCommitThreads) commit_kernel(const __grid_constant__ CommitArgs a)
{
    __shared__ int32_t from_page[kNodes], from_row[kNodes], to_page[kNodes], to_row[kNodes];   // of the i-th move; page -1: none
    __shared__ int32_t end;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t l = blockIdx.x;
    const int tid = threadIdx.x;
    const int32_t c0 = __ldg(a.cu + l), c1 = __ldg(a.cu + l + 1), n = c1 > c0 ? c1 - c0 : 0;
    const int32_t ctx = __ldg(a.seq_lens + l) - n;
    int32_t moves = __ldg(a.accept + l);
    moves = moves < 0 ? 0 : moves > a.depth ? a.depth : moves;
    if (tid == 0) end = n > 0 ? moves : 0;
    __syncthreads();
    if (tid < moves) {
        const int32_t i = tid + 1, node = __ldg(a.path + l * (a.depth + 1) + i);
        if (node < i || node >= n) atomicMin(&end, tid);
        const int64_t from = (int64_t)ctx + node, to = (int64_t)ctx + i;
        int32_t fp = -1, tp = -1;
        if (from != to && ctx >= 0 && node >= i && node < n) {
            const int64_t f = udiv(from, a.page_size), t = udiv(to, a.page_size);
            if (f < a.max_pages && t < a.max_pages) {
                fp = __ldg(a.block_table + l * a.max_pages + f);
                tp = __ldg(a.block_table + l * a.max_pages + t);
                from_row[tid] = (int32_t)(from - f * a.page_size);
                to_row[tid] = (int32_t)(to - t * a.page_size);
            }
        }
        const bool on = fp >= 0 && fp < a.pages && tp >= 0 && tp < a.pages;
        from_page[tid] = on ? fp : -1;
        to_page[tid] = tp;
    }
    __syncthreads();
    moves = end;
    if (tid == 0 && a.context_out) a.context_out[l] = n > 0 ? ctx + 1 + moves : ctx;
    if (moves == 0) return;

    const int per = a.heads * a.vector;
    for (int p = tid; p < 2 * per; p += kCommitThreads) {
        const bool value = p >= per;
        const int r = value ? p - per : p, h = r / a.vector, e = (r - h * a.vector) * 16;
        const int64_t *st = value ? a.v_strides : a.k_strides;
        const int64_t s0 = st[0], s1 = st[1];
        uint8_t *base = (value ? a.v : a.k) + h * st[2] + e;
        for (int i0 = 0; i0 < moves; i0 += kAhead) {
            uint4 x[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (i0 + u < moves && from_page[i0 + u] >= 0)
                    x[u] = *reinterpret_cast<const uint4 *>(base + from_page[i0 + u] * s0 + from_row[i0 + u] * s1);
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (i0 + u < moves && from_page[i0 + u] >= 0)
                    *reinterpret_cast<uint4 *>(base + to_page[i0 + u] * s0 + to_row[i0 + u] * s1) = x[u];
        }
    }
    if (!a.k_scales) return;
    for (int p = tid; p < 2 * a.heads; p += kCommitThreads) {
        const bool value = p >= a.heads;
        const int h = value ? p - a.heads : p;
        uint8_t *s = value ? a.v_scales : a.k_scales;
        for (int i0 = 0; i0 < moves; i0 += kAhead) {
            uint8_t x[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (i0 + u < moves && from_page[i0 + u] >= 0)
                    x[u] = s[((int64_t)from_page[i0 + u] * a.heads + h) * a.page_size + from_row[i0 + u]];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (i0 + u < moves && from_page[i0 + u] >= 0)
                    s[((int64_t)to_page[i0 + u] * a.heads + h) * a.page_size + to_row[i0 + u]] = x[u];
        }
    }
}

}  // namespace tree
