// Penalties for repeated tokens, biases and grammar masks on bf16 logits.
//
// Column j of a lane, token t, in fp32 and rounded once:
//   x = t seen ? (x > 0 ? x / r : x * r) : x        (prompt, output, drafts before j)
//   x -= f * n + p * (n > 0)                        (n: output and drafts before j)
//   x += bias(t);   x = -inf where the grammar's bit is clear.
#pragma once

#include "common.cuh"

namespace rules {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kSlice = 4096;             // tokens of a slice
constexpr int kPieces = 4;               // of a slice: a warp works on one piece of one column at a time
constexpr int kPiece = kSlice / kPieces;
constexpr int kPer = kPiece / 8 / 32;    // 16-byte vectors a lane has in a piece
constexpr int kWindow = kSlice + 8;      // a column's vectors may start up to 7 tokens before the slice
constexpr int kRing = 2;                 // pieces a warp has in shared memory
constexpr int kList = kPiece + 8;        // listed tokens of a piece, in any phase
constexpr int kMaxCols = SPEC_MAX_GAMMA + 1;
constexpr uint32_t kSeen = 0x80000000u;  // the token is in the prompt
constexpr uint32_t kDraft = 0x40000000u; // the token is one of the drafts
constexpr uint32_t kBiased = 0x20000000u; // the token has a bias; the other bits count the output
constexpr int32_t kNoId = INT32_MIN;        // an id of no window
constexpr uint32_t kMasked = 0xFF80FF80u;   // two bf16 -inf
static_assert(kWindow % 4 == 0, "");
static_assert(kWarps % kPieces == 0, "a warp stays with one piece");

struct Args {
    const uint16_t *logits;
    uint16_t *out;
    int64_t lanes, V;
    int32_t cols;
    const int32_t *history;
    int64_t history_stride;
    const int32_t *prompt_lens, *history_lens, *drafts;
    const float *penalties;
    const int32_t *bias_ids;
    const float *bias_vals;
    int64_t max_bias;
    const int32_t *bias_lens;
    const uint32_t *mask;
    int64_t mask_count;
    const int32_t *mask_rows;
};

// dynamic shared memory: the warps' rings, the counts, the lists, and the biases if any
constexpr int kCountAt = kWarps * kRing * kPiece * 2, kListAt = kCountAt + kWindow * 4;
constexpr int kBiasAt = kListAt + kPieces * kList * 2;
constexpr int smem_bytes(bool biases) { return kBiasAt + (biases ? kWindow * 4 : 0); }

__device__ __forceinline__ uint16_t to_bf16(float f)
{
    uint16_t h;
    asm("{\n\t.reg .b16 r;\n\tcvt.rn.bf16.f32 r, %1;\n\tmov.b16 %0, r;\n\t}" : "=h"(h) : "f"(f));
    return h;
}

struct Yes { static constexpr bool value = true; };
struct No { static constexpr bool value = false; };

// bytes of the sign bits that the selector's nibbles (8 + byte) name
__device__ __forceinline__ uint32_t copies(uint32_t v, uint32_t selector)
{
    uint32_t d;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(d) : "r"(v), "r"(selector));
    return d;
}

// One bulk copy shared -> global, and the bulk groups of the issuing thread.
__device__ __forceinline__ void bulk_s2g(void *dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// all but the newest n groups have read their shared memory
template <int n>
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(n) : "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ int64_t clamp_len(int32_t n, int64_t most) { return n < 0 ? 0 : n > most ? most : n; }

// One CTA per (slice of the vocabulary, lane).  It counts the lane's history
// over its slice in shared memory and lists the tokens that anything but the
// mask can change.  From there on its warps work alone, without barriers: a warp
// takes one piece of the slice through the lane's columns, each piece brought
// into the warp's ring by a bulk copy, its listed tokens rewritten and its vectors masked
// in place, and taken out by a bulk copy, with the next pieces on
// their way in.  Instructions so go to listed tokens and masks only.  (With every
// vector in registers and tested for seen tokens, 64 x 16 columns of 248,046 took 243 us,
// bound by instructions; with columns staged by the whole CTA 257 us, bound by barriers.)
// 64 x 16 columns now take 146 us copied (1.0 of a measured copy), 153 with masks, 180 with
// histories of up to 16,000 ids, 214 with everything, at two thirds of the issue slots:
// reading the history in every slice and rewriting its tokens in every column.  One lane's
// column takes 4.9 us.  Two CTAs of 16 warps an SM; a third ring place, which leaves one,
// cost 312 us.
__global__ void __launch_bounds__(kThreads, 2) process_kernel(const __grid_constant__ Args a)
{
    extern __shared__ __align__(128) uint8_t smem[];
    uint32_t *count = reinterpret_cast<uint32_t *>(smem + kCountAt);
    uint16_t *lists = reinterpret_cast<uint16_t *>(smem + kListAt);   // [kPieces][kList]
    float *bias = reinterpret_cast<float *>(smem + kBiasAt);          // only with biases
    __shared__ uint32_t touched[kWindow / 32 + 1];
    __shared__ int n_listed[kPieces];
    __shared__ int32_t draft_entry[kMaxCols], mask_row[kMaxCols];
    __shared__ uint64_t full[kWarps][kRing];
    __shared__ int bias_again;
    const int tid = threadIdx.x, warp = tid >> 5, wl = tid & 31;
    const int64_t lane = blockIdx.y, t0 = (int64_t)blockIdx.x * kSlice;
    const int64_t w0 = t0 - 8;   // the token of window entry 0
    pdl_launch_dependents();
    {
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        for (int i = tid; i < kWindow / 4; i += kThreads) {
            reinterpret_cast<uint4 *>(count)[i] = zero;
            if (a.bias_ids) reinterpret_cast<uint4 *>(bias)[i] = zero;
        }
    }
    for (int i = tid; i < kWindow / 32 + 1; i += kThreads) touched[i] = 0u;
    if (tid < kWarps * kRing) mbar_init(&full[0][0] + tid, 1);
    if (tid == 0) {
        s_gave_up = 0u;
        bias_again = 0;
    }
    fence_mbar_init();
    pdl_wait();
    __syncthreads();

    // Vectors are 8 tokens, 16-byte aligned: the column's part of the slice starts
    // at token t0 - mis.  Element i of piece q is token t0 - mis + q * kPiece + i.
    const int64_t col0 = lane * a.cols;
    const int mis0 = (int)(((reinterpret_cast<uintptr_t>(a.logits) & 15) / 2 + col0 * a.V + t0) & 7), v7 = (int)(a.V & 7);
    const bool same_phase = ((reinterpret_cast<uintptr_t>(a.logits) ^ reinterpret_cast<uintptr_t>(a.out)) & 15) == 0;
    const int64_t left = a.V - t0;                        // tokens from t0 to the column's end
    const int end = left > kSlice ? kSlice : (int)left, begin = t0 > 0 ? -8 : 0;   // tokens [begin, end) are the column's
    const int piece = warp % kPieces, col_step = kWarps / kPieces, first_col = warp / kPieces;
    struct Part {
        int lo, hi;        // elements [lo, hi) are the column's
        int v0, v1;        // vectors wholly inside: by bulk copy (the rest token by token)
    };
    auto part = [&](int mis) -> Part {
        Part p;
        p.lo = begin + mis - piece * kPiece;
        p.hi = end + mis - piece * kPiece;
        p.v0 = p.lo > 0 ? 1 : 0;                          // lo is at most 7
        const int n = p.hi >> 3;
        p.v1 = n > kPiece / 8 ? kPiece / 8 : n < p.v0 ? p.v0 : n;
        return p;
    };
    // the slice lies inside its columns, in whatever phase: every piece is whole
    const bool inner = t0 >= 8 && t0 + kSlice <= a.V;
    uint16_t *ring = reinterpret_cast<uint16_t *>(smem) + warp * kRing * kPiece;
    // one thread: the piece at element `at` of the logits (its phase taken off) into a place of the ring
    auto fetch = [&](int place, int64_t at, int mis) {
        uint64_t *bar = &full[warp][place];
        uint16_t *to = ring + place * kPiece;
        if (inner) {
            mbar_arrive_expect_tx(bar, kPiece * 2);
            bulk_g2s(to, a.logits + at, kPiece * 2, bar);
            return;
        }
        const Part p = part(mis);
        const uint32_t bytes = (uint32_t)(p.v1 - p.v0) * 16;
        mbar_arrive_expect_tx(bar, bytes);
        if (bytes) bulk_g2s(to + 8 * p.v0, a.logits + at + 8 * p.v0, bytes, bar);
    };
    // from one of the warp's columns to the next
    const int64_t col_stride = (int64_t)col_step * a.V, at_first = (col0 + first_col) * a.V + t0 + piece * kPiece;
    const int mis_first = (mis0 + first_col * v7) & 7, mis_stride = (col_step * v7) & 7;
    const int mine = a.cols > first_col ? (a.cols - first_col + col_step - 1) / col_step : 0;   // pieces of this warp
    if (wl == 0)
        for (int k = 0; k < kRing && k < mine; ++k) {
            const int mis = (mis_first + k * mis_stride) & 7;
            fetch(k, at_first + k * col_stride - mis, mis);
        }

    // Window entry of an id, or at least `limit`: one unsigned comparison keeps ids
    // outside the window and the vocabulary out (where the window starts below
    // zero, ids -8 .. -1 land on entries that are no column's).
    const uint32_t limit = (uint32_t)(a.V - w0 < kWindow ? a.V - w0 : kWindow);
    auto entry = [&](int32_t id) -> uint32_t { return (uint32_t)id - (uint32_t)w0; };
    auto touch = [&](uint32_t e) {   // (common tokens set their bit once)
        const uint32_t bit = 1u << (e & 31);
        if (!(*reinterpret_cast<volatile uint32_t *>(&touched[e >> 5]) & bit)) atomicOr(&touched[e >> 5], bit);
    };
    if (tid < a.cols) {
        // the draft that counts as output from column tid on; the column's mask
        const uint32_t e = tid > 0 && a.drafts ? entry(__ldg(a.drafts + lane * (a.cols - 1) + tid - 1)) : limit;
        draft_entry[tid] = e < limit ? (int)e : -1;
        if (e < limit) {
            atomicOr(&count[e], kDraft);
            touch(e);
        }
        const int32_t row = a.mask ? __ldg(a.mask_rows + lane * a.cols + tid) : -1;
        mask_row[tid] = row >= 0 && row < a.mask_count ? row : -1;
    }
    if (a.history) {
        const int32_t *h = a.history + lane * a.history_stride;
        const int64_t whole = clamp_len(__ldg(a.history_lens + lane), a.history_stride);
        const int64_t prompt = clamp_len(__ldg(a.prompt_lens + lane), whole);
        auto met = [&](int32_t id, int64_t i) {
            const uint32_t e = entry(id);
            if (e < limit) {
                if (i < prompt) atomicOr(&count[e], kSeen);
                else atomicAdd(&count[e], 1u);
                touch(e);
            }
        };
        // Four ids a load from the first 16-byte boundary on, kAhead loads in
        // flight.  Few ids fall into the slice: a bit each, and the code that counts
        // one stands once (unrolled for every id it was 13 KB, and
        // fetching it took a CTA 3 us).
        const int64_t head0 = (16 - (reinterpret_cast<uintptr_t>(h) & 15)) / 4 % 4, head = head0 < whole ? head0 : whole;
        const int64_t quads = (whole - head) / 4;
        const int4 *h4 = reinterpret_cast<const int4 *>(h + head);
        constexpr int kAhead = 8;
#pragma unroll 1
        for (int64_t q = tid; q < quads; q += kAhead * kThreads) {
            int4 id[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                id[u] = q + u * kThreads < quads ? __ldg(h4 + q + u * kThreads) : make_int4(kNoId, kNoId, kNoId, kNoId);
            uint32_t hits = 0u;
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                hits |= (entry(id[u].x) < limit ? 1u << (4 * u) : 0u) | (entry(id[u].y) < limit ? 2u << (4 * u) : 0u) |
                        (entry(id[u].z) < limit ? 4u << (4 * u) : 0u) | (entry(id[u].w) < limit ? 8u << (4 * u) : 0u);
#pragma unroll 1
            while (hits) {
                const int u = (__ffs(hits) - 1) >> 2;
                const uint32_t some = hits >> (4 * u);
                const int64_t at = q + u * kThreads, i = head + 4 * at;
                const int4 four = __ldg(h4 + at);         // (from L1)
                if (some & 1u) met(four.x, i);
                if (some & 2u) met(four.y, i + 1);
                if (some & 4u) met(four.z, i + 2);
                if (some & 8u) met(four.w, i + 3);
                hits &= ~(15u << (4 * u));
            }
        }
        const int64_t tail = head + 4 * quads, i = tid < head ? tid : tail + tid - head;
        if (i < whole && (tid < head || i >= tail)) met(__ldg(h + i), i);
    }
    const int32_t *bias_ids = a.bias_ids + lane * a.max_bias;
    const float *bias_vals = a.bias_vals + lane * a.max_bias;
    const int64_t biases = a.bias_ids ? clamp_len(__ldg(a.bias_lens + lane), a.max_bias) : 0;
    if (biases > 0) {
        for (int64_t i = tid; i < biases; i += kThreads) {
            const uint32_t e = entry(__ldg(bias_ids + i));
            if (e < limit) {
                if (atomicOr(&count[e], kBiased) & kBiased) bias_again = 1;
                else bias[e] = __ldg(bias_vals + i);
                touch(e);
            }
        }
    }
    float r = 1.f, f = 0.f, p = 0.f;
    if (a.penalties) {
        r = __ldg(a.penalties + 3 * lane);
        f = __ldg(a.penalties + 3 * lane + 1);
        p = __ldg(a.penalties + 3 * lane + 2);
    }
    const float over_r = 1.f / r;   // one divide a lane; x * (1 / r) is within 1.5 fp32 units of x / r
    const int64_t words = (a.V + 31) / 32;
    const uint32_t *mask0 = a.mask ? a.mask + (t0 >> 5) : nullptr;
    __syncthreads();

    // An id given twice: the first of its places adds them all up, in their order.
    if (bias_again)
        for (int64_t i = tid; i < biases; i += kThreads) {
            const int32_t id = __ldg(bias_ids + i);
            if (entry(id) >= limit) continue;
            int64_t j = 0;
            while (j < i && __ldg(bias_ids + j) != id) ++j;
            if (j < i) continue;
            float sum = __ldg(bias_vals + i);
            for (j = i + 1; j < biases; ++j)
                if (__ldg(bias_ids + j) == id) sum = __fadd_rn(sum, __ldg(bias_vals + j));
            bias[entry(id)] = sum;
        }

    // The pieces' lists, in order, from the bits.  Entry e is element e - 8 + mis
    // of the slice: a piece's list has the first eight entries of the next piece too.
    uint16_t *list = lists + piece * kList;
    if (warp < kPieces) {
        constexpr int kBits = kPiece / 32;
        const uint32_t *bits = touched + piece * kBits;
        int n = 0;
        for (int w0 = 0; w0 <= kBits; w0 += 32) {
            uint32_t own = w0 + wl < kBits ? bits[w0 + wl] : w0 + wl == kBits ? bits[kBits] & 0xFFu : 0u;
            for (uint32_t some = __ballot_sync(kFull, own != 0u); some; some &= some - 1) {
                const int w = __ffs(some) - 1;
                const uint32_t word = __shfl_sync(kFull, own, w);
                if ((word >> wl) & 1u) list[n + __popc(word & lanemask_lt())] = (uint16_t)(piece * kPiece + 32 * (w0 + w) + wl);
                n += __popc(word);
            }
        }
        if (wl == 0) n_listed[piece] = n;
    }
    __syncthreads();
    const int n = n_listed[piece];

    auto stream = [&](auto inner_tag) {
        constexpr bool kInner = decltype(inner_tag)::value;
        // The mask words of a lane's vectors, a piece ahead of their use (a column's
        // mask lies in memory of its own, read once).
        auto mask_words = [&](int row, int mis, uint2 (&m)[kPer]) {
            if (row < 0) return;
            const int rel = piece * kPiece + 8 * wl - mis, w = rel >> 5;   // w: floor, also below 0
            const uint32_t *q = mask0 + row * words + w;
            const bool both = (rel & 31) > 24;            // a vector's bits lie in two words
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                m[u] = make_uint2(0u, 0u);
                if (!kInner && rel + 256 * u >= end) break;
                if (kInner || u > 0 || t0 > 0 || w >= 0) m[u].x = __ldg(q + 8 * u);
                if (both && (kInner || 32 * (w + 8 * u + 1) < end)) m[u].y = __ldg(q + 8 * u + 1);
            }
        };
        uint2 words_now[kPer], words_next[kPer];
        int mis = mis_first, row = mine > 0 ? mask_row[first_col] : -1;
        int64_t at = at_first;
        mask_words(row, mis, words_now);
#pragma unroll 1
        for (int k = 0, j = first_col; k < mine; ++k, j += col_step) {
            const Part pt = kInner ? Part{0, kPiece, 0, kPiece / 8} : part(mis);
            const int64_t at0 = at - mis;
            const int place = k % kRing, mis_next = (mis + mis_stride) & 7, row_next = k + 1 < mine ? mask_row[j + col_step] : -1;
            uint16_t *x = ring + place * kPiece;
            mask_words(row_next, mis_next, words_next);
            mbar_wait(&full[warp][place], (k / kRing) & 1);
            if (!kInner && (pt.v0 > 0 || pt.v1 < kPiece / 8)) {   // the ends of the column
                const int e = wl < 8 ? 8 * (pt.v0 - 1) + wl : 8 * pt.v1 + wl - 8;
                if (wl < 16 && e >= 0 && e < kPiece && e >= pt.lo && e < pt.hi) x[e] = a.logits[at0 + e];
                __syncwarp();
            }
            const int first = pt.lo > 0 ? pt.lo : 0, many = (pt.hi < kPiece ? pt.hi : kPiece) - first;
            const int shift = 8 + piece * kPiece - mis + first;   // from an entry to its place past `first`
#pragma unroll 1
            for (int i = wl; i < n; i += 32) {
                const int e = list[i], at = e - shift;
                if ((uint32_t)at >= (uint32_t)many || (!kInner && many <= 0)) continue;
                const uint32_t c = count[e];
                uint32_t m = c & ~(kSeen | kDraft | kBiased);
                if (c & kDraft)                            // its count grows along the columns
                    for (int d = 1; d <= j; ++d) m += draft_entry[d] == e;
                const float v = bf16_as_float(x[at + first]);
                const float factor = (c & kSeen) || m ? (v > 0.f ? over_r : r) : 1.f;
                const float take = __fadd_rn(__fmul_rn(f, (float)m), m ? p : 0.f);
                const float z = __fsub_rn(__fmul_rn(v, factor), take);
                x[at + first] = to_bf16(a.bias_ids ? __fadd_rn(z, bias[e]) : z);
            }
            if (row >= 0) {
                __syncwarp();
                uint4 *vec = reinterpret_cast<uint4 *>(x) + wl;
                const uint32_t bit = (uint32_t)(8 * wl - mis) & 31u;
#pragma unroll
                for (int u = 0; u < kPer; ++u) {
                    const uint32_t allowed = __funnelshift_r(words_now[u].x, words_now[u].y, bit) & 0xFFu;
                    if (allowed == 0xFFu || (!kInner && 8 * (wl + 32 * u) >= pt.hi)) continue;
                    uint4 q = make_uint4(kMasked, kMasked, kMasked, kMasked);
                    if (allowed != 0u) {
                        q = vec[32 * u];
                        // bit k of four to the top of byte k, then 16 copies of each top bit: the words' masks
                        const uint32_t l = (allowed & 15u) * 0x10204080u, h = (allowed >> 4) * 0x10204080u;
                        auto keep = [](uint32_t w, uint32_t m) { return (w & m) | (kMasked & ~m); };
                        q.x = keep(q.x, copies(l, 0x9988));
                        q.y = keep(q.y, copies(l, 0xBBAA));
                        q.z = keep(q.z, copies(h, 0x9988));
                        q.w = keep(q.w, copies(h, 0xBBAA));
                    }
                    vec[32 * u] = q;
                }
            }
            if (n > 0 || row >= 0 || !kInner) fence_proxy_async();
            __syncwarp();
            if (same_phase) {
                if (!kInner && (pt.v0 > 0 || pt.v1 < kPiece / 8)) {
                    const int e = wl < 8 ? 8 * (pt.v0 - 1) + wl : 8 * pt.v1 + wl - 8;
                    if (wl < 16 && e >= 0 && e < kPiece && e >= pt.lo && e < pt.hi) a.out[at0 + e] = x[e];
                }
                if (wl == 0) {
                    if (kInner || pt.v1 > pt.v0) bulk_s2g(a.out + at0 + 8 * pt.v0, x + 8 * pt.v0, (uint32_t)(pt.v1 - pt.v0) * 16);
                    bulk_commit();                         // a group a piece, empty or not
                }
            } else {
                for (int e = wl; e < kPiece; e += 32)
                    if (e >= pt.lo && e < pt.hi) a.out[at0 + e] = x[e];
                fence_proxy_async();                       // (the next copy comes over what was read)
                __syncwarp();
            }
#pragma unroll
            for (int u = 0; u < kPer; ++u) words_now[u] = words_next[u];
            // The place of the piece before this one takes the next load: its store has
            // had this piece's time to read it, and the warp's own reads are past a
            // barrier (and a proxy fence).
            if (wl == 0 && k > 0 && k - 1 + kRing < mine) {
                bulk_wait_read<1>();
                const int steps = kRing - 1, mis_then = (mis + steps * mis_stride) & 7;
                fetch((k - 1) % kRing, at + steps * col_stride - mis_then, mis_then);
            }
            mis = mis_next;
            row = row_next;
            at += col_stride;
        }
    };
    if (inner) stream(Yes());
    else stream(No());
    if (wl == 0) {
        bulk_wait_all();
        // given up on a load: it may still be on its way into this CTA's memory (bounded)
        if (*reinterpret_cast<volatile unsigned int *>(&s_gave_up))
            for (int k = mine > kRing ? mine - kRing : 0; k < mine; ++k) {
                const uint64_t since = global_ns();
                while (!mbar_try_wait(&full[warp][k % kRing], (k / kRing) & 1) && global_ns() - since < kWaitLimitNs) {}
            }
    }
}

}  // namespace rules
