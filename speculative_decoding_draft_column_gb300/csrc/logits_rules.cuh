// Penalties for repeated tokens, biases and grammar masks on bf16 logits.
//
// Column j of a lane, token t, in fp32 and rounded once:
//   x = t seen ? (x > 0 ? x / r : x * r) : x        (prompt, output, drafts before j)
//   x -= f * n + p * (n > 0)                        (n: output and drafts before j)
//   x += bias(t);   x = -inf where the grammar's bit is clear.
#pragma once

#include "common.cuh"

namespace rules {

constexpr int kThreads = 512;
constexpr int kSlice = 8 * kThreads;     // tokens of a slice: one 16-byte vector a thread and column
constexpr int kWindow = kSlice + 8;      // a column's vectors may start up to 7 elements before the slice
constexpr int kBatch = 4;                // columns whose loads are in flight together
// Counts and biases lie by token mod 8: element i of every thread's vector is
// read by consecutive threads from consecutive words.
constexpr int kPitch = kWindow / 8;
__device__ __forceinline__ int place(int e) { return (e & 7) * kPitch + (e >> 3); }
constexpr uint32_t kSeen = 0x80000000u;  // the token is in the prompt; the other bits count the output

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

struct Yes { static constexpr bool value = true; };
struct No { static constexpr bool value = false; };

__device__ __forceinline__ uint16_t to_bf16(float f)
{
    uint16_t h;
    asm("{\n\t.reg .b16 r;\n\tcvt.rn.bf16.f32 r, %1;\n\tmov.b16 %0, r;\n\t}" : "=h"(h) : "f"(f));
    return h;
}

// bytes of the sign bits that the selector's nibbles (8 + byte) name
__device__ __forceinline__ uint32_t copies(uint32_t v, uint32_t selector)
{
    uint32_t d;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(d) : "r"(v), "r"(selector));
    return d;
}

__device__ __forceinline__ int64_t clamp_len(int32_t n, int64_t most) { return n < 0 ? 0 : n > most ? most : n; }

// One CTA per (slice of the vocabulary, lane): it counts the lane's history
// over its slice in shared memory, then streams the slice of every column of
// the lane.  A bit per token says whether anything but the mask can change it:
// a vector none of whose tokens was seen costs one test, and only the seen
// tokens of the others go through the rules, one after the other.  The mask is read first,
// and a vector that it leaves nothing of is not read at all.
__global__ void __launch_bounds__(kThreads, 3) process_kernel(const __grid_constant__ Args a)
{
    __shared__ uint32_t count[kWindow];
    __shared__ float bias[kWindow];
    __shared__ uint32_t touched[kWindow / 32 + 2];
    __shared__ int32_t draft_entry[SPEC_MAX_GAMMA + 1], mask_row[SPEC_MAX_GAMMA + 1];
    const int tid = threadIdx.x;
    const int64_t lane = blockIdx.y, t0 = (int64_t)blockIdx.x * kSlice;
    const int64_t w0 = t0 - 8;   // the token of window entry 0
    pdl_launch_dependents();
    for (int i = tid; i < kWindow; i += kThreads) {
        count[i] = 0u;
        bias[i] = 0.f;
    }
    if (tid < kWindow / 32 + 2) touched[tid] = 0u;
    pdl_wait();
    __syncthreads();

    auto entry = [&](int32_t id) -> int {   // window entry of an id, -1 outside
        const int64_t e = (int64_t)id - w0;
        return id >= 0 && id < a.V && e >= 0 && e < kWindow ? (int)e : -1;
    };
    auto touch = [&](int e) { atomicOr(&touched[e >> 5], 1u << (e & 31)); };
    if (tid < a.cols) {
        // the draft that counts as output from column tid on; the column's mask
        draft_entry[tid] = tid > 0 && a.drafts ? entry(__ldg(a.drafts + lane * (a.cols - 1) + tid - 1)) : -1;
        const int32_t row = a.mask ? __ldg(a.mask_rows + lane * a.cols + tid) : -1;
        mask_row[tid] = row >= 0 && row < a.mask_count ? row : -1;
    }
    if (a.history) {
        const int64_t whole = clamp_len(__ldg(a.history_lens + lane), a.history_stride);
        const int64_t prompt = clamp_len(__ldg(a.prompt_lens + lane), whole);
        const int32_t *h = a.history + lane * a.history_stride;
        constexpr int kAhead = 8;   // ids in flight a thread
        for (int64_t i0 = tid; i0 < whole; i0 += kAhead * kThreads) {
            int32_t id[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) id[u] = i0 + u * kThreads < whole ? __ldg(h + i0 + u * kThreads) : -1;
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int e = entry(id[u]);
                if (e >= 0) {
                    if (i0 + u * kThreads < prompt) atomicOr(&count[place(e)], kSeen);
                    else atomicAdd(&count[place(e)], 1u);
                    touch(e);
                }
            }
        }
    }
    if (a.bias_ids) {
        const int64_t nb = clamp_len(__ldg(a.bias_lens + lane), a.max_bias);
        for (int64_t i = tid; i < nb; i += kThreads) {
            const int e = entry(__ldg(a.bias_ids + lane * a.max_bias + i));
            if (e >= 0) {
                atomicAdd(&bias[place(e)], __ldg(a.bias_vals + lane * a.max_bias + i));
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
    __syncthreads();

    auto rule = [&](uint32_t raw, int at) -> uint32_t {   // at: the token's place
        const uint32_t c = count[at], n = c & ~kSeen;
        const float x = bf16_as_float(raw);
        const float y = __fmul_rn(x, c == 0u ? 1.f : x > 0.f ? over_r : r);
        const float z = __fsub_rn(y, __fadd_rn(__fmul_rn(f, (float)n), n ? p : 0.f));
        return to_bf16(__fadd_rn(z, bias[at]));
    };
    const int64_t words = (a.V + 31) / 32;
    const bool same_phase = ((reinterpret_cast<uintptr_t>(a.logits) ^ reinterpret_cast<uintptr_t>(a.out)) & 15) == 0;
    const int base_mis = (int)((reinterpret_cast<uintptr_t>(a.logits) & 15) / 2);
    const int64_t col0 = lane * a.cols;

    // A vector starts at token t0 + rel of its column; rel = 8 * tid - mis, where
    // mis (the same for the whole CTA) is the column's phase.
    const uint16_t *in0 = a.logits + col0 * a.V + t0;
    uint16_t *out0 = a.out + col0 * a.V + t0;
    const uint32_t *mask0 = a.mask ? a.mask + (t0 >> 5) : nullptr;
    const int mis0 = (int)((base_mis + col0 * a.V + t0) & 7), v7 = (int)(a.V & 7);
    const int64_t left = a.V - t0;                  // tokens from t0 to the column's end
    const int end = left > kSlice ? kSlice + 8 : (int)left, begin = t0 > 0 ? -8 : 0;   // tokens [begin, end) are the column's

    // kInner: no vector of the slice reaches over an end of its column, in
    // whatever phase, and input and output vectors line up
    auto stream = [&](auto inner) {
        constexpr bool kInner = decltype(inner)::value;
        for (int j0 = 0; j0 < a.cols; j0 += kBatch) {
            uint4 x[kBatch];
            uint32_t allowed[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                allowed[u] = 0xFFu;
                const int j = j0 + u, row = j < a.cols ? mask_row[j] : -1;
                if (row < 0) continue;
                const int rel = 8 * tid - ((mis0 + j * v7) & 7), w = rel >> 5;   // w: floor, also below 0
                const uint32_t *m = mask0 + row * words + w;
                uint32_t lo = 0u, hi = 0u;
                if (kInner || (rel < end && (t0 > 0 || w >= 0))) lo = __ldg(m);
                if ((rel & 31) > 24 && (kInner || 32 * (w + 1) < end)) hi = __ldg(m + 1);
                allowed[u] = __funnelshift_r(lo, hi, (uint32_t)(rel & 31)) & 0xFFu;
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                x[u] = make_uint4(0, 0, 0, 0);
                const int j = j0 + u;
                if (j >= a.cols || allowed[u] == 0u) continue;
                const int rel = 8 * tid - ((mis0 + j * v7) & 7);
                const uint16_t *src = in0 + j * a.V + rel;
                if (kInner || (rel >= begin && rel + 8 <= end)) x[u] = __ldcs(reinterpret_cast<const uint4 *>(src));
                else if (rel + 8 > begin && rel < end) x[u] = load_edge(src, 0, 0, begin - rel, end - rel);
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int j = j0 + u;
                if (j >= a.cols) break;
                const int e = draft_entry[j];
                if (e >= 0) {          // the same for the whole CTA
                    __syncthreads();
                    if (tid == 0) {
                        count[place(e)] += 1u;
                        touched[e >> 5] |= 1u << (e & 31);
                    }
                    __syncthreads();
                }
                const int rel = 8 * tid - ((mis0 + j * v7) & 7);
                if (!kInner && (rel + 8 <= begin || rel >= end)) continue;
                const int e0 = rel + 8;
                uint32_t todo = __funnelshift_r(touched[e0 >> 5], touched[(e0 >> 5) + 1], (uint32_t)(e0 & 31)) & allowed[u];
                uint4 w = x[u];
                // many seen tokens in one of the warp's vectors: all eight of
                // each at once, so that their reads overlap (a vector with few goes
                // one by one: a third of the instructions)
                if (__any_sync(__activemask(), __popc(todo) > 2)) {
                    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
                    uint32_t out[4];
                    const int low = e0 & 7, at0 = e0 >> 3;   // low: the same for every thread
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int p0 = (low + 2 * k) & 7, p1 = (low + 2 * k + 1) & 7;
                        const uint32_t a0 = rule(in[k] & 0xFFFFu, p0 * kPitch + at0 + (low + 2 * k >= 8));
                        const uint32_t a1 = rule(in[k] >> 16, p1 * kPitch + at0 + (low + 2 * k + 1 >= 8));
                        out[k] = ((todo >> (2 * k)) & 1u ? a0 : in[k] & 0xFFFFu) |
                                 ((todo >> (2 * k + 1)) & 1u ? a1 << 16 : in[k] & 0xFFFF0000u);
                    }
                    w = make_uint4(out[0], out[1], out[2], out[3]);
                    todo = 0u;
                }
                while (todo) {
                    const int i = __ffs(todo) - 1;
                    todo &= todo - 1;
                    const uint32_t old = i < 4 ? (i < 2 ? w.x : w.y) : (i < 6 ? w.z : w.w);
                    const uint32_t raw = rule((i & 1) ? old >> 16 : old & 0xFFFFu, place(e0 + i));
                    const uint32_t now = __byte_perm(old, raw, (i & 1) ? 0x5410 : 0x3254);
                    if (i < 2) w.x = now;
                    else if (i < 4) w.y = now;
                    else if (i < 6) w.z = now;
                    else w.w = now;
                }
                if (allowed[u] != 0xFFu) {
                    // bit k of four to the top of byte k, then 16 copies of each
                    // top bit: the words' masks
                    const uint32_t lo = (allowed[u] & 15u) * 0x10204080u, hi = (allowed[u] >> 4) * 0x10204080u;
                    auto keep = [](uint32_t v, uint32_t m) { return (v & m) | (0xFF80FF80u & ~m); };
                    w.x = keep(w.x, copies(lo, 0x9988));
                    w.y = keep(w.y, copies(lo, 0xBBAA));
                    w.z = keep(w.z, copies(hi, 0x9988));
                    w.w = keep(w.w, copies(hi, 0xBBAA));
                }
                uint16_t *dst = out0 + j * a.V + rel;
                if (kInner || (same_phase && rel >= begin && rel + 8 <= end)) {
                    __stcs(reinterpret_cast<uint4 *>(dst), w);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t word = i < 4 ? (i < 2 ? w.x : w.y) : (i < 6 ? w.z : w.w);
                        if (rel + i >= begin && rel + i < end) dst[i] = (uint16_t)(word >> (16 * (i & 1)));
                    }
                }
            }
        }
    };
    if (same_phase && t0 >= 8 && t0 + kSlice <= a.V) stream(Yes());
    else stream(No());
}

}  // namespace rules
