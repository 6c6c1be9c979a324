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
                    if (i0 + u * kThreads < prompt) atomicOr(&count[e], kSeen);
                    else atomicAdd(&count[e], 1u);
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
                atomicAdd(&bias[e], __ldg(a.bias_vals + lane * a.max_bias + i));
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

    auto rule = [&](uint32_t raw, int e) -> uint32_t {
        const uint32_t c = count[e];
        float x = bf16_as_float(raw);
        if (c) {
            x = __fmul_rn(x, x > 0.f ? over_r : r);
            const uint32_t n = c & ~kSeen;
            x = __fsub_rn(x, __fadd_rn(__fmul_rn(f, (float)n), n ? p : 0.f));
        }
        return to_bf16(__fadd_rn(x, bias[e]));
    };
    const int64_t words = (a.V + 31) / 32;
    const bool same_phase = ((reinterpret_cast<uintptr_t>(a.logits) ^ reinterpret_cast<uintptr_t>(a.out)) & 15) == 0;
    const int base_mis = (int)((reinterpret_cast<uintptr_t>(a.logits) & 15) / 2);
    const int64_t col0 = lane * a.cols;

    // kInner: no vector of the slice reaches over an end of its column, in
    // whatever phase, and input and output vectors line up
    auto stream = [&](auto inner) {
        constexpr bool kInner = decltype(inner)::value;
        for (int j0 = 0; j0 < a.cols; j0 += kBatch) {
            uint4 x[kBatch];
            uint32_t allowed[kBatch];
            int mis[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                allowed[u] = 0xFFu;
                mis[u] = (int)((base_mis + (col0 + j0 + u) * a.V + t0) & 7);
                const int row = j0 + u < a.cols ? mask_row[j0 + u] : -1;
                if (row < 0) continue;
                const int64_t t = t0 + 8 * tid - mis[u], w = t >> 5;   // floor, also below 0
                const uint32_t *m = reinterpret_cast<const uint32_t *>(a.mask) + row * words + w;
                uint32_t lo = 0u, hi = 0u;
                if (kInner || (w >= 0 && w < words)) lo = __ldg(m);
                if ((t & 31) > 24 && (kInner || (w + 1 >= 0 && w + 1 < words))) hi = __ldg(m + 1);
                allowed[u] = __funnelshift_r(lo, hi, (uint32_t)(t & 31)) & 0xFFu;
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                x[u] = make_uint4(0, 0, 0, 0);
                if (j0 + u >= a.cols || allowed[u] == 0u) continue;
                const int64_t t = t0 + 8 * tid - mis[u];
                const uint16_t *src = a.logits + (col0 + j0 + u) * a.V + t;
                if (kInner || (t >= 0 && t + 8 <= a.V)) x[u] = __ldcs(reinterpret_cast<const uint4 *>(src));
                else if (t + 8 > 0 && t < a.V) x[u] = load_edge(src, 0, 0, -t, a.V - t);
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (j0 + u >= a.cols) break;
                const int e = draft_entry[j0 + u];
                if (e >= 0) {          // the same for the whole CTA
                    __syncthreads();
                    if (tid == 0) {
                        count[e] += 1u;
                        touched[e >> 5] |= 1u << (e & 31);
                    }
                    __syncthreads();
                }
                const int64_t t = t0 + 8 * tid - mis[u];
                if (!kInner && (t + 8 <= 0 || t >= a.V)) continue;
                const int e0 = 8 + 8 * tid - mis[u];
                uint32_t todo = __funnelshift_r(touched[e0 >> 5], touched[(e0 >> 5) + 1], (uint32_t)(e0 & 31)) & allowed[u];
                uint4 w = x[u];
                while (todo) {
                    const int i = __ffs(todo) - 1;
                    todo &= todo - 1;
                    const uint32_t old = i < 4 ? (i < 2 ? w.x : w.y) : (i < 6 ? w.z : w.w);
                    const uint32_t raw = rule((i & 1) ? old >> 16 : old & 0xFFFFu, e0 + i);
                    const uint32_t now = __byte_perm(old, raw, (i & 1) ? 0x5410 : 0x3254);
                    if (i < 2) w.x = now;
                    else if (i < 4) w.y = now;
                    else if (i < 6) w.z = now;
                    else w.w = now;
                }
                auto keep = [&](uint32_t v, int k) -> uint32_t {   // 16 bits per allowed bit, else -inf
                    const uint32_t two = (allowed[u] >> (2 * k)) & 3u;
                    const uint32_t m = (two & 1u) * 0xFFFFu + (two >> 1) * 0xFFFF0000u;
                    return (v & m) | (0xFF80FF80u & ~m);
                };
                if (allowed[u] != 0xFFu) w = make_uint4(keep(w.x, 0), keep(w.y, 1), keep(w.z, 2), keep(w.w, 3));
                uint16_t *dst = a.out + (col0 + j0 + u) * a.V + t;
                if (kInner || (same_phase && t >= 0 && t + 8 <= a.V)) {
                    __stcs(reinterpret_cast<uint4 *>(dst), w);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t word = i < 4 ? (i < 2 ? w.x : w.y) : (i < 6 ? w.z : w.w);
                        if (t + i >= 0 && t + i < a.V) dst[i] = (uint16_t)(word >> (16 * (i & 1)));
                    }
                }
            }
        }
    };
    if (same_phase && t0 >= 8 && t0 + kSlice <= a.V) stream(Yes());
    else stream(No());
}

}  // namespace rules
