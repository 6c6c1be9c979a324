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

__device__ __forceinline__ uint16_t to_bf16(float f)
{
    uint16_t h;
    asm("{\n\t.reg .b16 r;\n\tcvt.rn.bf16.f32 r, %1;\n\tmov.b16 %0, r;\n\t}" : "=h"(h) : "f"(f));
    return h;
}

__device__ __forceinline__ int64_t clamp_len(int32_t n, int64_t most) { return n < 0 ? 0 : n > most ? most : n; }

// One CTA per (slice of the vocabulary, lane): it counts the lane's history
// over its slice in shared memory, then streams the slice of every column of
// the lane.  A bit per token says whether anything but the mask can change it,
// so that a vector none of whose tokens was seen costs one test.
__global__ void __launch_bounds__(kThreads, 4) process_kernel(const __grid_constant__ Args a)
{
    pdl_launch_dependents();
    pdl_wait();
    __shared__ uint32_t count[kWindow];
    __shared__ float bias[kWindow];
    __shared__ uint32_t touched[kWindow / 32 + 2];
    const int tid = threadIdx.x;
    const int64_t lane = blockIdx.y, t0 = (int64_t)blockIdx.x * kSlice;
    const int64_t w0 = t0 - 8;   // the token of window entry 0
    for (int i = tid; i < kWindow; i += kThreads) {
        count[i] = 0u;
        bias[i] = 0.f;
    }
    if (tid < kWindow / 32 + 2) touched[tid] = 0u;
    __syncthreads();

    auto entry = [&](int32_t id) -> int {   // window entry of an id, -1 outside
        const int64_t e = (int64_t)id - w0;
        return id >= 0 && id < a.V && e >= 0 && e < kWindow ? (int)e : -1;
    };
    auto touch = [&](int e) { atomicOr(&touched[e >> 5], 1u << (e & 31)); };
    if (a.history) {
        const int64_t whole = clamp_len(__ldg(a.history_lens + lane), a.history_stride);
        const int64_t prompt = clamp_len(__ldg(a.prompt_lens + lane), whole);
        const int32_t *h = a.history + lane * a.history_stride;
        for (int64_t i = tid; i < whole; i += kThreads) {
            const int e = entry(__ldg(h + i));
            if (e >= 0) {
                if (i < prompt) atomicOr(&count[e], kSeen);
                else atomicAdd(&count[e], 1u);
                touch(e);
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
    __syncthreads();

    auto rule = [&](uint32_t raw, int e) -> uint16_t {
        const uint32_t c = count[e];
        float x = bf16_as_float(raw);
        if (c) {
            x = x > 0.f ? __fdiv_rn(x, r) : __fmul_rn(x, r);
            const uint32_t n = c & ~kSeen;
            x = __fsub_rn(x, __fadd_rn(__fmul_rn(f, (float)n), n ? p : 0.f));
        }
        return to_bf16(__fadd_rn(x, bias[e]));
    };
    const int words = (int)((a.V + 31) / 32);
    const bool same_phase = ((reinterpret_cast<uintptr_t>(a.logits) ^ reinterpret_cast<uintptr_t>(a.out)) & 15) == 0;
    const int base_mis = (int)((reinterpret_cast<uintptr_t>(a.logits) & 15) / 2);

    // the column's vector of this thread: it starts at token t (maybe below 0)
    auto first_token = [&](int64_t c) -> int64_t {
        const int mis = (int)((base_mis + c * a.V + t0) & 7);
        return t0 - mis + 8 * tid;
    };
    for (int j0 = 0; j0 < a.cols; j0 += kBatch) {
        uint4 x[kBatch];
        uint32_t allowed[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            x[u] = make_uint4(0, 0, 0, 0);
            allowed[u] = 0xFFu;
            const int j = j0 + u;
            if (j >= a.cols) continue;
            const int64_t c = lane * a.cols + j, t = first_token(c);
            const uint16_t *src = a.logits + c * a.V;
            if (t >= 0 && t + 8 <= a.V) x[u] = __ldcs(reinterpret_cast<const uint4 *>(src + t));
            else if (t + 8 > 0 && t < a.V) x[u] = load_edge(src + t, 0, 0, -t, a.V - t);
            if (a.mask && t + 8 > 0 && t < a.V) {
                const int32_t row = __ldg(a.mask_rows + c);
                if (row >= 0 && row < a.mask_count) {
                    const uint32_t *m = a.mask + (int64_t)row * words;
                    const int64_t w = t >> 5;   // floor, also below 0
                    const uint32_t lo = w >= 0 ? __ldg(m + w) : 0u, hi = w + 1 < words ? __ldg(m + w + 1) : 0u;
                    allowed[u] = __funnelshift_r(lo, hi, (uint32_t)(t & 31)) & 0xFFu;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int j = j0 + u;
            if (j >= a.cols) break;
            if (j > 0 && a.drafts) {   // the draft before this column counts as output from here on
                const int e = entry(__ldg(a.drafts + lane * (a.cols - 1) + j - 1));
                if (e >= 0) {          // the same for the whole CTA
                    __syncthreads();
                    if (tid == 0) {
                        count[e] += 1u;
                        touched[e >> 5] |= 1u << (e & 31);
                    }
                    __syncthreads();
                }
            }
            const int64_t c = lane * a.cols + j, t = first_token(c);
            if (t + 8 <= 0 || t >= a.V) continue;
            const int e0 = (int)(t - w0);
            const uint32_t hit = __funnelshift_r(touched[e0 >> 5], touched[(e0 >> 5) + 1], (uint32_t)(e0 & 31)) & 0xFFu;
            uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            const uint32_t act = hit | (~allowed[u] & 0xFFu);
            if (act) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (!((act >> i) & 1u)) continue;
                    uint32_t raw = (w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
                    if (!((allowed[u] >> i) & 1u)) raw = 0xFF80u;
                    else raw = rule(raw, e0 + i);
                    w[i >> 1] = (i & 1) ? (w[i >> 1] & 0xFFFFu) | (raw << 16) : (w[i >> 1] & 0xFFFF0000u) | raw;
                }
            }
            uint16_t *dst = a.out + c * a.V;
            if (same_phase && t >= 0 && t + 8 <= a.V) {
                __stcs(reinterpret_cast<uint4 *>(dst + t), make_uint4(w[0], w[1], w[2], w[3]));
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (t + i >= 0 && t + i < a.V) dst[t + i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
            }
        }
    }
}

}  // namespace rules
