// Attention of a chunk of new tokens over the paged cache: the simplest form,
// one warp per (new token, query head), keys one after the other.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace attn {

struct Args {
    const uint16_t *q;
    int64_t tokens, qs_t, qs_h;
    int32_t heads_q, group;
    spec_paged_cache c;
    const int32_t *block_table, *cu_new, *seq_lens;
    int32_t lanes;
    int64_t max_pages;
    float scale;
    int64_t window;
    uint16_t *out;
    float *lse;
};

template <bool F16>
__device__ __forceinline__ float widen(uint16_t x)
{
    if (F16) return __half2float(__ushort_as_half(x));
    return __bfloat162float(__ushort_as_bfloat16(x));
}

template <bool F16>
__device__ __forceinline__ uint16_t narrow(float x)
{
    if (F16) return __half_as_ushort(__float2half_rn(x));
    return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

template <bool F16>
__global__ void __launch_bounds__(128) simple_kernel(const __grid_constant__ Args a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, per = a.c.head_dim / 32;
    const int64_t nw = (int64_t)gridDim.x * 4;
    const int64_t total = min((int64_t)__ldg(a.cu_new + a.lanes), a.tokens);
    for (int64_t w = (int64_t)blockIdx.x * 4 + threadIdx.x / 32; w < total * a.heads_q; w += nw) {
        const int64_t t = w / a.heads_q;
        const int h = (int)(w % a.heads_q), kh = h / a.group;
        int lo = 0, hi = a.lanes - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (__ldg(a.cu_new + mid) <= t) lo = mid; else hi = mid - 1;
        }
        const int64_t n = __ldg(a.cu_new + lo + 1) - __ldg(a.cu_new + lo);
        const int64_t pos = __ldg(a.seq_lens + lo) - n + (t - __ldg(a.cu_new + lo));
        const int64_t first = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
        float q[8], o[8] = {0.f}, m = -INFINITY, l = 0.f;
        for (int i = 0; i < per; ++i) q[i] = widen<F16>(a.q[t * a.qs_t + h * a.qs_h + lane * per + i]);
        for (int64_t j = first; j <= pos; ++j) {
            const int64_t pi = j / a.c.page_size;
            const int32_t page = pi < a.max_pages ? __ldg(a.block_table + lo * a.max_pages + pi) : -1;
            const bool real = page >= 0 && page < a.c.pages;
            const uint16_t *k = static_cast<const uint16_t *>(a.c.k) + page * a.c.k_strides[0] +
                                (j % a.c.page_size) * a.c.k_strides[1] + kh * a.c.k_strides[2] + lane * per;
            const uint16_t *v = static_cast<const uint16_t *>(a.c.v) + page * a.c.v_strides[0] +
                                (j % a.c.page_size) * a.c.v_strides[1] + kh * a.c.v_strides[2] + lane * per;
            float s = 0.f;
            for (int i = 0; i < per; ++i) s += q[i] * (real ? widen<F16>(k[i]) : 0.f);
            for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
            s *= a.scale;
            const float mn = fmaxf(m, s), f = __expf(m - mn), p = __expf(s - mn);
            l = l * f + p;
            m = mn;
            for (int i = 0; i < per; ++i) o[i] = o[i] * f + p * (real ? widen<F16>(v[i]) : 0.f);
        }
        for (int i = 0; i < per; ++i)
            a.out[(t * a.heads_q + h) * a.c.head_dim + lane * per + i] = narrow<F16>(l > 0.f ? o[i] / l : 0.f);
        if (lane == 0 && a.lse) a.lse[t * a.heads_q + h] = l > 0.f ? m + logf(l) : -INFINITY;
    }
}

}  // namespace attn
