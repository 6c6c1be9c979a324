// Checks of arguments that the paged and tree entry points share.
#pragma once

#include <stdint.h>

#include "host.h"

namespace {

inline bool misaligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// A call's buffer, for the checks of what must not overlap.
struct Range {
    const void *p;
    int64_t bytes;
    const char *name;
};
inline bool overlap(const Range &a, const Range &b)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.bytes > 0 && b.bytes > 0 && x < y + (uint64_t)b.bytes && y < x + (uint64_t)a.bytes;
}

constexpr int64_t kMaxStride = 1ll << 39;

inline bool bad_stride(int64_t s) { return s < 0 || s >= kMaxStride || s % 8 != 0; }

inline spec_status check_cache(const spec_paged_cache *c)
{
    if (!c || !c->k || !c->v) return host::fail(SPEC_ERR_ARG, "cache: null pointer");
    if (c->dtype != SPEC_BF16 && c->dtype != SPEC_F16) return host::fail(SPEC_ERR_ARG, "cache: unknown dtype %d", c->dtype);
    if (misaligned(c->k, 16) || misaligned(c->v, 16))
        return host::fail(SPEC_ERR_ARG, "cache: keys and values must be 16-byte aligned");
    if (c->pages < 1 || c->pages > INT32_MAX) return host::fail(SPEC_ERR_ARG, "cache: pages = %lld", (long long)c->pages);
    if (c->page_size < 1) return host::fail(SPEC_ERR_ARG, "cache: page_size = %d < 1", c->page_size);
    if (c->heads < 1) return host::fail(SPEC_ERR_ARG, "cache: heads = %d < 1", c->heads);
    if (c->head_dim < 8 || c->head_dim > 256 || c->head_dim % 8 != 0)
        return host::fail(SPEC_ERR_ARG, "cache: head_dim = %d, need a multiple of 8 up to 256", c->head_dim);
    if ((int64_t)c->heads * c->head_dim > INT32_MAX)
        return host::fail(SPEC_ERR_ARG, "cache: heads * head_dim = %lld exceeds 2^31-1", (long long)c->heads * c->head_dim);
    for (int i = 0; i < 3; ++i)
        if (bad_stride(c->k_strides[i]) || bad_stride(c->v_strides[i]))
            return host::fail(SPEC_ERR_ARG, "cache: strides must be non-negative multiples of 8 elements below 2^39");
    return SPEC_OK;
}

inline spec_status check_cache8(const spec_paged_cache8 *c)
{
    if (!c || !c->k || !c->v || !c->k_scales || !c->v_scales) return host::fail(SPEC_ERR_ARG, "cache: null pointer");
    if (c->dtype != SPEC_BF16 && c->dtype != SPEC_F16) return host::fail(SPEC_ERR_ARG, "cache: unknown dtype %d", c->dtype);
    if (misaligned(c->k, 16) || misaligned(c->v, 16) || misaligned(c->k_scales, 16) || misaligned(c->v_scales, 16))
        return host::fail(SPEC_ERR_ARG, "cache: codes and scales must be 16-byte aligned");
    if (c->pages < 1 || c->pages > INT32_MAX) return host::fail(SPEC_ERR_ARG, "cache: pages = %lld", (long long)c->pages);
    if (c->page_size < 1) return host::fail(SPEC_ERR_ARG, "cache: page_size = %d < 1", c->page_size);
    if (c->heads < 1) return host::fail(SPEC_ERR_ARG, "cache: heads = %d < 1", c->heads);
    if (c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16 != 0)
        return host::fail(SPEC_ERR_ARG, "cache: head_dim = %d, need a multiple of 16 up to 256", c->head_dim);
    if ((int64_t)c->heads * c->head_dim > INT32_MAX)
        return host::fail(SPEC_ERR_ARG, "cache: heads * head_dim = %lld exceeds 2^31-1", (long long)c->heads * c->head_dim);
    if ((__int128)c->pages * c->heads * c->page_size > INT64_MAX / 2)
        return host::fail(SPEC_ERR_ARG, "cache: pages * heads * page_size is too large");
    for (int i = 0; i < 3; ++i)
        if (bad_stride(c->k_strides[i]) || bad_stride(c->v_strides[i]) || c->k_strides[i] % 16 || c->v_strides[i] % 16)
            return host::fail(SPEC_ERR_ARG, "cache: strides must be non-negative multiples of 16 elements below 2^39");
    return SPEC_OK;
}

inline spec_status check_batch(const spec_paged_batch *b)
{
    if (!b) return host::fail(SPEC_ERR_ARG, "batch: null pointer");
    if (b->lanes < 0 || b->lanes > SPEC_PAGED_MAX_LANES)
        return host::fail(SPEC_ERR_ARG, "batch: lanes = %lld outside [0, %d]", (long long)b->lanes, SPEC_PAGED_MAX_LANES);
    if (b->max_pages < 1 || b->max_pages > INT32_MAX)
        return host::fail(SPEC_ERR_ARG, "batch: max_pages = %lld", (long long)b->max_pages);
    if (b->page_size < 1) return host::fail(SPEC_ERR_ARG, "batch: page_size = %d < 1", b->page_size);
    return SPEC_OK;
}

// New keys and values, and their slots (0 tokens: nothing else is looked at).
inline spec_status check_new(const void *k, const void *v, int64_t tokens, int64_t k_token_stride, int64_t k_head_stride,
                             int64_t v_token_stride, int64_t v_head_stride, const int64_t *slots)
{
    if (tokens < 0 || tokens > INT32_MAX) return host::fail(SPEC_ERR_ARG, "tokens = %lld", (long long)tokens);
    if (tokens == 0) return SPEC_OK;
    if (!k || !v || !slots) return host::fail(SPEC_ERR_ARG, "null pointer");
    if (misaligned(k, 16) || misaligned(v, 16) || misaligned(slots, 8))
        return host::fail(SPEC_ERR_ARG, "misaligned pointer (keys and values need 16 bytes, slots 8)");
    if (bad_stride(k_token_stride) || bad_stride(k_head_stride) || bad_stride(v_token_stride) ||
        bad_stride(v_head_stride))
        return host::fail(SPEC_ERR_ARG, "strides must be non-negative multiples of 8 elements below 2^39");
    return SPEC_OK;
}

}  // namespace
