// libspecsel: the paged key/value cache (plan of a step, store, attention of a
// chunk of new tokens) and the rules applied to logits -- argument checks,
// launches and the C ABI.

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <initializer_list>
#include <mutex>

#include "specsel.h"
#include "checks.h"
#include "common.cuh"
#include "paged.cuh"
#include "attention_launch.cuh"
#include "logits_rules.cuh"
#include "host.h"

using host::cuda_fail;
using host::fail;

namespace {

using attn::kMaxDevices;

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct Device {
    bool init = false;
    int index = 0, sms = 0;
    EncodeTiled encode = nullptr;
};

std::mutex g_paged_mu;
Device g_devices[kMaxDevices];

spec_status device(Device **out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(SPEC_ERR_CUDA, "device ordinal %d unsupported", dev);
    Device &d = g_devices[dev];
    std::lock_guard<std::mutex> lock(g_paged_mu);
    if (!d.init) {
        e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
        e = cudaFuncSetAttribute(paged::plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)paged::plan_smem(SPEC_PAGED_MAX_LANES));
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
        e = cudaFuncSetAttribute(rules::process_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, rules::smem_bytes(true));
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
        size_t smem = 0;   // (the kernels are loaded now, not inside a capture)
        const spec_status made[] = {attn::prepare<64, 1, false, false, false>(dev, &smem), attn::prepare<64, 1, true, false, false>(dev, &smem),
                                    attn::prepare<64, 2, false, false, false>(dev, &smem), attn::prepare<64, 2, true, false, false>(dev, &smem),
                                    attn::prepare<128, 1, false, false, false>(dev, &smem), attn::prepare<128, 1, true, false, false>(dev, &smem),
                                    attn::prepare<128, 2, false, false, false>(dev, &smem), attn::prepare<128, 2, true, false, false>(dev, &smem),
                                    attn::prepare<256, 1, false, false, false>(dev, &smem), attn::prepare<256, 1, true, false, false>(dev, &smem)};
        for (const spec_status st : made)
            if (st != SPEC_OK) return st;
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
        e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
        if (e != cudaSuccess) return cuda_fail(e, "cudaGetDriverEntryPointByVersion");
        if (!fn || found != cudaDriverEntryPointSuccess) return fail(SPEC_ERR_CUDA, "the driver has no cuTensorMapEncodeTiled");
        d.encode = reinterpret_cast<EncodeTiled>(fn);
        d.index = dev;
        d.init = true;
    }
    *out = &d;
    return SPEC_OK;
}

template <typename K, typename A>
spec_status launch(K kernel, dim3 grid, unsigned block, size_t smem, const A &a)
{
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = host::stream();
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e != cudaSuccess) return cuda_fail(e, "kernel launch");
    host::count_launch();
    return SPEC_OK;
}

constexpr int64_t max2(int64_t a, int64_t b) { return a > b ? a : b; }
constexpr int64_t kPartFloats = max2(attn::Shape<128, 2>::kPartFloats, attn::Shape<256, 1>::kPartFloats);

static_assert(SPEC_PAGED_WORKSPACE_ZEROED == 2 * attn::kMaxSms * sizeof(unsigned int), "the counters");

int attention_grid(const Device &d) { return d.sms < attn::kMaxSms ? d.sms : attn::kMaxSms; }

// The cache as TMA sees it: [page][head][block of 64][token][64], boxes of one
// page's tokens (at most a tile's) by 64 elements -- all blocks at once where
// the box has a whole tile's rows, so that its blocks land a tile apart.
spec_status page_map(const Device &d, const spec_paged_cache &c, void *base, const int64_t *strides, CUtensorMap *map)
{
    const int tile = c.head_dim == 256 ? attn::Shape<256, 1>::BK : attn::Shape<128, 1>::BK;
    const cuuint32_t rows = (cuuint32_t)(c.page_size < tile ? c.page_size : tile);
    const cuuint64_t dims[5] = {64, (cuuint64_t)c.page_size, (cuuint64_t)c.head_dim / 64, (cuuint64_t)c.heads,
                                (cuuint64_t)c.pages};
    const cuuint64_t st[4] = {(cuuint64_t)strides[1] * 2, 128, (cuuint64_t)strides[2] * 2, (cuuint64_t)strides[0] * 2};
    const cuuint32_t box[5] = {64, rows, (int)rows == tile ? (cuuint32_t)c.head_dim / 64 : 1u, 1, 1};
    const cuuint32_t one[5] = {1, 1, 1, 1, 1};
    const CUresult r = d.encode(map, c.dtype == SPEC_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                                5, base, dims, st, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(SPEC_ERR_ARG, "cache: its layout has no tensor map (driver error %d)", (int)r);
    return SPEC_OK;
}


// The 8-bit cache as TMA sees it: codes [page][head][token][head_dim], boxes of one page's
// tokens (at most a tile's), and scales [page][head][1][token].
spec_status code_maps(const Device &d, const spec_paged_cache8 &c, void *codes, const int64_t *strides, void *scales,
                      CUtensorMap *map, CUtensorMap *smap)
{
    const int tile = c.head_dim == 256 ? attn::Shape<256, 1>::BK : attn::Shape<128, 1>::BK;
    const cuuint32_t rows = (cuuint32_t)(c.page_size < tile ? c.page_size : tile);
    const cuuint32_t one[4] = {1, 1, 1, 1};
    const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.heads, (cuuint64_t)c.pages};
    const cuuint64_t st[3] = {(cuuint64_t)strides[1], (cuuint64_t)strides[2], (cuuint64_t)strides[0]};
    const cuuint32_t box[4] = {(cuuint32_t)c.head_dim, rows, 1, 1};
    CUresult r = d.encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, codes, dims, st, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS) {
        const cuuint64_t dims2[4] = {(cuuint64_t)c.page_size, 1, (cuuint64_t)c.heads, (cuuint64_t)c.pages};
        const cuuint64_t st2[3] = {(cuuint64_t)c.page_size, (cuuint64_t)c.page_size, (cuuint64_t)c.page_size * c.heads};
        const cuuint32_t box2[4] = {rows, 1, 1, 1};
        r = d.encode(smap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, scales, dims2, st2, box2, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    }
    if (r != CUDA_SUCCESS) return fail(SPEC_ERR_ARG, "cache: its layout has no tensor map (driver error %d)", (int)r);
    return SPEC_OK;
}

// A call of attention, whichever entry point it came through (its cache is checked there).
struct AttentionCall {
    const void *q;
    int64_t tokens;
    int32_t heads_q;
    int64_t q_token_stride, q_head_stride;
    const spec_paged_cache *cache;      // one of the two
    const spec_paged_cache8 *cache8;
    const spec_paged_batch *batch;
    const uint32_t *masks;
    int32_t mask_words;
    bool tree;
    float scale;
    int64_t window, max_new;
    void *out;
    float *lse;
    void *workspace;
    int64_t workspace_bytes;
};

spec_status attention_call(const AttentionCall &call)
{
    spec_status st = check_batch(call.batch);
    if (st != SPEC_OK) return st;
    const spec_paged_batch &b = *call.batch;
    const bool eight = call.cache8 != nullptr;
    struct { int32_t page_size, heads, head_dim, dtype; } c;   // of either cache
    if (eight) c = {call.cache8->page_size, call.cache8->heads, call.cache8->head_dim, call.cache8->dtype};
    else c = {call.cache->page_size, call.cache->heads, call.cache->head_dim, call.cache->dtype};
    const int64_t tokens = call.tokens, window = call.window, max_new = call.max_new;
    const int32_t heads_q = call.heads_q;
    const void *q = call.q;
    void *out = call.out, *workspace = call.workspace;
    float *lse = call.lse;
    if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256)
        return fail(SPEC_ERR_ARG, "head_dim = %d: attention takes 64, 128 or 256", c.head_dim);
    if (c.page_size < (eight ? 16 : 8) || (c.page_size & (c.page_size - 1)) != 0)
        return fail(SPEC_ERR_ARG, "page_size = %d: attention takes powers of two from %d", c.page_size, eight ? 16 : 8);
    if (b.page_size != c.page_size)
        return fail(SPEC_ERR_ARG, "page_size of batch (%d) and cache (%d) differ", b.page_size, c.page_size);
    if (tokens < 0 || tokens > INT32_MAX) return fail(SPEC_ERR_ARG, "tokens = %lld", (long long)tokens);
    if (heads_q < 1 || heads_q % c.heads != 0)
        return fail(SPEC_ERR_ARG, "heads_q = %d: need a positive multiple of the cache's %d heads", heads_q, c.heads);
    if ((int64_t)tokens * heads_q > INT32_MAX) return fail(SPEC_ERR_ARG, "tokens * heads_q exceeds 2^31-1");
    // the items of the step at most: row tiles of 128 rows, a partial one for each head of a lane with tokens
    const int64_t items = tokens * heads_q / 128 + (tokens < b.lanes ? tokens : b.lanes) * c.heads;
    if (items >= 1ll << (63 - attn::kItemBit))
        return fail(SPEC_ERR_ARG, "tokens, lanes and heads make up to %lld row tiles, need fewer than 2^%d", (long long)items,
                    63 - attn::kItemBit);
    if (!(call.scale > 0.f) || !isfinite(call.scale))
        return fail(SPEC_ERR_ARG, "scale = %g: must be positive and finite", call.scale);
    if (window < 0) return fail(SPEC_ERR_ARG, "window = %lld < 0", (long long)window);
    if (call.tree && window > 0 && window < SPEC_TREE_MAX_NODES)
        return fail(SPEC_ERR_ARG, "window = %lld: a tree's is 0 or at least %d", (long long)window, SPEC_TREE_MAX_NODES);
    if (call.tree && (call.mask_words < 1 || call.mask_words > SPEC_TREE_MAX_NODES / 32))
        return fail(SPEC_ERR_ARG, "mask_words = %d outside [1, %d]", call.mask_words, SPEC_TREE_MAX_NODES / 32);
    if (max_new < 0) return fail(SPEC_ERR_ARG, "max_new = %lld < 0", (long long)max_new);
    if (bad_stride(call.q_token_stride) || bad_stride(call.q_head_stride))
        return fail(SPEC_ERR_ARG, "strides must be non-negative multiples of 8 elements below 2^39");
    if (tokens == 0 || b.lanes == 0) return SPEC_OK;
    if (!q || !out || !b.block_table || !b.cu_new || !b.seq_lens || !workspace || (call.tree && !call.masks))
        return fail(SPEC_ERR_ARG, "null pointer");
    if (misaligned(q, 16) || misaligned(out, 16) || misaligned(workspace, 16) || misaligned(lse, 4) ||
        misaligned(b.block_table, 4) || misaligned(b.cu_new, 4) || misaligned(b.seq_lens, 4) ||
        misaligned(call.masks, 4))
        return fail(SPEC_ERR_ARG, "misaligned pointer (q, out and workspace need 16 bytes, int32, masks and lse 4)");
    // from q's first element to its last, whatever lies between its rows
    const __int128 span = ((__int128)(tokens - 1) * call.q_token_stride + (__int128)(heads_q - 1) * call.q_head_stride + c.head_dim) * 2;
    const Range in[] = {{q, span < INT64_MAX ? (int64_t)span : INT64_MAX, "q"}, {b.block_table, b.lanes * b.max_pages * 4, "block_table"},
                        {b.cu_new, (b.lanes + 1) * 4, "cu_new"}, {b.seq_lens, b.lanes * 4, "seq_lens"},
                        {call.masks, call.tree ? tokens * call.mask_words * 4 : 0, "masks"}};
    const Range o = {out, tokens * heads_q * c.head_dim * 2, "out"}, ls = {lse, tokens * heads_q * 4, "lse"};
    for (const Range &i : in)
        for (const Range *w : {&o, &ls})
            if (overlap(*w, i)) return fail(SPEC_ERR_ARG, "%s overlaps %s", w->name, i.name);
    if (overlap(o, ls)) return fail(SPEC_ERR_ARG, "out overlaps lse");
    const int64_t need = spec_paged_attention_workspace();
    if (need < 0) return (spec_status)need;
    if (call.workspace_bytes < need)
        return fail(SPEC_ERR_ARG, "workspace: %lld bytes, the call needs %lld", (long long)call.workspace_bytes,
                    (long long)need);
    if (overlap(o, {workspace, need, ""}) || overlap(ls, {workspace, need, ""}))
        return fail(SPEC_ERR_ARG, "out or lse overlaps workspace");
    Device *d = nullptr;
    st = device(&d);
    if (st != SPEC_OK) return st;
    attn::Args8 a;
    memset(&a, 0, sizeof a);
    if (eight) {
        const spec_paged_cache8 &c8 = *call.cache8;
        st = code_maps(*d, c8, c8.k, c8.k_strides, c8.k_scales, &a.kmap, &a.ksmap);
        if (st == SPEC_OK) st = code_maps(*d, c8, c8.v, c8.v_strides, c8.v_scales, &a.vmap, &a.vsmap);
    } else {
        st = page_map(*d, *call.cache, call.cache->k, call.cache->k_strides, &a.kmap);
        if (st == SPEC_OK) st = page_map(*d, *call.cache, call.cache->v, call.cache->v_strides, &a.vmap);
    }
    if (st != SPEC_OK) return st;
    a.q = static_cast<const uint16_t *>(q);
    a.tokens = tokens; a.qs_t = call.q_token_stride; a.qs_h = call.q_head_stride;
    a.heads_q = heads_q; a.heads_kv = c.heads; a.group = heads_q / c.heads;
    while ((1 << a.log_page) < c.page_size) ++a.log_page;
    while ((1u << a.group_shift) < (uint32_t)a.group) ++a.group_shift;
    a.group_magic = (uint32_t)((((1ull << a.group_shift) - a.group) << 32) / a.group + 1);
    a.block_table = b.block_table; a.cu_new = b.cu_new; a.seq_lens = b.seq_lens;
    a.lanes = (int32_t)b.lanes; a.max_pages = b.max_pages;
    const int64_t hint = max_new < tokens ? max_new : tokens, chunk = hint > 0 ? hint : (tokens + b.lanes - 1) / b.lanes;
    const bool two = chunk * a.group > 128;   // more rows than one tile: two tiles share every K/V tile
    // Few rows (8 bits, heads of 128): items of 16 rows, if the step's can be counted.  A lane of more reads its cache again for
    // every 16, so the lanes' most is to be known, or a token each.
    const int64_t most = hint > 0 ? hint : tokens <= b.lanes ? 1 : tokens;
    const int64_t few_items = tokens * heads_q / 16 + (tokens < b.lanes ? tokens : b.lanes) * c.heads;
    const bool few = eight && c.head_dim == 128 && most * a.group <= 16 && few_items < 1ll << (63 - attn::kItemBit);
    // (of tiles of 64 keys, the smaller; 2^31 - 2^16 unless there are 2^15 items)
    const int64_t tiles = (1ll << attn::kItemBit) / (few ? few_items : items) - 2;
    a.most_keys = (int32_t)(tiles < (0x7FFF0000 >> 6) ? tiles << 6 : 0x7FFF0000);
    a.c = call.scale * attn::kLog2e;
    a.window = window > INT32_MAX ? 0 : window;   // past every position: none (and positions less it stay within 64 bits)
    a.out = static_cast<uint16_t *>(out); a.lse = lse;
    a.counters = static_cast<unsigned int *>(workspace);
    a.parts = reinterpret_cast<float *>(static_cast<char *>(workspace) + SPEC_PAGED_WORKSPACE_ZEROED);
    a.masks = call.tree ? call.masks : nullptr;
    a.mask_words = call.mask_words;
    const attn::Pick pick = {c.head_dim, two, few, c.dtype == SPEC_F16, chunk, d->index, attention_grid(*d)};
    if (eight) return attn::launch8(a, pick, call.tree);
    const attn::Args &a16 = a;
    return call.tree ? attn::launch_tree(a16, pick) : attn::launch<false, false>(a16, pick);
}

}  // namespace

namespace host {

cudaError_t take_paged_timeouts(unsigned int *flags) { return take_flag(g_wait_timeouts, flags); }

}  // namespace host

extern "C" {

spec_status spec_paged_plan(const spec_paged_batch *batch, const int32_t *free_pages, int64_t num_free,
                            const int32_t *cursor)
{
    host::clear_error();
    spec_status st = check_batch(batch);
    if (st != SPEC_OK) return st;
    const spec_paged_batch &b = *batch;
    if (b.tokens < 0) return fail(SPEC_ERR_ARG, "batch: tokens = %lld < 0", (long long)b.tokens);
    if (num_free < 0 || num_free > INT32_MAX) return fail(SPEC_ERR_ARG, "num_free = %lld", (long long)num_free);
    if (!b.cu_new || !b.info ||
        (b.lanes > 0 && (!b.context_lens || !b.new_lens || !b.held || !b.block_table || !b.seq_lens || !b.held_out)) ||
        (b.tokens > 0 && (!b.positions || !b.slots)) || (num_free > 0 && !free_pages))
        return fail(SPEC_ERR_ARG, "null pointer");
    const void *words[] = {b.context_lens, b.new_lens, b.held,      b.block_table, b.cu_new,   b.seq_lens,
                           b.held_out,     b.info,     b.positions, free_pages,    cursor};
    for (const void *p : words)
        if (misaligned(p, 4)) return fail(SPEC_ERR_ARG, "misaligned pointer (int32 arrays need 4 bytes)");
    if (misaligned(b.slots, 8)) return fail(SPEC_ERR_ARG, "misaligned pointer (slots need 8 bytes)");
    // every CTA reads the inputs while others write the outputs
    const int64_t l4 = b.lanes * 4, t4 = b.tokens < INT64_MAX / 8 ? b.tokens * 4 : INT64_MAX / 2;
    const Range in[] = {{b.context_lens, l4, "context_lens"}, {b.new_lens, l4, "new_lens"}, {b.held, l4, "held"},
                        {free_pages, num_free * 4, "free_pages"}, {cursor, 4, "cursor"}};
    const Range out[] = {{b.info, 16, "info"}, {b.held_out, l4, "held_out"}, {b.seq_lens, l4, "seq_lens"},
                         {b.cu_new, l4 + 4, "cu_new"}, {b.positions, t4, "positions"}, {b.slots, 2 * t4, "slots"},
                         {b.block_table, l4 * b.max_pages, "block_table"}};
    for (const Range &o : out)
        for (const Range &i : in)
            if (overlap(o, i)) return fail(SPEC_ERR_ARG, "outputs must not alias inputs (%s and %s)", o.name, i.name);
    Device *d = nullptr;
    st = device(&d);
    if (st != SPEC_OK) return st;
    paged::PlanArgs a = {b, free_pages, num_free, cursor};
    int64_t grid = (b.tokens + paged::kPlanThreads - 1) / paged::kPlanThreads;
    const int64_t by_lanes = (b.lanes + paged::kPlanWarps - 1) / paged::kPlanWarps;
    if (grid < by_lanes) grid = by_lanes;
    if (grid < 1) grid = 1;
    if (grid > d->sms) grid = d->sms;
    return launch(paged::plan_kernel, dim3((unsigned)grid), paged::kPlanThreads, paged::plan_smem(b.lanes), a);
}

spec_status spec_paged_store(const void *k, const void *v, int64_t tokens, int64_t k_token_stride,
                             int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                             const int64_t *slots, const spec_paged_cache *cache)
{
    host::clear_error();
    spec_status st = check_cache(cache);
    if (st != SPEC_OK) return st;
    st = check_new(k, v, tokens, k_token_stride, k_head_stride, v_token_stride, v_head_stride, slots);
    if (st != SPEC_OK || tokens == 0) return st;
    Device *d = nullptr;
    st = device(&d);
    if (st != SPEC_OK) return st;
    paged::StoreArgs a = {static_cast<const uint16_t *>(k), static_cast<const uint16_t *>(v), tokens,
                          k_token_stride, k_head_stride, v_token_stride, v_head_stride, slots, *cache};
    const int64_t nv = tokens * cache->heads * (cache->head_dim / 8);
    int64_t grid = (nv + paged::kStoreThreads - 1) / paged::kStoreThreads;
    if (grid > 8 * d->sms) grid = 8 * d->sms;
    return launch(paged::store_kernel, dim3((unsigned)grid), paged::kStoreThreads, 0, a);
}

int64_t spec_paged_attention_workspace(void)
{
    host::clear_error();
    Device *d = nullptr;
    const spec_status st = device(&d);
    if (st != SPEC_OK) return st;
    return SPEC_PAGED_WORKSPACE_ZEROED + (int64_t)attention_grid(*d) * 2 * kPartFloats * 4;
}

spec_status spec_paged_attention(const void *q, int64_t tokens, int32_t heads_q, int64_t q_token_stride,
                                 int64_t q_head_stride, const spec_paged_cache *cache, const spec_paged_batch *batch,
                                 float scale, int64_t window, int64_t max_new, void *out, float *lse,
                                 void *workspace, int64_t workspace_bytes)
{
    host::clear_error();
    const spec_status st = check_cache(cache);
    if (st != SPEC_OK) return st;
    return attention_call({q, tokens, heads_q, q_token_stride, q_head_stride, cache, nullptr, batch, nullptr, 0, false, scale,
                           window, max_new, out, lse, workspace, workspace_bytes});
}

spec_status spec_paged_attention8(const void *q, int64_t tokens, int32_t heads_q, int64_t q_token_stride,
                                  int64_t q_head_stride, const spec_paged_cache8 *cache, const spec_paged_batch *batch,
                                  float scale, int64_t window, int64_t max_new, void *out, float *lse,
                                  void *workspace, int64_t workspace_bytes)
{
    host::clear_error();
    const spec_status st = check_cache8(cache);
    if (st != SPEC_OK) return st;
    return attention_call({q, tokens, heads_q, q_token_stride, q_head_stride, nullptr, cache, batch, nullptr, 0, false, scale,
                           window, max_new, out, lse, workspace, workspace_bytes});
}

spec_status spec_tree_attention(const void *q, int64_t tokens, int32_t heads_q, int64_t q_token_stride,
                                int64_t q_head_stride, const spec_paged_cache *cache, const spec_paged_batch *batch,
                                const uint32_t *masks, int32_t mask_words, float scale, int64_t window, int64_t max_new,
                                void *out, float *lse, void *workspace, int64_t workspace_bytes)
{
    host::clear_error();
    const spec_status st = check_cache(cache);
    if (st != SPEC_OK) return st;
    return attention_call({q, tokens, heads_q, q_token_stride, q_head_stride, cache, nullptr, batch, masks, mask_words, true,
                           scale, window, max_new, out, lse, workspace, workspace_bytes});
}

spec_status spec_tree_attention8(const void *q, int64_t tokens, int32_t heads_q, int64_t q_token_stride,
                                 int64_t q_head_stride, const spec_paged_cache8 *cache, const spec_paged_batch *batch,
                                 const uint32_t *masks, int32_t mask_words, float scale, int64_t window, int64_t max_new,
                                 void *out, float *lse, void *workspace, int64_t workspace_bytes)
{
    host::clear_error();
    const spec_status st = check_cache8(cache);
    if (st != SPEC_OK) return st;
    return attention_call({q, tokens, heads_q, q_token_stride, q_head_stride, nullptr, cache, batch, masks, mask_words, true,
                           scale, window, max_new, out, lse, workspace, workspace_bytes});
}

spec_status spec_logits_process(const uint16_t *logits, int64_t lanes, int32_t cols, int64_t V,
                                const int32_t *history, int64_t history_stride, const int32_t *prompt_lens,
                                const int32_t *history_lens, const int32_t *drafts, const float *penalties,
                                const int32_t *bias_ids, const float *bias_vals, int64_t max_bias,
                                const int32_t *bias_lens, const uint32_t *mask, int64_t mask_count,
                                const int32_t *mask_rows, uint16_t *out)
{
    host::clear_error();
    if (lanes < 0 || lanes > 65535) return fail(SPEC_ERR_ARG, "lanes = %lld outside [0, 65535]", (long long)lanes);
    if (cols < 1 || cols > SPEC_MAX_GAMMA + 1)
        return fail(SPEC_ERR_ARG, "cols = %d outside [1, %d]", cols, SPEC_MAX_GAMMA + 1);
    if (V < 1 || V > INT32_MAX) return fail(SPEC_ERR_ARG, "V = %lld outside [1, 2^31-1]", (long long)V);
    if (history_stride < 0 || max_bias < 0 || mask_count < 0)
        return fail(SPEC_ERR_ARG, "history_stride, max_bias and mask_count must not be negative");
    if (lanes == 0) return SPEC_OK;
    if (!logits || !out) return fail(SPEC_ERR_ARG, "null pointer");
    // (a table of no entries has no address: with its lengths or rows it is a rule that changes nothing)
    if (!!prompt_lens != !!history_lens || (history_stride > 0 ? !!history != !!prompt_lens : history && !prompt_lens))
        return fail(SPEC_ERR_ARG, "history, prompt_lens and history_lens go together");
    if (max_bias > 0 ? !!bias_ids != !!bias_vals || !!bias_ids != !!bias_lens : (bias_ids || bias_vals) && !bias_lens)
        return fail(SPEC_ERR_ARG, "bias_ids, bias_vals and bias_lens go together");
    if (mask_count > 0 ? !!mask != !!mask_rows : mask && !mask_rows)
        return fail(SPEC_ERR_ARG, "mask and mask_rows go together");
    if (misaligned(logits, 2) || misaligned(out, 2)) return fail(SPEC_ERR_ARG, "misaligned pointer (logits need 2 bytes)");
    const void *words[] = {history, prompt_lens, history_lens, drafts, penalties, bias_ids, bias_vals, bias_lens, mask, mask_rows};
    for (const void *p : words)
        if (misaligned(p, 4)) return fail(SPEC_ERR_ARG, "misaligned pointer (32-bit arrays need 4 bytes)");
    const int64_t bytes = lanes * cols * V * 2;   // below 2^16 * 2^4 * 2^31 * 2
    const char *x = reinterpret_cast<const char *>(logits), *y = reinterpret_cast<const char *>(out);
    if (x != y && x < y + bytes && y < x + bytes)
        return fail(SPEC_ERR_ARG, "out overlaps logits without being them");
    Device *d = nullptr;
    spec_status st = device(&d);
    if (st != SPEC_OK) return st;
    rules::Args a = {logits, out, lanes, V, cols, history, history_stride, prompt_lens, history_lens, drafts,
                     penalties, bias_ids, bias_vals, max_bias, bias_lens, mask, mask_count, mask_rows};
    const unsigned slices = (unsigned)((V + 7 + rules::kSlice - 1) / rules::kSlice);
    return launch(rules::process_kernel, dim3(slices, (unsigned)lanes), rules::kThreads, (size_t)rules::smem_bytes(bias_ids != nullptr), a);
}

}  // extern "C"
