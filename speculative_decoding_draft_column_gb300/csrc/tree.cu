// libspecsel: rounds whose drafts form a tree (masks and positions, verification, the accepted path
// moved into place) and the store of the 8-bit cache -- argument checks, launches and the C ABI.

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "specsel.h"
#include "checks.h"
#include "tree_verify.cuh"
#include "host.h"

using host::cuda_fail;
using host::fail;

namespace {

// `cluster`: CTAs of a thread-block cluster (1: none)
template <typename K, typename... A>
spec_status launch(K kernel, dim3 grid, unsigned block, size_t smem, unsigned cluster, const A &...a)
{
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = host::stream();
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a...);
    if (e != cudaSuccess) return cuda_fail(e, "kernel launch");
    host::count_launch();
    return SPEC_OK;
}

spec_status sm_count(int64_t *sms)
{
    int dev = 0, n = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
    *sms = n;
    return SPEC_OK;
}

spec_status commit(tree::CommitArgs &a, const spec_paged_batch *batch, int32_t page_size, const int32_t *path,
                   const int32_t *accept_lens, int32_t depth, int32_t *context_out)
{
    const spec_status st = check_batch(batch);
    if (st != SPEC_OK) return st;
    const spec_paged_batch &b = *batch;
    if (b.page_size != page_size)
        return fail(SPEC_ERR_ARG, "page_size of batch (%d) and cache (%d) differ", b.page_size, page_size);
    if (depth < 1 || depth >= SPEC_TREE_MAX_NODES)
        return fail(SPEC_ERR_ARG, "depth = %d outside [1, %d]", depth, SPEC_TREE_MAX_NODES - 1);
    if (b.lanes == 0) return SPEC_OK;
    if (!b.block_table || !b.cu_new || !b.seq_lens || !path || !accept_lens) return fail(SPEC_ERR_ARG, "null pointer");
    for (const void *p : {(const void *)b.block_table, (const void *)b.cu_new, (const void *)b.seq_lens, (const void *)path,
                          (const void *)accept_lens, (const void *)context_out})
        if (misaligned(p, 4)) return fail(SPEC_ERR_ARG, "misaligned pointer (int32 arrays need 4 bytes)");
    const int64_t l4 = b.lanes * 4;
    const Range o = {context_out, l4, "context_out"};
    for (const Range &i : {Range{b.block_table, l4 * b.max_pages, "block_table"}, Range{b.cu_new, l4 + 4, "cu_new"},
                           Range{b.seq_lens, l4, "seq_lens"}, Range{path, l4 * (depth + 1), "path"},
                           Range{accept_lens, l4, "accept_lens"}})
        if (overlap(o, i)) return fail(SPEC_ERR_ARG, "context_out overlaps %s", i.name);
    a.max_pages = b.max_pages; a.lanes = b.lanes;
    a.page_size = page_size; a.depth = depth;
    a.block_table = b.block_table; a.cu = b.cu_new; a.seq_lens = b.seq_lens;
    a.path = path; a.accept = accept_lens; a.context_out = context_out;
    return launch(tree::commit_kernel, dim3((unsigned)b.lanes), tree::kCommitThreads, 0, 1, a);
}

spec_status verify(const uint16_t *logits, const int32_t *drafts, const int32_t *parents, const int32_t *cu, int64_t tokens,
                   int64_t lanes, int32_t depth, int64_t V, int32_t top_k, double temperature, double top_p,
                   const double *uniforms, bool sampled, int32_t *accept, int32_t *commits, int32_t *path)
{
    if (lanes < 0 || lanes > 65535) return fail(SPEC_ERR_ARG, "lanes = %lld outside [0, 65535]", (long long)lanes);
    if (tokens < 0 || tokens > INT32_MAX) return fail(SPEC_ERR_ARG, "tokens = %lld", (long long)tokens);
    if (depth < 1 || depth >= SPEC_TREE_MAX_NODES)
        return fail(SPEC_ERR_ARG, "depth = %d outside [1, %d]", depth, SPEC_TREE_MAX_NODES - 1);
    if (V < 1 || V > INT32_MAX) return fail(SPEC_ERR_ARG, "V = %lld outside [1, 2^31-1]", (long long)V);
    if (tokens > INT64_MAX / 4 / V) return fail(SPEC_ERR_ARG, "tokens * V overflows");
    if (sampled) {
        if (!(temperature > 0.0) || !isfinite(temperature))
            return fail(SPEC_ERR_ARG, "temperature = %g: must be positive and finite", temperature);
        if (!(top_p > 0.0) || !(top_p <= 1.0)) return fail(SPEC_ERR_ARG, "top_p = %g outside (0, 1]", top_p);
        if (top_k < 1 || top_k > SPEC_MAX_K || (int64_t)top_k > V)
            return fail(SPEC_ERR_ARG, "top_k = %d outside [1, min(V, %d)]", top_k, SPEC_MAX_K);
    }
    if (lanes == 0) return SPEC_OK;
    if (!cu || !accept || !commits || !path || (tokens > 0 && (!logits || !drafts || !parents || (sampled && !uniforms))))
        return fail(SPEC_ERR_ARG, "null pointer");
    if (misaligned(logits, 2) || misaligned(uniforms, 8)) return fail(SPEC_ERR_ARG, "misaligned pointer (logits need 2 bytes, uniforms 8)");
    for (const void *p : {(const void *)drafts, (const void *)parents, (const void *)cu, (const void *)accept, (const void *)commits,
                          (const void *)path})
        if (misaligned(p, 4)) return fail(SPEC_ERR_ARG, "misaligned pointer (int32 arrays need 4 bytes)");
    const int64_t width = depth + 1;
    const Range out[] = {{accept, lanes * 4, "out_accept_len"}, {commits, lanes * width * 4, "out_commit_ids"},
                         {path, lanes * width * 4, "out_path"}};
    const Range in[] = {{logits, tokens * V * 2, "target_logits"}, {drafts, tokens * 4, "drafts"}, {parents, tokens * 4, "parents"},
                        {cu, lanes * 4 + 4, "cu"}, {uniforms, sampled ? tokens * 16 : 0, "uniforms"}};
    for (int i = 0; i < 3; ++i) {
        for (const Range &r : in)
            if (overlap(out[i], r)) return fail(SPEC_ERR_ARG, "%s overlaps %s", out[i].name, r.name);
        if (overlap(out[i], out[(i + 1) % 3])) return fail(SPEC_ERR_ARG, "%s overlaps %s", out[i].name, out[(i + 1) % 3].name);
    }
    int64_t sms = 0;
    const spec_status st = sm_count(&sms);
    if (st != SPEC_OK) return st;
    tree::VerifyArgs a;
    memset(&a, 0, sizeof a);
    a.logits = logits; a.drafts = drafts; a.parents = parents; a.cu = cu;
    a.tokens = tokens; a.lanes = lanes; a.V = V; a.depth = depth;
    a.k = sampled ? top_k : 1;
    a.temperature = temperature; a.top_p = top_p;
    a.inv_temperature = (float)(1.0 / temperature); a.top_p_single = (float)top_p;
    a.uniforms = sampled ? uniforms : nullptr;
    a.accept = accept; a.commit = commits; a.path = path;
    // CTAs of a column: more while all lanes' make up four turns of the GPU (two are on an SM) at most, and a part keeps
    // every thread at a vector or more (128 lanes of 16 nodes 88 us with four turns, 107 with one, 166 with a half)
    const int64_t vectors = (V + 14) / 8;
    unsigned ctas = 1;
    while (ctas < tree::kMostCtas && lanes * ctas * 2 <= 8 * sms && vectors >= 2 * ctas * tree::kThreads) ctas *= 2;
    // All nodes' columns at once, where they fit the GPU together; else the paths' only.
    std::unique_lock<std::mutex> hold;
    if (tokens * ctas <= 2 * sms && tokens > 0 && host::lane_scratch(lanes, tokens * a.k, &a.tickets, &a.lists, &hold))
        return launch(tree::verify_kernel<true>, dim3((unsigned)(tokens * ctas)), tree::kThreads, sizeof(tree::VerifySmem), ctas, a, (uint32_t)ctas);
    return launch(tree::verify_kernel<false>, dim3((unsigned)(lanes * ctas)), tree::kThreads, sizeof(tree::VerifySmem), ctas, a, (uint32_t)ctas);
}

}  // namespace

extern "C" {

spec_status spec_paged_store8(const void *k, const void *v, int64_t tokens, int64_t k_token_stride,
                              int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                              const int64_t *slots, const spec_paged_cache8 *cache)
{
    host::clear_error();
    spec_status st = check_cache8(cache);
    if (st != SPEC_OK) return st;
    st = check_new(k, v, tokens, k_token_stride, k_head_stride, v_token_stride, v_head_stride, slots);
    if (st != SPEC_OK || tokens == 0) return st;
    tree::StoreArgs a;
    memset(&a, 0, sizeof a);
    a.k = static_cast<const uint16_t *>(k); a.v = static_cast<const uint16_t *>(v);
    a.tokens = tokens;
    a.ks_t = k_token_stride; a.ks_h = k_head_stride; a.vs_t = v_token_stride; a.vs_h = v_head_stride;
    a.slots = slots; a.c = *cache;
    a.group = 1;
    while (a.group * 16 < cache->head_dim) a.group *= 2;
    const int32_t most = tree::kStoreThreads / a.group;
    a.heads = cache->heads < most ? cache->heads : most;
    a.per = most / a.heads;
    a.log_page = -1;
    if ((cache->page_size & (cache->page_size - 1)) == 0) a.log_page = 31 - __builtin_clz((unsigned)cache->page_size);
    // heads past a CTA's: more CTAs a token, as far as a grid's second dimension goes
    const int64_t parts = ((int64_t)cache->heads + a.heads - 1) / a.heads;
    if (parts > 65535) return fail(SPEC_ERR_ARG, "cache: heads = %d, the store takes %d of this size", cache->heads, 65535 * a.heads);
    int64_t sms = 0;
    st = sm_count(&sms);
    if (st != SPEC_OK) return st;
    int64_t grid = (tokens + a.per - 1) / a.per;
    const int64_t room = (tree::kStoreCtas * sms + parts - 1) / parts;
    if (grid > room) grid = room;
    return cache->dtype == SPEC_F16 ? launch(tree::store_kernel<true>, dim3((unsigned)grid, (unsigned)parts), tree::kStoreThreads, 0, 1, a)
                                    : launch(tree::store_kernel<false>, dim3((unsigned)grid, (unsigned)parts), tree::kStoreThreads, 0, 1, a);
}

spec_status spec_tree_plan(const int32_t *parents, int64_t tokens, const spec_paged_batch *batch, uint32_t *masks,
                           int32_t mask_words, int32_t *positions)
{
    host::clear_error();
    spec_status st = check_batch(batch);
    if (st != SPEC_OK) return st;
    const spec_paged_batch &b = *batch;
    if (tokens < 0 || tokens > INT32_MAX) return fail(SPEC_ERR_ARG, "tokens = %lld", (long long)tokens);
    if (mask_words < 1 || mask_words > SPEC_TREE_MAX_NODES / 32)
        return fail(SPEC_ERR_ARG, "mask_words = %d outside [1, %d]", mask_words, SPEC_TREE_MAX_NODES / 32);
    if (tokens == 0 || b.lanes == 0) return SPEC_OK;
    if (!parents || !b.cu_new || !b.seq_lens || !masks || !positions) return fail(SPEC_ERR_ARG, "null pointer");
    for (const void *p : {(const void *)parents, (const void *)b.cu_new, (const void *)b.seq_lens, (const void *)masks,
                          (const void *)positions})
        if (misaligned(p, 4)) return fail(SPEC_ERR_ARG, "misaligned pointer (32-bit arrays need 4 bytes)");
    const Range m = {masks, tokens * mask_words * 4, "masks"}, p = {positions, tokens * 4, "positions"};
    for (const Range &i : {Range{parents, tokens * 4, "parents"}, Range{b.cu_new, b.lanes * 4 + 4, "cu_new"},
                           Range{b.seq_lens, b.lanes * 4, "seq_lens"}})
        for (const Range *o : {&m, &p})
            if (overlap(*o, i)) return fail(SPEC_ERR_ARG, "%s overlaps %s", o->name, i.name);
    if (overlap(m, p)) return fail(SPEC_ERR_ARG, "masks overlaps positions");
    tree::PlanArgs a = {parents, b.cu_new, b.seq_lens, tokens, b.lanes, masks, mask_words, positions};
    return launch(tree::plan_kernel, dim3((unsigned)b.lanes), tree::kPlanThreads, 0, 1, a);
}

spec_status spec_tree_verify(const uint16_t *target_logits, const int32_t *drafts, const int32_t *parents,
                             const int32_t *cu, int64_t tokens, int64_t lanes, int32_t depth, int64_t V,
                             int32_t *out_accept_len, int32_t *out_commit_ids, int32_t *out_path)
{
    host::clear_error();
    return verify(target_logits, drafts, parents, cu, tokens, lanes, depth, V, 1, 1.0, 1.0, nullptr, false, out_accept_len,
                  out_commit_ids, out_path);
}

spec_status spec_tree_verify_sampled(const uint16_t *target_logits, const int32_t *drafts, const int32_t *parents,
                                     const int32_t *cu, int64_t tokens, int64_t lanes, int32_t depth, int64_t V,
                                     double temperature, double top_p, int32_t top_k, const double *uniforms,
                                     int32_t *out_accept_len, int32_t *out_commit_ids, int32_t *out_path)
{
    host::clear_error();
    return verify(target_logits, drafts, parents, cu, tokens, lanes, depth, V, top_k, temperature, top_p, uniforms, true,
                  out_accept_len, out_commit_ids, out_path);
}

spec_status spec_tree_commit(const spec_paged_cache *cache, const spec_paged_batch *batch, const int32_t *path,
                             const int32_t *accept_lens, int32_t depth, int32_t *context_out)
{
    host::clear_error();
    const spec_status st = check_cache(cache);
    if (st != SPEC_OK) return st;
    tree::CommitArgs a;
    memset(&a, 0, sizeof a);
    a.k = static_cast<uint8_t *>(cache->k); a.v = static_cast<uint8_t *>(cache->v);
    for (int i = 0; i < 3; ++i) {
        a.k_strides[i] = cache->k_strides[i] * 2;
        a.v_strides[i] = cache->v_strides[i] * 2;
    }
    a.pages = cache->pages; a.heads = cache->heads; a.vector = cache->head_dim / 8;
    return commit(a, batch, cache->page_size, path, accept_lens, depth, context_out);
}

spec_status spec_tree_commit8(const spec_paged_cache8 *cache, const spec_paged_batch *batch, const int32_t *path,
                              const int32_t *accept_lens, int32_t depth, int32_t *context_out)
{
    host::clear_error();
    const spec_status st = check_cache8(cache);
    if (st != SPEC_OK) return st;
    tree::CommitArgs a;
    memset(&a, 0, sizeof a);
    a.k = static_cast<uint8_t *>(cache->k); a.v = static_cast<uint8_t *>(cache->v);
    a.k_scales = cache->k_scales; a.v_scales = cache->v_scales;
    for (int i = 0; i < 3; ++i) {
        a.k_strides[i] = cache->k_strides[i];
        a.v_strides[i] = cache->v_strides[i];
    }
    a.pages = cache->pages; a.heads = cache->heads; a.vector = cache->head_dim / 16;
    return commit(a, batch, cache->page_size, path, accept_lens, depth, context_out);
}

}  // extern "C"
