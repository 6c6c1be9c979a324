// Launch of one variant of the attention kernel: its shared memory, and whether
// an item's parts are joined by all its CTAs.  Included by the translation units
// that hold the variants (paged.cu: a causal chunk over a 16-bit cache;
// attention_tree.cu: trees; attention8.cu: 8-bit caches).
#pragma once

#include <string.h>

#include <mutex>

#include "attention.cuh"
#include "host.h"

namespace attn {

constexpr int kMaxDevices = 64;

// Give an attention kernel all the shared memory a CTA can have (one CTA an SM,
// so that TMEM is never contended), and check what the kernel relies on: its
// static shared memory stays below the first 1,024-byte boundary.  Once a device.
template <int D, int QT, bool F16, bool Q8, bool TREE>
spec_status prepare(int dev, size_t *smem)
{
    using S = Shape<D, QT, Q8, TREE>;
    static std::mutex mu;
    static int dynamic[kMaxDevices];
    std::lock_guard<std::mutex> lock(mu);
    if (dynamic[dev] == 0) {
        auto kernel = attention_kernel<D, QT, F16, Q8, TREE>;
        int smem_max = 0;
        cudaError_t e = cudaDeviceGetAttribute(&smem_max, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
        if (e != cudaSuccess) return host::cuda_fail(e, "cudaDeviceGetAttribute");
        cudaFuncAttributes at;
        e = cudaFuncGetAttributes(&at, kernel);
        if (e != cudaSuccess) return host::cuda_fail(e, "cudaFuncGetAttributes");
        if (at.sharedSizeBytes > 1024 || 1024 + S::kPayload > smem_max)
            return host::fail(SPEC_ERR_CUDA, "attention: %d bytes of shared memory are not enough", smem_max);
        const int d = smem_max - (int)at.sharedSizeBytes;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, d);
        if (e != cudaSuccess) return host::cuda_fail(e, "cudaFuncSetAttribute");
        dynamic[dev] = d;
    }
    *smem = (size_t)dynamic[dev];
    return SPEC_OK;
}

// Whether an item's parts are joined by all its CTAs (a cooperative launch) or
// by the last part's CTA alone (an ordinary one: 2-4 us less a call in a
// stream, 1 in a graph; 8 lanes of 8 tokens at 8,000 keys 51.8 against 55.3 us, 64 lanes of
// 16 tokens at 3,000 keys 30.8 against 34.8, 8 lanes of a token at 2,000 keys of one head
// 12.0 against 14.4).  The lengths are on the device, so the number of parts is
// estimated twice: from the items that the lanes and heads make if they are
// even, and from one lane having all the keys (the others short, or without tokens, as in
// a padded batch), whose heads then share the GPU.  Both are bounded by the table's
// width and the window.  Alone, a CTA joins the even case's 128 KB in 2 us.  Of 64 lanes
// of 4 tokens, one with 60,000 keys, it takes 29.4 against 20.5 us in a stream where that lane has
// one head (152 parts of 8 KB), 26.6 against 23.5 where it has two (76 parts); of 64 lanes
// of 16 tokens, one with 131,072 keys of one head (152 parts of 32 KB), 66 against 24 in a graph.
template <typename S>
bool shares_joins(const Args &a, int64_t chunk, int64_t ctas)
{
    constexpr int64_t kAlone = 32 << 10, kAloneAll = 128 << 10, kAloneWorst = 1 << 20, kAloneParts = 96;
    const int64_t rows = chunk * a.group < S::kRows ? chunk * a.group : S::kRows;
    const int64_t table = a.max_pages << a.log_page, seen = a.window > 0 && a.window < table ? a.window + S::kRows / a.group + 2 : table;
    const int64_t widest = ((seen < table ? seen : table) / S::BK + 2) / S::kLeast + 2;
    const int64_t items = (int64_t)a.lanes * a.heads_kv, likely = ctas / items + 2, one = ctas / a.heads_kv + 2;
    const int64_t parts = widest < likely ? widest : likely, worst = widest < one ? widest : one, part = rows * S::D * 4;
    return part > kAlone || parts * part > kAloneAll || worst * part > kAloneWorst || worst > kAloneParts;
}

template <int D, int QT, bool F16, bool Q8, bool TREE, typename A>
spec_status launch_one(const A &a, int64_t chunk, int dev, int grid)
{
    using S = Shape<D, QT, Q8, TREE>;
    size_t smem = 0;
    const spec_status st = prepare<D, QT, F16, Q8, TREE>(dev, &smem);
    if (st != SPEC_OK) return st;
    A b = a;
    b.share_joins = shares_joins<S>(a, chunk, grid);
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = host::stream();
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeCooperative;
    attr[1].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = b.share_joins ? 2 : 1;   // CTAs wait for one another's parts
    const cudaError_t e = cudaLaunchKernelEx(&cfg, attention_kernel<D, QT, F16, Q8, TREE>, b);
    if (e != cudaSuccess) return host::cuda_fail(e, "kernel launch");
    host::count_launch();
    return SPEC_OK;
}

// What picks the variant besides the kind of cache and of mask.
struct Pick {
    int32_t head_dim;      // 64, 128 or 256
    bool two, few, f16;    // two row tiles share every K/V tile; at most 16 rows an item; fp16
    int64_t chunk;         // new tokens of a lane to expect
    int dev, grid;
};

template <bool Q8, bool TREE, typename A>
spec_status launch(const A &a, const Pick &p)
{
    auto go = [&](auto kernel) { return kernel(a, p.chunk, p.dev, p.grid); };
    if (p.head_dim == 256) return go(p.f16 ? launch_one<256, 1, true, Q8, TREE, A> : launch_one<256, 1, false, Q8, TREE, A>);
    if (p.head_dim == 128) {
        if constexpr (Q8)
            if (p.few) return go(p.f16 ? launch_one<128, 0, true, Q8, TREE, A> : launch_one<128, 0, false, Q8, TREE, A>);
        if (p.two) return go(p.f16 ? launch_one<128, 2, true, Q8, TREE, A> : launch_one<128, 2, false, Q8, TREE, A>);
        return go(p.f16 ? launch_one<128, 1, true, Q8, TREE, A> : launch_one<128, 1, false, Q8, TREE, A>);
    }
    if (p.two) return go(p.f16 ? launch_one<64, 2, true, Q8, TREE, A> : launch_one<64, 2, false, Q8, TREE, A>);
    return go(p.f16 ? launch_one<64, 1, true, Q8, TREE, A> : launch_one<64, 1, false, Q8, TREE, A>);
}

// The variants of the other translation units.
spec_status launch_tree(const Args &a, const Pick &p);
spec_status launch8(const Args8 &a, const Pick &p, bool tree);

}  // namespace attn
