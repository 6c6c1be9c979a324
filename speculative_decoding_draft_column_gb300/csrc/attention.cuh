// Attention of a chunk of new tokens over the paged cache, on the tensor
// cores (tcgen05) with the cache's pages brought in by TMA.
//
// Rows.  The query heads that share a key/value head are packed with the
// lane's new tokens: row r = token * group + head, 128 rows a tile, so one
// token of eight heads and an anchor with fifteen drafts of eight heads both
// fill one tile and read the cache once.  S = Q K^T (Q, K in shared memory, S
// in TMEM, fp32), P = exp2(c S - m) rounded to 16 bits over S in TMEM, and
// O += P V (P from TMEM, V in shared memory, O in TMEM, fp32).  A softmax
// thread owns one row.
//
// The running maximum m is a reference, not the exact maximum: it moves only
// when a tile exceeds it by more than 2^8 (kLag), and only then O and the sum
// are rescaled.  P stays below 2^8, where its 16-bit rounding is as relative
// as below 1, and the sum is kept in fp32 either way.
//
// Two streams hide the softmax of one behind the products of the other: with
// two row tiles in a CTA (QT = 2, chunks) each stream has its rows and both
// use every K/V tile; with one row tile (QT = 1) the streams take the K/V tiles
// in turn, each with its own m, sum and O, and are joined at the end.  Heads of 256
// leave TMEM for one O only: one stream over two S buffers.
//
// Work.  An item is (lane, key/value head, row tiles); its units are the K/V
// tiles in reach.  All units of the step, in item order, are cut into equal runs,
// one per CTA of a grid of one CTA per SM, from the lengths in device memory:
// ragged batches balance by themselves and a single long lane is split over
// the whole GPU.  A CTA whose run starts or ends inside an item leaves its part
// (m, sum, O) in the workspace, and the last part's CTA joins them in order.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace attn {

constexpr float kLag = 8.f;      // log2 units the running maximum may lag
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxSms = 512;     // tickets at the start of the workspace

template <int D_, int QT_>
struct Shape {
    static constexpr int D = D_, QT = QT_;
    static constexpr int BK = D == 256 ? 64 : 128;             // keys of a tile
    static constexpr int NS = D == 256 ? 1 : 2;                // streams (softmax warpgroups)
    static constexpr int NB = D / 64;                          // 128-byte-wide blocks of an operand
    static constexpr int kQBytes = 128 * D * 2;                // one row tile
    static constexpr int kStageBytes = BK * D * 2;             // a K or a V tile
    static constexpr int kStages = (224 * 1024 - QT * kQBytes) / kStageBytes < 12
                                       ? (224 * 1024 - QT * kQBytes) / kStageBytes : 12;
    static constexpr int kThreads = NS * 128 + 64;             // softmax warpgroups, loader, MMA
    static constexpr int kPayload = QT * kQBytes + kStages * kStageBytes + 2048;   // operands, then the streams' swap area
    static constexpr int kRows = QT * 128;
    // TMEM columns: S buffers, then O
    static constexpr int kO = 2 * BK;
    static constexpr int kPartFloats = kRows * (D + 2);        // O, then m and sum
    static_assert(D == 64 || D == 128 || (D == 256 && QT == 1), "");
    static_assert(kO + NS * D <= 512, "TMEM");
};

struct Args {
    CUtensorMap kmap, vmap;
    const uint16_t *q;
    int64_t tokens, qs_t, qs_h;
    int32_t heads_q, heads_kv, group, log_page;
    const int32_t *block_table, *cu_new, *seq_lens;
    int64_t max_pages;
    int32_t lanes;
    float c;               // scale * log2(e)
    int64_t window;
    uint16_t *out;
    float *lse;
    unsigned int *tickets;
    float *parts;          // [grid][2][kPartFloats]
};

// mbar_wait without the long suspension hint: the waits of this kernel's pipeline
// are a fraction of a microsecond each, on the critical path.  Bounded like it.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(smem_u32(bar)), "r"(parity)
                 : "memory");
    return ok != 0;
}
__device__ __noinline__ bool wait_slow(uint64_t *bar, uint32_t parity)
{
    const uint64_t t0 = global_ns();
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (mbar_test(bar, parity)) return true;
        if (*reinterpret_cast<volatile unsigned int *>(&s_gave_up)) return false;
        if (global_ns() - t0 > kWaitLimitNs) {
            s_gave_up = 1u;
            atomicOr(&g_wait_timeouts, 1u);
            return false;
        }
    }
}
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity)
{
    for (int i = 0; i < 16; ++i)
        if (mbar_test(bar, parity)) return true;
    return wait_slow(bar, parity);
}

// ---- tcgen05 ----------------------------------------------------------------

__device__ __forceinline__ void tmem_alloc(uint32_t *slot)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t base)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(base) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// arrive on bar when every MMA issued so far by this thread is complete
__device__ __forceinline__ void commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
// Operand descriptors travel as their low words (address and leading offset);
// the high word is the same for all.  One elected thread issues 16 products a unit,
// so what it computes between them counts.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);   // rows 1,024 bytes a group of 8; version; 128-byte swizzle
template <bool kAcc>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
                 "setp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc),
                 "n"(kAcc ? 1 : 0), "n"(kDescHi)
                 : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tmov.b64 y, {%2, %5};\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc),
                 "r"((uint32_t)acc), "n"(kDescHi)
                 : "memory");
}
__device__ __forceinline__ void mma_ts_acc(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tmov.b64 y, {%2, %5};\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc),
                 "n"(1), "n"(kDescHi)
                 : "memory");
}
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

#define R8(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), "=r"(r[o + 6]), "=r"(r[o + 7])
#define I8(r, o) "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), "r"(r[o + 5]), "r"(r[o + 6]), "r"(r[o + 7])

// 32 (or 64) columns of the warp's 32 lanes (a thread: its lane's row).  The
// wait is in the same statement, so that no use of the values can move before it.
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t a)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : R8(r, 0), R8(r, 8), R8(r, 16), R8(r, 24)
                 : "r"(a)
                 : "memory");
}
// The load alone, and the wait for it: the values pass through the wait, so that
// no use of them can move before it.
__device__ __forceinline__ void tmem_issue32(uint32_t (&r)[32], uint32_t a)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : R8(r, 0), R8(r, 8), R8(r, 16), R8(r, 24)
                 : "r"(a)
                 : "memory");
}
#define M8(r, o) "+r"(r[o]), "+r"(r[o + 1]), "+r"(r[o + 2]), "+r"(r[o + 3]), "+r"(r[o + 4]), "+r"(r[o + 5]), "+r"(r[o + 6]), "+r"(r[o + 7])
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" : M8(r, 0), M8(r, 8), M8(r, 16), M8(r, 24)::"memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t a, const uint32_t (&r)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::I8(r, 0), I8(r, 8), I8(r, 16),
                 I8(r, 24), "r"(a)
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
                 "%15};" ::I8(r, 0), I8(r, 8), "r"(a)
                 : "memory");
}

// On an edge tile the scores outside [from, to) of 32 are -inf.
__device__ __forceinline__ void mask_scores(uint32_t (&x)[32], int from, int to)
{
#pragma unroll
    for (int e = 0; e < 32; ++e)
        if (e < from || e >= to) x[e] = 0xFF800000u;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t two(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void halves(uint64_t v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Low word of a shared-memory operand descriptor.  Rows of 128 bytes in groups of
// 8; for K-major operands the leading offset is unused, for the MN-major V it is the
// distance between blocks of 64 head elements.
__device__ __forceinline__ uint32_t operand(uint32_t addr, uint32_t leading) { return ((addr & 0x3FFFFu) >> 4) | ((leading >> 4) << 16); }

// Instruction descriptor: fp32 accumulator, A and B both bf16 or both fp16, M =
// 128, N columns, B K-major or MN-major.
__host__ __device__ constexpr uint32_t instr(bool f16, int n, bool b_mn)
{
    return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap *map, int row, int block, int head, int page,
                                         uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
                 "%4, %5, %6}], [%7];" ::"r"(dst),
                 "l"(map), "r"(0), "r"(row), "r"(block), "r"(head), "r"(page), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    if (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// ---- the step's items ---------------------------------------------------------

// A row-tile group of a lane: the keys any of its rows attends, and the K/V tiles.
struct Reach {
    int32_t lo, hi;    // keys [lo, hi); hi <= lo: none
    int32_t tile0;     // first tile
    int32_t tiles;     // at least 1, so that rows with no key are still answered
};

template <typename S>
__device__ __forceinline__ Reach reach_of(const Args &a, int n, int seq, int rt)
{
    const int64_t row0 = (int64_t)rt * S::kRows;
    const int f = (int)(row0 / a.group);
    const int64_t last = (row0 + S::kRows - 1) / a.group;
    const int e = last < n - 1 ? (int)last : n - 1;
    Reach r;
    r.hi = seq - n + e + 1;
    const int64_t lo = a.window > 0 ? (int64_t)(seq - n + f) - a.window + 1 : 0;
    r.lo = lo > 0 ? (int)lo : 0;
    if (r.hi > r.lo) {
        r.tile0 = r.lo / S::BK;
        r.tiles = (r.hi + S::BK - 1) / S::BK - r.tile0;
    } else {
        r.hi = r.lo;
        r.tile0 = r.lo / S::BK;
        r.tiles = 1;
    }
    return r;
}

struct Lane {
    int32_t first, n, seq;   // first row of q, new tokens, keys
};

__device__ __forceinline__ Lane lane_of(const Args &a, int l)
{
    Lane r;
    int32_t c0 = __ldg(a.cu_new + l), c1 = __ldg(a.cu_new + l + 1);
    const int32_t t = (int32_t)a.tokens;
    r.first = c0 < 0 ? 0 : c0 > t ? t : c0;
    const int32_t end = c1 < r.first ? r.first : c1 > t ? t : c1;
    r.n = end - r.first;
    // a lane cut by the buffer keeps its tokens' positions
    const int32_t seq = __ldg(a.seq_lens + l);
    r.seq = (seq < 0 ? 0 : seq) - (c1 > end && r.n > 0 ? c1 - end : 0);
    return r;
}

template <typename S>
__device__ __forceinline__ int row_tiles(const Args &a, int n) { return (int)(((int64_t)n * a.group + S::kRows - 1) / S::kRows); }

template <typename S>
__device__ __forceinline__ int64_t head_units(const Args &a, const Lane &l)
{
    int64_t u = 0;
    const int rts = row_tiles<S>(a, l.n);
    for (int rt = 0; rt < rts; ++rt) u += reach_of<S>(a, l.n, l.seq, rt).tiles;
    return u;
}

// A CTA's run of units [u, end): where it stands.
struct Run {
    int64_t u, end;        // next unit, end of the run
    int64_t item0;         // first unit of the current item
    int32_t lane, head, rt;
    Lane ln;
    int32_t rts;
};

struct Segment {           // the part of an item that this CTA computes
    Reach r;
    int32_t tile, tiles;   // first tile, number of tiles
    int64_t item0;
    int32_t item_tiles;
    int32_t lane, head, rt;
    Lane ln;
};

template <typename S>
__device__ __forceinline__ bool next_segment(const Args &a, Run &w, Segment &s)
{
    if (w.u >= w.end) return false;
    while (w.rt >= w.rts) {           // the next head, or the next lane that has tokens
        w.rt = 0;
        if (w.rts > 0 && ++w.head < a.heads_kv) break;
        w.head = 0;
        ++w.lane;
        w.ln = lane_of(a, w.lane);
        w.rts = row_tiles<S>(a, w.ln.n);
    }
    s.r = reach_of<S>(a, w.ln.n, w.ln.seq, w.rt);
    s.item0 = w.item0;
    s.item_tiles = s.r.tiles;
    const int64_t skip = w.u - w.item0, left = s.r.tiles - skip, room = w.end - w.u;
    s.tile = s.r.tile0 + (int)skip;
    s.tiles = (int)(left < room ? left : room);
    s.lane = w.lane; s.head = w.head; s.rt = w.rt; s.ln = w.ln;
    w.u += s.tiles;
    w.item0 += s.r.tiles;
    ++w.rt;
    return true;
}

struct Plan {
    int64_t total;         // units of the step
    int64_t lane_u;        // units before the lane where this CTA's run starts
    int32_t lane, grid;    // that lane; CTAs that have a run
};

__device__ __forceinline__ int64_t run_start(int64_t cta, int64_t total, int64_t grid) { return cta * total / grid; }
// the CTA whose run holds unit u
__device__ __forceinline__ int64_t run_owner(int64_t u, int64_t total, int64_t grid) { return ((u + 1) * grid + total - 1) / total - 1; }

// ---- the kernel ---------------------------------------------------------------

template <typename S>
struct Bars {
    uint64_t full[S::kStages], empty[S::kStages];
    uint64_t s_full[2], p_full[2], o_done[2], q_full, drain;
};

template <int D, int QT, bool F16>
__global__ void __launch_bounds__(Shape<D, QT>::kThreads, 1) attention_kernel(const __grid_constant__ Args a)
{
    using S = Shape<D, QT>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars<S> bar;
    __shared__ uint32_t tmem_slot;
    __shared__ Plan plan;
    __shared__ int64_t warp_units[S::kThreads / 32];
    __shared__ unsigned int last_part;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kLoader = S::NS * 4, kMma = kLoader + 1;

    pdl_launch_dependents();
    if (tid == 0) {
        s_gave_up = 0u;
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.p_full[i], 4);
            mbar_init(&bar.o_done[i], 1);
        }
        mbar_init(&bar.q_full, S::NS * 4);
        mbar_init(&bar.drain, 1);
        fence_mbar_init();
    }
    if (warp == kLoader && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&a.kmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&a.vmap) : "memory");
    }
    pdl_wait();

    // Units of the step and the lane where this CTA's run starts: each thread
    // sums a contiguous share of the lanes.
    {
        const int per = (a.lanes + S::kThreads - 1) / S::kThreads;
        const int l0 = min(tid * per, a.lanes), l1 = min(l0 + per, a.lanes);
        int64_t mine = 0;
        for (int l = l0; l < l1; ++l) mine += head_units<S>(a, lane_of(a, l)) * a.heads_kv;
        int64_t incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(kFull, incl, d);
            if (lane >= d) incl += y;
        }
        if (lane == 31) warp_units[warp] = incl;
        __syncthreads();
        int64_t before = incl - mine, total = 0;
        for (int w = 0; w < S::kThreads / 32; ++w) {
            if (w < warp) before += warp_units[w];
            total += warp_units[w];
        }
        const int64_t grid = total < (int64_t)gridDim.x ? total : (int64_t)gridDim.x;
        if (tid == 0) {
            plan.total = total;
            plan.grid = (int32_t)grid;
        }
        if ((int64_t)blockIdx.x < grid) {
            const int64_t u0 = run_start(blockIdx.x, total, grid);
            if (u0 >= before && u0 < before + mine) {
                int64_t at = before;
                int l = l0;
                for (;; ++l) {
                    const int64_t u = head_units<S>(a, lane_of(a, l)) * a.heads_kv;
                    if (u0 < at + u) break;
                    at += u;
                }
                plan.lane = l;
                plan.lane_u = at;
            }
        }
        __syncthreads();
    }
    if ((int64_t)blockIdx.x >= plan.grid) return;

    if (warp == kMma) tmem_alloc(&tmem_slot);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;

    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *q_smem = smem, *kv_smem = smem + QT * S::kQBytes;
    float2 *ml_swap = reinterpret_cast<float2 *>(kv_smem + S::kStages * S::kStageBytes);   // [2][128]

    Run run;
    {
        const int64_t total = plan.total;
        run.u = run_start(blockIdx.x, total, plan.grid);
        run.end = run_start(blockIdx.x + 1, total, plan.grid);
        run.lane = plan.lane;
        run.ln = lane_of(a, run.lane);
        run.rts = row_tiles<S>(a, run.ln.n);
        const int64_t per_head = head_units<S>(a, run.ln), off = run.u - plan.lane_u;
        run.head = (int)(off / per_head);
        run.item0 = plan.lane_u + run.head * per_head;
        run.rt = 0;
        for (;;) {
            const int t = reach_of<S>(a, run.ln.n, run.ln.seq, run.rt).tiles;
            if (run.u < run.item0 + t) break;
            run.item0 += t;
            ++run.rt;
        }
    }

    if (warp == kLoader) {
        // ---- K and V tiles: a lane of the warp per page, in the order K0 V0 K1 V1 ...
        const int rows = min(1 << a.log_page, S::BK);            // rows of a box
        const int boxes = S::BK / rows;
        const bool whole = rows == S::BK;                        // one box brings all blocks
        const uint32_t box_bytes = (uint32_t)rows * D * 2;
        uint32_t idx = 0;                                        // stage uses so far
        bool ok = true;
        Segment s;
        while (ok && next_segment<S>(a, run, s)) {
            for (int t = 0; t < s.tiles && ok; ++t) {
                const int key0 = (s.tile + t) * S::BK, k0 = key0 + lane * rows;
                const bool mine = lane < boxes && k0 < s.r.hi && k0 + rows > s.r.lo;
                int page = -1;
                if (mine) {
                    const int64_t pi = k0 >> a.log_page;
                    if (pi < a.max_pages) page = __ldg(a.block_table + s.lane * a.max_pages + pi);
                }
                const uint32_t bytes = __popc(__ballot_sync(kFull, mine)) * box_bytes;
                const int row = k0 & ((1 << a.log_page) - 1);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv, ++idx) {
                    const uint32_t st = idx % S::kStages, use = idx / S::kStages;
                    ok = ok && wait(&bar.empty[st], (use & 1) ^ 1);
                    ok = __all_sync(kFull, ok);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&bar.full[st], bytes);
                    __syncwarp();
                    if (mine) {
                        const CUtensorMap *map = kv ? &a.vmap : &a.kmap;
                        const uint32_t dst = smem_u32(kv_smem) + st * S::kStageBytes + lane * rows * 128;
                        if (whole) tma_page(dst, map, row, 0, s.head, page, &bar.full[st]);
                        else
#pragma unroll
                            for (int b = 0; b < S::NB; ++b)
                                tma_page(dst + b * S::BK * 128, map, row, b, s.head, page, &bar.full[st]);
                    }
                    __syncwarp();
                }
            }
        }
        if (!ok) {
            // given up: the copies in flight still have to land (each stage's
            // last use; bounded, whatever the other waits did)
            for (uint32_t i = idx > (uint32_t)S::kStages ? idx - S::kStages : 0; i < idx; ++i) {
                const uint64_t t0 = global_ns();
                while (!mbar_try_wait(&bar.full[i % S::kStages], (i / S::kStages) & 1) && global_ns() - t0 < kWaitLimitNs) {}
            }
        }
    } else if (warp == kMma) {
        // ---- the products, issued by one thread (the warp walks along with it)
        constexpr uint32_t kQk = instr(F16, S::BK, false), kPv = instr(F16, D, true);
        const bool leader = elect_one();
        uint32_t items = 0, units[2] = {0, 0};               // items so far; units per S buffer
        uint32_t k_stage = 0, k_phase = 0, v_stage = 1, v_phase = 0;   // of the next K and V tile (every second stage use)
        static_assert(S::kStages >= 3, "");
        auto advance = [](uint32_t &st, uint32_t &ph) {
            st += 2;
            if (st >= (uint32_t)S::kStages) {
                st -= S::kStages;
                ph ^= 1;
            }
        };
        bool ok = true;
        Segment s;
        const uint32_t q_desc = operand(smem_u32(q_smem), 16), k_desc = operand(smem_u32(kv_smem), 16),
                       v_desc = operand(smem_u32(kv_smem), S::BK * 128);
        while (ok && next_segment<S>(a, run, s)) {
            const int U = QT == 2 ? 2 * s.tiles : s.tiles;
            auto qk = [&](int i) -> bool {
                const int b = i & 1;
                if (!wait(&bar.full[k_stage], k_phase)) return false;
                fence_after();
                if (leader) {
                    const uint32_t qa = q_desc + (QT == 2 ? b * (S::kQBytes >> 4) : 0), ka = k_desc + k_stage * (S::kStageBytes >> 4);
                    const uint32_t d = tmem + b * S::BK;
                    mma_ss<false>(d, qa, ka, kQk);
#pragma unroll
                    for (int k = 1; k < D / 16; ++k)
                        mma_ss<true>(d, qa + (k >> 2) * (128 * 128 >> 4) + (k & 3) * 2, ka + (k >> 2) * (S::BK * 128 >> 4) + (k & 3) * 2, kQk);
                    commit(&bar.s_full[b]);
                    if (QT == 1 || b == 1) commit(&bar.empty[k_stage]);
                }
                __syncwarp();
                if (QT == 1 || b == 1) advance(k_stage, k_phase);
                return true;
            };
            ok = wait(&bar.q_full, items & 1);
            fence_after();
            ok = ok && qk(0);
            for (int i = 0; i < U && ok; ++i) {
                if (i + 1 < U) ok = qk(i + 1);
                const int b = i & 1, ob = S::NS == 2 ? b : 0;
                ok = ok && wait(&bar.full[v_stage], v_phase);
                ok = ok && wait(&bar.p_full[b], units[b] & 1);
                if (!ok) break;
                ++units[b];
                fence_after();
                if (leader) {
                    const uint32_t va = v_desc + v_stage * (S::kStageBytes >> 4), d = tmem + S::kO + ob * D, pa = tmem + b * S::BK;
                    mma_ts(d, pa, va, kPv, S::NS == 2 ? i >= 2 : i >= 1);
#pragma unroll
                    for (int k = 1; k < S::BK / 16; ++k) mma_ts_acc(d, pa + k * 8, va + k * (2048 >> 4), kPv);
                    commit(&bar.o_done[ob]);
                    if (QT == 1 || b == 1) commit(&bar.empty[v_stage]);
                }
                __syncwarp();
                if (QT == 1 || b == 1) advance(v_stage, v_phase);
            }
            ++items;
        }
        // everything issued is complete before TMEM is freed
        if (leader) {
            commit(&bar.drain);
            const uint64_t t0 = global_ns();
            while (!mbar_try_wait(&bar.drain, 0) && global_ns() - t0 < kWaitLimitNs) {}
        }
        __syncwarp();
    } else {
        // ---- softmax, correction and epilogue: warpgroup `st` is stream st
        const int st = warp >> 2, row = tid & 127;                // row of the tile
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const int wg_rows = QT == 2 ? 128 : 128 * S::NS;          // threads that load one Q tile together
        uint32_t tile_n = 0, s_n[2] = {0, 0}, pv_n = 0;           // tiles so far, units per S buffer, PVs of this stream
        Segment s;
        while (next_segment<S>(a, run, s)) {
            const int64_t rows_all = (int64_t)s.ln.n * a.group;
            const int64_t tile_row0 = (int64_t)s.rt * S::kRows + (QT == 2 ? st * 128 : 0);
            // Q: 16-byte pieces, consecutive threads on consecutive pieces of a row
            {
                constexpr int kPieces = D / 8;
                uint8_t *dst = q_smem + (QT == 2 ? st * S::kQBytes : 0);
                const int t0 = QT == 2 ? row : tid;
                const int64_t have = rows_all - tile_row0;
                const int valid = have < 0 ? 0 : have < 128 ? (int)have : 128;
                for (int i = t0; i < valid * kPieces; i += wg_rows) {
                    const int r = i / kPieces, p = i % kPieces;
                    const int64_t gr = tile_row0 + r, tok = gr / a.group;
                    const int h = s.head * a.group + (int)(gr - tok * a.group);
                    const uint4 x = __ldg(reinterpret_cast<const uint4 *>(a.q + (s.ln.first + tok) * a.qs_t + h * a.qs_h) + p);
                    *reinterpret_cast<uint4 *>(dst + (p >> 3) * (128 * 128) + r * 128 + (((p & 7) ^ (r & 7)) << 4)) = x;
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.q_full);
            }
            const int64_t gr = tile_row0 + row;
            const bool valid = gr < rows_all;
            const int64_t tok = valid ? gr / a.group : 0;
            const int h = s.head * a.group + (int)(valid ? gr - tok * a.group : 0);
            const int pos = s.ln.seq - s.ln.n + (int)tok;
            const int64_t klo64 = a.window > 0 ? (int64_t)pos - a.window + 1 : 0;
            const int klo = klo64 > 0 ? (int)klo64 : 0, khi = valid ? pos + 1 : klo;   // keys of this row
            const bool live = __any_sync(kFull, khi > klo);

            float m = -INFINITY, l = 0.f;
            int done = 0;                                          // units of this stream so far
            const int U = QT == 2 || S::NS == 1 ? s.tiles : (s.tiles - st + 1) >> 1;
            for (int i = 0; i < U; ++i, ++done) {
                const int t = QT == 2 || S::NS == 1 ? i : 2 * i + st;
                const int b = S::NS == 2 ? st : i & 1;
                const int key0 = (s.tile + t) * S::BK;
                wait(&bar.s_full[b], s_n[b] & 1);
                ++s_n[b];
                fence_after();
                if (live) {
                    const uint32_t sa = tmem + lane_base + b * S::BK;
                    // columns of this row in the tile; what a row past the item's holds is nobody's
                    const int from = valid ? klo - key0 : 0, to = valid ? khi - key0 : S::BK;
                    const bool edge = __any_sync(kFull, from > 0 || to < S::BK);
                    // Two passes over S in TMEM, 32 columns at a time with the next 32
                    // on their way (a row's whole tile in registers would spill).
                    uint32_t xa[32], xb[32];
                    float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    auto top_of = [&](uint32_t (&x)[32], int c) {
                        if (edge) mask_scores(x, from - c, to - c);
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                top4[k] = max3(top4[k], __uint_as_float(x[e + k]), __uint_as_float(x[e + 4 + k]));
                    };
                    tmem_issue32(xa, sa);
#pragma unroll
                    for (int c = 0; c < S::BK; c += 64) {
                        tmem_wait32(xa);
                        tmem_issue32(xb, sa + c + 32);
                        top_of(xa, c);
                        tmem_wait32(xb);
                        tmem_issue32(xa, c + 64 < S::BK ? sa + c + 64 : sa);   // at the end: the second pass's first
                        top_of(xb, c + 32);
                    }
                    float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
                    top *= a.c;
                    // a new reference only past the lag (or for a row's first key)
                    const bool move = valid && (top > m + kLag || (m == -INFINITY && top > -INFINITY));
                    if (__any_sync(kFull, move)) {
                        const float f = move ? exp2_fast(m - top) : 1.f;
                        if (move) m = top;
                        l *= f;
                        if (done > 0) {
                            wait(&bar.o_done[st], (pv_n - 1) & 1);
                            fence_after();
                            const uint32_t oa = tmem + lane_base + S::kO + st * D;
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                uint32_t o[32];
                                tmem_ld32(o, oa + c * 32);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tmem_st32(oa + c * 32, o);
                            }
                        }
                    }
                    const float ref = m == -INFINITY ? 0.f : m;
                    const uint64_t cc = two(a.c, a.c), mm = two(-ref, -ref);
                    uint64_t sum[2] = {0ull, 0ull};
                    // P of columns c .. c+31 covers columns c/2 .. c/2+15 of S, read before
                    auto weights = [&](uint32_t (&x)[32], int c) {
                        if (edge) mask_scores(x, from - c, to - c);
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float p0, p1;
                            halves(fma2(two(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), cc, mm), p0, p1);
                            p0 = exp2_fast(p0);
                            p1 = exp2_fast(p1);
                            sum[e & 1] = add2(sum[e & 1], two(p0, p1));
                            pk[e] = pack2<F16>(p0, p1);
                        }
                        tmem_st16(sa + c / 2, pk);
                    };
#pragma unroll
                    for (int c = 0; c < S::BK; c += 64) {
                        tmem_wait32(xa);
                        tmem_issue32(xb, sa + c + 32);
                        weights(xa, c);
                        tmem_wait32(xb);
                        if (c + 64 < S::BK) tmem_issue32(xa, sa + c + 64);
                        weights(xb, c + 32);
                    }
                    float s0, s1;
                    halves(add2(sum[0], sum[1]), s0, s1);
                    l += s0 + s1;
                }
                // V rows that no row of the item may see hold anything, NaN
                // included: 0 * NaN must not reach O
                if (key0 < s.r.lo || key0 + S::BK > s.r.hi) {
                    const uint32_t idx = 2 * (tile_n + t) + 1, vs = idx % S::kStages;
                    wait(&bar.full[vs], (idx / S::kStages) & 1);
                    uint8_t *v = kv_smem + vs * S::kStageBytes;
                    constexpr int kPer = 128 / S::BK;               // threads of a key row
                    const int kr = row / kPer, part = row % kPer;
                    if (key0 + kr < s.r.lo || key0 + kr >= s.r.hi) {
#pragma unroll
                        for (int blk = 0; blk < S::NB; ++blk)
#pragma unroll
                            for (int p = part; p < 8; p += kPer)
                                *reinterpret_cast<uint4 *>(v + blk * (S::BK * 128) + kr * 128 + p * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async();
                }
                // One stream over two S buffers: S of this unit says nothing about the
                // product before it, and a barrier's parity tells only its last two phases
                // apart, so that every phase is waited for.  (With two streams, S of a
                // stream's unit comes after its last product.)
                if (S::NS == 1 && done > 0) wait(&bar.o_done[st], (pv_n - 1) & 1);
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_full[b]);
                ++pv_n;
            }
            tile_n += s.tiles;
            if (U > 0) wait(&bar.o_done[st], (pv_n - 1) & 1);
            fence_after();

            // where the rows go: the output, or this CTA's part of the item
            const bool split = s.tiles < s.item_tiles;
            const int slot = s.tile == s.r.tile0 ? 1 : 0;          // an item begun here, or one begun before
            float *part = a.parts + ((int64_t)blockIdx.x * 2 + slot) * S::kPartFloats + (QT == 2 ? st * 128 * (D + 2) : 0);
            float f0 = 1.f, f1 = 0.f;                              // weights of the two streams' O
            int c0 = 0, c1 = D;                                    // columns this thread writes
            if (QT == 1 && S::NS == 2) {
                // join the streams: the same row of the other warpgroup; each takes half the columns
                ml_swap[st * 128 + row] = make_float2(m, l);
                fence_before();
                asm volatile("bar.sync 1, 256;" ::: "memory");
                fence_after();
                const float2 e0 = ml_swap[row], e1 = ml_swap[128 + row];
                m = fmaxf(e0.x, e1.x);
                f0 = e0.x == -INFINITY ? 0.f : exp2_fast(e0.x - m);
                f1 = e1.x == -INFINITY ? 0.f : exp2_fast(e1.x - m);
                l = e0.y * f0 + e1.y * f1;
                c0 = st * (D / 2);
                c1 = c0 + D / 2;
            }
            const float inv = split ? 1.f : l > 0.f ? 1.f / l : 0.f;
            const int64_t out_row = ((int64_t)s.ln.first + tok) * a.heads_q + h;
            if (live) {
                const uint32_t oa = tmem + lane_base + S::kO + (QT == 2 ? st * D : 0);
#pragma unroll 1
                for (int c = c0; c < c1; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(o, oa + c);
                    if (QT == 1 && S::NS == 2 && s.tiles > 1) {
                        uint32_t o1[32];
                        tmem_ld32(o1, oa + D + c);
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float v0 = f0 > 0.f ? __uint_as_float(o[e]) * f0 : 0.f;
                            const float v1 = f1 > 0.f ? __uint_as_float(o1[e]) * f1 : 0.f;
                            o[e] = __float_as_uint(v0 + v1);
                        }
                    }
                    if (l <= 0.f) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0u;
                    }
                    if (!valid) continue;
                    if (split) {
                        float4 *dst = reinterpret_cast<float4 *>(part) + (c / 4) * 128 + row;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            dst[e * 128] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                       __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
                    } else {
                        uint4 *dst = reinterpret_cast<uint4 *>(a.out + out_row * D + c);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                w[k] = pack2<F16>(__uint_as_float(o[8 * e + 2 * k]) * inv, __uint_as_float(o[8 * e + 2 * k + 1]) * inv);
                            dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
            } else if (valid && !split) {                          // a warp of rows without keys
                for (int c = c0; c < c1; c += 8) *reinterpret_cast<uint4 *>(a.out + out_row * D + c) = make_uint4(0, 0, 0, 0);
            }
            if (valid && c0 == 0) {
                if (split) {
                    float *ml = part + 128 * D;
                    ml[row] = live ? m : -INFINITY;
                    ml[128 + row] = live ? l : 0.f;
                } else if (a.lse) {
                    a.lse[out_row] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
                }
            }
            fence_before();

            if (split) {
                // publish, and the last part's CTA joins all parts in order
                constexpr int kT = S::NS * 128;
                const int64_t first_cta = run_owner(s.item0, plan.total, plan.grid);
                const int n_parts = (int)(run_owner(s.item0 + s.item_tiles - 1, plan.total, plan.grid) - first_cta) + 1;
                __threadfence();
                asm volatile("bar.sync 2, %0;" ::"n"(kT) : "memory");
                if (tid == 0) {
                    last_part = atom_add_acq_rel(a.tickets + first_cta, 1u) == (unsigned)n_parts - 1 ? 1u : 0u;
                    if (last_part) a.tickets[first_cta] = 0u;
                }
                asm volatile("bar.sync 2, %0;" ::"n"(kT) : "memory");
                if (last_part) {
                    __threadfence();
                    for (int qt = 0; qt < QT; ++qt) {
                        const int64_t r0 = (int64_t)s.rt * S::kRows + qt * 128;
                        const int64_t have = rows_all - r0;
                        const int nr = have < 0 ? 0 : have < 128 ? (int)have : 128;
                        for (int i = tid; i < nr * (D / 8); i += kT) {
                            const int r = i % nr, c = i / nr * 8;
                            auto part_of = [&](int p) -> const float * {
                                return a.parts + ((first_cta + p) * 2 + (p == 0 ? 1 : 0)) * S::kPartFloats + qt * 128 * (D + 2);
                            };
                            float M = -INFINITY;
#pragma unroll 4
                            for (int p = 0; p < n_parts; ++p) M = fmaxf(M, __ldcg(part_of(p) + 128 * D + r));
                            float L = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
                            for (int p = 0; p < n_parts; ++p) {
                                const float *pp = part_of(p);
                                const float mp = __ldcg(pp + 128 * D + r), lp = __ldcg(pp + 128 * D + 128 + r);
                                if (mp == -INFINITY) continue;
                                const float f = exp2_fast(mp - M);
                                const float4 x = __ldcg(reinterpret_cast<const float4 *>(pp) + (c / 4) * 128 + r);
                                const float4 y = __ldcg(reinterpret_cast<const float4 *>(pp) + (c / 4 + 1) * 128 + r);
                                L = fmaf(lp, f, L);
                                o[0] = fmaf(x.x, f, o[0]); o[1] = fmaf(x.y, f, o[1]);
                                o[2] = fmaf(x.z, f, o[2]); o[3] = fmaf(x.w, f, o[3]);
                                o[4] = fmaf(y.x, f, o[4]); o[5] = fmaf(y.y, f, o[5]);
                                o[6] = fmaf(y.z, f, o[6]); o[7] = fmaf(y.w, f, o[7]);
                            }
                            const float iv = L > 0.f ? 1.f / L : 0.f;
                            const int64_t g = r0 + r, tk = g / a.group;
                            const int64_t orow = ((int64_t)s.ln.first + tk) * a.heads_q + s.head * a.group + (g - tk * a.group);
                            *reinterpret_cast<uint4 *>(a.out + orow * D + c) =
                                make_uint4(pack2<F16>(o[0] * iv, o[1] * iv), pack2<F16>(o[2] * iv, o[3] * iv),
                                           pack2<F16>(o[4] * iv, o[5] * iv), pack2<F16>(o[6] * iv, o[7] * iv));
                            if (c == 0 && a.lse) a.lse[orow] = L > 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
                        }
                    }
                }
            }
            if (S::NS == 2 && QT == 1) {
                // Q and the swap area are reused by the next item
                asm volatile("bar.sync 1, 256;" ::: "memory");
            }
        }
    }
    __syncthreads();
    if (warp == kMma) {
        fence_after();
        tmem_free(tmem);
    }
}

}  // namespace attn
