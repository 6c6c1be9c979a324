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
// when a tile exceeds it by more than 2^8 (kLag; 2^4 in fp16), and only then O and the sum
// are rescaled.  A bf16 weight rounds relative to itself at any size.  An fp16 one does
// from 2^-14 on and is lost below 2^-25, while a long context's weights may add up
// to something at 2^-25 of the largest each; so fp16's reference lies 2^7 below the
// maximum (kRaise): the largest weight is 2^7 .. 2^11, and the others round relative to
// themselves down to 2^-21 of it, to 2^-32 of it below that.  (Above 2^11 there is
// room up to fp16's 65,504 for what fp32 leaves open between a score and the maximum it was
// compared with: 2^4 where scores reach 2^27.)  The sum is kept in fp32, of unrounded weights.
//
// Two streams hide the softmax of one behind the products of the other: with
// two row tiles in a CTA (QT = 2, chunks) each stream has its rows and both
// use every K/V tile; with one row tile (QT = 1) the streams take the K/V tiles
// in turn, each with its own m, sum and O, and are joined at the end.  Heads of 256
// leave TMEM for one O only: one stream over two S buffers.  Each stream has two
// warpgroups, one for each half of a tile's columns: a softmax thread holds half a row's
// scores, and the pair agrees on the maximum through shared memory.
//
// Work.  An item is (lane, key/value head, row tiles); its units are the K/V
// tiles in reach, and kExtra for what it costs beside them.  All units of the step,
// in item order, are cut into equal runs, one per CTA of a grid of one CTA per SM, from the lengths in device memory:
// ragged batches balance by themselves and a single long lane is split over
// the whole GPU.  A CTA whose run starts or ends inside an item leaves its part
// (m, sum, O) in the workspace; when its run is done it waits for the item's
// other parts and joins its share of the item's elements, in an order of sums that
// follows from the item and the CTA's place in it, not from timing.  (The
// launch is cooperative, so all CTAs are there; runs are equal, so the wait is
// short, and it is bounded.  Items in 152 parts, in a graph: one token of one head of 128 over
// 38,912 keys 16 us, 24 with the last part's CTA joining alone; 128 rows of 256 over
// 19,456 keys 30 against 284.  A second kernel for the joins cost every call 4 us.)  Where the parts of an item are small,
// the last part's CTA does join alone, and the launch is an ordinary one (the
// host's rule is at the launch).  The loader warp works the items out and hands them
// to the others through a ring in shared memory.
//
// What bounds it, on GB300 (graph-replayed; fractions of a measured copy, 6,788 GB/s, and
// of a cuBLAS bf16 product, 1,886 TFLOP/s).  Many cached keys for few rows: the cache's bytes --
// 16 lanes of 8 tokens over 16,000 keys, 32 query on 8 key/value heads of 128, 167 us, 0.93; 16
// tokens over 262,144 keys 162 us, 0.98.  Chunks: the chain of a stream from one S to
// the next (product, softmax, product) with the tensor pipe 50-60% busy -- 2,048 tokens over
// 30,000 keys 708 us, 1,470 TFLOP/s, 0.78; heads of 64 870 TFLOP/s (the same softmax for half
// the products), heads of 256 1,130 (K and V tiles of 64 keys from L2 for one row tile).  A prompt of
// 2,048 at 0 keys 52 us, 660 TFLOP/s: rows of Q, edges, outputs and joins as much as tiles.  Little
// work: the chain of one tile, 8 us (lengths 1.0, runs 1.5, first tile 1.5, scores 0.4, softmax
// 1-2, product 0.4, output 1), and 3 us more where parts are joined.  Neither the exponentials (a polynomial for a
// quarter of them: 748 -> 804 us) nor the second pass over S (held back in registers: 745 -> 769 us)
// nor the weights' last columns (their product in two lots: 733 -> 742 us) is what a chunk waits for.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace attn {

template <bool F16>
constexpr float kLag = F16 ? 4.f : 8.f;     // log2 units the running maximum may lag
template <bool F16>
constexpr float kRaise = F16 ? 7.f : 0.f;   // log2 units of the reference below the maximum it was taken from
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kItemBit = 40;     // a step's tiles are counted below this bit of a word, its items above (the host checks that they fit)
constexpr int kMaxSms = 512;     // counters at the start of the workspace: [2][kMaxSms]

template <int D_, int QT_>
struct Shape {
    static constexpr int D = D_, QT = QT_;
    static constexpr int BK = D == 256 ? 64 : 128;             // keys of a tile
    static constexpr int NS = D == 256 ? 1 : 2;                // streams (softmax warpgroups)
    static constexpr int NB = D / 64;                          // 128-byte-wide blocks of an operand
    static constexpr int kQBytes = 128 * D * 2;                // one row tile
    static constexpr int kStageBytes = BK * D * 2;             // a K or a V tile
    static constexpr int QB = QT == 1 && D <= 128 ? 2 : 1;     // Q buffers
    static constexpr int kStages = (224 * 1024 - QB * QT * kQBytes) / kStageBytes < 12
                                       ? (224 * 1024 - QB * QT * kQBytes) / kStageBytes : 12;
    static constexpr int kSoftmaxWarps = NS * 8;
    static constexpr int kThreads = kSoftmaxWarps * 32 + 128;  // softmax; K/V loader, MMA, two Q loaders
    static constexpr int kSwap = 512;                          // floats that softmax warps exchange through
    static constexpr int kPayload = QB * QT * kQBytes + kStages * kStageBytes + kSwap * 4;
    static constexpr int kRows = QT * 128;
    static constexpr int kExtra = QT == 2 ? 4 : 3;             // tiles that an item's other work costs
    static constexpr int kLeast = QT == 1 ? 2 : 1;             // units of a run that an item is cut into, at least
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
    uint32_t group_magic, group_shift;   // n / group = (umulhi(n, magic) + n) >> shift for n below 2^31
    const int32_t *block_table, *cu_new, *seq_lens;
    int64_t max_pages;
    int32_t lanes;
    int32_t most_keys;     // what a lane's length is cut to, so that the step has at most 2^kItemBit tiles
    int32_t share_joins;   // the CTAs of an item share its join (a cooperative launch); else its last part's CTA does it
    float c;               // scale * log2(e)
    int64_t window;
    uint16_t *out;
    float *lse;
    unsigned int *counters;   // [2][kMaxSms], zero between calls: parts published, and joiners done, of the item begun by a CTA
    float *parts;          // [grid][2][kPartFloats]
};

// An item in parts that this CTA has one of: the second slot's part of CTA
// `first_cta` (which begins the item) and the first slots' of the n - 1 CTAs after it.
struct Join {
    int32_t n;             // 0: none
    int32_t first_cta;
    int32_t rows;          // of the item's row tiles, in use
    int32_t first, head, rt;
    int32_t from, count;   // elements (16 columns of a row) this CTA joins: its share, or all if its part comes last
    int32_t lg;            // log2 of the threads that share an element's parts, two of them each at least
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
__device__ __forceinline__ void tmem_st32(uint32_t a, const uint32_t (&r)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::I8(r, 0), I8(r, 8), I8(r, 16),
                 I8(r, 24), "r"(a)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t (&r)[16], uint32_t a)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : R8(r, 0), R8(r, 8)
                 : "r"(a)
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

// 16 bytes global -> shared, and the wait for all of the thread's
__device__ __forceinline__ void copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_landed() { asm volatile("cp.async.wait_all;" ::: "memory"); }

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

// Rows of all new tokens are below 2^31 (checked by the host), and the divisor is
// the same for all: a multiplication by its reciprocal, rounded up to 33 bits.  (The
// plan of the runs and the loads of Q wait for these divides; the 64-bit ones of a
// first version took 3 us of a call.)
__device__ __forceinline__ uint32_t div_group(const Args &a, uint32_t n) { return (__umulhi(n, a.group_magic) + n) >> a.group_shift; }

// A row-tile group of a lane: the keys any of its rows attends, and the K/V tiles.
struct Reach {
    int32_t lo, hi;    // keys [lo, hi); hi <= lo: none
    int32_t tile0;     // first tile
    int32_t tiles;     // at least 1, so that rows with no key are still answered
};

template <typename S>
__device__ __forceinline__ Reach reach_of(const Args &a, int n, int seq, int rt)
{
    const uint32_t row0 = (uint32_t)rt * S::kRows;
    const int last = (int)div_group(a, row0 + S::kRows - 1), e = last < n - 1 ? last : n - 1;
    Reach r;
    r.hi = seq - n + e + 1;
    r.lo = 0;
    if (a.window > 0) {
        const int64_t lo = (int64_t)(seq - n + (int)div_group(a, row0)) - a.window + 1;
        r.lo = lo > 0 ? (int)lo : 0;
    }
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
    // a lane cut by the buffer keeps its tokens' positions; a length that is no
    // length must not overflow the tiles' arithmetic
    const int32_t seq = __ldg(a.seq_lens + l);
    r.seq = (seq < 0 ? 0 : seq > a.most_keys ? a.most_keys : seq) - (c1 > end && r.n > 0 ? c1 - end : 0);
    return r;
}

template <typename S>
__device__ __forceinline__ int row_tiles(const Args &a, int n) { return (int)(((uint32_t)n * (uint32_t)a.group + S::kRows - 1) / S::kRows); }

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
    int32_t extra;         // units of an item before its tiles'
    int32_t lane, head, rt;
    Lane ln;
    int32_t rts;
};

struct Segment {           // the part of an item that this CTA computes
    Reach r;
    int32_t tile, tiles;   // first tile, number of tiles
    int64_t item0;         // unit of the item's first tile
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
    s.item0 = w.item0 + w.extra;
    s.item_tiles = s.r.tiles;
    const int64_t left = s.r.tiles - (w.u - s.item0), room = w.end - w.u, to = w.u + (left < room ? left : room);
    const int from = w.u > s.item0 ? (int)(w.u - s.item0) : 0;
    s.tile = s.r.tile0 + from;
    s.tiles = (int)(to - s.item0) - from;
    s.lane = w.lane; s.head = w.head; s.rt = w.rt; s.ln = w.ln;
    w.u = to;
    w.item0 = s.item0 + s.r.tiles;
    ++w.rt;
    return s.tiles > 0;    // (a run that ends before an item's first tile leaves it to the next)
}

// Run c is units [floor(c * total / grid), floor((c + 1) * total / grid)).
struct Plan {
    int64_t total;         // units of the step: the tiles, and `extra` for every item
    int64_t each;          // total / grid
    int64_t lane_u;        // units before the lane where this CTA's run starts
    int64_t per_head;      // units of one head of that lane
    int32_t more, lane, grid;   // total % grid; that lane; CTAs that have a run
    int32_t extra;
};

__device__ __forceinline__ int64_t run_start(int cta, int64_t each, int32_t more, int32_t grid) { return cta * each + (uint32_t)(cta * more) / (uint32_t)grid; }
// the CTA whose run holds unit u
__device__ __forceinline__ int run_owner(int64_t u, int64_t total, int32_t grid) { return (int)udiv((u + 1) * grid + total - 1, total) - 1; }

// ---- the kernel ---------------------------------------------------------------

// What the other warps need of a segment.
struct Item {
    int32_t first, n, seq, head, rt;
    int32_t lo, hi, tile, tiles;   // tiles == 0: no more items
    int32_t slot;                  // -1: a whole item; else where its part goes
    int32_t pad[2];
};
constexpr int kItems = 4;

template <typename S>
struct Bars {
    uint64_t full[S::kStages], empty[S::kStages];
    uint64_t s_full[2], p_full[2], o_done[2];
    uint64_t q_full[2], q_empty[2], item_full[kItems], item_empty[kItems], drain;
    uint64_t part_full[2], part_known[2];   // the part in a slot is written; the others know
};

__device__ __forceinline__ void named_barrier(int id, int threads)
{
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// a barrier that tells every thread whether any of them says so
__device__ __forceinline__ bool named_barrier_any(int id, int threads, bool mine)
{
    uint32_t any;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.or.pred q, %1, %2, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(any)
                 : "r"(id), "r"(threads), "r"((uint32_t)mine)
                 : "memory");
    return any != 0;
}
__device__ __forceinline__ uint32_t ld_acquire(const unsigned int *p)
{
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
constexpr int kAllSoftmax = 9;   // barrier ids: 1 .. 8 a pair of warps with the same rows, 9 all softmax warps

template <int D, int QT, bool F16>
__global__ void __launch_bounds__(Shape<D, QT>::kThreads, 1) attention_kernel(const __grid_constant__ Args a)
{
    using S = Shape<D, QT>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars<S> bar;
    __shared__ Item items[kItems];
    __shared__ Join joins[2];      // of the parts in this CTA's first and second slot
    __shared__ int32_t came_last[2];   // this CTA's part was the item's last (where joins are not shared)
    __shared__ uint32_t tmem_slot;
    __shared__ Plan plan;
    __shared__ __align__(16) int64_t warp_units[S::kThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kLoader = S::kSoftmaxWarps, kMma = kLoader + 1, kQLoader = kLoader + 2;

    pdl_launch_dependents();
    if (tid == 0) {
        s_gave_up = 0u;
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.p_full[i], 8);
            mbar_init(&bar.o_done[i], 1);
            mbar_init(&bar.q_full[i], 2);
            mbar_init(&bar.q_empty[i], 1);
            mbar_init(&bar.part_full[i], S::kSoftmaxWarps);
            mbar_init(&bar.part_known[i], 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&bar.item_full[i], 1);
            mbar_init(&bar.item_empty[i], S::kSoftmaxWarps + 3);
        }
        mbar_init(&bar.drain, 1);
        fence_mbar_init();
    }
    if (warp == kLoader && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&a.kmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&a.vmap) : "memory");
    }
    if (warp == kMma) tmem_alloc(&tmem_slot);
    pdl_wait();

    // Units of the step and the lane where this CTA's run starts.  Few lanes: a
    // warp each, its threads sharing the row tiles; many: each thread sums a
    // contiguous share of them.
    {
        constexpr int kWarps = S::kThreads / 32;
        const bool by_warp = a.lanes <= kWarps;
        const int per = (a.lanes + S::kThreads - 1) / S::kThreads;
        const int l0 = by_warp ? warp : min(tid * per, a.lanes), l1 = by_warp ? min(warp + 1, a.lanes) : min(l0 + per, a.lanes);
        // units in the low bits, items (a CTA of its own each, if there are enough) above
        constexpr int64_t kUnits = (1ll << kItemBit) - 1;
        int64_t mine = 0, head = 0, incl;
        if (by_warp) {
            if (l0 < l1) {
                const Lane ln = lane_of(a, l0);
                const int rts = row_tiles<S>(a, ln.n);
                for (int rt = lane; rt < rts; rt += 32) head += reach_of<S>(a, ln.n, ln.seq, rt).tiles + (1ll << kItemBit);
            }
#pragma unroll
            for (int d = 16; d; d >>= 1) head += __shfl_xor_sync(kFull, head, d);
            incl = mine = head * a.heads_kv;
        } else {
            for (int l = l0; l < l1; ++l) {
                const Lane ln = lane_of(a, l);
                head = head_units<S>(a, ln) + ((int64_t)row_tiles<S>(a, ln.n) << kItemBit);
                mine += head * a.heads_kv;
            }
            incl = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t y = __shfl_up_sync(kFull, incl, d);
                if (lane >= d) incl += y;
            }
        }
        if (lane == 31) warp_units[warp] = incl;
        fence_before();
        __syncthreads();
        fence_after();
        int64_t all = 0, below = 0;                              // of all warps, of those before this one
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const int64_t x = warp_units[w];
            all += x;
            below += w < warp ? x : 0;
        }
        // An item costs more than its tiles: its rows of Q, its first scores and its output
        // take the time of kExtra tiles, and a run is cut by that too (a prompt of 2,048 at 0
        // keys 84.3 us without, 72.3 with 1, 63.0 with 2, 59.1 with 3, 58.5 with 4; 8 lanes of
        // 8 tokens 57.5, 55.0, 54.4, 54.0, 54.5).  Not where there are too few tiles for
        // runs of two each: there the cuts are even ones of the tiles (one token at 1,000
        // keys 12.9 us, with extra units its first part would be shorter than the others).
        const int32_t extra = (all & kUnits) >= 2 * (int64_t)gridDim.x ? S::kExtra : 0;
        auto units_of = [&](int64_t x) { return (x & kUnits) + extra * (x >> kItemBit); };
        const int64_t total = units_of(all), before = units_of(below + incl - mine);
        mine = units_of(mine);
        head = units_of(head);
        // As many runs as there are CTAs, but not so many that an item has to be
        // cut into runs of less than kLeast units: the streams of a CTA work on two
        // tiles at once, and parts have to be joined.
        int64_t grid = all >> kItemBit;
        const int64_t some = (total + S::kLeast - 1) / S::kLeast;
        if (grid < some) grid = some;
        if (grid > (int64_t)gridDim.x) grid = gridDim.x;
        const int64_t each = grid > 0 ? udiv(total, grid) : 0;
        const int32_t more = (int32_t)(total - each * grid);
        if (tid == 0) {
            plan.total = total;
            plan.each = each;
            plan.more = more;
            plan.grid = (int32_t)grid;
            plan.extra = extra;
        }
        if ((int64_t)blockIdx.x < grid) {
            const int64_t u0 = run_start(blockIdx.x, each, more, (int32_t)grid);
            if (u0 >= before && u0 < before + mine && (!by_warp || lane == 0)) {
                int64_t at = before;
                int l = l0;
                if (l1 - l0 > 1)
                    for (;; ++l) {
                        const Lane ln = lane_of(a, l);
                        head = head_units<S>(a, ln) + extra * row_tiles<S>(a, ln.n);
                        if (u0 < at + head * a.heads_kv) break;
                        at += head * a.heads_kv;
                    }
                plan.lane = l;
                plan.lane_u = at;
                plan.per_head = head;
            }
        }
        __syncthreads();
    }
    const uint32_t tmem = tmem_slot;

    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *q_smem = smem, *kv_smem = smem + S::QB * QT * S::kQBytes;
    float *swap = reinterpret_cast<float *>(kv_smem + S::kStages * S::kStageBytes);

    if (warp == kLoader) {
        // ---- the items of this CTA's run, and their K and V tiles: a lane of
        // the warp per page, in the order K0 V0 K1 V1 ...
        Run run;
        run.u = run.end = 0;
        if ((int64_t)blockIdx.x < plan.grid) {
            run.u = run_start(blockIdx.x, plan.each, plan.more, plan.grid);
            run.end = run_start(blockIdx.x + 1, plan.each, plan.more, plan.grid);
            run.extra = plan.extra;
            run.lane = plan.lane;
            run.ln = lane_of(a, run.lane);
            run.rts = row_tiles<S>(a, run.ln.n);
            const int64_t off = run.u - plan.lane_u;
            run.head = (int)udiv(off, plan.per_head);
            run.item0 = plan.lane_u + run.head * plan.per_head;
            // the row tile: 32 at a time
            run.rt = 0;
            for (; run.rts > 1; run.rt += 32) {
                const int rt = run.rt + lane;
                int all;
                const int tiles = rt < run.rts ? reach_of<S>(a, run.ln.n, run.ln.seq, rt).tiles + run.extra : 0;
                const int before = warp_exclusive_sum(tiles, lane, all);
                if (run.u < run.item0 + all) {
                    const uint32_t past = __ballot_sync(kFull, run.u < run.item0 + before + tiles);
                    const int k = __ffs(past) - 1;
                    run.rt += k;
                    run.item0 += __shfl_sync(kFull, before, k);
                    break;
                }
                run.item0 += all;
            }
        }
        const int rows = min(1 << a.log_page, S::BK);            // rows of a box
        const int boxes = S::BK / rows;
        const bool whole = rows == S::BK;                        // one box brings all blocks
        const uint32_t box_bytes = (uint32_t)rows * D * 2;
        auto page_of = [&](const Segment &s, int t) -> int {     // of this lane's box of tile t
            const int64_t k0 = (int64_t)(s.tile + t) * S::BK + lane * rows, pi = k0 >> a.log_page;
            return lane < boxes && k0 < s.r.hi && k0 + rows > s.r.lo && pi < a.max_pages
                       ? __ldg(a.block_table + s.lane * a.max_pages + pi) : -1;
        };
        uint32_t idx = 0;                                        // stage uses so far
        bool ok = true;
        if (lane < 2) joins[lane].n = joins[lane].count = joins[lane].lg = came_last[lane] = 0;
        __syncwarp();
        for (uint32_t n = 0; ok; ++n) {
            Segment s;
            const bool more = next_segment<S>(a, run, s);
            int page = more ? page_of(s, 0) : -1;                // on its way while the item is handed out
            ok = __all_sync(kFull, wait(&bar.item_empty[n % kItems], ((n / kItems) & 1) ^ 1));
            if (!ok) break;
            if (lane == 0) {
                Item &it = items[n % kItems];
                it.tiles = 0;
                if (more) {
                    const bool split = s.tiles < s.item_tiles, begins = s.tile == s.r.tile0;
                    it.first = s.ln.first; it.n = s.ln.n; it.seq = s.ln.seq; it.head = s.head; it.rt = s.rt;
                    it.lo = s.r.lo; it.hi = s.r.hi; it.tile = s.tile; it.tiles = s.tiles;
                    it.slot = !split ? -1 : begins ? 1 : 0;
                }
                mbar_arrive(&bar.item_full[n % kItems]);
            }
            __syncwarp();
            if (!more) break;
            for (int t = 0; t < s.tiles && ok; ++t) {
                const int k0 = (s.tile + t) * S::BK + lane * rows;
                const bool mine = lane < boxes && k0 < s.r.hi && k0 + rows > s.r.lo;
                if (t > 0) page = page_of(s, t);
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
            if (lane == 0 && s.tiles < s.item_tiles) {           // (seen with the next item, or with the end)
                const int64_t left = (int64_t)s.ln.n * a.group - (int64_t)s.rt * S::kRows;
                Join &jn = joins[s.tile == s.r.tile0 ? 1 : 0];
                jn.first_cta = run_owner(s.item0, plan.total, plan.grid);
                jn.n = run_owner(s.item0 + s.item_tiles - 1, plan.total, plan.grid) - jn.first_cta + 1;
                jn.rows = (int32_t)(left < S::kRows ? left : S::kRows);
                jn.first = s.ln.first; jn.head = s.head; jn.rt = s.rt;
                const int all = jn.rows * (D / 16), sharers = a.share_joins ? jn.n : 1, mine = a.share_joins ? (int)blockIdx.x - jn.first_cta : 0;
                jn.from = (int32_t)((uint32_t)(all * mine) / (uint32_t)sharers);
                jn.count = (int32_t)((uint32_t)(all * (mine + 1)) / (uint32_t)sharers) - jn.from;
                // The threads of an element order its sums, and so follow from the item
                // alone -- whether this CTA comes last at an item, or at two, is timing -- or, in
                // a shared join, from the two items that the CTA joins at once.
                const bool both = a.share_joins && joins[0].n > 0 && joins[1].n > 0;
                const int work = both ? joins[0].count + joins[1].count : jn.count, most = both ? max(joins[0].n, joins[1].n) : jn.n;
                int lg = 0;
                while (lg < 5 && (4 << lg) <= most && work << (lg + 1) <= S::kSoftmaxWarps * 32) ++lg;
                jn.lg = lg;
                if (both) joins[0].lg = lg;
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
        uint32_t units[2] = {0, 0};                          // units per S buffer
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
        const uint32_t q_desc = operand(smem_u32(q_smem), 16), k_desc = operand(smem_u32(kv_smem), 16),
                       v_desc = operand(smem_u32(kv_smem), S::BK * 128);
        for (uint32_t n = 0; ok; ++n) {
            if (!__all_sync(kFull, wait(&bar.item_full[n % kItems], (n / kItems) & 1))) break;
            const int tiles = items[n % kItems].tiles;
            __syncwarp();
            if (tiles == 0) break;
            if (lane == 0) mbar_arrive(&bar.item_empty[n % kItems]);
            const int U = QT == 2 ? 2 * tiles : tiles;
            const uint32_t qb = n % S::QB;
            auto qk = [&](int i) -> bool {
                const int b = i & 1;
                if ((QT == 1 || b == 0) && !wait(&bar.full[k_stage], k_phase)) return false;
                fence_after();
                if (leader) {
                    const uint32_t qa = q_desc + (qb * QT + (QT == 2 ? b : 0)) * (S::kQBytes >> 4), ka = k_desc + k_stage * (S::kStageBytes >> 4);
                    const uint32_t d = tmem + b * S::BK;
                    mma_ss<false>(d, qa, ka, kQk);
#pragma unroll
                    for (int k = 1; k < D / 16; ++k)
                        mma_ss<true>(d, qa + (k >> 2) * (128 * 128 >> 4) + (k & 3) * 2, ka + (k >> 2) * (S::BK * 128 >> 4) + (k & 3) * 2, kQk);
                    commit(&bar.s_full[b]);
                    if (QT == 1 || b == 1) commit(&bar.empty[k_stage]);
                    if (i == U - 1) commit(&bar.q_empty[qb]);
                }
                __syncwarp();
                if (QT == 1 || b == 1) advance(k_stage, k_phase);
                return true;
            };
            ok = wait(&bar.q_full[qb], (n / S::QB) & 1);
            fence_after();
            ok = ok && qk(0);
            for (int i = 0; i < U && ok; ++i) {
                if (i + 1 < U) ok = qk(i + 1);
                const int b = i & 1, ob = S::NS == 2 ? b : 0;
                if (QT == 1 || b == 0) ok = ok && wait(&bar.full[v_stage], v_phase);
                ok = ok && wait(&bar.p_full[b], units[b] & 1);
                if (!ok) break;
                ++units[b];
                fence_after();
                if (leader) {
                    const uint32_t va = v_desc + v_stage * (S::kStageBytes >> 4), d = tmem + S::kO + ob * D, pa = tmem + b * S::BK;
                    mma_ts(d, pa, va, kPv, S::NS == 2 ? i >= 2 : i >= 1);
#pragma unroll
                    for (int k = 1; k < S::BK / 16; ++k)   // the halves' weights lie half a tile apart
                        mma_ts_acc(d, pa + k / (S::BK / 32) * (S::BK / 2) + k % (S::BK / 32) * 8, va + k * (2048 >> 4), kPv);
                    commit(&bar.o_done[ob]);
                    if (QT == 1 || b == 1) commit(&bar.empty[v_stage]);
                }
                __syncwarp();
                if (QT == 1 || b == 1) advance(v_stage, v_phase);
            }
            ok = __all_sync(kFull, ok);
        }
        // everything issued is complete before TMEM is freed
        if (leader) {
            commit(&bar.drain);
            const uint64_t t0 = global_ns();
            while (!mbar_try_wait(&bar.drain, 0) && global_ns() - t0 < kWaitLimitNs) {}
        }
        __syncwarp();
    } else if (warp >= kQLoader) {
        // ---- Q: 16-byte pieces of the item's rows, consecutive lanes on
        // consecutive pieces, all of them on their way together; rows past the item's
        // keep what is there.  (Through registers, 8 at a time, 256 rows took 4 us.)
        constexpr int kPieces = D / 8, kStep = 64 / kPieces;       // kStep rows a pass
        const int p = (tid - kQLoader * 32) % kPieces, r0 = (tid - kQLoader * 32) / kPieces;
        // kStep rows on: step_t tokens and step_h heads, less a token's heads for one more token
        const int step_t = (int)div_group(a, kStep), step_h = kStep - step_t * a.group;
        const int64_t step = step_t * a.qs_t + step_h * a.qs_h, carry = a.qs_t - a.group * a.qs_h;
        // The last of these warps also tells the other CTAs of this CTA's parts, an item
        // late: a fence waits for the part's writes, 1-2 us in which the softmax warps go on.
        int part = -1;                                             // slot of the last item's part
        auto tell = [&]() -> bool {
            if (part < 0 || warp == kQLoader) return true;
            if (!__all_sync(kFull, wait(&bar.part_full[part], 0))) return false;
            if (lane == 0) {
                __threadfence();
                const Join &j = joins[part];
                const uint32_t before = atom_add_acq_rel(a.counters + j.first_cta, 1u);
                if (!a.share_joins && before == (uint32_t)j.n - 1) {
                    came_last[part] = 1;
                    a.counters[j.first_cta] = 0u;
                }
                mbar_arrive(&bar.part_known[part]);
            }
            __syncwarp();
            return true;
        };
        for (uint32_t n = 0;; ++n) {
            if (!__all_sync(kFull, wait(&bar.item_full[n % kItems], (n / kItems) & 1))) break;
            const Item it = items[n % kItems];
            __syncwarp();
            if (it.tiles == 0) {
                tell();
                break;
            }
            if (lane == 0) mbar_arrive(&bar.item_empty[n % kItems]);
            const uint32_t qb = n % S::QB;
            if (!__all_sync(kFull, wait(&bar.q_empty[qb], ((n / S::QB) & 1) ^ 1))) break;
            const int64_t row0 = (int64_t)it.rt * S::kRows, have = (int64_t)it.n * a.group - row0;
            const int valid = have < S::kRows ? (int)have : S::kRows;
            const uint32_t dst = smem_u32(q_smem) + qb * QT * S::kQBytes + (p >> 3) * (128 * 128);
            const uint32_t gr = (uint32_t)row0 + r0, tok = div_group(a, gr);
            int h = (int)(gr - tok * a.group);
            const uint16_t *src = a.q + (int64_t)(it.first + (int)tok) * a.qs_t + (int64_t)(it.head * a.group + h) * a.qs_h + p * 8;
#pragma unroll 4
            for (int r = r0; r < valid; r += kStep) {
                copy16(dst + (r >> 7) * S::kQBytes + (r & 127) * 128 + (((p & 7) ^ (r & 7)) << 4), src);
                h += step_h;
                src += step;
                if (h >= a.group) {
                    h -= a.group;
                    src += carry;
                }
            }
            copies_landed();
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.q_full[qb]);
            if (!tell()) break;
            part = it.slot;
        }
    } else {
        // ---- softmax, correction and epilogue: stream `st`, columns [half * kW, half * kW + kW) of its tiles
        constexpr int kW = S::BK / 2;
        const int st = warp >> 3, half = (warp >> 2) & 1, quad = warp & 3, row = quad * 32 + lane;   // row of the tile
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        const int pair = 1 + st * 4 + quad;                       // barrier of the two warps with these rows
        uint32_t tile_n = 0, s_n[2] = {0, 0}, pv_n = 0;           // tiles so far, units per S buffer, PVs of this stream
        bool stop = false;                                        // a wait gave up: no parts, no joins
        for (uint32_t n = 0;; ++n) {
            const bool ok = wait(&bar.item_full[n % kItems], (n / kItems) & 1);
            // all softmax warps go on or none does: the barriers below count on it
            stop = named_barrier_any(kAllSoftmax, S::kSoftmaxWarps * 32, !ok);
            if (stop) break;
            const Item &it = items[n % kItems];
            const int tiles = it.tiles;
            if (tiles == 0) break;
            const int lo = it.lo, hi = it.hi, tile0 = it.tile;
            const int64_t gr = (int64_t)it.rt * S::kRows + (QT == 2 ? st * 128 : 0) + row;
            const bool valid = gr < (int64_t)it.n * a.group;
            const int tok = valid ? (int)div_group(a, (uint32_t)gr) : 0;
            const int pos = it.seq - it.n + tok;
            const int64_t klo64 = a.window > 0 ? (int64_t)pos - a.window + 1 : 0;
            const int klo = klo64 > 0 ? (int)klo64 : 0, khi = valid ? pos + 1 : klo;   // keys of this row
            const bool live = __any_sync(kFull, khi > klo);
            // the quads of rows in use, and this thread's place among those who clear V rows
            const int64_t rows_left = (int64_t)it.n * a.group - (int64_t)it.rt * S::kRows - (QT == 2 ? st * 128 : 0);
            const int quads = rows_left >= 97 ? 4 : rows_left <= 0 ? 0 : (int)(rows_left + 31) >> 5, idle = quads < 4 ? quads : 0;
            const bool clears = quad >= idle;
            const int clear_id = ((quad - idle) * 2 + half) * 32 + lane, clear_of = (4 - idle) * 64;

            float m = -INFINITY, l = 0.f;                          // l: of this half's columns
            const int U = QT == 2 || S::NS == 1 ? tiles : (tiles - st + 1) >> 1;
            for (int i = 0; i < U; ++i) {
                const int t = QT == 2 || S::NS == 1 ? i : 2 * i + st;
                const int b = S::NS == 2 ? st : i & 1;
                const int key0 = (tile0 + t) * S::BK;
                if (S::NS == 2 || b == 0) wait(&bar.s_full[b], s_n[0]++ & 1);
                else wait(&bar.s_full[1], s_n[1]++ & 1);
                fence_after();
                if (live) {
                    const uint32_t sa = tmem + lane_base + b * S::BK + half * kW;
                    // columns of this row in the half tile; what a row past the item's holds is nobody's
                    const int from = valid ? klo - key0 - half * kW : 0, to = valid ? khi - key0 - half * kW : kW;
                    const bool edge = __any_sync(kFull, from > 0 || to < kW);
                    // two passes over S in TMEM (other warps hide the loads; the
                    // half row in registers would not fit), rolled: the kernel's
                    // code is read from L2 once a launch, and its size counts
                    float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int c = 0; c < kW; c += 32) {
                        uint32_t x[32];
                        tmem_ld32(x, sa + c);
                        if (edge) mask_scores(x, from - c, to - c);
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                top4[k] = max3(top4[k], __uint_as_float(x[e + k]), __uint_as_float(x[e + 4 + k]));
                    }
                    float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])) * a.c;
                    // the other half's maximum; a row's two threads decide alike.  (One
                    // stream: a slot per S buffer, since S of the next unit may be there
                    // before the other half has read this one's.)
                    float *mx = swap + (S::NS == 2 ? st : b) * 256 + row;
                    mx[half * 128] = top;
                    named_barrier(pair, 64);
                    top = fmaxf(top, mx[(half ^ 1) * 128]);
                    // a new reference only past the lag (or for a row's first key)
                    const bool move = valid && (top > m + (kLag<F16> + kRaise<F16>) || (m == -INFINITY && top > -INFINITY));
                    if (__any_sync(kFull, move)) {
                        const float to = top - kRaise<F16>, f = move ? exp2_fast(m - to) : 1.f;
                        if (move) m = to;
                        l *= f;
                        if (i > 0) {
                            wait(&bar.o_done[st], (pv_n - 1) & 1);
                            fence_after();
                            const uint32_t oa = tmem + lane_base + S::kO + st * D + half * (D / 2);
#pragma unroll 1
                            for (int c = 0; c < D / 2; c += 32) {
                                uint32_t o[32];
                                tmem_ld32(o, oa + c);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tmem_st32(oa + c, o);
                            }
                        }
                    }
                    const float ref = m == -INFINITY ? 0.f : m;
                    const uint64_t cc = two(a.c, a.c), mm = two(-ref, -ref);
                    uint64_t sum[2] = {0ull, 0ull};
#pragma unroll 1
                    for (int c = 0; c < kW; c += 32) {
                        // P of columns c .. c+31 covers columns c/2 .. c/2+15 of this half's S, read before
                        uint32_t x[32], pk[16];
                        tmem_ld32(x, sa + c);
                        if (edge) mask_scores(x, from - c, to - c);
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
                    }
                    float s0, s1;
                    halves(add2(sum[0], sum[1]), s0, s1);
                    l += s0 + s1;
                }
                // V rows that no row of the item may see hold anything, NaN
                // included: 0 * NaN must not reach O.  Warps without rows clear
                // them while the others compute, or all do.
                if ((key0 < lo || key0 + S::BK > hi) && clears) {
                    const uint32_t idx = 2 * (tile_n + t) + 1, vs = idx % S::kStages;
                    wait(&bar.full[vs], (idx / S::kStages) & 1);
                    uint8_t *v = kv_smem + vs * S::kStageBytes;
                    const int below = lo > key0 ? min(lo - key0, S::BK) : 0, above = hi < key0 + S::BK ? max(hi - key0, below) : S::BK;
                    const int gone = below + S::BK - above;         // rows [0, below) and [above, BK)
                    for (int k = clear_id; k < gone * (D / 8); k += clear_of) {
                        const int g = k / (D / 8), p = k % (D / 8), kr = g < below ? g : g - below + above;
                        *reinterpret_cast<uint4 *>(v + (p >> 3) * (S::BK * 128) + kr * 128 + (p & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async();
                }
                // One stream over two S buffers: S of this unit says nothing about the
                // product before it, and a barrier's parity tells only its last two phases
                // apart, so that every phase is waited for.  (With two streams, S of a
                // stream's unit comes after its last product.)
                if (S::NS == 1 && i > 0) wait(&bar.o_done[st], (pv_n - 1) & 1);
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_full[b]);
                ++pv_n;
            }
            tile_n += tiles;
            if (U > 0) wait(&bar.o_done[st], (pv_n - 1) & 1);
            fence_after();

            // the row's sum over the halves (and the streams), and the columns this thread writes
            float f0 = 1.f, f1 = 0.f;                              // weights of the streams' O
            int c0 = half * (D / 2);
            constexpr bool kStreams = QT == 1 && S::NS == 2;
            const bool streams = kStreams && tiles > 1;            // (an item of one tile has the first stream's only)
            const int cols = streams ? D / 4 : kStreams && st == 1 ? 0 : D / 2;
            if (streams) {
                swap[st * 256 + half * 128 + row] = l;
                fence_before();
                named_barrier(kAllSoftmax, S::kSoftmaxWarps * 32);
                fence_after();
                const float l0 = swap[row] + swap[128 + row], l1 = swap[256 + row] + swap[384 + row];
                named_barrier(kAllSoftmax, S::kSoftmaxWarps * 32);
                if (half == 0) swap[st * 128 + row] = m;
                named_barrier(kAllSoftmax, S::kSoftmaxWarps * 32);
                const float m0 = swap[row], m1 = swap[128 + row];
                m = fmaxf(m0, m1);
                f0 = m0 == -INFINITY ? 0.f : exp2_fast(m0 - m);
                f1 = m1 == -INFINITY ? 0.f : exp2_fast(m1 - m);
                l = l0 * f0 + l1 * f1;
                c0 = (st * 2 + half) * (D / 4);
            } else if (live) {
                float *mx = swap + st * 256 + row;
                mx[half * 128] = l;
                named_barrier(pair, 64);
                l += mx[(half ^ 1) * 128];
            }

            // where the rows go: the output, or this CTA's part of the item
            const int slot = it.slot;
            const bool split = slot >= 0;
            float *part = a.parts + ((int64_t)blockIdx.x * 2 + slot) * S::kPartFloats + (QT == 2 ? st * 128 * (D + 2) : 0);
            const float inv = split ? 1.f : l == 0.f ? 0.f : 1.f / l;   // (NaN scores: NaN)
            const int h = it.head * a.group + (int)(valid ? gr - (int64_t)tok * a.group : 0);
            const int64_t out_row = ((int64_t)it.first + tok) * a.heads_q + h;
            if (live) {
                const uint32_t oa = tmem + lane_base + S::kO + (QT == 2 ? st * D : 0);
#pragma unroll 1
                for (int c = c0; c < c0 + cols; c += 16) {
                    uint32_t o[16];
                    tmem_ld16(o, oa + c);
                    if (streams) {
                        uint32_t o1[16];
                        tmem_ld16(o1, oa + D + c);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float v0 = f0 > 0.f ? __uint_as_float(o[e]) * f0 : 0.f;
                            const float v1 = f1 > 0.f ? __uint_as_float(o1[e]) * f1 : 0.f;
                            o[e] = __float_as_uint(v0 + v1);
                        }
                    }
                    if (l == 0.f) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = 0u;
                    }
                    if (!valid) continue;
                    if (split) {
                        float4 *dst = reinterpret_cast<float4 *>(part) + (c / 4) * 128 + row;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            dst[e * 128] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                       __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
                    } else {
                        uint4 *dst = reinterpret_cast<uint4 *>(a.out + out_row * D + c);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            uint32_t w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                w[k] = pack2<F16>(__uint_as_float(o[8 * e + 2 * k]) * inv, __uint_as_float(o[8 * e + 2 * k + 1]) * inv);
                            dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
            } else if (valid) {                                    // a warp of rows without keys
                for (int c = c0; c < c0 + cols; c += 8)
                    if (!split) *reinterpret_cast<uint4 *>(a.out + out_row * D + c) = make_uint4(0, 0, 0, 0);
                    else
                        for (int e = 0; e < 2; ++e)                // (what was there, a NaN perhaps, times 0 is not 0)
                            *(reinterpret_cast<float4 *>(part) + (c / 4 + e) * 128 + row) = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            if (valid && c0 == 0 && cols > 0) {
                if (split) {
                    float *ml = part + 128 * D;
                    ml[row] = live ? m : -INFINITY;
                    ml[128 + row] = live ? l : 0.f;
                } else if (a.lse) {
                    a.lse[out_row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) {
                if (split) mbar_arrive(&bar.part_full[slot]);
                mbar_arrive(&bar.item_empty[n % kItems]);
            }
            // (O, the swap area and the pair barriers are used again only past the
            // barrier at the next item's start)
        }

        // ---- the items in parts: wait for the others' and join this CTA's share.
        // A thread takes sixteen columns of a row (four cost a chunk of 2,048 at 0 keys 5 us
        // more: the maxima and scales of a part are worked out for every element); where
        // there are threads to spare, up to 32 of them share an element's parts, each with
        // its own running maximum, and their sums are added up in pairs.
        constexpr int kT = S::kSoftmaxWarps * 32;
        bool failed = false;
        if (!stop && a.share_joins && lane == 0 && warp < 2 && joins[warp].n > 0) {   // a warp waits for each of the two items
            const Join &j = joins[warp];
            const uint64_t t0 = global_ns();
            while (ld_acquire(a.counters + j.first_cta) < (unsigned)j.n) {
                failed = *reinterpret_cast<volatile unsigned int *>(&s_gave_up) != 0u;
                if (failed) break;
                if (global_ns() - t0 > kWaitLimitNs) {
                    s_gave_up = 1u;
                    atomicOr(&g_wait_timeouts, 1u);
                }
            }
            __threadfence();
            // the last joiner leaves the counters at zero for the next call
            if (atom_add_acq_rel(a.counters + kMaxSms + j.first_cta, 1u) == (unsigned)j.n - 1) {
                a.counters[j.first_cta] = 0u;
                a.counters[kMaxSms + j.first_cta] = 0u;
            }
        }
        if (!stop && !a.share_joins && lane == 0 && warp < 2 && joins[warp].n > 0) failed = !wait(&bar.part_known[warp], 0);
        if (!stop && joins[0].n + joins[1].n > 0) stop = named_barrier_any(kAllSoftmax, kT, failed);
        // this CTA's elements of both items; a warp's threads are all at one item
        const int count0 = !stop && (a.share_joins || came_last[0]) ? joins[0].count : 0;
        const int count1 = !stop && (a.share_joins || came_last[1]) ? joins[1].count : 0;
        const int second = ((count0 << joins[0].lg) + 31) & ~31, work = second + (count1 << joins[1].lg);
        for (int base = 0; base < work; base += kT) {
            const int at = base + tid, sl = at < second ? 0 : 1;
            const Join &j = joins[sl];
            const int step = 1 << j.lg, p0 = tid & (step - 1), k = (sl ? at - second : at) >> j.lg;
            const bool mine = k < (sl ? count1 : count0);
            const int e = j.from + k, n = mine ? j.n : 0;
            const int g = mine ? (int)((uint32_t)e / (uint32_t)j.rows) : 0, r = mine ? e - g * j.rows : 0;   // columns 16 g on; over the item's row tiles
            // the first part; the others are one slot on, then every second
            const float *first_part = a.parts + ((int64_t)j.first_cta * 2 + 1) * S::kPartFloats + (r >> 7) * 128 * (D + 2);
            float M = -INFINITY, L = 0.f, o[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = 0.f;
            auto scales = [&](float mp, float lp, float &fo, float &fp) {
                const float Mn = fmaxf(M, mp), ref = Mn == -INFINITY ? 0.f : Mn;
                fo = exp2_fast(M - ref);
                fp = exp2_fast(mp - ref);
                M = Mn;
                L = L * fo + lp * fp;
            };
#pragma unroll 2
            for (int p = p0; p < n; p += step) {
                const float *q = p == 0 ? first_part : first_part + (int64_t)(2 * p - 1) * S::kPartFloats;
                const float mp = q[128 * D + (r & 127)], lp = q[128 * D + 128 + (r & 127)];
                float4 x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = __ldcg(reinterpret_cast<const float4 *>(q) + (4 * g + i) * 128 + (r & 127));
                float fo, fp;
                scales(mp, lp, fo, fp);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    o[4 * i] = o[4 * i] * fo + x[i].x * fp;
                    o[4 * i + 1] = o[4 * i + 1] * fo + x[i].y * fp;
                    o[4 * i + 2] = o[4 * i + 2] * fo + x[i].z * fp;
                    o[4 * i + 3] = o[4 * i + 3] * fo + x[i].w * fp;
                }
            }
#pragma unroll 1
            for (int d = 1; d < step; d <<= 1) {                   // (an element's threads are neighbours in a warp; the first's result counts)
                float fo, fp;
                scales(__shfl_xor_sync(kFull, M, d), __shfl_xor_sync(kFull, L, d), fo, fp);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = o[i] * fo + __shfl_xor_sync(kFull, o[i], d) * fp;
            }
            if (n == 0 || p0 != 0) continue;
            const uint32_t gr = (uint32_t)j.rt * S::kRows + r, tok = div_group(a, gr);
            const int64_t orow = ((int64_t)j.first + tok) * a.heads_q + (int64_t)j.head * a.group + (gr - tok * a.group);
            const float iv = L == 0.f ? 0.f : 1.f / L;
            uint4 *dst = reinterpret_cast<uint4 *>(a.out + orow * D + g * 16);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                dst[i] = make_uint4(pack2<F16>(o[8 * i] * iv, o[8 * i + 1] * iv), pack2<F16>(o[8 * i + 2] * iv, o[8 * i + 3] * iv),
                                    pack2<F16>(o[8 * i + 4] * iv, o[8 * i + 5] * iv), pack2<F16>(o[8 * i + 6] * iv, o[8 * i + 7] * iv));
            if (g == 0 && a.lse) a.lse[orow] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
        }
    }
    __syncthreads();
    if (warp == kMma) {
        fence_after();
        tmem_free(tmem);
    }
}

}  // namespace attn
