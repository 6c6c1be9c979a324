// Few rows over an 8-bit cache of heads of 128: at most 16 rows an item.  Included by attention.cuh,
// inside its namespace.
//
// Codes widened and scaled in 16 bits, as the other 8-bit variants have them, take 4.5
// instructions a pair of codes, two thirds of them of the ALU pipe, and made a token's step slower than over the
// 16-bit cache (64 tokens of 4 rows a head at 500-16,000 keys 369 us against 320).  Here the products are
// transposed, S^T = K Q^T and O^T += V^T P^T: a softmax thread has one key, so that the key's scale is one
// factor of all its scores, and its value's scale one of all its weights.  Codes then go to fp16 as they
// are, one instruction a pair, and a thread's 16 columns (rows of q) are read from TMEM once for both passes over
// them.  275 us, 3.9 TB/s.  What bounds it: chains, none of them full.  A pair of tiles takes 1.27 us; the loader's
// copies are issued in 0.6 (eight, for pages of 64), the issuing warp works for 0.75, a converting team for 0.65, a stream's
// softmax for 1.5 every second pair.  640 threads leave 96 registers each, and 36 to 48 bytes of a thread's are kept in
// local memory (of its counters and places; with more of them there the same loop took 279 to 293 us).  With 32 rows (two
// columns' groups) or 64 a thread's sums went there: 440 and 496 us.  Scores two tiles ahead of the weights' products
// instead of one: 2 % slower.  More converting warps take its registers: 16 373 us, three
// teams of four 341.  Codes brought to L2 two tiles ahead cost the loader what they save.
//
// All products are fp16's.  A bf16 row of q is taken times a power of two that brings its largest element to
// 2^14 (its eight bits fit; what lies below 2^-38 of the largest is lost, far below what the
// sums lose).  With t the score in log2 units and v that of the value's scale, the running maximum is of t + v, a weight
// 2^(t + v - m) is what multiplies the code, and the sum is of weight * 2^-v, that is of
// 2^(t - m), unrounded.  v runs from -127 (the store gives -120 to a vector of zeros) to 7, so keys of equal scores lie up to 2^134
// apart: a weight below 2^-126 would be 0 and its key gone from the sum.  So keys with v below kTiny have weights 2^kLift
// above in the sum (what is lost then has t - m below -63, and of other keys below -86; the largest weight's is 0 or
// more; lifted, an exponent is rounded as a number near 64 is).  The sum is kept times 2^-kDown, and where references move or
// meet it is multiplied by 2^x in two factors, as x may be below -126.  (2^-kDown over a sum may be, too: O^T is
// multiplied by each.)
// Weights are fp16 as elsewhere: against a reference 2^7 below the maximum, lag 2^4.

constexpr int kDown = 48, kLift = 64, kTiny = -40;
constexpr float kUp = 0x1p-48f, kUnlift = 0x1p-64f;   // what takes out kDown, kLift

// 2^x as a product of two factors, neither subnormal for x from -190 on (the first is all of it from -64 on).
__device__ __forceinline__ float2 exp2_pair(float x)
{
    const float a = fmaxf(x, -64.f);
    return make_float2(exp2_fast(a), exp2_fast(x - a));
}

// m + log2(sum * 2^kDown), exponent and fraction apart: the logarithm of a sum near 2^-kDown would be rounded
// as a number near kDown is.
__device__ __forceinline__ float log2_up(float m, float sum)
{
    const uint32_t b = __float_as_uint(sum);
    if ((b & 0x7F800000u) == 0x7F800000u) return sum;         // (no number)
    return (m + (float)((int)(b >> 23) - 127 + kDown)) + log2f(__uint_as_float((b & 0x007FFFFFu) | 0x3F800000u));
}

// What the softmax threads, the converting warps and the Q loaders exchange.
struct Few {
    float factors[kPairs][2][128];      // of a pair of tiles' keys: of the score; what the sums have of the value's
    float row_factor[kItems][16];       // log2 units of a score of the row's, but for its key's factor
    float ref[2][16];                   // a stream's references
    float2 moved[2][16];                // what its sums are to be multiplied by: the root, and the whole (O^T)
    float top[2][4][16];                // maxima of 32 keys
    float sum[2][4][16];                // sums over 32 keys
    float w0[16], w1[16], inv[16];      // weights of the streams' O^T, and 1 over the sum
    int32_t klo[16], khi[16], token[16];   // keys of a row; its token's row of masks
    int64_t out_row[16];
};

// Four codes to four fp16 values, without a scale.
__device__ __forceinline__ uint2 bare4(uint32_t w)
{
    uint2 r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(r.x), "=r"(r.y) : "r"(w));
    return r;
}

// The factor of a key's scores.
template <bool F16>
__device__ __forceinline__ float key_factor(uint32_t byte)
{
    const uint32_t bits = F16 ? (byte < 113u ? 113u : byte) << 23 : byte > 0u ? byte << 23 : 0x00400000u;   // (2^-127 is subnormal)
    return byte > 134u ? __uint_as_float(0x7FC00000u) : __uint_as_float(bits);
}
// Of a value's scale what takes it (and the lift) out of a weight, times 2^-kDown, and its log2: the upper halves of two floats.
// The log2 of a scale of no number is none: the scores of the rows that see the key are then no numbers (the others' are
// masked), and with them their outputs.
template <bool F16>
__device__ __forceinline__ float value_factors(uint32_t byte)
{
    const uint32_t b = F16 && byte < 113u ? 113u : byte > 134u ? 127u : byte;
    const float log2v = byte > 134u ? __uint_as_float(0x7FC00000u) : (float)((int)b - 127);
    return __uint_as_float((254u - kDown - b - ((int)b < 127 + kTiny ? kLift : 0)) << 23 | __float_as_uint(log2v) >> 16);
}

// The converting warps: a team of four the K tiles, another the V tiles, a thread 16 codes of a row at a time (as
// convert_tiles, whose comments hold here too).  Stages and barriers of slots are even in number, so that a
// team meets every use of its own.
template <typename S, bool F16>
__device__ __forceinline__ void convert_bare(Bars<S> &bar, const Item *items, const uint8_t *raw_smem, uint8_t *kv_smem, Few &few,
                                             int rows, int warp, int lane)
{
    constexpr int kPieces = S::D / 16, kStep = 128 / kPieces, kPasses = S::BK / kStep;
    static_assert(kStep % 8 == 0 && S::BK == 128 && S::kConverters == 8, "");
    // A key's factors are written over those of the key kPairs tiles before, which the softmax of that tile must have read
    // (its weights were waited for).  A team writes those of tile n once it has converted tile n - 1, that is, once the
    // product of tile n - 1 - kStages / 2 has read that tile's stage: the weights' product for V; for K the scores',
    // which are issued once the weights of the tile kAhead + 1 before theirs were waited for.
    static_assert(S::kStages % 2 == 0 && kPairs >= S::kStages / 2 + 2 + S::kAhead, "factors that are still read");
    const int team = warp >> 2, id = (warp & 3) * 32 + lane, p = id % kPieces, r0 = id / kPieces;
    const int block = p >> 2, piece = (p & 3) * 2, flip = block & 1;
    const uint32_t x0 = ((piece + flip) ^ (r0 & 7)) << 4, x1 = x0 ^ 16;
    uint8_t *const to = kv_smem + block * (S::BK * 128) + r0 * 128;
    const int log_rows = 31 - __clz(rows), scale_at = S::kRawCodes + (id >> log_rows) * 128 + (id & (rows - 1));   // of key id
    uint32_t rb = team, rb_phase = 0, st = team, st_phase = 0, pair = 0;   // barrier of the tile's slot, its stage, its factors
    for (uint32_t n = 0;; ++n) {
        if (!__all_sync(kFull, wait(&bar.item_full[n % kItems], (n / kItems) & 1))) return;
        const int tiles = items[n % kItems].tiles;
        __syncwarp();
        if (tiles == 0) return;
        if (lane == 0) mbar_arrive(&bar.item_empty[n % kItems]);
        for (int t = 0; t < tiles; ++t) {
            const uint32_t rs = rb < (uint32_t)S::kRaw ? rb : rb - S::kRaw;
            if (!__all_sync(kFull, wait(&bar.raw_full[rb], rb_phase))) return;
            const uint8_t *raw = raw_smem + rs * S::kRawBytes;
            uint4 w[kPasses];
#pragma unroll
            for (int i = 0; i < kPasses; ++i) w[i] = *reinterpret_cast<const uint4 *>(raw + id * 16 + i * (kStep * S::D));
            const uint32_t byte = raw[scale_at];
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.raw_empty[rs]);
            // the factors are there before the tile is: the softmax need not wait for a stage
            few.factors[pair][team][id] = team ? value_factors<F16>(byte) : key_factor<F16>(byte);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.scaled[pair]);
            pair = pair + 1 < kPairs ? pair + 1 : 0;
            if (!__all_sync(kFull, wait(&bar.empty[st], st_phase ^ 1))) return;
            uint8_t *tile = to + st * S::kStageBytes;
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const uint2 b0 = bare4(w[i].x), b1 = bare4(w[i].y), b2 = bare4(w[i].z), b3 = bare4(w[i].w);
                const uint4 u = make_uint4(b0.x, b0.y, b1.x, b1.y), v = make_uint4(b2.x, b2.y, b3.x, b3.y);
                *reinterpret_cast<uint4 *>(tile + i * (kStep * 128) + x0) = flip ? v : u;
                *reinterpret_cast<uint4 *>(tile + i * (kStep * 128) + x1) = flip ? u : v;
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.full[st]);
            rb += 2;
            if (rb >= 2u * S::kRaw) {
                rb -= 2 * S::kRaw;
                rb_phase ^= 1;
            }
            st += 2;
            if (st >= (uint32_t)S::kStages) {
                st -= S::kStages;
                st_phase ^= 1;
            }
        }
    }
}

// An item's rows of q, which the lanes copied: bf16 to fp16 in place, each with its factor.  A
// row's pieces are with kPieces neighbouring lanes, each with what it copied itself.
template <bool F16, int kPieces, int kStep, int kRows>
__device__ __forceinline__ void scale_rows(uint8_t *q, float *factor, float c, int valid, int r0, int p)
{
    const int columns = (valid + 15) & ~15;
    for (int r = r0; r - r0 < columns; r += kStep) {     // (a warp's lanes go on together)
        int up = 0;
        if (!F16) {
            uint4 *at = reinterpret_cast<uint4 *>(q + (p >> 3) * (kRows * 128) + r * 128 + (((p & 7) ^ (r & 7)) << 4));
            uint4 x = make_uint4(0, 0, 0, 0);
            if (r < valid) x = *at;
            uint32_t most = 0u;
#pragma unroll
            for (uint32_t w : {x.x, x.y, x.z, x.w}) most = max(most, max(w & 0x7FFFu, w >> 16 & 0x7FFFu));
#pragma unroll
            for (int d = 1; d < kPieces; d <<= 1) most = max(most, __shfl_xor_sync(kFull, most, d));
            const int e = (int)(most >> 7);              // the largest's exponent + 127
            up = e == 255 ? 0 : min(141 - e, 126);       // (no numbers: as they are)
            const float f = __uint_as_float((uint32_t)(127 + up) << 23);
            auto two16 = [&](uint32_t w) { return pack2<true>(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f); };
            if (r < valid) *at = make_uint4(two16(x.x), two16(x.y), two16(x.z), two16(x.w));
        }
        if (p == 0 && r < columns) factor[r] = r < valid ? c * __uint_as_float((uint32_t)(127 - up) << 23) : 0.f;
    }
}

// Softmax, correction and epilogue of the softmax warps, four a stream: a thread a key of its tiles.  Returns
// whether a wait gave up.
template <typename S, bool F16>
__device__ __forceinline__ bool few_rows(const Args &a, Bars<S> &bar, const Item *items, Few &few, uint8_t *p_smem, uint8_t *kv_smem,
                                         uint32_t tmem, int warp, int lane)
{
    constexpr int kAll = S::kSoftmaxWarps * 32;
    constexpr float kPast = kLag<true> + kRaise<true>;
    const int st = warp >> 2, quad = warp & 3, key = quad * 32 + lane, tid = warp * 32 + lane, stream_barrier = 1 + st;
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    uint8_t *const weights = p_smem + key * 128;              // 16 columns of either stream
    uint32_t tile_n = 0, unit = 0;                            // tiles so far, those of this stream
    for (uint32_t n = 0;; ++n) {
        const bool ok = wait(&bar.item_full[n % kItems], (n / kItems) & 1);
        // all softmax warps go on or none does: the barriers below count on it
        if (named_barrier_any(kAllSoftmax, kAll, !ok)) return true;
        const Item &it = items[n % kItems];
        const int tiles = it.tiles;
        if (tiles == 0) return false;
        const int tile0 = it.tile, ctx = it.seq - it.n;
        const int64_t row0 = (int64_t)it.rt * S::kRows, left = (int64_t)it.n * a.group - row0;
        const int rows = left < S::kRows ? (int)left : S::kRows;
        if (tid < S::kRows) {
            const bool valid = tid < rows;
            const uint32_t gr = (uint32_t)row0 + (valid ? tid : 0), tok = div_group(a, gr);
            const uint32_t *mask = S::kTree ? a.masks + (int64_t)(it.first + (int)tok) * a.mask_words : nullptr;
            const int64_t klo = a.window > 0 ? (int64_t)ctx + (S::kTree ? node_depth(mask, a.mask_words, (int)tok) : (int)tok) - a.window + 1 : 0;
            few.klo[tid] = klo > 0 ? (int)klo : 0;
            few.khi[tid] = valid ? ctx + (int)tok + 1 : -1;
            few.token[tid] = it.first + (int)tok;
            few.out_row[tid] = ((int64_t)it.first + tok) * a.heads_q + (int64_t)it.head * a.group + (gr - tok * a.group);
        }
        if (tid < 32) few.ref[tid >> 4][tid & 15] = -INFINITY;
        named_barrier(kAllSoftmax, kAll);
        // no tile within these has a key that some row does not see
        const int tok0 = (int)div_group(a, (uint32_t)row0), tok1 = (int)div_group(a, (uint32_t)row0 + rows - 1);
        const int64_t last = a.window > 0 ? (int64_t)ctx + tok1 - a.window + 1 : 0;
        const int last_lo = last > 0 ? (int)last : 0;
        const int first_hi = S::kTree ? ctx : ctx + tok0 + 1;

        uint64_t l[8];                                         // two columns' sums each
#pragma unroll
        for (int e = 0; e < 8; ++e) l[e] = 0ull;
        const int U = (tiles - st + 1) >> 1;
        for (int i = 0; i < U; ++i) {
            const int t = 2 * i + st, key0 = (tile0 + t) * S::BK, at = key0 + key;
            const uint32_t pair = tile_n + t;
            wait(&bar.scaled[pair % kPairs], (pair / kPairs) & 1);
            const float *f = few.factors[pair % kPairs][0] + key;
            const float ks = f[0];
            const uint32_t vf = __float_as_uint(f[128]);
            const float v = __uint_as_float(vf << 16), over = __uint_as_float(vf & 0xFFFF0000u);
            const bool tiny = !F16 && v < kTiny;                      // (fp16's are -14 or more)
            const float lift = tiny ? (float)kLift : 0.f, unlift = tiny ? kUnlift : 1.f;
            wait(&bar.s_full[st], unit & 1);
            // the weights of the last tile are read, and its product may be multiplied
            if (i > 0) wait(&bar.o_done[st], (unit - 1) & 1);
            fence_after();
            const bool edge = key0 < last_lo || key0 + S::BK > first_hi;
            {
                uint32_t x[16];
                float u[16];
                tmem_ld16(x, tmem + lane_base + st * S::kRows);
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float4 c = *reinterpret_cast<const float4 *>(&few.row_factor[n % kItems][e]);
                    u[e] = fmaf(__uint_as_float(x[e]) * ks, c.x, v);
                    u[e + 1] = fmaf(__uint_as_float(x[e + 1]) * ks, c.y, v);
                    u[e + 2] = fmaf(__uint_as_float(x[e + 2]) * ks, c.z, v);
                    u[e + 3] = fmaf(__uint_as_float(x[e + 3]) * ks, c.w, v);
                }
                if (edge) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        bool sees = at >= few.klo[e] && at < few.khi[e];
                        if (S::kTree && sees && at >= ctx) {
                            const int node = at - ctx;
                            sees = (node >> 5) < a.mask_words &&
                                   (__ldg(a.masks + (int64_t)few.token[e] * a.mask_words + (node >> 5)) >> (node & 31) & 1u);
                        }
                        if (!sees) u[e] = -INFINITY;
                    }
                }
                bool past = false;
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float4 m = *reinterpret_cast<const float4 *>(&few.ref[st][e]);
                    past = past || u[e] > m.x + kPast || u[e + 1] > m.y + kPast || u[e + 2] > m.z + kPast || u[e + 3] > m.w + kPast;
                }
                if (named_barrier_any(stream_barrier, 128, past)) {
                    // new references, for the columns that are past the lag (or have their first key)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float top;
                        asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(top) : "f"(u[e]));
                        if (lane == 0) few.top[st][quad][e] = top;
                    }
                    named_barrier(stream_barrier, 128);
                    if (quad == 0 && lane < 16) {
                        const float top = fmaxf(fmaxf(few.top[st][0][lane], few.top[st][1][lane]), fmaxf(few.top[st][2][lane], few.top[st][3][lane]));
                        const float m = few.ref[st][lane], to = top - kRaise<true>;
                        const bool move = top > m + kPast;     // (m = -inf: any key's)
                        const float f = move ? exp2_fast(0.5f * (m - to)) : 1.f;
                        few.moved[st][lane] = make_float2(f, f * f);
                        if (move) few.ref[st][lane] = to;
                    }
                    named_barrier(stream_barrier, 128);
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float4 f = *reinterpret_cast<const float4 *>(&few.moved[st][e]);
                        const uint64_t f2 = two(f.x, f.z);
                        l[e / 2] = mul2(mul2(l[e / 2], f2), f2);
                    }
                    if (i > 0) {
                        const uint32_t oa = tmem + lane_base + S::kO + st * S::kRows;
                        uint32_t o[16];
                        tmem_ld16(o, oa);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * few.moved[st][e].y);
                        }
                        tmem_st16(oa, o);
                    }
                }
                uint32_t pk[8];
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float2 m = *reinterpret_cast<const float2 *>(&few.ref[st][e]);
                    float p0 = exp2_fast(u[e] - (m.x == -INFINITY ? 0.f : m.x) + lift),
                          p1 = exp2_fast(u[e + 1] - (m.y == -INFINITY ? 0.f : m.y) + lift);
                    const uint64_t p = two(p0, p1);
                    l[e / 2] = fma2(p, two(over, over), l[e / 2]);
                    halves(mul2(p, two(unlift, unlift)), p0, p1);
                    pk[e / 2] = pack2<true>(p0, p1);
                }
                *reinterpret_cast<uint4 *>(weights + ((2 * st ^ (key & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                *reinterpret_cast<uint4 *>(weights + ((2 * st + 1 ^ (key & 7)) << 4)) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
            }
            // V rows that no row of the item may see hold anything, NaN included: 0 * NaN must not reach O
            if (edge && (key0 < it.lo || key0 + S::BK > it.hi)) {
                const uint32_t idx = 2 * pair + 1, vs = idx % S::kStages;
                wait(&bar.full[vs], (idx / S::kStages) & 1);
                if (at < it.lo || at >= it.hi) {
                    uint8_t *row = kv_smem + vs * S::kStageBytes + key * 128;
#pragma unroll
                    for (int k = 0; k < 2 * 8; ++k) *reinterpret_cast<uint4 *>(row + (k >> 3) * (S::BK * 128) + (k & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
            }
            fence_proxy_async();
            wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.p_full[st]);
            ++unit;
        }
        tile_n += tiles;
        if (U > 0) wait(&bar.o_done[st], (unit - 1) & 1);

        // the columns' sums over the keys and the streams
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            float a0, a1;
            halves(l[e / 2], a0, a1);
            a0 = warp_sum_f(a0);
            a1 = warp_sum_f(a1);
            if (lane == 0) *reinterpret_cast<float2 *>(&few.sum[st][quad][e]) = make_float2(a0, a1);
        }
        fence_before();
        named_barrier(kAllSoftmax, kAll);
        fence_after();
        const int slot = it.slot;
        const bool split = slot >= 0;
        float *part = a.parts + ((int64_t)blockIdx.x * 2 + slot) * S::kPartFloats;
        if (tid < S::kRows) {
            const float m0 = few.ref[0][tid], m1 = few.ref[1][tid], m = fmaxf(m0, m1);
            const float2 f0 = m0 == -INFINITY ? make_float2(0.f, 0.f) : exp2_pair(m0 - m),
                         f1 = m1 == -INFINITY ? make_float2(0.f, 0.f) : exp2_pair(m1 - m);
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                s0 += few.sum[0][q][tid];
                s1 += few.sum[1][q][tid];
            }
            const float sum = s0 * f0.x * f0.y + s1 * f1.x * f1.y;
            few.w0[tid] = f0.x * f0.y;
            few.w1[tid] = tiles > 1 ? f1.x * f1.y : 0.f;
            few.inv[tid] = sum == 0.f ? 0.f : split ? 1.f : 1.f / sum;   // (NaN scores: NaN)
            if (tid < rows) {
                if (split) {
                    part[128 * S::D + tid] = m;
                    part[128 * S::D + 128 + tid] = sum;
                } else if (a.lse) {
                    a.lse[few.out_row[tid]] = sum == 0.f ? -INFINITY : log2_up(m, sum) * kLn2;
                }
            }
        }
        named_barrier(kAllSoftmax, kAll);
        // O^T: this thread has an element of every row; each stream's warps write half the rows
        if (st * 8 < rows) {
            uint32_t o0[16], o1[16];
            tmem_ld16(o0, tmem + lane_base + S::kO);
            if (tiles > 1) tmem_ld16(o1, tmem + lane_base + S::kO + S::kRows);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int row = e;
                if ((e >> 3) != st) continue;
                const float f0 = few.w0[row], f1 = few.w1[row], inv = few.inv[row];
                const float v = (f0 > 0.f ? __uint_as_float(o0[e]) * f0 : 0.f) + (f1 > 0.f ? __uint_as_float(o1[e]) * f1 : 0.f);
                if (row >= rows) continue;
                if (split) part[((key >> 2) * 128 + row) * 4 + (key & 3)] = inv == 0.f ? 0.f : v;
                else a.out[few.out_row[row] * S::D + key] = (uint16_t)pack2<F16>(inv == 0.f ? 0.f : v * kUp * inv, 0.f);
            }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) {
            if (split) mbar_arrive(&bar.part_full[slot]);
            mbar_arrive(&bar.item_empty[n % kItems]);
        }
        // (O, Few and the barriers are used again only past the barrier at the next item's start)
    }
}
