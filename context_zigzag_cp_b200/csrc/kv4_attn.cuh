// Attention of the newest tokens over the 4-bit K/V cache (kv4.cuh).
//
// For query row q of KV head h and key k:  s = scale * q.K_k,
// O = sum_k 2^(s' - m) V_k / l,  LSE = m + ln l,  with a running maximum m and
// sum l in one pass over the keys (online softmax).  Both products run on the
// codes, which are exact in fp16, and the group scales are applied outside:
//   s  = sum_groups (scale_g * (q . codes)_g + zero_g * (sum of q)_g)
//   O  = sum_k (p scale_k) (code_k - 8) + sum_k p (zero_k + 8 scale_k)
// so no dequantised value is ever rounded.
//
// Bound by HBM in principle (18 D / 16 bytes a key and head); what it has to watch
// is instruction issue, since every 4-bit code has to become an operand.
//   - The query rows of a KV head (its query heads x query tokens) are the N = 8 side
//     of warp-wide products and the keys the M side: S^T = K Q^T, O^T = V^T P^T.  With a few
//     rows tcgen05's 128-row tiles would be nearly empty, and the operands
//     would have to go through shared memory once more; here the codes go
//     from registers straight into fragments.
//   - Codes to fp16 without arithmetic: bits 0-3 of a half alone are the subnormal
//     n 2^-24 and bits 4-7 alone are 16 n 2^-24, both exact, so a word of eight codes
//     takes one shift and four ANDs.  The powers of two go into the query (16 q against
//     low places), the score's factor and the end of a segment; -8 sum(p scale) is summed
//     from the rounded p scale beside the products and taken in every four stages.
//     The tensor cores align products by nominal exponents, so a step of 16 is cut at 2^-15
//     of its largest weight (or query value) times one code: less than the weights' own
//     rounding to 11 bits does, and a bf16 query value loses bits only below 2^-8 of the largest.
//     (Integer products on bytes take half the ANDs for K: with the query in two
//     bytes 64 ragged sequences were 6 % faster but the LSE of a handful of keys was off by
//     4e-6, where fp32 has 5e-8; with three bytes they were slower.  e4m3 holds a bf16
//     value as two exact parts, but runs as conversions and fp16 products here: 20 % slower.)
//   - Up to four rows (PAIR): columns 2r and 2r + 1 both belong to row r.  The two halves
//     of a masked word are dims i and i + 4 of one token, so for O^T the reduction index
//     is (token, half), eight tokens a step, and column 2r + s takes P of half s and 0 of
//     the other.  No two tokens' words have to be interleaved, each lane keeps the scores
//     of one row instead of two, and O takes half the registers.
//   - P^T fragments come from S^T ones by a transposed 8x8 move (movmatrix).
//   - Every warp streams its own run of 16-key blocks (contiguous records) through a
//     ring of bulk copies of its own, with its own m, l and O: no barrier between
//     warps until all of a CTA's tiles are done.
//   - m is a lazily moved reference: a stage raises it only when some score
//     exceeds it by 8 (base 2), so the common stage needs one vote and no shuffles.
//     p <= 2^8 then; P goes to fp16 as p scale 2^(6 - E), E the largest exponent of the V
//     scales of the same 64 dims so far (a key without weight does not count), hence at most
//     2^15: 11 bits down to 2^-20 of that scale, steps of 2^-30 of it below.  (One E for all
//     dims gave 64 dims with values 2^30 below the others' an O of zeros.  An E for each 64
//     costs nothing; leaving keys without weight out costs 0.1 of 5.2 us for 301 keys, 0.5 of
//     119 us for 64 ragged sequences, 1 to 1.6 of 44 to 52 us at head_dim 256.)
//   - One CTA of eight warps an SM and 64 keys computed together: two warps a scheduler fill
//     the integer pipe as well as more do, and what a stage costs is paid half as often (64
//     ragged sequences of up to 16k keys, 32 / 8 heads of 128 dims: 115 us; 16 warps and 32
//     keys 125 us, 11 and 12 warps 118 to 123).  That is 5.9 TB/s with an L2 that nothing else
//     writes; among other kernels it is 133 us, 5.1 TB/s.  128k keys of one sequence: 34.5 us, of
//     which 25 stream at 6.0 TB/s and the rest is start, join and merge.
//   - Rows beyond a block of 16 (8 at D 256) pass over the keys again: 8 tokens of 16 heads a KV
//     head, 16 sequences of up to 8k keys, take 69 us for 3.8 us of bytes (D 256: 150 for 7.6).
//
// Work split.  The warps of all CTAs share all key tiles of all (sequence, KV head, row
// block) units evenly: with the units laid end to end, warp v of n takes the tiles
// [v total / n, (v + 1) total / n), whatever the lengths.  A unit inside one warp is finished
// there; the parts of one that runs over several warps are joined at the end of the CTA;
// of one that runs over several CTAs, each writes a partial (m, l, O) into its slot, the
// first leaves a job, and kv4_merge_kernel joins them in order: the result does not
// depend on timing.  Where the table holds KV4_WHOLE tiles of a sequence at most and there
// are no more units than SMs, every unit is one CTA's and there is nothing to join.
#pragma once
#include <cuda_fp16.h>
#include "exp2_poly.cuh"
#include "kv4.cuh"

namespace cpattn {

constexpr int KV4_TILE = 64;         // keys of a scheduling tile (four 16-key blocks)
constexpr uint32_t KV4_NONE = 0xffffffffu;
// Tiles that one CTA takes alone: two stages a warp, no more than a join and its launch cost.  Whole / split, us, one
// sequence and 18 of 32 / 8 heads of 128 dims, 4 rows a unit: up to 447 keys 5.8 / 9.0 and 6.1 / 11.0, 1023 keys 7.8 / 9.0
// and 8.2 / 13.6; above it one sequence is behind, 1279 keys 9.4 / 9.1 and 9.7 / 13.8, 2047 keys 11.4 / 9.0 and 11.7 /
// 15.3.  At 1023 keys of 256 dims 11.8 / 11.5 for one and 12.3 / 14.5 for 30, of 64 dims 6.2 / 7.5 for one.
constexpr int KV4_WHOLE = 16;

// ROWS: query rows a unit, 4 (PAIR), 8, or 16 (two n-tiles; not at D 256, where O alone would take
// 128 registers).  BPS: blocks of a stage, in which they are copied and
// waited for; STEP: blocks computed together (two where the registers hold the second one's scores and weights).
template <int D, int ROWS_>
struct Kv4AttnCfg {
    static constexpr int ROWS = ROWS_;
    static constexpr bool PAIR = ROWS == 4;
    static constexpr int NT = ROWS == 16 ? 2 : 1;    // n-tiles
    static constexpr int NC = PAIR ? 1 : 2;          // rows of a lane in each
    static constexpr int OT = PAIR ? D / 32 : D / 16;   // m-tiles of O^T
    static constexpr int WARPS = 8;
    static constexpr int BPS = D == 256 ? 2 : 4;
    static constexpr int STEP = D == 256 ? 1 : NT == 1 ? 4 : D == 64 ? 2 : 1;
    static constexpr int MSTEP = 1;   // the same where keys are masked: rare, and short code
    static constexpr int STAGES = 2;
    static constexpr int BLOCK = 18 * D;
    static constexpr int STAGE = BPS * BLOCK;
    static constexpr int O_LD = D + 4;
    static constexpr int RING = WARPS * STAGES * STAGE;
    static constexpr int PART = ROWS * (O_LD + 2);   // floats of a part: O [ROWS][O_LD], (m, l) [ROWS]
    static constexpr int MERGE = WARPS * PART * 4;
    static constexpr int BODY = RING > MERGE ? RING : MERGE;
    static constexpr int SMEM_BYTES = BODY + MERGE + WARPS * STAGES * 8;   // ring (then kept parts), parked parts, barriers
    static_assert(SMEM_BYTES <= 225 * 1024, "with the static arrays, what a CTA may have");
};

struct Kv4AttnParams {
    Kv4Cache C;
    const __nv_bfloat16* q;     // [B][Hq][T][D], strides below
    int64_t qs[3];
    const int32_t* lens;        // [B]
    __nv_bfloat16* o;           // [B][Hq][T][D], or null:
    float* o_part;              // the same in fp32
    float* lse;                 // [B][Hq][T]
    float* slots;               // [2 * grid] partials of CTAs: O [ROWS][D], (m, l) [ROWS]
    int4* jobs;                 // [grid] (sequence, KV head, row block, parts) of the unit that begins in a CTA
    int32_t Hq, T, rows, row_blocks, causal, window, whole;   // and runs on; 0 parts: none
    float scale_log2;
    Kv4Div by_t, by_row_blocks, by_page;   // n_queries, row blocks, blocks of a page
};

// ---------------------------------------------------------------- schedule

// First and last + 1 tile of sequence b (at least one, so that an empty sequence's
// outputs are written too) and its clamped length.
struct Kv4Span {
    int len, t0, n;
};

__device__ __forceinline__ Kv4Span kv4_span_of(const Kv4AttnParams& P, int len)
{
    Kv4Span s;
    s.len = len;
    const int lo = P.window > 0 ? max(0, s.len - P.T - P.window + 1) : 0;   // oldest key of query 0
    s.t0 = lo / KV4_TILE;
    s.n = max(1, (s.len + KV4_TILE - 1) / KV4_TILE - s.t0);
    return s;
}

__device__ __forceinline__ Kv4Span kv4_span(const Kv4AttnParams& P, int b, bool report)
{
    const int len = P.lens[b], room = P.C.width * P.C.page_size;   // at most 2^30
    const int cut = min(max(len, 0), room);
    if (report && cut != len) record_status(1 /* CP_ERR_INVALID_ARG */);
    return kv4_span_of(P, cut);
}

// Exclusive sum over the CTA's threads, all of which take part; sh holds 32 ints.
__device__ inline int kv4_scan(int v, int* sh, int& total)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    __syncthreads();
    if (lane == 31) sh[w] = x;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int i = 0; i < nw; ++i) {
        const int y = sh[i];
        if (i < w) before += y;
        total += y;
    }
    return before + x - v;
}

// -> tiles of one thread's chunk of sequences, scanned.  units: Hkv * row_blocks.
struct Kv4Chunk {
    int b0, b1, before, total;
};

__device__ inline Kv4Chunk kv4_chunk(const Kv4AttnParams& P, int units, int* sh, bool report)
{
    Kv4Chunk c;
    const int per = (P.C.B + blockDim.x - 1) / blockDim.x;
    c.b0 = min(static_cast<int>(threadIdx.x) * per, P.C.B);
    c.b1 = min(c.b0 + per, P.C.B);
    int n = 0;
    for (int b = c.b0; b < c.b1; ++b) n += kv4_span(P, b, report).n * units;
    c.before = kv4_scan(n, sh, c.total);
    return c;
}

// The same for up to 128 sequences, by every warp for itself: lane i holds sequences i, 32 + i, ...  (No barriers: 0.2 of
// 7.8 us for one sequence, 0.5 of 51.5 us in a step over 32.)
constexpr int KV4_FEW = 128;

struct Kv4Lane {
    int len[4], n[4], upto[4], total;   // tiles, and tiles up to its end

    __device__ __forceinline__ Kv4Lane(const Kv4AttnParams& P, int units, bool report)
    {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            Kv4Span s = {0, 0, 0};
            if (32 * k + lane < P.C.B) s = kv4_span(P, 32 * k + lane, report);
            len[k] = s.len;
            upto[k] = n[k] = s.n * units;
        }
#pragma unroll
        for (int off = 1; off < 32; off <<= 1)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int y = __shfl_up_sync(0xffffffffu, upto[k], off);
                if (lane >= off) upto[k] += y;
            }
        total = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            upto[k] += total;
            total = __shfl_sync(0xffffffffu, upto[k], 31);
        }
    }
    // (sequence, tiles before it, its length) for tile x < total
    __device__ __forceinline__ int4 find(int x) const
    {
        int4 r = make_int4(-1, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t after = __ballot_sync(0xffffffffu, upto[k] > x);
            if (r.x < 0 && after) {
                const int i = __ffs(after) - 1;
                r = make_int4(32 * k + i, __shfl_sync(0xffffffffu, upto[k] - n[k], i),
                              __shfl_sync(0xffffffffu, len[k], i), 0);
            }
        }
        return r;
    }
};

// total items over n takers: taker i begins at i total / n.
struct Kv4Split {
    int total, n, each, rest;
    __device__ __forceinline__ Kv4Split(int total_, int n_) : total(total_), n(n_)
    {
        each = total / n;
        rest = total - each * n;
    }
    __device__ __forceinline__ int at(int i) const { return i * each + i * rest / n; }   // n is a few thousand at most
    __device__ __forceinline__ int taker(int x) const   // the last one that begins at x or before
    {
        return static_cast<int>((static_cast<int64_t>(x + 1) * n - 1) / total);
    }
};

// The sequence that holds tile x: (its number, tiles before it, its length), the same on every lane.  pre: the tiles
// before each thread's chunk.
__device__ __forceinline__ int4 kv4_find(const Kv4AttnParams& P, int units, const int* pre, int x)
{
    const int lane = threadIdx.x & 31, per = (P.C.B + blockDim.x - 1) / blockDim.x;
    const int used = per == 1 ? P.C.B : static_cast<int>(blockDim.x);   // chunks that may hold a sequence
    int chunk = -1;
    for (int i = 0; i < used; i += 32) chunk += __popc(__ballot_sync(0xffffffffu, i + lane < used && pre[i + lane] <= x));
    int at = pre[chunk];
    for (int b = chunk * per;; ++b) {
        const Kv4Span s = kv4_span(P, b, false);
        const int n = s.n * units;
        if (x < at + n || b + 1 >= P.C.B) return make_int4(b, at, s.len, 0);
        at += n;
    }
}

// ---------------------------------------------------------------- fragments

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The same with an accumulator of 0.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// fp16 subnormals of the codes in bits 0-3 (n 2^-24) and bits 4-7 (16 n 2^-24) of each half
__device__ __forceinline__ uint32_t nibble16(uint32_t x) { return x & 0x00f000f0u; }
__device__ __forceinline__ uint32_t nibble1(uint32_t x) { return x & 0x000f000fu; }

__device__ __forceinline__ float f16_half(uint32_t x, int high)
{
    __half2 h;
    memcpy(&h, &x, 4);
    return high ? __high2float(h) : __low2float(h);
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// The query operand of one unit: per n-tile the fragments of D / 16 k-steps and, for the
// lane's score columns, the sum of q a group and the factor from accumulator to base-2 score.
// The accumulator counts 2^-20 q.code: codes in high places come as 16 n, those in low ones as n
// against 16 q.
template <int D, int ROWS>
struct Kv4Query {
    using Cfg = Kv4AttnCfg<D, ROWS>;
    uint32_t f[Cfg::NT][D / 32][4];
    float sum[Cfg::NT][D / 64][Cfg::NC];     // 2^-20 * sum of q over the group
    float mul[Cfg::NT][Cfg::NC];
};

// The lane's words of the rows of column g; of a row that is not there NaN, which counts in no maximum and no vote.
template <int D, int ROWS>
__device__ __forceinline__ void kv4_load_query(const Kv4AttnParams& P, int b, int h, int rb,
                                               uint4 (&x)[Kv4AttnCfg<D, ROWS>::NT][D / 32])
{
    using Cfg = Kv4AttnCfg<D, ROWS>;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint4 none = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
#pragma unroll
    for (int nt = 0; nt < Cfg::NT; ++nt) {
        const int r = rb * ROWS + nt * 8 + (Cfg::PAIR ? g >> 1 : g);
        const bool live = r < P.rows;
        const int hg = live ? P.by_t.of(r) : 0, tok = live ? r - hg * P.T : 0;
        const uint4* src =
            reinterpret_cast<const uint4*>(P.q + b * P.qs[0] + (h * (P.Hq / P.C.Hkv) + hg) * P.qs[1] + tok * P.qs[2]);
#pragma unroll
        for (int w = 0; w < D / 32; ++w) x[nt][w] = live ? src[4 * w + t] : none;
    }
}

template <int D, int ROWS>
__device__ __forceinline__ void kv4_make_query(const Kv4AttnParams& P, const uint4 (&x)[Kv4AttnCfg<D, ROWS>::NT][D / 32],
                                               Kv4Query<D, ROWS>& Q)
{
    using Cfg = Kv4AttnCfg<D, ROWS>;
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int nt = 0; nt < Cfg::NT; ++nt) {
        uint32_t top = 0;   // largest magnitude, as bits
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
            const uint32_t v[4] = {x[nt][w].x, x[nt][w].y, x[nt][w].z, x[nt][w].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) top = max(top, max(v[i] & 0x7fffu, (v[i] >> 16) & 0x7fffu));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // The row times a power of two, its largest value in [2^11, 2^12) (times 16 in the low places):
        // bf16 values are then exact in fp16 down to 2^-26 of it.
        const int e = min(max(static_cast<int>(top >> 7) - 127 - 11, -110), 116);
        const float down = pow2i(-e);
        float sums[D / 64];
#pragma unroll
        for (int i = 0; i < D / 64; ++i) sums[i] = 0.f;
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
            const uint32_t v[4] = {x[nt][w].x, x[nt][w].y, x[nt][w].z, x[nt][w].w};
            float y[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[2 * i] = bf_lo(v[i]) * down;
                y[2 * i + 1] = bf_hi(v[i]) * down;
            }
            // word of codes: values (0,4) low, (1,5) high for the first k-step, (2,6) low, (3,7) high
            // for the second
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float up = i & 1 ? 1.f : 16.f;
                const uint32_t p = pack_f16(up * y[i], up * y[i + 4]);
                Q.f[nt][w][i] = p;
                __half2 hp;
                memcpy(&hp, &p, 4);
                const float both = __low2float(hp) + __high2float(hp);
                sums[w / 2] += i & 1 ? 16.f * both : both;
            }
        }
        // (infinite for values beyond 2^119 / scale; a row with an infinity or a NaN sees NaN scores)
        const float mul = top >= 0x7f80u ? __uint_as_float(0x7fc00000u) : P.scale_log2 * 1048576.f * pow2i(e);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            sums[i] += __shfl_xor_sync(0xffffffffu, sums[i], 1);
            sums[i] += __shfl_xor_sync(0xffffffffu, sums[i], 2);
        }
        // from the lanes of column g to the lanes of columns 2t, 2t + 1
#pragma unroll
        for (int c = 0; c < Cfg::NC; ++c) {
            const int from = (2 * t + c) * 4;
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
                Q.sum[nt][i][c] = __shfl_sync(0xffffffffu, sums[i], from) * 5.9604644775390625e-8f;
            Q.mul[nt][c] = __shfl_sync(0xffffffffu, mul, from);
        }
    }
}

// Running state of a warp.  O^T accumulators, m-tile by m-tile, in units of 2^-24 2^(e - 133), e that of the group:
//   PAIR: tile 2 gd + m, dims 64 gd + 8 g + (2m, 2m + 4; 2m + 1, 2m + 5) of row t;
//   else: tile 4 gd + i, dims 64 gd + 8 g + 2i (and 2i + 1 in c + 2), columns 2t, 2t + 1;
// the odd dims count 16 times.  Reference -m, and the lane's share of l, of the sum of p scale (as rounded
// for the products, in units of 2^(e - 133)) and of sum p (zero + 8 scale).
template <int D, int ROWS>
struct Kv4State {
    using Cfg = Kv4AttnCfg<D, ROWS>;
    float o[Cfg::NT][Cfg::OT][4];
    float nm[Cfg::NT][Cfg::NC], l[Cfg::NT][Cfg::NC], ps[Cfg::NT][D / 64][Cfg::NC], z[Cfg::NT][D / 64][Cfg::NC];
    float down[D / 64];   // 2^(133 - e), e the biased exponent that the V scales of a group are relative to in o and ps
};

// From 2^(133 - e): 2^(e - 133), and e.
__device__ __forceinline__ float kv4_up(float down) { return __uint_as_float((254u << 23) - __float_as_uint(down)); }
__device__ __forceinline__ int kv4_exp(float down) { return 260 - static_cast<int>(__float_as_uint(down) >> 23); }

template <int D, int ROWS>
__device__ __forceinline__ void kv4_clear(Kv4State<D, ROWS>& S)
{
    using Cfg = Kv4AttnCfg<D, ROWS>;
#pragma unroll
    for (int nt = 0; nt < Cfg::NT; ++nt) {
#pragma unroll
        for (int i = 0; i < Cfg::OT; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) S.o[nt][i][c] = 0.f;
#pragma unroll
        for (int c = 0; c < Cfg::NC; ++c) {
            S.nm[nt][c] = INFINITY;
            S.l[nt][c] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) S.ps[nt][i][c] = S.z[nt][i][c] = 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < D / 64; ++i) S.down[i] = pow2i(106);   // e = 27
}

// (scale, zero) pairs of one key.
template <int NG>
__device__ __forceinline__ void kv4_pairs(const uint8_t* meta, uint32_t (&m)[NG])
{
    if constexpr (NG == 1) {
        m[0] = *reinterpret_cast<const uint32_t*>(meta);
    } else if constexpr (NG == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(meta);
        m[0] = v.x; m[1] = v.y;
    } else {
        const uint4 v = *reinterpret_cast<const uint4*>(meta);
        m[0] = v.x; m[1] = v.y; m[2] = v.z; m[3] = v.w;
    }
}

// q . code of one block's keys g, g + 8 and the lane's columns, group scales applied: s[nt][column + NC * key].
template <int D, int ROWS>
__device__ __forceinline__ void kv4_scores(const uint8_t* blk, const Kv4Query<D, ROWS>& Q,
                                           float (&s)[Kv4AttnCfg<D, ROWS>::NT][2 * Kv4AttnCfg<D, ROWS>::NC])
{
    using Cfg = Kv4AttnCfg<D, ROWS>;
    constexpr int NG = D / 64, NW = D / 32, NC = Cfg::NC;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint32_t kw[2][NW], km[2][NG];   // keys g, g + 8: codes, (scale, zero)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint8_t* row = blk + (g + 8 * j) * (D / 2);
        if constexpr (D == 64) {
            const uint2 v = *reinterpret_cast<const uint2*>(row + t * 8);
            kw[j][0] = v.x; kw[j][1] = v.y;
        } else if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(row + t * 16);
            kw[j][0] = v.x; kw[j][1] = v.y; kw[j][2] = v.z; kw[j][3] = v.w;
        } else {
#pragma unroll
            for (int p = 0; p < 2; ++p) {   // rows g and g + 8 have the parity of g
                const uint4 v = *reinterpret_cast<const uint4*>(row + ((p ^ (g & 1)) << 6) + t * 16);
                kw[j][4 * p] = v.x; kw[j][4 * p + 1] = v.y; kw[j][4 * p + 2] = v.z; kw[j][4 * p + 3] = v.w;
            }
        }
        kv4_pairs<NG>(blk + 8 * D + (g + 8 * j) * (NG * 4), km[j]);
    }
#pragma unroll
    for (int i = 0; i < NG; ++i) {
        float acc[Cfg::NT][4];
#pragma unroll
        for (int w = 2 * i; w < 2 * i + 2; ++w) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t x = k ? kw[0][w] >> 8 : kw[0][w], y = k ? kw[1][w] >> 8 : kw[1][w];
                const uint32_t a[4] = {nibble1(x), nibble1(y), nibble16(x), nibble16(y)};
#pragma unroll
                for (int nt = 0; nt < Cfg::NT; ++nt) {
                    if (w == 2 * i && k == 0)
                        mma_f16_first(acc[nt], a, Q.f[nt][w][0], Q.f[nt][w][1]);
                    else
                        mma_f16(acc[nt], a, Q.f[nt][w][2 * k], Q.f[nt][w][2 * k + 1]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float sc = bf_lo(km[j][i]), ze = bf_hi(km[j][i]);
#pragma unroll
            for (int nt = 0; nt < Cfg::NT; ++nt)
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    float& to = s[nt][NC * j + c];
                    const float v = i == 0 ? ze * Q.sum[nt][i][c] : fmaf(ze, Q.sum[nt][i][c], to);
                    to = fmaf(sc, acc[nt][2 * j + c], v);
                }
        }
    }
}

// STEP blocks from shared memory.  MASK: keys outside [lo, hi) of a column are
// not seen (what their cache holds may be anything), nor those of the blocks in `gone`; pos: position of key 0.
template <int D, int ROWS, int STEP, bool MASK>
__device__ __forceinline__ void kv4_step(const uint8_t* blk, const Kv4Query<D, ROWS>& Q, Kv4State<D, ROWS>& S, int pos, uint32_t gone,
                                          const int (&lo)[Kv4AttnCfg<D, ROWS>::NT][Kv4AttnCfg<D, ROWS>::NC],
                                          const int (&hi)[Kv4AttnCfg<D, ROWS>::NT][Kv4AttnCfg<D, ROWS>::NC])
{
    using Cfg = Kv4AttnCfg<D, ROWS>;
    constexpr int NG = D / 64, BLOCK = 18 * D, NT = Cfg::NT, NC = Cfg::NC;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

    // ---- scores against the reference: x = s - m (base 2)
    float s[STEP][NT][2 * NC], x[STEP][NT][2 * NC];
    uint32_t vm[STEP][2][NG];   // V's (scale, zero) of keys g, g + 8
    float vd[STEP][2][NG];      // V's scales times S.down
    uint32_t hidden[STEP];      // MASK: bit 2 NC nt + NC j + c where a column does not see a key of the lane
    float most = -INFINITY, top = 0.f;
#pragma unroll
    for (int k = 0; k < STEP; ++k) {
        kv4_scores<D, ROWS>(blk + k * BLOCK, Q, s[k]);
        hidden[k] = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            bool seen = !MASK;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    float& y = x[k][nt][NC * j + c];
                    y = fmaf(s[k][nt][NC * j + c], Q.mul[nt][c], S.nm[nt][c]);
                    if (MASK) {
                        const int key = pos + 16 * k + g + 8 * j;
                        if (key < lo[nt][c] || key >= hi[nt][c] || (gone >> k & 1)) {
                            y = -INFINITY;
                            hidden[k] |= 1u << (2 * NC * nt + NC * j + c);
                        } else {
                            seen = true;
                        }
                    }
                }
            kv4_pairs<NG>(blk + k * BLOCK + 17 * D + (g + 8 * j) * (NG * 4), vm[k][j]);
#pragma unroll
            for (int i = 0; i < NG; ++i)
                if (MASK && !seen) vm[k][j][i] = 0;   // whatever it holds
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2 * NC; c += 2) most = fmax3(most, x[k][nt][c], x[k][nt][c + 1]);
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            vd[k][0][i] = bf_lo(vm[k][0][i]) * S.down[i];
            vd[k][1][i] = bf_lo(vm[k][1][i]) * S.down[i];
            top = fmax3(top, vd[k][0][i], vd[k][1][i]);
        }
    }

    // ---- a new reference, or other exponents of V's scales (which are not negative)
    if (__any_sync(0xffffffffu, most > 8.f || top >= 128.f)) {
        float f[NT][NC];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                float m = -S.nm[nt][c];
                const float old = m;
#pragma unroll
                for (int k = 0; k < STEP; ++k)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (!MASK || x[k][nt][c + NC * j] != -INFINITY)
                            m = fmaxf(m, s[k][nt][c + NC * j] * Q.mul[nt][c]);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
                f[nt][c] = old == -INFINITY ? 0.f : ex2(old - m);
                S.nm[nt][c] = -m;
#pragma unroll
                for (int k = 0; k < STEP; ++k)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (!MASK || x[k][nt][c + NC * j] != -INFINITY)
                            x[k][nt][c + NC * j] = fmaf(s[k][nt][c + NC * j], Q.mul[nt][c], -m);
                S.l[nt][c] *= f[nt][c];
            }
        // The exponent of a group's scales follows the largest, but not that of a key without weight, beside which the
        // others would lose their bits: no further than 2^8 above the smallest of the lanes' largest scales or 2^10 above
        // the largest p scale of the step.  It falls where it was 2^8 too large.  p <= 1 here, so p scale 2^(6 - E) < 2^7.
        float p[STEP][2];   // largest weight of a key
#pragma unroll
        for (int k = 0; k < STEP; ++k)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float y = x[k][0][NC * j];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < NC; ++c) y = fmaxf(y, x[k][nt][NC * j + c]);
                p[k][j] = ex2(y);
            }
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            float v = 0.f, w = 0.f;
#pragma unroll
            for (int k = 0; k < STEP; ++k) {
                v = fmax3(v, bf_lo(vm[k][0][i]), bf_lo(vm[k][1][i]));
                w = fmax3(w, p[k][0] * bf_lo(vm[k][0][i]), p[k][1] * bf_lo(vm[k][1][i]));
            }
            const int most_e = min(__reduce_max_sync(0xffffffffu, __float_as_uint(v)) >> 23, 254u);
            const int least_e = __reduce_min_sync(0xffffffffu, v > 0.f ? __float_as_uint(v) : 0x7f800000u) >> 23;
            const int w_e = __reduce_max_sync(0xffffffffu, __float_as_uint(w)) >> 23;
            const int old = kv4_exp(S.down[i]);
            // most_e where that is no more than old; a scale times S.down stays finite, 2^(most_e + 7 - e) at most
            int e = min(most_e, max(max(max(w_e + 10, least_e + 8), old), most_e - 120));
            e = e >= old ? e : e > 0 && e + 7 < old ? max(e, max(old - 60, 27)) : old;
            const float fe = pow2i(max(old - e, -126));
            S.down[i] = pow2i(133 - e);
#pragma unroll
            for (int k = 0; k < STEP; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j) vd[k][j][i] = bf_lo(vm[k][j][i]) * S.down[i];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    S.z[nt][i][c] *= f[nt][c];
                    S.ps[nt][i][c] *= f[nt][c] * fe;
                }
#pragma unroll
                for (int t = i * (Cfg::OT / NG); t < (i + 1) * (Cfg::OT / NG); ++t)
#pragma unroll
                    for (int c = 0; c < 4; ++c) S.o[nt][t][c] *= f[nt][c & (NC - 1)] * fe;
            }
        }
    }

    // ---- weights, and O^T += V^T P^T
    // PAIR: P of the lane's column goes into its half (column 2r: the low one), 0 into the other; as a product, since
    // the integer pipe has the ANDs to do
    const __half2 half_of = g & 1 ? __halves2half2(__ushort_as_half(0), __ushort_as_half(0x3c00))
                                  : __halves2half2(__ushort_as_half(0x3c00), __ushort_as_half(0));
#pragma unroll
    for (int k = 0; k < STEP; ++k) {
        float p[NT][2 * NC];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int c = 0; c < 2 * NC; ++c) p[nt][c] = ex2(x[k][nt][c]);
#pragma unroll
            for (int c = 0; c < NC; ++c) S.l[nt][c] += p[nt][c] + p[nt][c + NC];
        }
        uint32_t pf[NT][NG][2];   // keys 2t, 2t + 1 and 2t + 8, 2t + 9 of column g
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float sc = bf_lo(vm[k][j][i]), ze = fmaf(8.f, sc, bf_hi(vm[k][j][i])), sd = vd[k][j][i];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float ps[NC];
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const float w = p[nt][NC * j + c];
                        // a key that another column sees may hold a NaN that this one must not; under a weight that came
                        // out as 0 it is a NaN here too
                        const bool none = MASK && (hidden[k] >> (2 * NC * nt + NC * j + c) & 1);
                        ps[c] = none ? 0.f : w * sd;
                        S.z[nt][i][c] = none ? S.z[nt][i][c] : fmaf(w, ze, S.z[nt][i][c]);
                    }
                    const uint32_t pk = pack_f16(ps[0], ps[NC - 1]);
#pragma unroll
                    for (int c = 0; c < NC; ++c) S.ps[nt][i][c] += f16_half(pk, c);
                    pf[nt][i][j] = transpose8(pk);
                }
            }
        uint32_t vw[2][2][NG];   // pair of tokens (2t, 2t + 8), token of the pair, group
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint8_t* base = blk + k * BLOCK + 9 * D + g * D;
            const int pair = t + 4 * j;
            if constexpr (D == 64) {
                const uint2 v = *reinterpret_cast<const uint2*>(base + (pair ^ (((g >> 1) & 1) << 2)) * 8);
                vw[j][0][0] = v.x; vw[j][1][0] = v.y;
            } else if constexpr (D == 128) {
                const uint4 v = *reinterpret_cast<const uint4*>(base + (pair ^ ((g & 1) << 2)) * 16);
                vw[j][0][0] = v.x; vw[j][0][1] = v.y; vw[j][1][0] = v.z; vw[j][1][1] = v.w;
            } else {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint4 v = *reinterpret_cast<const uint4*>(base + pair * 32 + ((q ^ (g & 1)) << 4));
                    vw[j][q][0] = v.x; vw[j][q][1] = v.y; vw[j][q][2] = v.z; vw[j][q][3] = v.w;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            if constexpr (Cfg::PAIR) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {   // tokens 2t, 2t + 1 (+ 8)
                    __half2 both, first, second;
                    memcpy(&both, &pf[0][i][j], 4);
                    first = __hmul2(__low2half2(both), half_of);
                    second = __hmul2(__high2half2(both), half_of);
                    uint32_t b0, b1;
                    memcpy(&b0, &first, 4);
                    memcpy(&b1, &second, 4);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const uint32_t v = m ? (vw[j][0][i] >> 8) : vw[j][0][i];
                        const uint32_t y = m ? (vw[j][1][i] >> 8) : vw[j][1][i];
                        const uint32_t a[4] = {nibble1(v), nibble16(v), nibble1(y), nibble16(y)};
                        mma_f16(S.o[0][2 * i + m], a, b0, b1);
                    }
                }
            } else {
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    uint32_t a[2][4];   // two m-tiles
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t v = __byte_perm(vw[j][0][i], vw[j][1][i], hf ? 0x7632 : 0x5410);
                        const uint32_t y = (v >> 8);
                        a[0][2 * j] = nibble1(v);
                        a[0][2 * j + 1] = nibble16(v);
                        a[1][2 * j] = nibble1(y);
                        a[1][2 * j + 1] = nibble16(y);
                    }
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_f16(S.o[nt][4 * i + 2 * hf + m], a[m], pf[nt][i][0], pf[nt][i][1]);
                }
            }
        }
    }
}

// Takes -8 sum(p scale) into O.  The running sums are cut, not rounded, to 24 bits, and sums of codes 0..15 grow with
// the keys: after 16k keys of even weights the cuts had come to 1.6 % of O, after 64k to 3.6 %.  Taken to their middle
// every few hundred keys they stay small (2e-4, which is P's rounding).
template <int D, int ROWS>
__device__ __forceinline__ void kv4_center(Kv4State<D, ROWS>& S)
{
    using Cfg = Kv4AttnCfg<D, ROWS>;
    constexpr float kEven = -8.f / 16777216.f, kOdd = 16.f * kEven;   // odd dims count 16 times
#pragma unroll
    for (int nt = 0; nt < Cfg::NT; ++nt)
#pragma unroll
        for (int c = 0; c < Cfg::NC; ++c)
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                float p = S.ps[nt][i][c];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) p += __shfl_xor_sync(0xffffffffu, p, off);
                S.ps[nt][i][c] = 0.f;
                if constexpr (Cfg::PAIR) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int m = 0; m < 2; ++m) S.o[0][2 * i + m][k] = fmaf(p, k < 2 ? kEven : kOdd, S.o[0][2 * i + m][k]);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        S.o[nt][4 * i + k][c] = fmaf(p, kEven, S.o[nt][4 * i + k][c]);
                        S.o[nt][4 * i + k][c + 2] = fmaf(p, kOdd, S.o[nt][4 * i + k][c + 2]);
                    }
                }
            }
}

// f(row of the unit, first dim, its 8 dims of O, m, l) for what the lane holds of a finished segment.
template <int D, int ROWS, class F>
__device__ __forceinline__ void kv4_rows_of(const Kv4State<D, ROWS>& S, F&& f)
{
    using Cfg = Kv4AttnCfg<D, ROWS>;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < Cfg::NT; ++nt)
#pragma unroll
        for (int c = 0; c < Cfg::NC; ++c)
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const float up = kv4_up(S.down[i]);
                float x[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if constexpr (Cfg::PAIR) {   // tile 2i + (k & 1): dims 2m (c 0), + 4 (c 1), + 1 (c 2), + 5 (c 3)
                        x[2 * k] = S.o[0][2 * i + (k & 1)][k >> 1];
                        x[2 * k + 1] = S.o[0][2 * i + (k & 1)][2 + (k >> 1)];
                    } else {
                        x[2 * k] = S.o[nt][4 * i + k][c];
                        x[2 * k + 1] = S.o[nt][4 * i + k][c + 2];
                    }
                }
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    x[k] = fmaf(fmaf(x[k], k & 1 ? 1048576.f : 16777216.f, -8.f * S.ps[nt][i][c]), up, S.z[nt][i][c]);
                f(nt * 8 + Cfg::NC * t + c, 64 * i + 8 * g, x, -S.nm[nt][c], S.l[nt][c]);
            }
}

template <int D, int ROWS>
__device__ __forceinline__ void kv4_store_part(const Kv4State<D, ROWS>& S, float* to)
{
    using Cfg = Kv4AttnCfg<D, ROWS>;
    kv4_rows_of(S, [&](int r, int d, const float (&x)[8], float m, float l) {
        float4* d4 = reinterpret_cast<float4*>(to + r * Cfg::O_LD + d);
        d4[0] = make_float4(x[0], x[1], x[2], x[3]);
        d4[1] = make_float4(x[4], x[5], x[6], x[7]);
        if (d == 0) *reinterpret_cast<float2*>(to + ROWS * Cfg::O_LD + 2 * r) = make_float2(m, l);
    });
}

template <int D, int ROWS>
__global__ void __launch_bounds__(Kv4AttnCfg<D, ROWS>::WARPS * 32, 1)
kv4_attn_kernel(Kv4AttnParams P)
{
    using Cfg = Kv4AttnCfg<D, ROWS>;
    constexpr int W = Cfg::WARPS, ST = Cfg::STAGES, BPS = Cfg::BPS, STEP = Cfg::STEP, MSTEP = Cfg::MSTEP, NT = Cfg::NT, NC = Cfg::NC, NG = D / 64;
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ int sh_scan[32], sh_before[W * 32], sh_groups;
    __shared__ int4 sh_group[2 * W];
    __shared__ int4 sh_part[2 * W];   // (first tile, sequence, unit of the sequence, tiles) of the parts to be joined
    __shared__ volatile int sh_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = lane & 3;
    uint8_t* ring = sm + warp * ST * Cfg::STAGE;
    const uint32_t bars = smem_u32(sm + Cfg::BODY + Cfg::MERGE) + warp * ST * 8;
    float* parked = reinterpret_cast<float*>(sm + Cfg::BODY);   // [W] parts of units that end inside a warp's tiles
    const uint32_t ring32 = smem_u32(ring);

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join may take its place and wait
    if (threadIdx.x == 0) sh_abort = 0;
    if (threadIdx.x < 2 * W) sh_part[threadIdx.x] = make_int4(-1, 0, 0, 0);
    if (lane == 0) {
        for (int i = 0; i < ST; ++i) mbar_init(bars + 8 * i, 1);
        fence_barrier_init();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");   // what was launched before is done: its outputs may be read
    const int units = P.C.Hkv * P.row_blocks;
    int cta0, cta1, begin, end;   // tiles of the CTA and of the warp
    int b, before;                // the warp's sequence and the tiles before it
    Kv4Span span;
    int ctas = 1, total = 1;
    if (P.whole) {
        b = blockIdx.x / units;
        const int u = blockIdx.x - b * units;
        span = kv4_span(P, b, u == 0);
        before = 0;
        cta0 = u * span.n;
        cta1 = cta0 + span.n;
        const Kv4Split split(span.n, W);
        begin = cta0 + split.at(warp);
        end = cta0 + split.at(warp + 1);
        __syncthreads();   // the barriers and shared arrays are set
    } else {
        if (threadIdx.x == 0) P.jobs[blockIdx.x] = make_int4(0, 0, 0, 0);
        int4 where;   // of a warp without tiles: of the next tile, or of the last
        auto share = [&] {
            ctas = min(static_cast<int>(gridDim.x), (total - 1) / W + 1);   // each has a tile at least
            const Kv4Split split(total, ctas * W);
            const int v = blockIdx.x * W;
            cta0 = split.at(v);
            cta1 = split.at(v + W);
            begin = split.at(v + warp);
            end = split.at(v + warp + 1);
        };
        if (P.C.B <= KV4_FEW) {
            const Kv4Lane all(P, units, blockIdx.x == 0 && warp == 0);
            total = all.total;
            share();
            if (blockIdx.x >= ctas) return;
            where = all.find(min(begin, total - 1));
            __syncthreads();   // the barriers and shared arrays are set
        } else {
            const Kv4Chunk chunk = kv4_chunk(P, units, sh_scan, blockIdx.x == 0);
            total = chunk.total;
            share();
            if (blockIdx.x >= ctas) return;
            sh_before[threadIdx.x] = chunk.before;
            __syncthreads();
            where = kv4_find(P, units, sh_before, min(begin, total - 1));
        }
        b = where.x;
        before = where.y;
        span = kv4_span_of(P, where.z);
    }
    uint32_t slot = 0, parity = 0;   // of the warp's next stage in its ring
    Kv4State<D, ROWS> S;
    bool ok = true, kept = false;   // kept: the last part is in S

    for (int at = begin; at < end;) {
        while (at >= before + span.n * units) {
            before += span.n * units;
            ++b;
            span = kv4_span(P, b, false);
        }
        const int u = (at - before) / span.n, first = before + u * span.n;   // unit and its first tile
        const int stop = min(end, first + span.n);
        const int h = P.by_row_blocks.of(u), rb = u - h * P.row_blocks;
        // the segment's 16-key blocks [blk0, blk1) of the sequence, in n stages
        const int blk0 = (span.t0 + at - first) * (KV4_TILE / 16);
        const int blk1 = min((span.t0 + stop - first) * (KV4_TILE / 16), (span.len + 15) / 16);
        const int n = blk1 > blk0 ? (blk1 - blk0 + BPS - 1) / BPS : 0;
        const int bpp = P.C.page_size >> 4;   // blocks a page

        // Lane i holds the i-th of the next 32 blocks: its place in the pool in blocks, or KV4_NONE: no such block,
        // or its page is not in the pool (bit in `bad`: nothing of it is seen).
        constexpr int PER = 32 / BPS;   // stages of a lookup
        uint32_t place = KV4_NONE, runs = 0, bad = 0, bad_next = 0;   // bit i of runs: block i + 1 follows block i
        auto lookup = [&](int i0) {   // i0: first stage, a multiple of PER
            const int blk = blk0 + i0 * BPS + lane;
            bool wrong = false;
            place = KV4_NONE;
            if (blk < blk1) {
                const int i = P.by_page.of(blk);   // below the table's width: blk * 16 is below the length
                const int page = P.C.table[static_cast<int64_t>(b) * P.C.width + i];
                wrong = page < 0 || page >= P.C.num_pages;
                if (wrong)
                    record_status(1 /* CP_ERR_INVALID_ARG */);
                else
                    place = (static_cast<uint32_t>(page) * P.C.Hkv + h) * bpp + (blk - i * bpp);
            }
            bad_next = __ballot_sync(0xffffffffu, wrong);
            const uint32_t next = __shfl_down_sync(0xffffffffu, place, 1);
            runs = __ballot_sync(0xffffffffu, place != KV4_NONE && next == place + 1);
        };
        auto issue = [&](int i, uint32_t to) {   // stage i of the warp into slot `to`
            const uint32_t bar = bars + 8 * to, dst = ring32 + to * Cfg::STAGE;
            const int at = (i * BPS) & 31;
            const uint32_t p0 = __shfl_sync(0xffffffffu, place, at);
            if ((~(runs >> at) & ((1u << (BPS - 1)) - 1)) == 0) {   // one run of blocks
                if (elect_one()) {
                    mbar_arrive_expect_tx(bar, Cfg::STAGE);
                    bulk_load(dst, P.C.pages + static_cast<int64_t>(p0) * Cfg::BLOCK, Cfg::STAGE, bar);
                }
            } else {
                uint32_t p[BPS];
                int there = 0;
#pragma unroll
                for (int k = 0; k < BPS; ++k) {
                    p[k] = __shfl_sync(0xffffffffu, place, at + k);
                    there += p[k] != KV4_NONE;
                }
                if (elect_one()) {
                    mbar_arrive_expect_tx(bar, there * Cfg::BLOCK);
#pragma unroll
                    for (int k = 0; k < BPS; ++k)
                        if (p[k] != KV4_NONE)
                            bulk_load(dst + k * Cfg::BLOCK, P.C.pages + static_cast<int64_t>(p[k]) * Cfg::BLOCK,
                                      Cfg::BLOCK, bar);
                }
            }
            __syncwarp();
        };
        uint4 words[NT][D / 32];   // asked for before the table's entries are waited for
        kv4_load_query<D, ROWS>(P, b, h, rb, words);
        if (n > 0) lookup(0);
        {
            uint32_t to = slot;
            for (int i = 0; i < min(n, ST); ++i) {
                issue(i, to);
                if (++to == ST) to = 0;
            }
        }

        Kv4Query<D, ROWS> Q;
        kv4_make_query<D, ROWS>(P, words, Q);
        kv4_clear(S);
        // the lane's rows see keys [lo, hi); every row sees [all_lo, all_hi)
        int lo[NT][NC], hi[NT][NC];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int r = rb * ROWS + nt * 8 + NC * t + c;
                const int p = span.len - P.T + r - P.by_t.of(r) * P.T;   // the row's position
                hi[nt][c] = P.causal ? p + 1 : span.len;
                lo[nt][c] = P.window > 0 ? p - P.window + 1 : 0;
            }
        const int all_hi = P.causal ? span.len - P.T + 1 : span.len;
        const int all_lo = P.window > 0 ? span.len - P.window : 0;

        // Stages [open, close) see every key, whatever the row.
        const int pos0 = blk0 * 16;
        constexpr int step = BPS * 16;
        const int open = all_lo > pos0 ? (all_lo - pos0 + step - 1) / step : 0;
        const int close = all_hi >= pos0 + 16 * BPS ? (all_hi - 16 * BPS - pos0) / step + 1 : 0;
        int left = 0;   // copies in flight where a wait gave up
        for (int i = 0; i < n; ++i) {
            if ((i & (PER - 1)) == 0) bad = bad_next;
            if (__any_sync(0xffffffffu, !mbar_try_wait(bars + 8 * slot, parity)))
                if (!mbar_wait_warp(bars + 8 * slot, parity, &sh_abort)) {
                    ok = false;
                    left = min(ST, n - i);
                    break;
                }
            const uint8_t* blk = ring + slot * Cfg::STAGE;
            if (i >= open && i < close && bad == 0) {
#pragma unroll 1
                for (int k = 0; k < BPS; k += STEP)
                    kv4_step<D, ROWS, STEP, false>(blk + k * Cfg::BLOCK, Q, S, 0, 0, lo, hi);
            } else {
#pragma unroll 1
                for (int k = 0; k < BPS; k += MSTEP) {
                    const int pos = pos0 + i * step + 16 * k;
                    if (pos >= span.len) break;
                    const uint32_t gone = bad >> ((i * BPS + k) & 31);
                    kv4_step<D, ROWS, MSTEP, true>(blk + k * Cfg::BLOCK, Q, S, pos, gone, lo, hi);
                }
            }
            __syncwarp();   // all lanes have read the slot
            if ((i & 3) == 3) kv4_center(S);
            if (i + ST < n) {
                if (((i + ST) & (PER - 1)) == 0) lookup(i + ST);
                issue(i + ST, slot);
            }
            if (++slot == ST) {
                slot = 0;
                parity ^= 1;
            }
        }
        if (!ok) {
            // a wait gave up: let this warp's copies land before the CTA's memory goes
            for (; left > 0; --left) {
                mbar_wait_drain(bars + 8 * slot, parity);
                if (++slot == ST) {
                    slot = 0;
                    parity ^= 1;
                }
            }
            break;
        }

        // ---- the end of a segment: the lanes' shares of the sums
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    S.l[nt][c] += __shfl_xor_sync(0xffffffffu, S.l[nt][c], off);
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
                        S.z[nt][i][c] += __shfl_xor_sync(0xffffffffu, S.z[nt][i][c], off);
                        S.ps[nt][i][c] += __shfl_xor_sync(0xffffffffu, S.ps[nt][i][c], off);
                    }
                }
            }
        const int4 part = make_int4(first, b, u, span.n);
        if (at == first && stop == first + span.n) {   // a whole unit
            const int64_t row0 = (static_cast<int64_t>(b) * P.Hq + h * (P.Hq / P.C.Hkv)) * P.T + rb * ROWS;
            kv4_rows_of(S, [&](int r, int d, const float (&x)[8], float m, float l) {
                if (rb * ROWS + r >= P.rows) return;
                const float inv = l == 0.f ? 0.f : 1.f / l;
                if (P.o) {
                    uint4 y;
                    y.x = pack_bf16(x[0] * inv, x[1] * inv);
                    y.y = pack_bf16(x[2] * inv, x[3] * inv);
                    y.z = pack_bf16(x[4] * inv, x[5] * inv);
                    y.w = pack_bf16(x[6] * inv, x[7] * inv);
                    *reinterpret_cast<uint4*>(P.o + (row0 + r) * D + d) = y;
                } else {
                    float4* dst = reinterpret_cast<float4*>(P.o_part + (row0 + r) * D + d);
                    dst[0] = make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
                    dst[1] = make_float4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
                }
                if (d == 0) P.lse[row0 + r] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            });
        } else if (stop == end) {
            kept = true;
            if (lane == 0) sh_part[2 * warp + 1] = part;
        } else {
            kv4_store_part(S, parked + warp * Cfg::PART);
            if (lane == 0) sh_part[2 * warp] = part;
        }
        at = stop;
    }

    // ---- join the warps' parts of each unit, in the order of the tiles
    __syncthreads();   // every warp is done with its ring
    if (sh_abort) return;
    float* parts = reinterpret_cast<float*>(sm);
    if (kept) kv4_store_part(S, parts + warp * Cfg::PART);
    if (warp == 0) {
        // entries of one unit: kept parts (bits 2 warp + 1 of y) and then a parked one (of warp z), if any
        const int x = lane < 2 * W ? sh_part[lane].x : -1;
        const uint32_t all = __ballot_sync(0xffffffffu, x >= 0), below = (1u << lane) - 1;
        const int prev = __shfl_sync(0xffffffffu, x, 31 - __clz(all & below | 1u));
        const bool leads = x >= 0 && ((all & below) == 0 || prev != x);
        const uint32_t leaders = __ballot_sync(0xffffffffu, leads), after = leaders & ~below & ~(1u << lane);
        const uint32_t mine = all & ~below & (after ? (after & -after) - 1 : 0xffffffffu);
        const uint32_t kept_parts = mine & 0xaaaaaaaau, parked = mine & 0x55555555u;
        if (leads)
            sh_group[__popc(leaders & below)] =
                make_int4(lane, static_cast<int>(kept_parts), parked ? __ffs(parked) >> 1 : -1, 0);
        if (lane == 0) sh_groups = __popc(leaders);
    }
    __syncthreads();
    for (int at = threadIdx.x; at < sh_groups * (ROWS * D / 4); at += W * 32) {
        const int k = at / (ROWS * D / 4), i = at - k * (ROWS * D / 4), r = i / (D / 4), d = (i - r * (D / 4)) * 4;
        const int4 group = sh_group[k], unit = sh_part[group.x];
        const int b = unit.y, h = P.by_row_blocks.of(unit.z), rb = unit.z - h * P.row_blocks;
        const bool begins = unit.x >= cta0, ends = unit.x + unit.w <= cta1;
        if (begins && !ends && i == 0)
            P.jobs[blockIdx.x] = make_int4(
                b, h, rb, Kv4Split(total, ctas * W).taker(unit.x + unit.w - 1) / W - static_cast<int>(blockIdx.x) + 1);
        if (rb * ROWS + r >= P.rows) continue;
        const float* src[W + 1];
        float2 ml[W + 1];
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w <= W; ++w) {
            const bool is = w < W ? (group.y >> (2 * w + 1)) & 1 : group.z >= 0;
            src[w] = w < W ? parts + w * Cfg::PART : parked + max(group.z, 0) * Cfg::PART;
            ml[w] = is ? *reinterpret_cast<const float2*>(src[w] + ROWS * Cfg::O_LD + 2 * r) : make_float2(0.f, 0.f);
            if (ml[w].y != 0.f) m = fmaxf(m, ml[w].x);   // l = 0: no key there
        }
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w <= W; ++w) {
            if (ml[w].y == 0.f) continue;
            const float f = ex2(ml[w].x - m);
            const float4 x = *reinterpret_cast<const float4*>(src[w] + r * Cfg::O_LD + d);
            l = fmaf(f, ml[w].y, l);
            o.x = fmaf(f, x.x, o.x); o.y = fmaf(f, x.y, o.y); o.z = fmaf(f, x.z, o.z); o.w = fmaf(f, x.w, o.w);
        }
        if (begins && ends) {
            const int64_t row = (static_cast<int64_t>(b) * P.Hq + h * (P.Hq / P.C.Hkv)) * P.T + rb * ROWS + r;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            if (P.o)
                *reinterpret_cast<uint2*>(P.o + row * D + d) =
                    make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
            else
                *reinterpret_cast<float4*>(P.o_part + row * D + d) =
                    make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
            if (d == 0) P.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        } else {
            // a unit that began before goes to slot 2c, one that begins here and runs on to 2c + 1
            float* to = P.slots + (2 * static_cast<int64_t>(blockIdx.x) + (begins ? 1 : 0)) * ROWS * (D + 2);
            *reinterpret_cast<float4*>(to + r * D + d) = o;
            if (d == 0) *reinterpret_cast<float2*>(to + ROWS * D + 2 * r) = make_float2(m, l);
        }
    }
}

// Joins the partials of the unit that begins in CTA blockIdx.x's share and runs on into the next CTAs':
// WPR warps a row, a batch of parts in flight in each, then one row at a time through shared memory.
template <int ROWS>
constexpr int KV4_MERGE_WARPS = ROWS == 16 ? 16 : 8;   // few: they find room beside the kernel before

template <int D, int ROWS>
__global__ void __launch_bounds__(KV4_MERGE_WARPS<ROWS> * 32, ROWS == 16 ? 2 : 4) kv4_merge_kernel(Kv4AttnParams P)
{
    constexpr int W = KV4_MERGE_WARPS<ROWS>, WPR = W / ROWS, V = D / 32, U = D == 256 ? 4 : 8;
    __shared__ float sh_o[W][D];
    __shared__ float2 sh_ml[W];
    // every CTA waits, also those with nothing to join: the grid must not be over before the first one
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 job = P.jobs[blockIdx.x];   // written by the kernel before
    const int parts = job.w;
    if (parts == 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = warp / WPR, w0 = warp % WPR;
    const bool live = job.z * ROWS + r < P.rows;
    float m = -INFINITY, l = 0.f, o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = 0.f;
    const float* slots = P.slots + static_cast<int64_t>(blockIdx.x) * 2 * ROWS * (D + 2);
    for (int i0 = w0; live && i0 < parts; i0 += U * WPR) {
        float2 ml[U];
        float x[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * WPR;
            ml[u] = make_float2(0.f, 0.f);
            if (i >= parts) continue;
            // part 0 in slot 2c + 1 of this CTA, the others in slots 2c of the next ones
            const int part = (2 * i + (i == 0 ? 1 : 0)) * ROWS * (D + 2);
            ml[u] = *reinterpret_cast<const float2*>(slots + part + ROWS * D + 2 * r);
            const float* src = slots + part + r * D + lane * V;
#pragma unroll
            for (int v = 0; v < V; v += 2) {
                const float2 y = *reinterpret_cast<const float2*>(src + v);
                x[u][v] = y.x;
                x[u][v + 1] = y.y;
            }
        }
        float top = m;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (ml[u].y != 0.f) top = fmaxf(top, ml[u].x);   // l = 0: no key there
        const float f = l == 0.f ? 0.f : ex2(m - top);
        m = top;
        l *= f;
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] *= f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (ml[u].y == 0.f) continue;
            const float e = ex2(ml[u].x - m);
            l = fmaf(e, ml[u].y, l);
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] = fmaf(e, x[u][v], o[v]);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) sh_o[warp][lane * V + v] = o[v];
    if (lane == 0) sh_ml[warp] = make_float2(m, l);
    __syncthreads();
    const int G = P.Hq / P.C.Hkv;
    for (int i = threadIdx.x; i < ROWS * D; i += W * 32) {
        const int row = i / D, d = i - row * D;
        if (job.z * ROWS + row >= P.rows) break;
        float top = -INFINITY, sum = 0.f, y = 0.f;
#pragma unroll
        for (int w = 0; w < WPR; ++w)
            if (sh_ml[row * WPR + w].y != 0.f) top = fmaxf(top, sh_ml[row * WPR + w].x);
#pragma unroll
        for (int w = 0; w < WPR; ++w) {
            const float2 ml = sh_ml[row * WPR + w];
            if (ml.y == 0.f) continue;
            const float e = ex2(ml.x - top);
            sum = fmaf(e, ml.y, sum);
            y = fmaf(e, sh_o[row * WPR + w][d], y);
        }
        const int64_t at = (static_cast<int64_t>(job.x) * P.Hq + job.y * G) * P.T + job.z * ROWS + row;
        y *= sum == 0.f ? 0.f : 1.f / sum;
        if (P.o)
            P.o[at * D + d] = __float2bfloat16_rn(y);
        else
            P.o_part[at * D + d] = y;
        if (d == 0) P.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    }
}

}  // namespace cpattn
