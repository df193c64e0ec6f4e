// Rotary positions on rows of q, k (any tensors [B][heads][rows][D]), one launch
// for up to four tensors.
//
// Pair i of a row (the values i and i + R/2, or 2i and 2i + 1) turns by the
// angle position[axis(i)] * inv_freq[i]:
//   y1 = x1 cos - x2 sin,  y2 = x1 sin + x2 cos,
// and by minus that angle for the gradients (a rotation's transpose).  Values
// from the rotary dim on are copied.  fp32 arithmetic, one rounding to bf16.
//
// The angle.  Only its fraction of a full turn matters, so it is taken in
// 64-bit fixed point: F = frac(inv_freq / 2 pi) * 2^64, and position * F modulo
// 2^64 is that fraction, exact for every int32 position (a far position in fp32
// would lose it: 1e6 * 2^-24 rad).  What it has beyond the nearest quarter turn is taken
// with 24 bits of its own, so that a small sine or cosine is right relative to itself (the
// top 32 bits of the turn were not: 6e-4 of the sine of 2.5e-6 rad).
//
// Bound by HBM (4 bytes a value against 3 flops).  A thread keeps one octet of
// pairs (16 values, two 16-byte vectors) of one token and walks the heads of
// every tensor, four heads' loads in flight, so the angles are computed once a
// token and not once a head; few tokens split the heads over the grid instead.
// 128k tokens of 40 heads of 128 dims: 406 us, 6.6 TB/s.
#pragma once
#include <cuda_bf16.h>
#include "ptx.cuh"

namespace cpattn {

constexpr int ROPE_MAX_BUFS = 4;
constexpr int ROPE_MAX_AXES = 4;

struct RopeParams {
    int32_t B, N, R, n_axes;
    int32_t sec_end[ROPE_MAX_AXES];        // pairs before sec_end[a] turn by axis a
    int32_t inverse, n_bufs, total_heads, heads_per_block, row_base;
    const double* inv_freq;                // [R/2]
    const int32_t* positions;              // null: the row's (document) position
    int64_t pos_batch, pos_axis;           // strides of positions
    int32_t pos_len;                       // rows of positions
    // rows: orig(n) = orig_map ? orig_map[n] : n indexes positions (or, row_base added, is the position);
    // doc_start is by shard row, shard_map ? shard_map[n] : n; in_map: the input's row
    const int32_t *orig_map, *shard_map, *doc_start, *in_map;
    const __nv_bfloat16* in[ROPE_MAX_BUFS];
    __nv_bfloat16* out[ROPE_MAX_BUFS];
    int32_t heads[ROPE_MAX_BUFS];
    int64_t s_batch[ROPE_MAX_BUFS], s_head[ROPE_MAX_BUFS], s_row[ROPE_MAX_BUFS];
    int32_t in_rows;                       // rows of the inputs (bound of in_map)
};

// frac(f / 2 pi) * 2^64 (two-part product: 1 / 2 pi to 106 bits)
__device__ __forceinline__ unsigned long long rope_turns(double f)
{
    constexpr double c_hi = 0.15915494309189535, c_lo = -9.839338337591243e-18;
    const double p = f * c_hi;
    const double e = fma(f, c_hi, -p) + f * c_lo;
    const double fr = p - floor(p);
    const unsigned long long hi = static_cast<unsigned long long>(fr * 18446744073709551616.0);
    return hi + static_cast<unsigned long long>(static_cast<long long>(e * 18446744073709551616.0));
}

// Sine and cosine of |x| <= pi / 4 by their Taylor series: what is left out is x^10 / 11! = 2.2e-9 and x^12 / 12! =
// 1.2e-10 of them at most, below fp32's own 6e-8.
__device__ __forceinline__ void rope_sincos(float x, float& s, float& c)
{
    const float z = x * x;
    float p = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
    p = fmaf(z, p, 1.f / 120.f);
    p = fmaf(z, p, -1.f / 6.f);
    s = fmaf(x * z, p, x);
    p = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
    p = fmaf(z, p, -1.f / 720.f);
    p = fmaf(z, p, 1.f / 24.f);
    p = fmaf(z, p, -0.5f);
    c = fmaf(z, p, 1.f);
}

__device__ __forceinline__ void rope_unpack(const uint4& v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 rope_pack(const float (&x)[8])
{
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// TPR = D / 16 threads a row; HALF: pairs (i, i + R/2), else (2i, 2i + 1).
template <int TPR, bool HALF>
__global__ void __launch_bounds__(256, HALF ? 2 : 4) rope_kernel(RopeParams P)
{
    // Heads in flight.  128k tokens of 40 heads, D 128, half: 405 us with four (126 registers), 410 with two; 24573
    // tokens of 10 heads, D 256, adjacent: 46 us with two and 64 registers, 52 with four.
    constexpr int U = HALF ? 4 : 2;
    grid_ahead();
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t row = idx / TPR;
    const int j = static_cast<int>(idx % TPR);
    if (row >= static_cast<int64_t>(P.B) * P.N) return;
    const int b = static_cast<int>(row / P.N), n = static_cast<int>(row - static_cast<int64_t>(b) * P.N);
    const int octets = P.R / 16;
    const bool turns = j < octets;
    const int v0 = turns && HALF ? j : 2 * j;                 // 16-byte vectors of the row
    const int v1 = turns && HALF ? j + octets : 2 * j + 1;

    int src = n;
    if (P.in_map) {
        src = P.in_map[n];
        if (src < 0 || src >= P.in_rows) {
            record_status(1 /* CP_ERR_INVALID_ARG */);
            return;
        }
    }
    float cs[8], sn[8];
    if (turns) {
        int orig = P.orig_map ? P.orig_map[n] : n;
        if (!P.positions) orig += P.row_base;
        int pos[ROPE_MAX_AXES];
        if (P.positions) {
            if (orig < 0 || orig >= P.pos_len) {
                record_status(1 /* CP_ERR_INVALID_ARG */);
                orig = 0;
            }
#pragma unroll
            for (int a = 0; a < ROPE_MAX_AXES; ++a)
                pos[a] = a < P.n_axes ? P.positions[b * P.pos_batch + a * P.pos_axis + orig] : 0;
        } else {
            if (P.doc_start) orig -= P.doc_start[P.shard_map ? P.shard_map[n] : n];
#pragma unroll
            for (int a = 0; a < ROPE_MAX_AXES; ++a) pos[a] = orig;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int pair = 8 * j + i;
            int p = pos[0];
#pragma unroll
            for (int a = 1; a < ROPE_MAX_AXES; ++a)
                if (a < P.n_axes && pair >= P.sec_end[a - 1]) p = pos[a];
            const unsigned long long t =
                static_cast<unsigned long long>(static_cast<long long>(p)) * rope_turns(P.inv_freq[pair]);
            const unsigned quarter = static_cast<unsigned>((t + (1ull << 61)) >> 62);
            const long long rest = static_cast<long long>(t - (static_cast<unsigned long long>(quarter) << 62));
            float s, c;
            rope_sincos(static_cast<float>(rest) * 3.4061215800865545e-19f, s, c);   // pi 2^-63
            const float a = quarter & 1 ? c : s, b = quarter & 1 ? s : c;
            cs[i] = (quarter + 1) & 2 ? -b : b;
            sn[i] = (quarter & 2) != 0 != (P.inverse != 0) ? -a : a;
        }
    }

    // this block's heads, counted over all tensors
    const int first = blockIdx.y * P.heads_per_block, last = min(first + P.heads_per_block, P.total_heads);
    int off = 0;
    for (int t = 0; t < P.n_bufs; off += P.heads[t], ++t) {
        const int h0 = max(first - off, 0), h1 = min(last - off, P.heads[t]);
        const uint4* in = reinterpret_cast<const uint4*>(P.in[t] + b * P.s_batch[t] + src * P.s_row[t]);
        const int64_t hs = P.s_head[t] / 8;
        uint4* out = reinterpret_cast<uint4*>(P.out[t]) +
                     (static_cast<int64_t>(b) * P.heads[t] * P.N + n) * (2 * TPR);
        const int64_t os = static_cast<int64_t>(P.N) * (2 * TPR);
        for (int h = h0; h < h1; h += U) {
            uint4 a[U], c[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (h + u < h1) {
                    a[u] = in[(h + u) * hs + v0];
                    c[u] = in[(h + u) * hs + v1];
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (h + u >= h1) break;
                if (turns) {
                    float x[8], y[8], p[8], q[8];
                    rope_unpack(a[u], x);
                    rope_unpack(c[u], y);
                    if (HALF) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            p[i] = x[i] * cs[i] - y[i] * sn[i];
                            q[i] = x[i] * sn[i] + y[i] * cs[i];
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            p[2 * i] = x[2 * i] * cs[i] - x[2 * i + 1] * sn[i];
                            p[2 * i + 1] = x[2 * i] * sn[i] + x[2 * i + 1] * cs[i];
                            q[2 * i] = y[2 * i] * cs[4 + i] - y[2 * i + 1] * sn[4 + i];
                            q[2 * i + 1] = y[2 * i] * sn[4 + i] + y[2 * i + 1] * cs[4 + i];
                        }
                    }
                    a[u] = rope_pack(p);
                    c[u] = rope_pack(q);
                }
                out[(h + u) * os + v0] = a[u];
                out[(h + u) * os + v1] = c[u];
            }
        }
    }
}

}  // namespace cpattn
