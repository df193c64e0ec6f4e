// The 4-bit K/V cache: its layout, the kernel that quantises rows into it and
// the one that reads them back.
//
// Pages hold page_size tokens (a multiple of 16) of every KV head, uint8
// [num_pages][Hkv][page_size / 16][18 D].  A block of 16 tokens is 18 D bytes:
//   [0, 8D)     codes of K        [8D, 9D)    (scale, zero) of K
//   [9D, 17D)   codes of V        [17D, 18D)  (scale, zero) of V
// Each 64 dims of a row are a group with a bf16 scale and zero (pair index
// row * D/64 + group); a value is zero + scale * code, code 0..15.  Eight codes
// of dims 8o .. 8o+7 (octet o of a row) form one 32-bit word, dim 8o + i at bits
// 4i; the words lie where the attention kernel's lanes read them (kv4_attn.cuh):
//   K  one row after the other; inside a row the octets with o mod 4 = t are
//      contiguous, for lane t of a quad (one 16-byte load at D 128).  At D 256
//      (two loads) odd rows swap the halves, so eight lanes cover every bank.
//   V  by g = o mod 8 (lane group), then by pairs of tokens, so that a lane gets
//      tokens 2t and 2t+1 in one load; the pair index or the token of the
//      pair is flipped by bits of g, again for the banks.
//
// Quantisation: zero = min, scale = bf16((max - min) / 15), code = (x - zero) /
// scale to nearest, ties to even (0 where the scale is below 2^-126).  A group
// with a NaN or an infinity, or whose range overflows, gets a NaN scale: it
// reads back as NaN rather than as something finite.
//
// Both kernels are bound by HBM: 4 D bytes of bf16 and 18 D / 16 of cache a token and
// head.  Four lanes share a token: lane t takes the octets with o mod 4 = t of K and of V, so
// its codes of K are one store, those of V two (octets t and t + 4 of every group), a
// group's minimum and maximum take two shuffles, and what is worked out once a group or a
// token serves eight octets.  (One octet of each a lane, as the first form had it, was
// bound by instruction issue.)  32k tokens of 8 heads of 128 dims: written in 36 us (4.8 TB/s,
// the issue slots 74 % taken; 76 before), read back in 27 (6.3 TB/s; 41 before).
#pragma once
#include <cuda_bf16.h>
#include "exp2_poly.cuh"
#include "ptx.cuh"

namespace cpattn {

// Byte of the word of (row r, octet o) inside the K codes / V codes of a block.
template <int D>
__host__ __device__ __forceinline__ int kv4_k_word(int r, int o)
{
    const int w = o >> 2, t = o & 3;
    if (D == 256) return r * 128 + (((w >> 2) ^ (r & 1)) << 6) + t * 16 + (w & 3) * 4;
    return r * (D / 2) + t * (D / 8) + w * 4;
}

template <int D>
__host__ __device__ __forceinline__ int kv4_v_word(int r, int o)
{
    const int gd = o >> 3, g = o & 7, pair = r >> 1, odd = r & 1;
    if (D == 64) return g * 64 + (pair ^ (((g >> 1) & 1) << 2)) * 8 + odd * 4;
    if (D == 128) return g * 128 + (pair ^ ((g & 1) << 2)) * 16 + odd * 8 + gd * 4;
    return g * 256 + pair * 32 + ((odd ^ (g & 1)) << 4) + gd * 4;
}

constexpr int KV4_ROWS_CTA = 64;   // tokens of a CTA of the kernels that write and read rows

struct Kv4Cache {
    uint8_t* pages;
    const int32_t* table;    // [B][width] page of each page_size tokens
    int32_t B, Hkv, page_size, num_pages, width;
    int64_t page_bytes;      // of one head: page_size / 16 * 18 D
};

// x / d for 0 <= x < 2^31 by a product: mul = ceil(2^(31 + s) / d) with 2^s >= d, so that the quotient is too
// large by less than x / 2^31 / d.
struct Kv4Div {
    uint32_t d, mul, shift;
    __host__ __device__ Kv4Div() : d(1), mul(0), shift(0) {}
    explicit Kv4Div(uint32_t d_) : d(d_), shift(0)
    {
        while ((uint64_t(1) << shift) < d) ++shift;
        mul = static_cast<uint32_t>(((uint64_t(1) << (31 + shift)) + d - 1) / d);
    }
    __device__ __forceinline__ int of(int x) const
    {
        return static_cast<int>(__umulhi(static_cast<uint32_t>(x) << 1, mul) >> shift);
    }
};

struct Kv4RowsParams {
    Kv4Cache C;
    int32_t T;                  // tokens of a sequence at most
    const int32_t* start;       // [B] position of token 0
    const int32_t* counts;      // [B] tokens of each sequence (null: T)
    const int32_t* rows;        // [T] row of token t in k, v (null: t)
    int32_t n_rows;             // rows of k, v
    const __nv_bfloat16 *k_in, *v_in;
    __nv_bfloat16 *k_out, *v_out;
    int64_t ks[3], vs[3];       // strides (batch, head, row) of k_in, v_in in values
    int32_t t_blocks;           // CTAs of a (sequence, head)
    Kv4Div by_t_blocks, by_heads, by_page;   // t_blocks, Hkv, blocks of a page
};

// Token t of sequence b and head h; false where there is nothing to do.
struct Kv4Token {
    int row;          // of k, v
    uint8_t* block;   // its block of 16 tokens
    int r;            // its row of the block
};

template <int D>
__device__ __forceinline__ bool kv4_token(const Kv4RowsParams& P, int b, int h, int t, Kv4Token& k)
{
    if (t >= P.T || (P.counts && t >= P.counts[b])) return false;
    k.row = P.rows ? P.rows[t] : t;
    if (k.row < 0 || k.row >= P.n_rows) {
        record_status(1 /* CP_ERR_INVALID_ARG */);
        return false;
    }
    const int s = P.start[b];
    if (s < 0 || s > 0x7fffffff - t) {
        record_status(1 /* CP_ERR_INVALID_ARG */);
        return false;
    }
    const int pos = s + t, blk = pos >> 4, i = P.by_page.of(blk);
    const int page = i < P.C.width ? P.C.table[static_cast<int64_t>(b) * P.C.width + i] : -1;
    if (page < 0 || page >= P.C.num_pages) {
        record_status(1 /* CP_ERR_INVALID_ARG */);
        return false;
    }
    k.block = P.C.pages + (static_cast<int64_t>(page) * P.C.Hkv + h) * P.C.page_bytes +
              static_cast<int64_t>(blk - i * (P.C.page_size >> 4)) * (18 * D);
    k.r = pos & 15;
    return true;
}

// What the four lanes of a group make of its 64 values (h: the lane's 16): its zero and 1 / scale, and (scale, zero) as
// two bf16.
struct Kv4Group {
    float zero, scale, inv;
    uint32_t meta;
};

__device__ __forceinline__ Kv4Group kv4_group(const uint32_t (&w)[8])
{
    __nv_bfloat162 h[8];
    memcpy(h, w, 32);
    // NaN-propagating packed minimum and maximum, then (min, -max) of the group by shuffles
    __nv_bfloat162 lo2 = h[0], hi2 = h[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo2 = __hmin2_nan(lo2, h[i]);
        hi2 = __hmax2_nan(hi2, h[i]);
    }
    __nv_bfloat162 mm = __halves2bfloat162(__hmin_nan(lo2.x, lo2.y), __hneg(__hmax_nan(hi2.x, hi2.y)));
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) mm = __hmin2_nan(mm, __shfl_xor_sync(0xffffffffu, mm, off));
    Kv4Group g;
    g.zero = __low2float(mm);
    const float range = -__high2float(mm) - g.zero;
    // range / 15 by the reciprocal and the exact remainder (Markstein's division)
    constexpr float kInv15 = 1.f / 15.f;
    const float quot = range * kInv15;
    __nv_bfloat16 sb = __float2bfloat16_rn(fmaf(fmaf(-quot, 15.f, range), kInv15, quot));
    g.scale = __bfloat162float(sb);
    if (!(g.scale >= 1.17549435e-38f)) {   // below 2^-126: one value (or NaN, handled next)
        sb = __float2bfloat16_rn(0.f);
        g.scale = 0.f;
    }
    if (!(range <= 3.402823466e38f)) {   // NaN or infinite
        sb = __ushort_as_bfloat16(0x7fc0);
        g.scale = 0.f;
    }
    g.inv = g.scale > 0.f ? __fdividef(1.f, g.scale) : 0.f;   // 2 ulp
    g.meta = static_cast<uint32_t>(__bfloat16_as_ushort(sb)) | (static_cast<uint32_t>(__bfloat16_as_ushort(mm.x)) << 16);
    return g;
}

// Codes of eight values.  The quotient d / scale by the reciprocal and one correction by its exact remainder is right to
// half a step (a little more where it is next to the middle of two), and exact where it is an integer and a half;
// adding 1.5 * 2^23 rounds it to the nearest integer, ties to even, and leaves that in the low bits.  (A quotient that
// is no tie can only round to one if d = x - zero takes more than 20 bits: values some 2^12 apart.)
__device__ __forceinline__ uint32_t kv4_codes(const uint32_t* w, const Kv4Group& g)
{
    const uint64_t nz = f2_pack(-g.zero, -g.zero), inv = f2_pack(g.inv, g.inv), ns = f2_pack(-g.scale, -g.scale);
    const uint64_t big = f2_pack(12582912.f, 12582912.f);   // 0x4b400000
    uint32_t codes = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
        const uint64_t d = f2_add(f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)), nz);
        const uint64_t q = f2_mul(d, inv), m = f2_add(f2_fma(f2_fma(q, ns, d), inv, q), big);
        codes = (codes * 16u + static_cast<uint32_t>(m >> 32)) * 16u + static_cast<uint32_t>(m);
    }
    return g.scale > 0.f ? codes - 0x4b400000u * 0x11111111u : 0u;
}

// CTA blockIdx.x: tokens from t0 on of sequence b and head h.
template <int D>
__device__ __forceinline__ void kv4_where(const Kv4RowsParams& P, int& b, int& h, int& t0)
{
    const int bh = P.by_t_blocks.of(blockIdx.x);
    b = P.by_heads.of(bh);
    h = bh - b * P.C.Hkv;
    t0 = (blockIdx.x - bh * P.t_blocks) * KV4_ROWS_CTA;
}

template <int D>
__global__ void __launch_bounds__(KV4_ROWS_CTA * 4) kv4_write_kernel(Kv4RowsParams P)
{
    constexpr int NW = D / 32, NG = D / 64;   // words (octets) of a lane, groups
    grid_ahead();
    int b, h, t0;
    kv4_where<D>(P, b, h, t0);
    const int t = threadIdx.x & 3;
    Kv4Token k;
    const bool live = kv4_token<D>(P, b, h, t0 + static_cast<int>(threadIdx.x >> 2), k);
    // K, then V: one of them in registers at a time leaves room for twice the warps
#pragma unroll 1
    for (int kv = 0; kv < 2; ++kv) {
        uint32_t x[4 * NW];   // octets 4w + t
        if (live) {
            const uint4* src = reinterpret_cast<const uint4*>(
                kv ? P.v_in + b * P.vs[0] + h * P.vs[1] + k.row * P.vs[2] : P.k_in + b * P.ks[0] + h * P.ks[1] + k.row * P.ks[2]);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const uint4 y = src[4 * w + t];
                x[4 * w] = y.x; x[4 * w + 1] = y.y; x[4 * w + 2] = y.z; x[4 * w + 3] = y.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4 * NW; ++i) x[i] = 0;
        }
        // every lane takes the shuffles; the lanes of a token are live together
        uint32_t c[NW], meta[NG];
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            uint32_t g[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = x[8 * i + j];
            const Kv4Group q = kv4_group(g);
            c[2 * i] = kv4_codes(g, q);
            c[2 * i + 1] = kv4_codes(g + 4, q);
            meta[i] = q.meta;
        }
        if (!live) continue;
        uint8_t* to = k.block + kv * 9 * D;
        if (kv == 0) {
            if constexpr (D == 64) {
                *reinterpret_cast<uint2*>(to + kv4_k_word<D>(k.r, t)) = make_uint2(c[0], c[1]);
            } else {
#pragma unroll
                for (int i = 0; i < NW; i += 4)
                    *reinterpret_cast<uint4*>(to + kv4_k_word<D>(k.r, t + 4 * i)) =
                        make_uint4(c[i], c[i + 1], c[i + 2], c[i + 3]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {   // octets t and t + 4 of every group
                uint8_t* at = to + kv4_v_word<D>(k.r, t + 4 * i);
                if constexpr (D == 64)
                    *reinterpret_cast<uint32_t*>(at) = c[i];
                else if constexpr (D == 128)
                    *reinterpret_cast<uint2*>(at) = make_uint2(c[i], c[2 + i]);
                else
                    *reinterpret_cast<uint4*>(at) = make_uint4(c[i], c[2 + i], c[4 + i], c[6 + i]);
            }
        }
#pragma unroll
        for (int i = 0; i < NG; ++i)   // lane t writes the pair of group t
            if (t == i) *reinterpret_cast<uint32_t*>(to + 8 * D + (k.r * NG + i) * 4) = meta[i];
    }
}

// Eight values of a word of codes.
__device__ __forceinline__ uint4 kv4_values(uint32_t codes, uint32_t meta)
{
    const float s = __uint_as_float(meta << 16), z = __uint_as_float(meta & 0xffff0000u);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)   // 2^23 + code, less 2^23
        x[i] = fmaf(__uint_as_float(((codes >> (4 * i)) & 15u) | 0x4b000000u) - 8388608.f, s, z);
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

template <int D>
__global__ void __launch_bounds__(KV4_ROWS_CTA * 4) kv4_read_kernel(Kv4RowsParams P)
{
    constexpr int NW = D / 32, NG = D / 64;
    grid_ahead();
    int b, h, t0;
    kv4_where<D>(P, b, h, t0);
    const int t = threadIdx.x & 3;
    Kv4Token k;
    if (!kv4_token<D>(P, b, h, t0 + static_cast<int>(threadIdx.x >> 2), k)) return;
    const uint8_t *kc = k.block, *vc = k.block + 9 * D;
    uint32_t code[2][NW], meta[2][NG];
    if constexpr (D == 64) {
        const uint2 y = *reinterpret_cast<const uint2*>(kc + kv4_k_word<D>(k.r, t));
        code[0][0] = y.x; code[0][1] = y.y;
        code[1][0] = *reinterpret_cast<const uint32_t*>(vc + kv4_v_word<D>(k.r, t));
        code[1][1] = *reinterpret_cast<const uint32_t*>(vc + kv4_v_word<D>(k.r, t + 4));
    } else {
#pragma unroll
        for (int i = 0; i < NW / 4; ++i) {
            const uint4 y = *reinterpret_cast<const uint4*>(kc + kv4_k_word<D>(k.r, t + 16 * i));
            code[0][4 * i] = y.x; code[0][4 * i + 1] = y.y; code[0][4 * i + 2] = y.z; code[0][4 * i + 3] = y.w;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint8_t* at = vc + kv4_v_word<D>(k.r, t + 4 * i);
            if constexpr (D == 128) {
                const uint2 y = *reinterpret_cast<const uint2*>(at);
                code[1][i] = y.x; code[1][2 + i] = y.y;
            } else {
                const uint4 y = *reinterpret_cast<const uint4*>(at);
                code[1][i] = y.x; code[1][2 + i] = y.y; code[1][4 + i] = y.z; code[1][6 + i] = y.w;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NG; ++i) {
        meta[0][i] = *reinterpret_cast<const uint32_t*>(kc + 8 * D + (k.r * NG + i) * 4);
        meta[1][i] = *reinterpret_cast<const uint32_t*>(vc + 8 * D + (k.r * NG + i) * 4);
    }
    const int64_t at = ((static_cast<int64_t>(b) * P.C.Hkv + h) * P.n_rows + k.row) * (D / 8) + t;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        reinterpret_cast<uint4*>(P.k_out)[at + 4 * w] = kv4_values(code[0][w], meta[0][w / 2]);
        reinterpret_cast<uint4*>(P.v_out)[at + 4 * w] = kv4_values(code[1][w], meta[1][w / 2]);
    }
}

}  // namespace cpattn
