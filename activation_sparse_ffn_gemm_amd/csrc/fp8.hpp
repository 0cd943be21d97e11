// Device helpers of the 8-bit (e4m3) matrices and of the row-wise kernels
// that write them: rows of any length and alignment in float32 or bfloat16,
// held in registers as chunks of eight elements per lane.
#pragma once

#include "common.hpp"

// twell_fp8_t: a scale for each FP8_BLK columns; |q| <= FP8_MAX (the largest
// finite e4m3 value); amax is taken as at least FP8_AMAX_MIN, so a block of
// zeros has a positive scale and no scale is denormal.
constexpr int FP8_BLK = TWELL_FP8_BLOCK;
constexpr float FP8_MAX = 448.f;
constexpr float FP8_AMAX_MIN = 0x1p-64f;

__host__ __device__ inline int fp8_blocks(int cols) { return (int)(((int64_t)cols + FP8_BLK - 1) / FP8_BLK); }
__host__ __device__ inline int64_t fp8_pitch(int cols) { return (int64_t)fp8_blocks(cols) * FP8_BLK; }

// Four values to four e4m3 bytes, nearest, ties to even (low byte first).
DEVI uint32_t f32x4_to_e4m3x4(float a, float b, float c, float d)
{
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

// Maximum over each group of 16 lanes, in every lane of the group (DPP moves
// within the 16-lane rows, as in wave_sum). Used on the bits of absolute
// values: as integers these order like the floats, with infinity above every
// finite value and NaN above infinity, so a NaN in a block reaches its scale.
DEVI uint32_t row16_umax(uint32_t v)
{
    auto step = [&](uint32_t o) { v = o > v ? o : v; };
    step((uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));
    step((uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));
    step((uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false));
    step((uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false));
    return v;
}

// Scale of a block from the bits of its largest absolute value, and a little
// over 1 / scale (2^-22 to 2^-20 of it). The scale is amax / 448 rounded once:
// the product's error is one fused step away (amax - q 448 is exact in the
// fused multiply-add). An infinite or NaN amax is the scale itself: it makes
// NaN of every code, zero among them. The codes are those of 1 / scale = 0
// then: NaN where the element is not finite, zeros elsewhere and past the edges.
struct BlockScale {
    float s, inv; // as e4m3_quotient takes them
    float held;   // the scale as it is stored
};
DEVI BlockScale fp8_scale(uint32_t amax_bits)
{
    const uint32_t lo = __float_as_uint(FP8_AMAX_MIN);
    const float amax = __uint_as_float(amax_bits > lo ? amax_bits : lo);
    const float q = amax * (1.f / FP8_MAX);
    const bool finite = amax_bits < 0x7f800000u;
    BlockScale b;
    b.s = finite ? fmaf(fmaf(-q, FP8_MAX, amax), 1.f / FP8_MAX, q) : 1.f;
    b.held = finite ? b.s : amax;
    const float y = __builtin_amdgcn_rcpf(b.s);
    b.inv = finite ? fmaf(fmaf(-b.s, y, 1.f + 0x1p-21f), y, y) : 0.f;
    return b;
}

// A float whose e4m3 rounding is that of v / s. The e4m3 values and the ties
// between them are points of a grid, of floats whose low 19 bits are clear. v
// inv is a little past the quotient, so its grid point t is the quotient's
// own, or the next one where the quotient lies just before that; v - t s, whose
// sign the fused multiply-add gives exactly, says which, or that the quotient
// is t. t moved by DELTA to that side is in the quotient's open interval of
// the grid and rounds like it: DELTA is more than half a unit of the largest
// quotients and less than the grid's step wherever a tie is near. Where a
// quotient matters (2^-10 and more) a remainder is 0 or at least 2^-110.
// (Rounding the float quotient instead rounds twice: of bfloat16 values over a
// bfloat16 amax, one in 250 lies that near to a tie.)
DEVI float e4m3_quotient(float v, BlockScale b)
{
    constexpr float DELTA = 0x1.8p-16f, SMALL = 0x1p-120f;
    const float t = __uint_as_float(__float_as_uint(v * b.inv) & 0xfff80000u);
    const float rest = __builtin_amdgcn_fmed3f(fmaf(-t, b.s, v), -SMALL, SMALL);
    return fmaf(rest, DELTA / SMALL, t);
}
DEVI uint32_t quant4(const float *v, BlockScale b)
{
    return f32x4_to_e4m3x4(e4m3_quotient(v[0], b), e4m3_quotient(v[1], b),
                           e4m3_quotient(v[2], b), e4m3_quotient(v[3], b));
}
DEVI uint2 quant8(const float *v, BlockScale b)
{
    return make_uint2(quant4(v, b), quant4(v + 4, b));
}

// Eight quotients in 64 bits, each to its nearest e4m3 value. Where a float32
// of one lies on a tie (its low 19 bits clear: seldom) and the quotient does
// not, the float is moved to the odd one of the two around the quotient, which
// is no tie and has the same neighbours.
DEVI uint2 quant8(const double *y)
{
    constexpr uint32_t TIE_BITS = 0x7ffff;
    float q[8];
    uint32_t low = TIE_BITS;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        q[i] = (float)y[i];
        const uint32_t t = __float_as_uint(q[i]) & TIE_BITS;
        low = t < low ? t : low;
    }
    if (low == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const double r = (double)q[i];
            if (y[i] != r)
                q[i] = __uint_as_float((__float_as_uint(q[i]) - (fabs(y[i]) < fabs(r))) | 1u);
        }
    }
    return make_uint2(f32x4_to_e4m3x4(q[0], q[1], q[2], q[3]),
                      f32x4_to_e4m3x4(q[4], q[5], q[6], q[7]));
}

// ---- rows of any alignment
// 16 bytes at an address that is only element-aligned: gfx950 takes unaligned
// vector accesses, so one instruction serves every row stride.
struct __attribute__((packed, aligned(2), may_alias)) bytes16 {
    uint32_t x, y, z, w;
};
DEVI uint4 ldg16u(const void *p)
{
    const bytes16 v = *(const bytes16 *)p;
    return make_uint4(v.x, v.y, v.z, v.w);
}
DEVI void stg16u(void *p, uint4 v)
{
    *(bytes16 *)p = bytes16{v.x, v.y, v.z, v.w};
}

// The same for results that are written once and not read here: they do not
// stay in L2, whose lines would otherwise be evicted one by one behind the
// loads. Measured on buffers in turn, with it and without: product of 8192 x
// 5632 over 2048 90.5 and 100.7 us, quantisation of 8192 x 2048 both ways 14.0
// and 15.6, norm of 8192 x 2048 29.0 and 31.3; a product that reads them next
// takes the same time. The norm's backward loses as often as it gains and keeps
// the ordinary store; loads of this kind are slower (norm 30.4).
typedef uint32_t u32x4u_t __attribute__((ext_vector_type(4), aligned(2), may_alias));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2), may_alias));
DEVI void stg16u_nt(void *p, uint4 v)
{
    __builtin_nontemporal_store(u32x4u_t{v.x, v.y, v.z, v.w}, (u32x4u_t *)p);
}
DEVI void stg8_nt(void *p, uint2 v)
{
    __builtin_nontemporal_store(u32x2_t{v.x, v.y}, (u32x2_t *)p);
}

// A row of d elements spread over LPR lanes: lane l holds elements
// 8 (l + LPR c) .. + 7 for c < C, zeros past d. Loads leave the raw bits in
// the registers (bf16: the first four words), so that the loads of several
// arrays are in flight together; widen() makes them floats in place.
// FULL: every lane has its elements, and loads are not tested (a row that is
// not there is the caller's to avoid); EIGHTS: some lanes may have none;
// RAGGED: d is no multiple of eight, and one lane's last chunk is cut.
enum RowKind { FULL, EIGHTS, RAGGED };
template <int LPR, int C, RowKind KIND> struct Row {
    static constexpr bool RAG = KIND == RAGGED;
    float v[C][8];

    DEVI void put(int c, int i, uint4 q)
    {
        v[c][i] = __uint_as_float(q.x), v[c][i + 1] = __uint_as_float(q.y);
        v[c][i + 2] = __uint_as_float(q.z), v[c][i + 3] = __uint_as_float(q.w);
    }
    DEVI uint4 bits(int c, int i) const
    {
        return make_uint4(__float_as_uint(v[c][i]), __float_as_uint(v[c][i + 1]),
                          __float_as_uint(v[c][i + 2]), __float_as_uint(v[c][i + 3]));
    }

    DEVI void load(const void *row, int dt, int d, int lane)
    {
        uint4 q[C], r[C]; // r: the second half of a float32 chunk
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (KIND != FULL)
                q[c] = r[c] = make_uint4(0, 0, 0, 0);
        if (dt == TWELL_BF16) {
            const uint16_t *p = (const uint16_t *)row;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int j = 8 * (lane + LPR * c);
                if (KIND == FULL || j + 8 <= d) {
                    q[c] = ldg16u(p + j);
                } else if (RAG && j < d) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = (j + 2 * i < d ? p[j + 2 * i] : 0) |
                               (j + 2 * i + 1 < d ? (uint32_t)p[j + 2 * i + 1] << 16 : 0);
                    q[c] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        } else {
            const uint32_t *p = (const uint32_t *)row;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int j = 8 * (lane + LPR * c);
                if (KIND == FULL || j + 8 <= d) {
                    q[c] = ldg16u(p + j);
                    r[c] = ldg16u(p + j + 4);
                } else if (RAG && j < d) {
                    uint32_t w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        w[i] = j + i < d ? p[j + i] : 0;
                    q[c] = make_uint4(w[0], w[1], w[2], w[3]);
                    r[c] = make_uint4(w[4], w[5], w[6], w[7]);
                }
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            put(c, 0, q[c]);
            if (KIND != FULL || dt != TWELL_BF16)
                put(c, 4, r[c]); // (FULL has none for bf16)
        }
    }

    // floats from the raw bits
    DEVI void widen(int dt)
    {
        if (dt == TWELL_BF16) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const uint4 q = bits(c, 0);
                v[c][0] = bf16_lo(q.x), v[c][1] = bf16_hi(q.x);
                v[c][2] = bf16_lo(q.y), v[c][3] = bf16_hi(q.y);
                v[c][4] = bf16_lo(q.z), v[c][5] = bf16_hi(q.z);
                v[c][6] = bf16_lo(q.w), v[c][7] = bf16_hi(q.w);
            }
        }
    }

    // bf16: rounded to nearest, ties to even
    template <bool NT> DEVI void store(void *row, int dt, int d, int lane) const
    {
        auto put16 = [](void *p, uint4 v) { NT ? stg16u_nt(p, v) : stg16u(p, v); };
        if (dt == TWELL_BF16) {
            uint16_t *p = (uint16_t *)row;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int j = 8 * (lane + LPR * c);
                const uint4 q = make_uint4(
                    f32x2_to_bf16x2(v[c][0], v[c][1]), f32x2_to_bf16x2(v[c][2], v[c][3]),
                    f32x2_to_bf16x2(v[c][4], v[c][5]), f32x2_to_bf16x2(v[c][6], v[c][7]));
                if (j + 8 <= d) {
                    put16(p + j, q);
                } else if (RAG && j < d) {
                    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int i = 0; i < 7; ++i)
                        if (j + i < d)
                            p[j + i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
                }
            }
        } else {
            float *p = (float *)row;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int j = 8 * (lane + LPR * c);
                if (j + 8 <= d) {
                    put16(p + j, bits(c, 0));
                    put16(p + j + 4, bits(c, 4));
                } else if (RAG && j < d) {
#pragma unroll
                    for (int i = 0; i < 7; ++i)
                        if (j + i < d)
                            p[j + i] = v[c][i];
                }
            }
        }
    }
};

// Element address of row r of a matrix of leading dimension ld.
DEVI const void *row_ptr(const void *p, int dt, int64_t ld, int64_t r)
{
    return (const uint8_t *)p + r * ld * (dt == TWELL_BF16 ? 2 : 4);
}
DEVI void *row_ptr(void *p, int dt, int64_t ld, int64_t r)
{
    return (uint8_t *)p + r * ld * (dt == TWELL_BF16 ? 2 : 4);
}
