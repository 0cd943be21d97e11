// Device helpers of the 4-bit (e2m1) matrices: codes, scales and the layout
// that the kernels of fp4_*.hip share.
#pragma once

#include "fp8.hpp" // rows of any alignment
#include "ntgemm.hpp"

constexpr int FP4_BLK = TWELL_FP4_BLOCK;
constexpr int FP4_BYTES = FP4_BLK / 2; // bytes of a row's block of columns
constexpr float FP4_MAX = 6.f;
constexpr float FP4_AMAX_MIN = 0x1p-64f, FP4_AMAX_MAX = 0x1p127f;

__host__ __device__ inline int fp4_blocks(int cols) { return (int)(((int64_t)cols + FP4_BLK - 1) / FP4_BLK); }
__host__ __device__ inline int64_t fp4_pitch(int cols) { return (int64_t)fp4_blocks(cols) * FP4_BYTES; }

// A 4-bit matrix as the kernels take it.
struct Fp4 {
    const uint8_t *q;
    const uint16_t *scale;
    int64_t pitch; // bytes of a row
    int rows, cols, nkb, group;
};
inline Fp4 fp4_arg(const twell_fp4_t *m)
{
    return {m->q, m->scale, fp4_pitch(m->cols), m->rows, m->cols, fp4_blocks(m->cols), m->group};
}

// Eight codes (low half of the low byte first) as bfloat16 values, exactly.
DEVI bf16x8_t fp4x8_to_bf16(uint32_t q)
{
    const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.f, 0);
    const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.f, 1);
    const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.f, 2);
    const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.f, 3);
    return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
// The same as floats.
DEVI void fp4x8_to_f32(uint32_t q, float *v)
{
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 0);
    const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 1);
    const f32x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 2);
    const f32x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 3);
    v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1];
    v[4] = c[0], v[5] = c[1], v[6] = d[0], v[7] = d[1];
}

// Eight elements of a row from column j, zeros past C.
DEVI void load8(const void *row, int dt, int j, int C, float *v)
{
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (dt == TWELL_BF16) {
        const uint16_t *p = (const uint16_t *)row;
        if (j + 8 <= C) {
            a = ldg16u(p + j);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = (j + 2 * i < C ? p[j + 2 * i] : 0) |
                       (j + 2 * i + 1 < C ? (uint32_t)p[j + 2 * i + 1] << 16 : 0);
            a = make_uint4(w[0], w[1], w[2], w[3]);
        }
        elem<TWELL_BF16>::widen(a, v);
    } else {
        const uint32_t *p = (const uint32_t *)row;
        if (j + 8 <= C) {
            a = ldg16u(p + j), b = ldg16u(p + j + 4);
        } else {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i] = j + i < C ? p[j + i] : 0;
            a = make_uint4(w[0], w[1], w[2], w[3]), b = make_uint4(w[4], w[5], w[6], w[7]);
        }
        elem<TWELL_F32>::widen(a, v), elem<TWELL_F32>::widen(b, v + 4);
    }
}

// Activations as the matrix instruction takes them: rows of bfloat16, padded
// with zeros to whole blocks of columns. A bfloat16 matrix whose rows are so
// already (16-byte aligned, whole blocks) is taken where it is. A float32 one
// becomes three rows a row, which add up to it exactly: its leading 8, the next
// 8 and the last 8 bits (cut, not rounded, so none overflows).
struct Acts {
    const uint8_t *data;
    int64_t pitch;     // bytes from a token's first row to the next token's
    int T, planes;     // planes: 1, or 3 rows a token, plane bytes apart
    int nkb;
    int64_t plane;
};
size_t fp4_pack_bytes(const twell_mat_t *x); // 0: taken where it is
Acts fp4_pack(const twell_mat_t *x, void *ws, hipStream_t s, bool *packed);

// The sparse layer's a = g u of an open gate (NaN opens too). A closed gate's is
// the one float that a sum with +0 of two floats is not: -0. The product is rounded
// before the sum, not fused with it: fused, one that underflows from below would
// round to -0 after it.
constexpr uint32_t FP4_CLOSED = 0x80000000u;
DEVI float fp4_act(float g, float u)
{
#pragma clang fp contract(off)
    return !(g <= 0.f) ? g * u + 0.f : __uint_as_float(FP4_CLOSED);
}

// out [T][w.rows] = x w^T for few tokens (any number is right); with up, of w's
// sizes, out is a of w's gates.
void fp4_rows(const Acts &x, const Fp4 &w, const Fp4 *up, void *out, int64_t ldo, int dto,
              hipStream_t s);
// Gates and up products of more tokens: [parts][T][2 wg.rows], parts 0 where
// fp4_rows takes the tokens. wg.rows is a multiple of 128.
int fp4_gates_parts(const twell_mat_t *x, int d_ff);
void fp4_gates(const Acts &x, const Fp4 &wg, const Fp4 &wu, float *parts, hipStream_t s);
