// Matrices in 4 bits (e2m1) with a scale for each group of 32, 64 or 128
// columns of a row, from float32 or bfloat16, and back.
//
// scale = amax / 6 with amax held within [2^-64, 2^127], rounded to six
// significant bits: three times a number of six bits has eight at most, so each
// of the 15 values times its scale is a bfloat16 number, and a product taken on
// bfloat16 copies is the product of the values themselves. The six bits move
// the largest element by at most 1/64 of it; the step of the codes there is 1/3.
#include "fp4.hpp"

namespace {

// Bits of a float's nearest number of six significant bits, ties to even.
DEVI uint32_t six_bits(float v)
{
    const uint32_t u = __float_as_uint(v);
    return (u + 0x1ffffu + (u >> 18 & 1u)) & 0xfffc0000u;
}

struct GroupScale {
    float s, inv; // inv: a little over 1 / s; 0 where the group is not finite
    uint16_t held; // the scale as it is stored
};
DEVI GroupScale fp4_scale(uint32_t amax_bits)
{
    const bool finite = amax_bits < 0x7f800000u;
    const float amax = fminf(fmaxf(__uint_as_float(finite ? amax_bits : 0u), FP4_AMAX_MIN),
                             FP4_AMAX_MAX);
    GroupScale g;
    const uint32_t bits = six_bits(amax / FP4_MAX);
    g.s = __uint_as_float(bits);
    g.held = finite ? (uint16_t)(bits >> 16) : (uint16_t)0x7fc0;
    const float y = __builtin_amdgcn_rcpf(g.s);
    g.inv = finite ? fmaf(fmaf(-g.s, y, 1.f + 0x1p-21f), y, y) : 0.f;
    return g;
}

// A float that rounds to the e2m1 value nearest to v / s. The values and the
// ties between them are points of a grid, of floats whose low 21 bits are clear
// (1.75, 3.5: three significant bits). v inv lies a little past the quotient, so
// its grid point t is the quotient's own, or the next where the quotient lies
// just before that one; the sign of v - t s, exact in a fused step, says which,
// and t moved to that side rounds like the quotient. (The float quotient would
// be rounded twice.) As e4m3_quotient, on its grid, but for where the minus stands:
// of an exact quotient the rest is -0, and the sum keeps the sign of a zero.
DEVI float e2m1_quotient(float v, GroupScale g)
{
    constexpr float DELTA = 0x1p-16f, SMALL = 0x1p-120f;
    const float t = __uint_as_float(__float_as_uint(v * g.inv) & 0xffe00000u);
    const float rest = __builtin_amdgcn_fmed3f(-fmaf(t, g.s, -v), -SMALL, SMALL);
    return fmaf(rest, DELTA / SMALL, t);
}
DEVI uint32_t quant8_fp4(const float *v, GroupScale g)
{
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, e2m1_quotient(v[0], g), e2m1_quotient(v[1], g), 1.f, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, e2m1_quotient(v[2], g), e2m1_quotient(v[3], g), 1.f, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, e2m1_quotient(v[4], g), e2m1_quotient(v[5], g), 1.f, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, e2m1_quotient(v[6], g), e2m1_quotient(v[7], g), 1.f, 3);
    return g.inv > 0.f ? q : 0u;
}

// Maximum over each LANES (4, 8, 16) neighbouring lanes, in every one of them.
template <int LANES> DEVI uint32_t lanes_umax(uint32_t v)
{
    auto step = [&](uint32_t o) { v = o > v ? o : v; };
    step((uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));
    step((uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));
    if constexpr (LANES >= 8)
        step((uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false));
    if constexpr (LANES >= 16)
        step((uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false));
    return v;
}

struct QuantArgs {
    const void *x;
    int64_t ld;
    int dt, R, C, nkb;
    uint8_t *q;
    uint16_t *scale;
    int64_t pitch, tiles;
    uint32_t grid;
};

// Workgroups of a launch (their threads are numbered in 32 bits): further tiles
// are taken by the same ones. The kernels are told their number: one that asks
// for it gets 256 bytes of arguments more, and a launch costs the host 0.5 us
// more for 150 bytes.
inline uint32_t groups(int64_t tiles) { return (uint32_t)(tiles < 1 << 22 ? tiles : 1 << 22); }

// A workgroup takes QR rows by QB blocks of columns; 16 lanes hold a block of a
// row, eight elements each, and a thread's rows are all in flight. The scales of
// the QR rows, which are neighbours in memory, meet in LDS and are written as runs.
// Bound by memory: 5632 x 2048 float32 in 10.3 us (52.4 MB, 5.1 TB/s), 8192 x 5632 in
// 41 (5.1); tiles of 32 rows, fewer workgroups with the same bytes each, took 14.3.
constexpr int QR = 8, QB = 4;
template <int G> __global__ __launch_bounds__(256) void fp4_quant_kernel(QuantArgs a)
{
    constexpr int NG = FP4_BLK / G; // groups of a block
    __shared__ uint16_t ss[QB * NG][QR];
    const int nbt = (a.nkb + QB - 1) / QB;
    const int l16 = threadIdx.x & 15, sub = threadIdx.x >> 4, cb = sub % QB, rr = sub / QB;
    constexpr int STEP = 16 / QB;
    for (int64_t tile = blockIdx.x; tile < a.tiles; tile += a.grid) {
        const int b0 = (int)(tile % nbt) * QB, b = b0 + cb, j = b * FP4_BLK + l16 * 8;
        const int64_t r0 = tile / nbt * QR;
        if (b < a.nkb) {
            float v[QR / STEP][8]; // (rows past the matrix read its last one)
#pragma unroll
            for (int i = 0; i < QR / STEP; ++i)
                load8(row_ptr(a.x, a.dt, a.ld, min(r0 + i * STEP + rr, (int64_t)a.R - 1)), a.dt, j,
                      a.C, v[i]);
#pragma unroll
            for (int i = 0; i < QR / STEP; ++i) {
                const int64_t r = r0 + i * STEP + rr;
                uint32_t m = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    m = max(m, __float_as_uint(v[i][e]) & 0x7fffffffu);
                const GroupScale g = fp4_scale(lanes_umax<G / 8>(m));
                if (r >= a.R)
                    continue;
                *(uint32_t *)(a.q + r * a.pitch + b * FP4_BYTES + l16 * 4) = quant8_fp4(v[i], g);
                if (l16 % (G / 8) == 0)
                    ss[cb * NG + l16 / (G / 8)][i * STEP + rr] = g.held;
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < QB * NG * QR; i += 256) {
            const int g = i / QR;
            const int64_t r = r0 + i % QR;
            if (r < a.R && b0 + g / NG < a.nkb)
                a.scale[((int64_t)b0 * NG + g) * a.R + r] = ss[g][i % QR];
        }
        __syncthreads();
    }
}

// Row i / n of piece i, n pieces a row: in 32 bits where they do.
DEVI int64_t row_of(int64_t i, int n)
{
    return i >> 32 ? i / n : (int64_t)((uint32_t)i / (uint32_t)n);
}

struct DequantArgs {
    Fp4 w;
    void *out;
    int64_t ld;
    int cn; // pieces of a row
    uint32_t grid;
    int64_t pieces;
};
// One thread takes 16 bytes of results of each of DR rows: eight bfloat16 or four
// float32 columns. Bound by memory: 6144 x 2304 to bfloat16 in 7.4 us (36 MB, 4.9
// TB/s). Threads are numbered over the whole matrix; a launch's threads by rows, a
// second workgroup for the last 32 of 288 pieces, took 8.8. Results go past L2's order.
constexpr int DR = 4;
template <class T> __global__ __launch_bounds__(256) void fp4_dequant_kernel(DequantArgs a)
{
    constexpr int N = 16 / sizeof(T);
    const int shift = 31 - __builtin_clz(a.w.group);
    for (int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x; i0 < a.pieces; i0 += (int64_t)a.grid * 256) {
        const int64_t rg = row_of(i0, a.cn);
        const int j = (int)(i0 - rg * a.cn) * N;
        const int64_t r0 = rg * DR;
        const uint16_t *sc = a.w.scale + (int64_t)(j >> shift) * a.w.rows;
        const uint8_t *q = a.w.q + j / 2;
        uint32_t code[DR];
        uint16_t s[DR];
#pragma unroll
        for (int i = 0; i < DR; ++i) {
            const int64_t r = min(r0 + i, (int64_t)a.w.rows - 1);
            code[i] = N == 8 ? *(const uint32_t *)(q + r * a.w.pitch)
                             : *(const uint16_t *)(q + r * a.w.pitch);
            s[i] = sc[r];
        }
#pragma unroll
        for (int i = 0; i < DR; ++i) {
            const int64_t r = r0 + i;
            if (r >= a.w.rows)
                break;
            float v[8];
            fp4x8_to_f32(code[i], v);
#pragma unroll
            for (int e = 0; e < N; ++e)
                v[e] *= bf16_to_f32(s[i]);
            uint4 u;
            if constexpr (N == 8)
                u = make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]),
                               f32x2_to_bf16x2(v[4], v[5]), f32x2_to_bf16x2(v[6], v[7]));
            else
                u = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]),
                               __float_as_uint(v[2]), __float_as_uint(v[3]));
            T *p = (T *)a.out + r * a.ld + j;
            if (j + N <= a.w.cols) {
                stg16u_nt(p, u);
            } else {
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < N - 1; ++e)
                    if (j + e < a.w.cols)
                        p[e] = (T)(w[e * sizeof(T) / 4] >> (8 * sizeof(T) * e % 32));
            }
        }
    }
}

// Columns 8c .. 8c + 7 of token t (see Acts).
DEVI void pack8(const void *x, int dt, int64_t ld, int64_t t, int c, int C, int nkb, uint8_t *out)
{
    float v[8];
    load8(row_ptr(x, dt, ld, t), dt, c * 8, C, v);
    const int64_t row = (int64_t)nkb * FP4_BLK * 2;
    auto put = [&](int64_t r, const float *f) { // f: bfloat16 numbers
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __float_as_uint(f[2 * i]) >> 16 | (__float_as_uint(f[2 * i + 1]) & 0xffff0000u);
        *(uint4 *)(out + r * row + c * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    };
    if (dt == TWELL_BF16)
        return put(t, v);
    float hi[8], mid[8], lo[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t u = __float_as_uint(v[e]);
        const bool finite = (u & 0x7f800000u) != 0x7f800000u;
        const bool nan = (u & 0x7fffffffu) > 0x7f800000u;
        hi[e] = __uint_as_float((u & 0xffff0000u) | (nan ? 0x400000u : 0u));
        const float r = finite ? v[e] - hi[e] : 0.f;
        mid[e] = __uint_as_float(__float_as_uint(r) & 0xffff0000u);
        lo[e] = r - mid[e];
    }
    put(3 * t, hi), put(3 * t + 1, mid), put(3 * t + 2, lo);
}

// Rows of bfloat16 padded to whole blocks, three rows a float32 row (see Acts). A
// launch and a trip to memory: 333 x 1090 float32 3 to 5 us, 17 x 6144 2.8.
__global__ __launch_bounds__(256) void fp4_pack_kernel(const void *x, int dt, int64_t ld, int C,
                                                       int nkb, int64_t pieces, uint32_t grid, uint8_t *out)
{
    const int n = nkb * (FP4_BLK / 8);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pieces; i += (int64_t)grid * 256) {
        const int64_t t = row_of(i, n);
        pack8(x, dt, ld, t, (int)(i - t * n), C, nkb, out);
    }
}

} // namespace

size_t fp4_pack_bytes(const twell_mat_t *x)
{
    // (the tile kernels address 256 rows by 32-bit offsets)
    const bool bf = x->dtype == TWELL_BF16, near = x->rows == 1 || x->ld < 1 << 23;
    if (bf && near && x->cols % FP4_BLK == 0 && (x->rows == 1 || x->ld % 8 == 0) &&
        (uintptr_t)x->data % 16 == 0)
        return 0;
    return (size_t)x->rows * fp4_blocks(x->cols) * FP4_BLK * 2 * (bf ? 1 : 3);
}

Acts fp4_pack(const twell_mat_t *x, void *ws, hipStream_t s, bool *packed)
{
    const int nkb = fp4_blocks(x->cols), planes = x->dtype == TWELL_BF16 ? 1 : 3;
    const int64_t row = (int64_t)nkb * FP4_BLK * 2;
    *packed = fp4_pack_bytes(x) != 0;
    if (!*packed)
        return {(const uint8_t *)x->data, x->ld * 2, x->rows, 1, nkb, 0};
    const int64_t pieces = (int64_t)nkb * (FP4_BLK / 8) * x->rows;
    const uint32_t grid = groups((pieces + 255) / 256);
    fp4_pack_kernel<<<grid, 256, 0, s>>>(x->data, x->dtype, x->ld, x->cols, nkb, pieces, grid,
                                         (uint8_t *)ws);
    return {(const uint8_t *)ws, row * planes, x->rows, planes, nkb, row};
}

hipError_t launch_fp4_quant(const twell_mat_t *x, const twell_fp4_t *o, twell_timing_t *timing,
                            hipStream_t s)
{
    Timer tm(timing, s);
    QuantArgs a = {x->data, x->ld, x->dtype, x->rows, x->cols, fp4_blocks(x->cols),
                   o->q, o->scale, fp4_pitch(x->cols), 0, 0};
    a.tiles = (int64_t)((a.nkb + QB - 1) / QB) * ((a.R + QR - 1) / QR);
    a.grid = groups(a.tiles);
    if (o->group == 32)
        fp4_quant_kernel<32><<<a.grid, 256, 0, s>>>(a);
    else if (o->group == 64)
        fp4_quant_kernel<64><<<a.grid, 256, 0, s>>>(a);
    else
        fp4_quant_kernel<128><<<a.grid, 256, 0, s>>>(a);
    tm.mark("fp4_quant");
    return hipGetLastError();
}

hipError_t launch_fp4_dequant(const twell_fp4_t *w, const twell_mat_t *out, twell_timing_t *timing,
                              hipStream_t s)
{
    Timer tm(timing, s);
    const int n = out->dtype == TWELL_BF16 ? 8 : 4, cn = (int)(((int64_t)w->cols + n - 1) / n);
    const int64_t pieces = (int64_t)cn * ((w->rows + DR - 1) / DR);
    const DequantArgs a = {fp4_arg(w), out->data, out->ld, cn, groups((pieces + 255) / 256), pieces};
    if (out->dtype == TWELL_BF16)
        fp4_dequant_kernel<uint16_t><<<a.grid, 256, 0, s>>>(a);
    else
        fp4_dequant_kernel<uint32_t><<<a.grid, 256, 0, s>>>(a);
    tm.mark("fp4_dequant");
    return hipGetLastError();
}
