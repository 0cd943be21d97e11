// out = X W^T of activations with weights in 4 bits, and dX = dY W:
//   out[t][n] = sum over groups g of s[g][n] sum_{k in g} x[t][k] c[n][k]
//   dx[t][k]  = sum over n of dy[t][n] s[g(k)][n] c[n][k]
// with c the code's value. Codes are bfloat16 numbers and float32 activations
// are three of them (see Acts), so the bfloat16 matrix instruction forms every
// product exactly; sums are float32.
#include <cmath>
#include <type_traits>

#include "fp4.hpp"
#include "fp4_plan.hpp"

namespace {

struct __attribute__((packed, aligned(2), may_alias)) bytes8 {
    uint32_t x, y;
};

// Eight codes times their scales, each rounded to bfloat16 (exact for scales of
// six bits).
DEVI bf16x8_t scaled8(uint32_t q, const float *s)
{
    float c[8];
    fp4x8_to_f32(q, c);
    return __builtin_bit_cast(bf16x8_t, make_uint4(f32x2_to_bf16x2(c[0] * s[0], c[1] * s[1]),
                                                   f32x2_to_bf16x2(c[2] * s[2], c[3] * s[3]),
                                                   f32x2_to_bf16x2(c[4] * s[4], c[5] * s[5]),
                                                   f32x2_to_bf16x2(c[6] * s[6], c[7] * s[7])));
}
// Two of them: those of byte h.
DEVI uint32_t scaled2(uint32_t q, int h, float lo, float hi)
{
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    const f32x2_t c = h == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 0)
                      : h == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 1)
                      : h == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 2)
                               : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 3);
    return f32x2_to_bf16x2(c[0] * lo, c[1] * hi);
}

// Four results of a row, from column n, as far as N goes.
DEVI void store4(void *out, int dto, int64_t ldo, int64_t row, int n, int N, floatx4_t v)
{
    if (dto == TWELL_BF16) {
        uint16_t *p = (uint16_t *)out + row * ldo + n;
        const uint2 u = make_uint2(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]));
        if (n + 4 <= N) {
            *(bytes8 *)p = bytes8{u.x, u.y};
        } else {
            for (int e = 0; e < 3; ++e)
                if (n + e < N)
                    p[e] = (uint16_t)((e < 2 ? u.x : u.y) >> (16 * (e & 1)));
        }
    } else {
        float *p = (float *)out + row * ldo + n;
        if (n + 4 <= N) {
            stg16u(p, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]),
                                 __float_as_uint(v[2]), __float_as_uint(v[3])));
        } else {
            for (int e = 0; e < 3; ++e)
                if (n + e < N)
                    p[e] = v[e];
        }
    }
}

// ---------------------------------------------------------------- few tokens
// A workgroup computes 16 NB rows of W for up to 16 columns (tokens, or a
// third of a float32 token each), its WV waves taking every WV-th block of 128
// k; their sums meet in LDS. A wave's rows of a block go to its own piece of
// LDS, NST blocks in turn, without a barrier: a wave waits for its own loads.
// The W rows are the instruction's first operand and the activations its
// second: a lane's four results are four rows of one column. A group's sum
// starts from zero and joins the accumulator times the group's scales: codes
// widened as they are (two an instruction) cost a quarter of scaled ones, which
// only many tokens pay back.
// A short product is a launch and two trips to memory (1 x 6144 over 2304 3.9 us);
// a long one is bound by memory (8 x 32768 over 4096, a scale for 32: 17 us, 75.5
// MB, 4.4 TB/s; 1 x 8192 over 8192 9.5 us). In between, on few CUs, by the 28
// vector instructions a set and block: 0.15 us of a wave beside another (2304 over
// 6144 with a scale for 32, 5.9 us; for 128, 4.7).
struct RowsArgs {
    const uint8_t *x;
    int64_t xrow;      // bytes from one column's row to the next
    int T, planes, R;  // R = T planes
    Fp4 w;
    void *out;
    int64_t ldo;
    int dto, tile0; // first tile of rows of this launch
    int tiles;      // tiles of rows of this launch
    int turn;       // log2 of the neighbouring rows that begin at the same block of k
    const uint8_t *q2; // BOTH: the up weights, of w's sizes
    const uint16_t *scale2;
};

// BOTH: of the NB sets of 16 rows every other one is of the sparse layer's up
// weights, the same neurons as the gates before it, and out is its a.
template <int G, int NB, int XR, int WV, int NST, bool BOTH>
__global__ __launch_bounds__(64 * WV) void fp4_rows_kernel(RowsArgs a)
{
    constexpr int STG = NB * 1024 + XR * 256, NG = FP4_BLK / G, MF = G / 32, LPF = NB + XR / 4;
    constexpr int SCB = 128 / NG; // blocks whose scales are staged at a time
    constexpr int BUF = WV * NST * STG;
    static_assert(BUF >= WV * NB * 1024, "the sums reuse the blocks' space");
    static_assert(XR % 4 == 0 && (NST - 1) * LPF < 64 && (NST & (NST - 1)) == 0, "stages");
    __shared__ __attribute__((aligned(16))) uint8_t L[BUF];
    __shared__ __attribute__((aligned(8))) uint16_t ss[SCB * NG][16 * NB];
    const int lane = threadIdx.x & 63, w = wave_id();
    const int l16 = lane & 15, q4 = lane >> 4;
    const int tile = (int)(blockIdx.x % (uint32_t)a.tiles), mt = (int)(blockIdx.x / (uint32_t)a.tiles);
    constexpr int SETS = BOTH ? NB / 2 : NB; // of 16 neurons
    const int n0 = (a.tile0 + tile) * (16 * SETS);
    const int tpt = a.planes == 3 ? 5 : 16; // tokens of a tile
    const int m0 = mt * tpt, c0 = m0 * a.planes;
    // W: lane l loads chunk l % 4 of row l / 4, as the swizzle places it; x: chunk
    // l % 16 of row 4 j + l / 16. Rows past an operand read its last row.
    const uint8_t *srcw = a.w.q + (int64_t)n0 * a.w.pitch, *srcx = a.x + (int64_t)c0 * a.xrow;
    const uint8_t *srcu = BOTH ? a.q2 + (int64_t)n0 * a.w.pitch : nullptr;
    uint32_t off[LPF];
#pragma unroll
    for (int i = 0; i < LPF; ++i) {
        if (i < NB) {
            const int r = (BOTH ? i / 2 : i) * 16 + lane / 4;
            off[i] = (uint32_t)min(r, a.w.rows - 1 - n0) * (uint32_t)a.w.pitch +
                     (((lane & 3) ^ (r >> 2 & 3)) << 4);
        } else {
            const int r = (i - NB) * 4 + lane / 16;
            off[i] = (uint32_t)min(r, a.R - 1 - c0) * (uint32_t)a.xrow + (((lane & 15) ^ r) << 4);
        }
    }
    uint8_t *Lw = L + w * NST * STG;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(ng::lds_u8 *)Lw;
    auto fetch = [&](int kb, int st) {
#pragma unroll
        for (int i = 0; i < LPF; ++i)
            ng::dma16(i < NB ? (BOTH && (i & 1) ? srcu : srcw) + (int64_t)kb * FP4_BYTES
                             : srcx + (int64_t)kb * FP4_BLK * 2,
                      off[i], lds0 + (uint32_t)(st * STG + i * 1024), kb, a.w.nkb);
    };
    floatx4_t acc[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i)
        acc[i] = floatx4_t{0.f, 0.f, 0.f, 0.f};
    const int xr = l16 % XR;
    // Workgroups begin at different blocks: rows whose pitch is a large power of two
    // would otherwise all be read from the same few memory channels at once. It goes
    // by the rows, in runs that do not depend on the number of tokens, and with it the
    // order of a token's sums does not depend on the tokens beside it here.
    const uint32_t turn = (uint32_t)n0 >> a.turn & 7;
    for (int k0 = 0; k0 < a.w.nkb; k0 += SCB) {
        const int nk = min(SCB, a.w.nkb - k0);
        const int n = (nk - w + WV - 1) / WV; // this wave's blocks
        auto block = [&](int i) { // the i-th of them, or none
            const int q = i + (int)(turn * (uint32_t)n >> 3);
            return i < n ? k0 + w + WV * (q < n ? q : q - n) : a.w.nkb;
        };
#pragma unroll
        for (int i = 0; i < NST - 1; ++i)
            fetch(block(i), i);
        if (k0)
            __syncthreads(); // the last scales are used
        for (int q = threadIdx.x; q < nk * NG * 4 * NB; q += 64 * WV) {
            const int g = q / (4 * NB), r = q % (4 * NB) * 4;
            const int i = r / 16, n = n0 + (BOTH ? i / 2 * 16 + r % 16 : r); // set, neuron
            const uint16_t *p = (BOTH && (i & 1) ? a.scale2 : a.w.scale) +
                                ((int64_t)k0 * NG + g) * a.w.rows;
            if (n + 4 <= a.w.rows) {
                const bytes8 v = *(const bytes8 *)(p + n);
                *(uint2 *)&ss[g][r] = make_uint2(v.x, v.y);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    ss[g][r + e] = p[min(n + e, a.w.rows - 1)];
            }
        }
        __syncthreads();
        for (int i = 0; i < n; ++i) {
            const int kc = block(i) - k0;
            fetch(block(i + NST - 1), (i + NST - 1) & (NST - 1));
            ng::wait_vm_steps<LPF, NST - 1>(min(n - 1 - i, NST - 1));
            asm volatile("" ::: "memory");
            const uint8_t *S = Lw + (i & (NST - 1)) * STG, *X = S + NB * 1024 + xr * 256;
            // all of the block's reads, then its products
            uint32_t wq[NB][4];
            bf16x8_t xf[4];
            uint2 sc[NB][NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const int o = g * (G / 2) + q4 * (G / 8);
                    const uint8_t *p = S + b * 1024 + l16 * 64 +
                                       (((o >> 4) ^ (l16 >> 2 & 3)) << 4) + (o & 15);
                    if constexpr (MF == 4) {
                        const uint4 u = *(const uint4 *)p;
                        wq[b][0] = u.x, wq[b][1] = u.y, wq[b][2] = u.z, wq[b][3] = u.w;
                    } else if constexpr (MF == 2) {
                        const uint2 u = *(const uint2 *)p;
                        wq[b][2 * g] = u.x, wq[b][2 * g + 1] = u.y;
                    } else {
                        wq[b][g] = *(const uint32_t *)p;
                    }
                    sc[b][g] = *(const uint2 *)&ss[kc * NG + g][b * 16 + q4 * 4];
                }
#pragma unroll
                for (int i = 0; i < MF; ++i) {
                    const int c = g * (G / 8) + q4 * MF + i;
                    xf[g * MF + i] = __builtin_bit_cast(bf16x8_t, *(const uint4 *)(X + ((c ^ xr) << 4)));
                }
            }
            floatx4_t d[NB][NG];
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    d[b][g] = floatx4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = g * MF; i < (g + 1) * MF; ++i)
                        d[b][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp4x8_to_bf16(wq[b][i]),
                                                                          xf[i], d[b][g], 0, 0, 0);
                }
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    acc[b][0] = fmaf(d[b][g][0], bf16_lo(sc[b][g].x), acc[b][0]);
                    acc[b][1] = fmaf(d[b][g][1], bf16_hi(sc[b][g].x), acc[b][1]);
                    acc[b][2] = fmaf(d[b][g][2], bf16_lo(sc[b][g].y), acc[b][2]);
                    acc[b][3] = fmaf(d[b][g][3], bf16_hi(sc[b][g].y), acc[b][3]);
                }
            // the reads are done before the piece is loaded again
            __builtin_amdgcn_s_waitcnt(0xC07F);
            asm volatile("" ::: "memory");
        }
    }
    __syncthreads();
    floatx4_t(*part)[NB][64] = (floatx4_t(*)[NB][64])L;
#pragma unroll
    for (int b = 0; b < NB; ++b)
        part[w][b][lane] = acc[b];
    __syncthreads();
    // joined in wave order
    const bool three = a.planes == 3;
    auto sum = [&](int b) {
        floatx4_t o = part[0][b][lane];
#pragma unroll
        for (int u = 1; u < WV; ++u)
            o += part[u][b][lane];
        if (three) // a token's three columns: the smallest two first
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float mid = __shfl(o[e], lane + 1, 64), lo = __shfl(o[e], lane + 2, 64);
                o[e] += mid + lo;
            }
        return o;
    };
    const int m = m0 + (three ? l16 / 3 : l16);
    const bool mine = (!three || (l16 % 3 == 0 && l16 < 15)) && m < a.T;
    for (int b = w; b < SETS; b += WV) {
        floatx4_t o = sum(BOTH ? 2 * b : b);
        if constexpr (BOTH) {
            const floatx4_t u = sum(2 * b + 1);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = fp4_act(o[e], u[e]);
        }
        if (mine)
            store4(a.out, a.dto, a.ldo, m, n0 + b * 16 + q4 * 4, a.w.rows, o);
    }
}

template <int G, int NB, int XR, int WV, int NST, bool BOTH> void rows_one(RowsArgs a, hipStream_t s)
{
    constexpr int NR = 16 * (BOTH ? NB / 2 : NB);
    const int tiles = (int)(((int64_t)a.w.rows + NR - 1) / NR);
    const int tpt = a.planes == 3 ? 5 : 16;
    const uint32_t mt = (uint32_t)((a.T + tpt - 1) / tpt);
    const int most = (1 << 22) / (int)mt; // threads of a launch are numbered in 32 bits
    for (a.tile0 = 0; a.tile0 < tiles; a.tile0 += a.tiles) {
        a.tiles = tiles - a.tile0 < most ? tiles - a.tile0 : most;
        fp4_rows_kernel<G, NB, XR, WV, NST, BOTH><<<mt * (uint32_t)a.tiles, 64 * WV, 0, s>>>(a);
    }
}
// Sets of 16 rows and waves of a workgroup. One set and eight waves, which share
// the contraction, while that gives no more than a workgroup a CU; two sets past
// that (1 x 6144 over 2304: 4.2 against 4.6 us; 1 x 4096 over 4096: 5.0 against 4.2),
// and with two workgroups a CU of these, four waves, so that one begins while
// another ends (1 x 32768 over 4096: 13.8 against 14.3). Sixteen columns of
// activations take four times the loads of a set: four sets share them there
// (16 x 32768 over 4096: 14.9 against 16.0; one set 28.8).
template <int G, int XR> void rows_x(RowsArgs a, hipStream_t s)
{
    const bool wide = a.w.rows >= 16384, two = wide || a.w.rows > 16 * 256;
    a.turn = a.q2 ? (wide ? 5 : 4) : wide ? 6 : two ? 5 : 4; // the most rows of a workgroup
    if (a.q2) {
        if (XR == 16 && wide)
            rows_one<G, 4, XR, 4, 2, true>(a, s);
        else
            rows_one<G, 2, XR, 4, 2, true>(a, s);
    } else if (wide) {
        rows_one<G, XR == 16 ? 4 : 2, XR, 4, 2, false>(a, s);
    } else if (two) {
        rows_one<G, 2, XR, 8, 2, false>(a, s);
    } else {
        rows_one<G, 1, XR, 8, 2, false>(a, s);
    }
}
template <int G> void rows_group(const RowsArgs &a, hipStream_t s)
{
    if (a.R <= 4)
        rows_x<G, 4>(a, s);
    else if (a.R <= 8)
        rows_x<G, 8>(a, s);
    else
        rows_x<G, 16>(a, s);
}

// ---------------------------------------------------------------- dY W, few tokens
// The contraction runs over W's rows here, so a lane needs the codes of eight
// rows at one column. It loads a dword, eight columns, of each of eight rows
// (16 lanes a row's 64 bytes, straight to registers) and turns the 8 x 8 codes
// in place: dword j then holds column 8 l + j of the eight rows, and gets the
// rows' scales (a bfloat16 number each, for six-bit scales exactly). Tile j of
// the eight 16 x 16 tiles is columns j, 8 + j, 16 + j ..., and a lane's results
// of one token are runs of eight columns.
// A workgroup takes a block of 128 columns and one of plan.parts runs of rows; its
// waves take 32 rows at a time. The activations of a step's rows are staged in LDS.
// What bounds it is trips to memory: at 6144 x 4096 (14 MB) vector instructions are 0.21
// of the issue slots, the matrix unit 0.02 busy, and waves wait for half of their time.
// Parts are joined by a second launch (2.3 us): a block of columns for each of 18
// CUs alone would take the whole contraction one trip after another.
// One token over 6144 x 2304 7.5 us, both launches and their trips (16 tokens 8.6, ten
// of float32 12.6 with their packing); over 16384 x 4096 15.4 us (35 MB).
struct ColsArgs {
    const uint8_t *x;
    int64_t xrow;
    int T, planes, nkx; // nkx: blocks of 128 that the activations are padded to
    Fp4 w;
    float *part; // [parts][T][128 nkb]
    ColsPlan plan;
    void *out; // of one part
    int64_t ldo;
    int dto;
};

// Eight rows of eight codes to eight columns of eight codes: neighbouring rows'
// nibbles to bytes, then 4 x 4 bytes by permutes.
DEVI void turn8(uint32_t *v)
{
    constexpr uint32_t M = 0x0f0f0f0fu;
    uint32_t a[2][4]; // [column's parity][pair of rows]: byte b is column 2b + parity
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const uint32_t lo = v[2 * p], hi = v[2 * p + 1];
        a[0][p] = (lo & M) | (hi << 4 & ~M);
        a[1][p] = (lo >> 4 & M) | (hi & ~M);
    }
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        const uint32_t t0 = __builtin_amdgcn_perm(a[o][1], a[o][0], 0x05010400);
        const uint32_t t1 = __builtin_amdgcn_perm(a[o][1], a[o][0], 0x07030602);
        const uint32_t t2 = __builtin_amdgcn_perm(a[o][3], a[o][2], 0x05010400);
        const uint32_t t3 = __builtin_amdgcn_perm(a[o][3], a[o][2], 0x07030602);
        v[o] = __builtin_amdgcn_perm(t2, t0, 0x05040100);
        v[2 + o] = __builtin_amdgcn_perm(t2, t0, 0x07060302);
        v[4 + o] = __builtin_amdgcn_perm(t3, t1, 0x05040100);
        v[6 + o] = __builtin_amdgcn_perm(t3, t1, 0x07060302);
    }
}

// TB: 16-column tiles of activations (five float32 tokens each); U: sets of 32
// rows that a wave has in flight, plan.sets. A part is whole steps of them, so only
// the last one ends inside a step, at the matrix's end.
constexpr int CWV = FP4_CWV, CN = FP4_CN;
template <int TB, int U> __global__ __launch_bounds__(64 * CWV) void fp4_cols_kernel(ColsArgs a)
{
    constexpr int ROWS = CN * U, XROW = ROWS * 2, XB = 16 * TB * XROW;
    constexpr int OROW = FP4_BLK + 4, OB = CWV * 16 * OROW * 4; // (OROW in floats)
    __shared__ __attribute__((aligned(16))) uint8_t L[XB > OB ? XB : OB];
    const int lane = threadIdx.x & 63, w = wave_id(), l16 = lane & 15, q4 = lane >> 4;
    // an XCD takes a run of neighbouring blocks: two share W's 128-byte lines
    const int total = a.w.nkb * a.plan.parts, each = (total + NXCD - 1) / NXCD;
    const int at = (int)blockIdx.x / NXCD, id = (int)(blockIdx.x % NXCD) * each + at;
    if (at >= each || id >= total)
        return;
    const int part = id / a.w.nkb, kb = id % a.w.nkb;
    const int n_lo = part * a.plan.per, n_hi = min(n_lo + a.plan.per, a.w.rows);
    const bool three = a.planes == 3;
    const uint8_t *wq = a.w.q + (int64_t)kb * FP4_BYTES + l16 * 4;
    const uint16_t *sc = a.w.scale + (int64_t)((kb * FP4_BLK + l16 * 8) / a.w.group) * a.w.rows;
    floatx4_t acc[8][TB];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int t = 0; t < TB; ++t)
            acc[j][t] = floatx4_t{0.f, 0.f, 0.f, 0.f};
    for (int n0 = n_lo; n0 < n_hi; n0 += ROWS) {
        // this wave's rows: past the matrix the last one, whose activations are zeros
        uint32_t v[U][8];
        uint4 s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int n = n0 + u * CN + w * 32 + q4 * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[u][i] = *(const uint32_t *)(wq + (int64_t)min(n + i, a.w.rows - 1) * a.w.pitch);
            if (n + 8 <= a.w.rows) {
                s[u] = ldg16u(sc + n);
            } else {
                uint32_t h[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    h[i] = sc[min(n + i, a.w.rows - 1)];
                s[u] = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16,
                                  h[6] | h[7] << 16);
            }
        }
        if (n0 > n_lo)
            __syncthreads(); // the last rows' activations are used
        constexpr int CH = ROWS / 8; // chunks of 16 bytes of a column
#pragma unroll
        for (int i = 0; i < 16 * TB * CH / (64 * CWV); ++i) {
            const int q = i * 64 * CWV + threadIdx.x, c = q / CH, k = q % CH, l = c & 15;
            const int r = three ? (c >> 4) * 15 + l : c; // its row of activations
            uint4 u = make_uint4(0, 0, 0, 0);
            if (r < a.T * a.planes && n0 + k * 8 < a.nkx * FP4_BLK)
                u = ldg16(a.x + r * a.xrow + (int64_t)(n0 + k * 8) * 2);
            *(uint4 *)(L + c * XROW + ((k ^ l) << 4)) = u;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            turn8(v[u]);
            float f[8];
            elem<TWELL_BF16>::widen(s[u], f);
            bf16x8_t xf[TB];
#pragma unroll
            for (int t = 0; t < TB; ++t)
                xf[t] = __builtin_bit_cast(
                    bf16x8_t, *(const uint4 *)(L + (t * 16 + l16) * XROW +
                                               (((u * CWV + w) * 4 + q4 ^ l16) << 4)));
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bf16x8_t c = scaled8(v[u][j], f);
#pragma unroll
                for (int t = 0; t < TB; ++t)
                    acc[j][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(c, xf[t], acc[j][t], 0, 0, 0);
            }
        }
    }
    // the waves' sums meet in LDS, 16 columns of activations at a time
    float(*O)[16][OROW] = (float(*)[16][OROW])L;
#pragma unroll
    for (int t = 0; t < TB; ++t) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float *p = &O[w][l16][(q4 * 4 + e) * 8];
            *(floatx4_t *)p = floatx4_t{acc[0][t][e], acc[1][t][e], acc[2][t][e], acc[3][t][e]};
            *(floatx4_t *)(p + 4) =
                floatx4_t{acc[4][t][e], acc[5][t][e], acc[6][t][e], acc[7][t][e]};
        }
        __syncthreads();
        const int c = threadIdx.x / 32, k = threadIdx.x % 32 * 4;
        auto sum = [&](int col) {
            floatx4_t o = *(const floatx4_t *)&O[0][col][k];
#pragma unroll
            for (int u = 1; u < CWV; ++u)
                o += *(const floatx4_t *)&O[u][col][k];
            return o;
        };
        const int m = three ? t * 5 + c : t * 16 + c;
        if (m < a.T && (!three || c < 5)) {
            const floatx4_t o = three ? (sum(3 * c + 2) + sum(3 * c + 1)) + sum(3 * c) : sum(c);
            if (a.plan.parts == 1)
                store4(a.out, a.dto, a.ldo, m, kb * FP4_BLK + k, a.w.cols, o);
            else
                *(floatx4_t *)(a.part + ((int64_t)part * a.T + m) * a.w.nkb * FP4_BLK +
                               kb * FP4_BLK + k) = o;
        }
    }
}

// out [T][N] = the sum of the parts, in order. Four columns a thread, eight parts in
// flight (17 x 2304 of 12 parts 2.3 us, a launch and a trip; one after another 10).
struct JoinArgs {
    const float *part;
    int parts, T, N;
    int64_t pitch; // floats of a row of a part, a multiple of four
    void *out;
    int64_t ldo;
    int dto;
    uint32_t grid; // workgroups
};
__global__ __launch_bounds__(64) void fp4_join_kernel(JoinArgs a)
{
    const int64_t n4 = (a.N + 3) / 4, total = n4 * a.T, stride = (int64_t)a.T * a.pitch;
    for (int64_t q = (int64_t)blockIdx.x * 64 + threadIdx.x; q < total; q += (int64_t)a.grid * 64) {
        const int64_t t = q / n4;
        const int n = (int)(q % n4) * 4;
        const float *src = a.part + t * a.pitch + n;
        floatx4_t sum = {0.f, 0.f, 0.f, 0.f};
        for (int p = 0; p < a.parts; p += 8) { // eight in flight
            floatx4_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = *(const floatx4_t *)(src + min(p + i, a.parts - 1) * stride);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (p + i < a.parts)
                    sum += v[i];
        }
        store4(a.out, a.dto, a.ldo, t, n, a.N, sum);
    }
}
void join(JoinArgs a, hipStream_t s)
{
    const int64_t wgs = ((int64_t)((a.N + 3) / 4) * a.T + 63) / 64;
    a.grid = (uint32_t)(wgs < 1 << 24 ? wgs : 1 << 24);
    fp4_join_kernel<<<a.grid, 64, 0, s>>>(a);
}

template <int TB> void cols_tb(const ColsArgs &a, hipStream_t s)
{
    const uint32_t grid = (uint32_t)((a.w.nkb * a.plan.parts + NXCD - 1) / NXCD * NXCD);
    if (a.plan.sets == 2)
        fp4_cols_kernel<TB, 2><<<grid, 64 * CWV, 0, s>>>(a);
    else
        fp4_cols_kernel<TB, 1><<<grid, 64 * CWV, 0, s>>>(a);
}
void cols(const ColsArgs &a, hipStream_t s)
{
    if (a.T <= (a.planes == 3 ? 5 : 16))
        cols_tb<1>(a, s);
    else
        cols_tb<2>(a, s);
}

// Which tiles, and in how many parts of the contraction: the least of the times
// that measured figures give (us; they order the choices, no more). A step of
// 128 takes `step` alone on its CU and `pair` beside another workgroup (both of
// them), a tile `ends` more for its beginning and end; parts add a launch and
// the partial sums' way through memory.
enum TileKind { TILE_64, TILE_128, TILE_256 };
struct TileTime {
    int bm, bn; // by TileKind
    double step, pair, ends;
};
struct TilePlan {
    TileKind k;
    int parts, per;
};
TilePlan tile_plan(const TileTime *kinds, int n_kinds, double T, double N, int nkb)
{
    TilePlan best = {TILE_64, 1, nkb};
    double least = 1e300;
    auto up = [](double a, double b) { return ceil(a / b); };
    for (int i = 0; i < n_kinds; ++i)
        for (int parts = 1; parts <= 32 && parts <= nkb; parts *= 2) {
            const TileTime &c = kinds[i];
            const double tiles = up(T, c.bm) * up(N, c.bn);
            if (parts > 1 && tiles >= 512)
                break; // the chip is full
            const double n = up(tiles * parts, 256), pairs = floor(n / 2);
            const double k = up(nkb, parts);
            const double t = pairs * (k * c.pair + c.ends) + (n - 2 * pairs) * (k * c.step + c.ends) +
                             (parts == 1 ? 0. : 3.0 + parts * T * N * 8 / 4e6);
            if (t < least)
                least = t, best = {(TileKind)i, parts, (nkb + parts - 1) / parts};
        }
    best.parts = best.per ? (nkb + best.per - 1) / best.per : 1;
    return best;
}
int64_t part_pitch(int N) { return ((int64_t)N + 3) / 4 * 4; }

// ---------------------------------------------------------------- X W^T, many tokens
// A workgroup computes BM tokens x BN rows of W. A step is 64 k: the tokens' 128
// bytes and W's 32 go straight from global memory to LDS, NST steps resident,
// the tokens' chunks XOR-swizzled so that the 16 rows of a fragment lie on
// distinct banks. A wave owns WM x WN of the tile, NI fragments of W (the first
// operand) by MI of tokens. W's codes become bfloat16 numbers times their scales
// in registers, a fragment at a time beside the products of the one before, so
// they cost LDS and memory a quarter of what values do.
// A step's codes are read two rows of products ahead and its tokens one, so at the
// step's one barrier, before its last two rows, all of it is in registers: its own
// stage is loaded anew behind the barrier, NST steps ahead.
// DX, of dY W: the contraction runs over W's rows, a step is 64 of them, 16 codes of a
// row in a lane, and the transposing LDS read of 4-bit elements (lane c of 16 gets
// code c of the 16 lanes' rows, as measured on the part) gives a lane its column's 16
// rows. Their scales, 16 to a lane, are the same for the 16 lanes of a row group.
// What bounds a large product is the matrix unit and the vector instructions that
// scale the codes (two an element, three of dY W, where each of a pair has its own
// scale), which take turns for the most part: busy 0.50 and 0.43 of the time of
// 8192 x 5632 over 2048, 160 us, 1180 TF (the library's bfloat16 product of these sizes
// without any codes: 164); dY W 155 us (library 131). Small ones: the steps' latency on
// one or two workgroups a CU (512 x 5632 over 2048 20 us, 64 x 4096 over 4096 of dY W 14).
// Tried without gain: two products at a time between the instructions of one, five
// stages, 128 x 128 tiles of 2 x 2 or 2 x 4 waves (5 to 15% slower: codes are scaled
// by two waves each).
template <int BM_, int BN_, int WGM_, int WGN_, int NST_, int KS_, int SG_> struct TileCfg {
    static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, NST = NST_, KS = KS_;
    static constexpr int NWV = WGM * WGN, NT = 64 * NWV;
    static constexpr int WM = BM / WGM, WN = BN / WGN, MI = WM / 16, NI = WN / 16;
    // bytes of a token's and of W's row of a step, 16-byte chunks of them, matrix
    // instructions of a step and tile
    static constexpr int RA = KS * 2, RW = KS / 2, CA = RA / 16, CW = RW / 16, NF = KS / 32;
    static constexpr int ABYTES = BM * RA, STAGE = ABYTES + BN * RW;
    static constexpr int WBA = ABYTES / 1024 / NWV, WBB = BN * RW / 1024 / NWV, WB = WBA + WBB;
    // what a row's chunks are XORed with, so that 16 rows lie on distinct banks
    DEVI static int swa(int r) { return KS == 64 ? r >> 1 & 7 : r & 15; }
    // DX: 16-byte chunks of a row of W's columns, and what they are XORed with
    static constexpr int CD = BN / 32;
    DEVI static int swd(int r) { return CD == 8 ? r >> 1 & 7 : r >> 2 & 3; }
    DEVI static int sww(int r) { return KS == 64 ? 0 : r >> 2 & 3; }
    static constexpr int SG = SG_; // groups of scales staged at a time
    static constexpr int OROW = 128 + 16, OUTB = 16 * OROW * NWV; // the epilogue's rows
    static_assert(ABYTES % (1024 * NWV) == 0 && BN * RW % (1024 * NWV) == 0, "whole loads");
    static_assert(KS == 64 || KS == 128, "a lane's codes share a scale");
    static constexpr int LPS = (WB + 2 * MI - 1) / (2 * MI); // loads beside a product after it
    static_assert(WN % 32 == 0 && NI % 2 == 0, "fragments in turn, whole runs of results");
    static_assert(NST >= 2 && (NST - 2) * WB < 64, "loads in flight must fit vmcnt");
    static_assert(OUTB <= NST * STAGE && NST * STAGE + SG * BN * 2 <= 160 * 1024, "LDS");
};

struct TileArgs {
    Acts x;
    Fp4 w;
    void *out;
    int64_t ldo;
    int dto;
    float *part; // split contraction: [parts][T][ldo of a part]
    int64_t ldp;
    int parts, per; // parts, blocks of 128 k in each
    // a second matrix of w's sizes, its rows after w's (whole tiles), or NULL
    const uint8_t *q2;
    const uint16_t *scale2;
};

// PL: rows of a token's activations. DX: of dY W, see above.
template <int G, class C, int PL, bool DX>
__global__ __launch_bounds__(C::NT, C::NWV / 4) void fp4_tile_kernel(TileArgs a)
{
    constexpr int NST = C::NST, MI = C::MI, NI = C::NI;
    __shared__ __attribute__((aligned(16))) uint8_t L[NST * C::STAGE];
    __shared__ __attribute__((aligned(16))) uint16_t ss[C::SG * C::BN];
    // an XCD takes a run of tiles, eight rows of them at a time
    constexpr int GM = 8;
    constexpr bool three = PL == 3;
    constexpr int tpt = three ? C::BM / 16 * 5 : C::BM; // tokens of a tile
    const int N = DX ? a.w.cols : a.q2 ? 2 * a.w.rows : a.w.rows;
    const int nt = (N + C::BN - 1) / C::BN, mt = (a.x.T + tpt - 1) / tpt;
    const int64_t total = (int64_t)nt * mt * a.parts, each = (total + NXCD - 1) / NXCD;
    const int64_t at = blockIdx.x / NXCD, q0 = blockIdx.x % NXCD * each + at;
    if (at >= each || q0 >= total)
        return;
    const int part = (int)(q0 / ((int64_t)nt * mt));
    const int64_t q = q0 % ((int64_t)nt * mt), gsz = (int64_t)GM * nt;
    const int grp = (int)(q / gsz), grows = min(GM, mt - grp * GM), gr = (int)(q % gsz);
    const int m0 = (grp * GM + gr % grows) * tpt, n0 = gr / grows * C::BN;
    const int lane = threadIdx.x & 63, w = wave_id(), l16 = lane & 15, q4 = lane >> 4;
    const int wm = w / C::WGN, wn = w % C::WGN;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(ng::lds_u8 *)L;

    // Rows past an operand read its last row; their results are dropped. Of
    // float32 activations a fragment holds five tokens, three rows each.
    const int64_t xrow = three ? a.x.plane : a.x.pitch;
    const uint8_t *srcx = a.x.data + (int64_t)m0 * a.x.pitch, *srcw;
    const bool second = !DX && n0 >= a.w.rows;
    const int nw0 = second ? n0 - a.w.rows : n0; // row of its matrix
    const uint16_t *scale = second ? a.scale2 : a.w.scale;
    srcw = DX ? a.w.q : (second ? a.q2 : a.w.q) + (int64_t)nw0 * a.w.pitch;
    uint32_t off[C::WB];
#pragma unroll
    for (int g = 0; g < C::WB; ++g) {
        if (g < C::WBA) {
            const int r = (w * C::WBA + g) * (64 / C::CA) + lane / C::CA;
            const int x = three ? (r >> 4) * 15 + (r & 15) : r; // this row's
            const int last = (a.x.T - m0) * PL - 1;
            off[g] = (uint32_t)min(x, last) * (uint32_t)xrow + (((lane % C::CA) ^ C::swa(r)) << 4);
        } else if (DX) { // row of the step, and the chunk of columns (past the last: the first)
            const int r = (w * C::WBB + g - C::WBA) * (64 / C::CD) + lane / C::CD;
            const uint32_t c = (uint32_t)n0 / 2 + (((lane % C::CD) ^ C::swd(r)) << 4);
            off[g] = c < (uint32_t)a.w.pitch ? c : 0;
        } else {
            const int r = (w * C::WBB + g - C::WBA) * (64 / C::CW) + lane / C::CW;
            off[g] = (uint32_t)min(r, a.w.rows - 1 - nw0) * (uint32_t)a.w.pitch +
                     (((lane % C::CW) ^ C::sww(r)) << 4);
        }
    }
    floatx4_t acc[NI][MI];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < MI; ++j)
            acc[i][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};

    // this lane's row of a fragment, its first chunk of tokens and its codes
    // The quarter of a step's k that its 16 lanes take, 0 3 1 2: a 16-byte read serves
    // four lanes, skips eight and goes on in the next 16, and quarters 0 and 1 (2 and 3)
    // of these rows would meet on their banks (conflicts 0.47 of LDS's cycles, so 0.14;
    // 2048 x 4096 over 4096 66.5 -> 63.3 us).
    constexpr int NF = C::NF;
    const int kq = (q4 & 1) * 3 ^ q4 >> 1;
    const uint8_t *Aw = L + (wm * C::WM + l16) * C::RA;
    // (DX: row 16 kq + l16 of the step, whose 16 codes of a tile the read turns)
    const uint8_t *Bw = L + C::ABYTES + (DX ? (kq * 16 + l16) * (C::BN / 2)
                                            : (wn * C::WN + l16) * C::RW +
                                                  (C::KS == 64 ? kq * 8 : (kq ^ C::sww(l16)) << 4));
    int f[NF];
#pragma unroll
    for (int e = 0; e < NF; ++e)
        f[e] = ((kq * NF + e) ^ C::swa(l16)) << 4;
    auto fence = [] {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
    };
    const int b0 = part * a.per, b1 = min(DX ? a.x.nkb : a.w.nkb, b0 + a.per);
    constexpr int CB = C::SG * G / FP4_BLK; // blocks of k whose scales are staged
    for (int c0 = b0; c0 < b1; c0 += CB) {
        const int nb = min(CB, b1 - c0), n_steps = FP4_BLK / C::KS * nb;
        int ls = 0; // the loads' own step
        auto load = [&](int g, int st) {
            const uint32_t dst = lds0 + (uint32_t)(st * C::STAGE);
            if (g < C::WBA)
                ng::dma16(srcx + (int64_t)c0 * 256 + ls * C::RA, off[g],
                          dst + (w * C::WBA + g) * 1024, ls, n_steps);
            else if (DX) {
                const int r = (w * C::WBB + g - C::WBA) * (64 / C::CD) + lane / C::CD;
                const int64_t n = min((int64_t)c0 * FP4_BLK + ls * C::KS + r, (int64_t)a.w.rows - 1);
                if (ls < n_steps)
                    ng::lds_dma16(srcw + n * a.w.pitch + off[g],
                                  dst + C::ABYTES + (w * C::WBB + g - C::WBA) * 1024);
            } else
                ng::dma16(srcw + (int64_t)c0 * FP4_BYTES + ls * C::RW, off[g],
                          dst + C::ABYTES + (w * C::WBB + g - C::WBA) * 1024, ls, n_steps);
        };
        if (c0 > b0)
            __syncthreads(); // the last scales and stages are used
#pragma unroll
        for (int s = 0; s < NST; ++s) {
#pragma unroll
            for (int g = 0; g < C::WB; ++g)
                load(g, s);
            ++ls;
        }
        // Scales, four rows a load, SL loads in flight: [group][row of the tile], or
        // (DX) [group of the tile][row].
        constexpr int SL = 4, NC = CB * FP4_BLK;
        const int per = DX ? nb * (FP4_BLK / 4) : C::BN / 4; // pieces of a group
        const int pieces = per * (DX ? C::BN / G : nb * (FP4_BLK / G));
        const int g0 = DX ? n0 / G : c0 * (FP4_BLK / G), r0 = DX ? c0 * FP4_BLK : nw0;
        for (int i = threadIdx.x; i < pieces; i += SL * C::NT) {
            bytes8 v[SL];
#pragma unroll
            for (int u = 0; u < SL; ++u) {
                const int q = min(i + u * C::NT, pieces - 1), r = r0 + q % per * 4;
                const int g = min(g0 + q / per, a.w.nkb * (FP4_BLK / G) - 1);
                const uint16_t *p = scale + (int64_t)g * a.w.rows;
                if (r + 4 <= a.w.rows) {
                    v[u] = *(const bytes8 *)(p + r);
                } else {
                    uint32_t h[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        h[e] = p[min(r + e, a.w.rows - 1)];
                    v[u] = bytes8{h[0] | h[1] << 16, h[2] | h[3] << 16};
                }
            }
#pragma unroll
            for (int u = 0; u < SL; ++u) {
                const int q = min(i + u * C::NT, pieces - 1);
                *(uint2 *)&ss[q / per * (DX ? NC : C::BN) + q % per * 4] =
                    make_uint2(v[u].x, v[u].y);
            }
        }
        ng::wait_vm<0>();
        __syncthreads();
        bf16x8_t xf[MI][NF];
        uint32_t wf[2][NF][4]; // fragments of W in turn
        uint32_t raw[2][NF];   // their codes and scales, read a row of products earlier
        float sc[2];
        uint32_t sp[4 * NF]; // DX: the scales of the lane's rows of a step
        auto ldx = [&](int j, int st) {
#pragma unroll
            for (int e = 0; e < NF; ++e)
                xf[j][e] = __builtin_bit_cast(
                    bf16x8_t, *(const uint4 *)(Aw + st * C::STAGE + j * 16 * C::RA + f[e]));
        };
        auto ldw = [&](int i, int st, int k) { // fragment i of step k
            uint32_t *q = raw[i & 1];
            if constexpr (DX) {
                typedef int intx2_t __attribute__((ext_vector_type(2)));
                typedef __attribute__((address_space(3))) intx2_t lds_i2;
                const int c = (wn * C::WN + i * 16) / 2; // byte of the row
                const uint8_t *p = Bw + st * C::STAGE + (((c >> 4) ^ C::swd(kq * 16 + l16)) << 4) + (c & 15);
                const intx2_t u = __builtin_amdgcn_ds_read_tr4_b64_v2i32((lds_i2 *)(uintptr_t)(ng::lds_u8 *)p);
                q[0] = (uint32_t)u[0], q[1] = (uint32_t)u[1];
                return;
            }
            const uint8_t *p = Bw + st * C::STAGE + i * 16 * C::RW;
            if constexpr (NF == 2) {
                const uint2 u = *(const uint2 *)p;
                q[0] = u.x, q[1] = u.y;
            } else {
                const uint4 u = *(const uint4 *)p;
                q[0] = u.x, q[1] = u.y, q[2] = u.z, q[3] = u.w;
            }
            sc[i & 1] = bf16_to_f32(
                ss[(k * C::KS + kq * (C::KS / 4)) / G * C::BN + wn * C::WN + i * 16 + l16]);
        };
        auto lds = [&](int i, int k) { // scales of fragment i of step k
            const uint4 *p = (const uint4 *)&ss[(wn * C::WN + i * 16) / G * NC + k * C::KS + kq * 16];
            const uint4 u = p[0], v = p[1];
            sp[0] = u.x, sp[1] = u.y, sp[2] = u.z, sp[3] = u.w;
            sp[4] = v.x, sp[5] = v.y, sp[6] = v.z, sp[7] = v.w;
        };
        auto conv = [&](int i, int p) { // dword p of fragment i
            const float lo = DX ? bf16_lo(sp[p]) : sc[i & 1], hi = DX ? bf16_hi(sp[p]) : sc[i & 1];
            wf[i & 1][p / 4][p % 4] = scaled2(raw[i & 1][p / 4], p % 4, lo, hi);
        };
#pragma unroll
        for (int j = 0; j < MI; ++j)
            ldx(j, 0);
        ldw(0, 0, 0);
        ldw(1, 0, 0);
        if (DX)
            lds(0, 0);
#pragma unroll
        for (int p = 0; p < 4 * NF; ++p)
            conv(0, p);
        for (int s = 0, st = 0; s < n_steps; ++s) {
            const int nxt = st == NST - 1 ? 0 : st + 1, sn = s + 1 < n_steps ? s + 1 : 0;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                if (i == NI - 2) {
                    fence();
                    if (s + NST - 1 < n_steps)
                        ng::wait_vm<(NST - 2) * C::WB>();
                    else
                        ng::wait_vm<0>();
                    __builtin_amdgcn_s_waitcnt(0xC07F); // lgkmcnt(0)
                    __builtin_amdgcn_s_barrier();
                    fence();
                }
                if (i < NI - 2)
                    ldw(i + 2, st, s);
                else
                    ldw(i + 2 - NI, nxt, sn);
                // DX: a fragment of other scales than the last, converted from the row's
                // middle on
                const int next = i < NI - 1 ? i + 1 : 0;
                const bool fresh = DX && (next == 0 || (C::WN > G && next * 16 % G == 0));
                if (fresh)
                    lds(next, next == 0 ? sn : s);
                const int from = fresh ? MI / 2 : 0;
#pragma unroll
                for (int j = 0; j < MI; ++j) {
#pragma unroll
                    for (int e = 0; e < NF; ++e)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8_t, *(const uint4 *)wf[i & 1][e]), xf[j][e],
                            acc[i][j], 0, 0, 0);
                    if (i == NI - 1)
                        ldx(j, nxt);
                    // the next fragment, piece by piece beside this row's products
#pragma unroll
                    for (int p = (j - from) * 4 * NF / (MI - from);
                         p < (j + 1 - from) * 4 * NF / (MI - from); ++p)
                        if (p >= 0)
                            conv(next, p);
                    // past the barrier the stage is free: all of its step is in registers
                    const int t = (i - (NI - 2)) * MI + j;
#pragma unroll
                    for (int g = t * C::LPS; g < (t + 1) * C::LPS && g < C::WB; ++g)
                        if (t >= 0)
                            load(g, st);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            ++ls;
            st = nxt;
        }
    }
    ng::wait_vm<0>();
    __syncthreads(); // the stages are free
    // ---- a lane's four results are one token's (j * 16 + l16), n i * 16 + q4 * 4:
    // through the wave's own piece of LDS, 128 bytes of 16 tokens at a time
    const int mw = m0 + (three ? wm * C::WM / 16 * 5 : wm * C::WM), nw = n0 + wn * C::WN;
    uint8_t *buf = L + w * 16 * C::OROW;
    auto store = [&](auto type, void *out, int64_t ld) {
        using T = decltype(type);
        constexpr int ES = sizeof(T), WE = 128 / ES < C::WN ? 128 / ES : C::WN;
        constexpr int VPL = 16 / ES, LPR = WE / VPL; // values a lane, lanes of a run
        const int c8 = lane % LPR, rr = lane / LPR;
#pragma unroll
        for (int j = 0; j < MI; ++j)
#pragma unroll
            for (int h = 0; h < C::WN / WE; ++h) {
#pragma unroll
                for (int i = 0; i < WE / 16; ++i) {
                    floatx4_t v = acc[h * (WE / 16) + i][j];
                    int row = l16;
                    if constexpr (three) { // a token's three rows, the smallest two first
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float mid = __shfl(v[e], lane + 1, 64), lo = __shfl(v[e], lane + 2, 64);
                            v[e] += mid + lo;
                        }
                        row = l16 % 3 == 0 && l16 < 15 ? l16 / 3 : 15;
                    }
                    uint8_t *p = buf + row * C::OROW + (i * 16 + q4 * 4) * ES;
                    if constexpr (ES == 4)
                        *(floatx4_t *)p = v;
                    else
                        *(uint2 *)p = make_uint2(f32x2_to_bf16x2(v[0], v[1]),
                                                 f32x2_to_bf16x2(v[2], v[3]));
                }
                const int c = nw + h * WE + c8 * VPL;
#pragma unroll
                for (int r0 = 0; r0 < 16; r0 += 64 / LPR) {
                    if (three && r0 + rr >= 5)
                        continue;
                    const int m = mw + j * (three ? 5 : 16) + r0 + rr;
                    const uint4 v = *(const uint4 *)(buf + (r0 + rr) * C::OROW + c8 * 16);
                    T *row = (T *)out + m * ld;
                    if (m < a.x.T && c + VPL <= N) {
                        stg16u_nt(row + c, v);
                    } else if (m < a.x.T) {
                        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < VPL; ++e)
                            if (c + e < N)
                                row[c + e] = (T)(u[e * ES / 4] >> (8 * ES * e % 32));
                    }
                }
            }
    };
    if (a.parts > 1)
        store(uint32_t(), a.part + (int64_t)part * a.x.T * a.ldp, a.ldp);
    else if (a.dto == TWELL_F32)
        store(uint32_t(), a.out, a.ldo);
    else
        store(uint16_t(), a.out, a.ldo);
}

using T64 = TileCfg<64, 128, 1, 4, 2, 128, 64>;  // waves of 64 tokens x 32 rows
using T64DX = TileCfg<64, 128, 1, 4, 3, 64, 64>;  // (dY W takes steps of 64)
using T128 = TileCfg<128, 128, 1, 4, 2, 64, 64>; // waves of 128 x 32
using T256 = TileCfg<256, 256, 2, 4, 3, 64, 64>; // waves of 128 x 64

template <int G, class C, bool DX> void tile_one(const TileArgs &a, hipStream_t s)
{
    const int tpt = a.x.planes == 3 ? C::BM / 16 * 5 : C::BM;
    const int64_t N = DX ? a.w.cols : (int64_t)a.w.rows * (a.q2 ? 2 : 1);
    const int64_t tiles = (N + C::BN - 1) / C::BN * ((a.x.T + tpt - 1) / tpt) * a.parts;
    const uint32_t grid = (uint32_t)((tiles + NXCD - 1) / NXCD * NXCD);
    if (a.x.planes == 3)
        fp4_tile_kernel<G, C, 3, DX><<<grid, C::NT, 0, s>>>(a);
    else
        fp4_tile_kernel<G, C, 1, DX><<<grid, C::NT, 0, s>>>(a);
}
template <int G, bool DX> void tile_group(const TileArgs &a, TileKind k, hipStream_t s)
{
    if (k == TILE_256)
        tile_one<G, T256, DX>(a, s);
    else if (k == TILE_128)
        tile_one<G, T128, DX>(a, s);
    else
        tile_one<G, std::conditional_t<DX, T64DX, T64>, DX>(a, s);
}
template <bool DX> void tiles(const TileArgs &a, TileKind k, hipStream_t s)
{
    if (a.w.group == 32)
        tile_group<32, DX>(a, k, s);
    else if (a.w.group == 64)
        tile_group<64, DX>(a, k, s);
    else
        tile_group<128, DX>(a, k, s);
}

// Tiles of X W^T. A float32 token takes 3.2 rows of a tile.
TilePlan fwd_plan(int T, int N, int nkb, int planes, bool both = false)
{
    static const TileTime kinds[] = {{64, 128, 0.75, 1.1, 2.5}, {128, 128, 1.1, 1.95, 3.0},
                                     {256, 256, 2.7, 5.4, 5.0}};
    // (of two matrices one after the other 256 rows may be of both)
    return tile_plan(kinds, both ? 2 : 3, planes == 3 ? T * 3.2 : T, N, nkb);
}
// Tiles of dY W.
TilePlan dx_plan(int T, int K, int nkb, int planes)
{
    static const TileTime kinds[] = {{64, 128, 0.9, 1.3, 2.5}, {128, 128, 1.3, 2.2, 3.0},
                                     {256, 256, 3.0, 6.0, 5.0}};
    return tile_plan(kinds, 3, planes == 3 ? T * 3.2 : T, K, nkb);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }
// Whether the few-token kernels take a product. Measured, us, by them and by the tile
// kernels: of X W^T over N rows of nkb blocks
// - up to two 16-column tiles of activations: 32 tokens over 6144 x 2304 7.1 and 11.1,
//   over 4096 x 4096 8.1 and 10.7, over 1024 x 1024 3.0 and 7.1;
// - more of them while all are little work, their tiles times rows / 16 times blocks at
//   most 22000: 64 tokens over 1024 x 1024 (2048) 3.5 and 8.1, 48 over 6144 x 2304
//   (20736) 9.9 and 11.7, 11 of float32 there (20736 too) 12.7 and 13.5; past it 64 over
//   4096 x 4096 (32768) 15.5 and 14.0, 128 over 2048 x 5632 (45056) 17.9 and 14.5. The
//   work alone does not see how many workgroups a CU gets: on the wrong side of the
//   limit lie 64 tokens over 6144 x 2304 (27648) 10.4 and 12.8, 33 over 11264 x 1024
//   (16896) 11.9 and 8.4, 128 over 2816 x 1024 (11264) 12.4 and 8.7.
// Of dY W up to two tiles: 32 tokens over 6144 x 2304 10.9 and 12.3, over 4096 x 4096
// 10.9 and 11.6, over 1024 x 1024 7.3 and 7.4 (48 over 6144 x 2304 15.3 and 13.0).
int token_tiles(int T, int planes) { return (T + (planes == 3 ? 4 : 15)) / (planes == 3 ? 5 : 16); }
bool few_fwd(int T, int planes, int64_t N, int nkb)
{
    const int64_t mt = token_tiles(T, planes);
    // (of no blocks the tiles store the zeros: rows_one's launches are for few tokens)
    return mt <= 2 || (nkb > 0 && mt * ((N + 15) / 16) * nkb <= 22000);
}
bool few_dx(int T, int planes) { return token_tiles(T, planes) <= 2; }
int planes_of(const twell_mat_t *x) { return x->dtype == TWELL_BF16 ? 1 : 3; }

} // namespace

void fp4_rows(const Acts &x, const Fp4 &w, const Fp4 *up, void *out, int64_t ldo, int dto,
              hipStream_t s)
{
    const RowsArgs a = {x.data, x.planes == 3 ? x.plane : x.pitch, x.T, x.planes, x.T * x.planes,
                        w, out, ldo, dto, 0, 0, 0, up ? up->q : nullptr, up ? up->scale : nullptr};
    if (w.group == 32)
        rows_group<32>(a, s);
    else if (w.group == 64)
        rows_group<64>(a, s);
    else
        rows_group<128>(a, s);
}

// Workspace: the packed activations, then the parts' sums.
size_t fp4_mm_workspace(const twell_mat_t *x, int rows, int cols, bool dx)
{
    const size_t pack = fp4_pack_bytes(x), pitch = (size_t)fp4_blocks(cols) * FP4_BLK;
    const int planes = planes_of(x);
    if (!dx && few_fwd(x->rows, planes, rows, fp4_blocks(cols)))
        return pack;
    if (dx && few_dx(x->rows, planes)) {
        const int parts = cols_plan(rows, fp4_blocks(cols)).parts;
        return parts == 1 ? pack : up256(pack) + (size_t)parts * x->rows * pitch * 4;
    }
    const int n = dx ? cols : rows, nkb = fp4_blocks(dx ? rows : cols);
    const TilePlan p = dx ? dx_plan(x->rows, n, nkb, planes) : fwd_plan(x->rows, n, nkb, planes);
    return p.parts == 1 ? pack : up256(pack) + (size_t)p.parts * x->rows * part_pitch(n) * 4;
}

int launch_fp4_mm(const twell_mat_t *x, const twell_fp4_t *w4, const twell_mat_t *out, bool dx,
                  void *ws, size_t ws_bytes, twell_timing_t *timing, hipStream_t s)
{
    const Fp4 w = fp4_arg(w4);
    const size_t need = fp4_mm_workspace(x, w.rows, w.cols, dx);
    if (need && (!ws || ws_bytes < need))
        return TWELL_E_WORKSPACE;
    Timer tm(timing, s);
    bool packed;
    const Acts a = fp4_pack(x, ws, s, &packed);
    if (packed)
        tm.mark("fp4_pack");
    uint8_t *ws2 = (uint8_t *)ws + up256(fp4_pack_bytes(x));
    const int dto = out->dtype, planes = planes_of(x);
    JoinArgs j = {(float *)ws2, 1, a.T, dx ? w.cols : w.rows, 0, out->data, out->ld, dto, 0};
    if (!dx && few_fwd(a.T, planes, w.rows, w.nkb)) {
        fp4_rows(a, w, nullptr, out->data, out->ld, dto, s);
        tm.mark("fp4_rows");
    } else if (dx && few_dx(a.T, planes)) {
        const ColsArgs c = {a.data, a.planes == 3 ? a.plane : a.pitch, a.T, a.planes, a.nkb, w,
                      (float *)ws2, cols_plan(w.rows, w.nkb), out->data, out->ld, dto};
        j.parts = c.plan.parts;
        j.pitch = (int64_t)w.nkb * FP4_BLK;
        cols(c, s);
        tm.mark("fp4_cols");
    } else {
        const TilePlan p = dx ? dx_plan(a.T, j.N, a.nkb, planes) : fwd_plan(a.T, j.N, a.nkb, planes);
        j.parts = p.parts, j.pitch = part_pitch(j.N);
        const TileArgs t = {a, w, out->data, out->ld, dto, (float *)ws2, j.pitch, p.parts, p.per,
                            nullptr, nullptr};
        dx ? tiles<true>(t, p.k, s) : tiles<false>(t, p.k, s);
        static const char *const names[] = {"fp4_tile64", "fp4_tile128", "fp4_tile256"};
        tm.mark(names[p.k]);
    }
    if (j.parts > 1) {
        join(j, s);
        tm.mark("fp4_join");
    }
    return hipGetLastError() == hipSuccess ? TWELL_OK : TWELL_E_HIP;
}

int fp4_gates_parts(const twell_mat_t *x, int d_ff)
{
    const int planes = planes_of(x);
    return few_fwd(x->rows, planes, 2 * d_ff, fp4_blocks(x->cols))
               ? 0 : fwd_plan(x->rows, 2 * d_ff, fp4_blocks(x->cols), planes, true).parts;
}

void fp4_gates(const Acts &x, const Fp4 &wg, const Fp4 &wu, float *parts, hipStream_t s)
{
    const TilePlan p = fwd_plan(x.T, 2 * wg.rows, wg.nkb, x.planes, true);
    const int64_t ld = 2 * (int64_t)wg.rows;
    tiles<false>({x, wg, parts, ld, TWELL_F32, parts, ld, p.parts, p.per, wu.q, wu.scale}, p.k, s);
}
