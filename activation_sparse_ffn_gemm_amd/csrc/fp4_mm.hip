// out = X W^T of activations with weights in 4 bits, and dX = dY W:
//   out[t][n] = sum over groups g of s[g][n] sum_{k in g} x[t][k] c[n][k]
//   dx[t][k]  = sum over n of dy[t][n] s[g(k)][n] c[n][k]
// with c the code's value. Codes are bfloat16 numbers and float32 activations
// are three of them (see Acts), so the bfloat16 matrix instruction forms every
// product exactly; sums are float32.
#include "fp4.hpp"

namespace {

// ---------------------------------------------------------------- few tokens
// A workgroup computes 16 NB rows of W for up to 16 columns (tokens, or a
// third of a float32 token each), its WV waves taking every WV-th block of 128
// k; their sums meet in LDS. A wave's rows of a block go to its own piece of
// LDS, NST blocks in turn, without a barrier: a wave waits for its own loads.
// The W rows are the instruction's first operand and the activations its
// second: a lane's four results are four rows of one column. A group's sum
// starts from zero and joins the accumulator times the group's scales.
struct RowsArgs {
    const uint8_t *x;
    int64_t xrow;      // bytes from one column's row to the next
    int T, planes, R;  // R = T planes
    Fp4 w;
    void *out;
    int64_t ldo;
    int dto, tile0; // first tile of rows of this launch
    int tiles;      // tiles of rows of this launch
};

template <int G, int NB, int XR, int WV, int NST>
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
    const int n0 = (a.tile0 + tile) * (16 * NB);
    const int tpt = a.planes == 3 ? 5 : 16; // tokens of a tile
    const int m0 = mt * tpt, c0 = m0 * a.planes;
    // W: lane l loads chunk l % 4 of row l / 4, as the swizzle places it; x: chunk
    // l % 16 of row 4 j + l / 16. Rows past an operand read its last row.
    const uint8_t *srcw = a.w.q + (int64_t)n0 * a.w.pitch, *srcx = a.x + (int64_t)c0 * a.xrow;
    uint32_t off[LPF];
#pragma unroll
    for (int i = 0; i < LPF; ++i) {
        if (i < NB) {
            const int r = i * 16 + lane / 4;
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
            ng::dma16(i < NB ? srcw + (int64_t)kb * FP4_BYTES : srcx + (int64_t)kb * FP4_BLK * 2,
                      off[i], lds0 + (uint32_t)(st * STG + i * 1024), kb, a.w.nkb);
    };
    floatx4_t acc[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i)
        acc[i] = floatx4_t{0.f, 0.f, 0.f, 0.f};
    const int xr = l16 % XR;
    const uint32_t turn = (uint32_t)(a.tile0 + tile) & 7;
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
            const uint16_t *p = a.w.scale + ((int64_t)k0 * NG + g) * a.w.rows;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                ss[g][r + e] = p[min(n0 + r + e, a.w.rows - 1)];
        }
        __syncthreads();
        for (int i = 0; i < n; ++i) {
            const int kc = block(i) - k0;
            fetch(block(i + NST - 1), (i + NST - 1) & (NST - 1));
            ng::wait_vm_steps<LPF, NST - 1>(min(n - 1 - i, NST - 1));
            asm volatile("" ::: "memory");
            const uint8_t *S = Lw + (i & (NST - 1)) * STG, *X = S + NB * 1024 + xr * 256;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                uint32_t wq[NB][MF];
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
                        wq[b][0] = u.x, wq[b][1] = u.y;
                    } else {
                        wq[b][0] = *(const uint32_t *)p;
                    }
                }
                bf16x8_t xf[MF];
#pragma unroll
                for (int i = 0; i < MF; ++i) {
                    const int c = g * (G / 8) + q4 * MF + i;
                    xf[i] = __builtin_bit_cast(bf16x8_t, *(const uint4 *)(X + ((c ^ xr) << 4)));
                }
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    floatx4_t d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < MF; ++i)
                        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp4x8_to_bf16(wq[b][i]), xf[i],
                                                                    d, 0, 0, 0);
                    const uint2 s = *(const uint2 *)&ss[kc * NG + g][b * 16 + q4 * 4];
                    acc[b][0] = fmaf(d[0], bf16_lo(s.x), acc[b][0]);
                    acc[b][1] = fmaf(d[1], bf16_hi(s.x), acc[b][1]);
                    acc[b][2] = fmaf(d[2], bf16_lo(s.y), acc[b][2]);
                    acc[b][3] = fmaf(d[3], bf16_hi(s.y), acc[b][3]);
                }
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
    for (int b = w; b < NB; b += WV) { // joined in wave order
        floatx4_t o = part[0][b][lane];
#pragma unroll
        for (int u = 1; u < WV; ++u)
            o += part[u][b][lane];
        int m = m0 + l16;
        bool mine = l16 < 16;
        if (a.planes == 3) { // a token's three columns: the smallest two first
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float mid = __shfl(o[e], lane + 1, 64), lo = __shfl(o[e], lane + 2, 64);
                o[e] += mid + lo;
            }
            m = m0 + l16 / 3;
            mine = l16 % 3 == 0 && l16 < 15;
        }
        if (!mine || m >= a.T)
            continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int n = n0 + b * 16 + q4 * 4 + e;
            if (n < a.w.rows) {
                if (a.dto == TWELL_BF16)
                    ((uint16_t *)a.out)[m * a.ldo + n] = (uint16_t)f32x2_to_bf16x2(o[e], 0.f);
                else
                    ((float *)a.out)[m * a.ldo + n] = o[e];
            }
        }
    }
}

template <int G, int NB, int XR, int WV, int NST> void rows_one(RowsArgs a, hipStream_t s)
{
    const int tiles = (int)(((int64_t)a.w.rows + 16 * NB - 1) / (16 * NB));
    const int tpt = a.planes == 3 ? 5 : 16;
    const uint32_t mt = (uint32_t)((a.T + tpt - 1) / tpt);
    const int most = (1 << 22) / (int)mt; // threads of a launch are numbered in 32 bits
    for (a.tile0 = 0; a.tile0 < tiles; a.tile0 += a.tiles) {
        a.tiles = tiles - a.tile0 < most ? tiles - a.tile0 : most;
        fp4_rows_kernel<G, NB, XR, WV, NST><<<mt * (uint32_t)a.tiles, 64 * WV, 0, s>>>(a);
    }
}
template <int G> void rows_group(const RowsArgs &a, hipStream_t s)
{
    const int cols = a.R < 16 ? a.R : 16;
    if (cols <= 4)
        rows_one<G, 1, 4, 8, 4>(a, s);
    else
        rows_one<G, 2, 16, 8, 2>(a, s);
}

// ---------------------------------------------------------------- many tokens
// The values as bfloat16 in the workspace, then a dense product on the shared
// main loop, over a float32 token's three rows in turn.
struct GemmArgs {
    Acts x;
    const uint8_t *w; // [n][k] (X W^T) or [k][n] (dY W), zeros past the contraction
    int64_t wpitch;
    int N, NW; // columns of the result, rows (X W^T) or columns (dY W) of w
    void *out;
    int64_t ldo;
    int dto;
};

template <class C, int LB> __global__ __launch_bounds__(C::NT) void fp4_gemm_kernel(GemmArgs a)
{
    __shared__ __attribute__((aligned(16))) uint8_t L[C::LDS];
    constexpr int KS = C::ROWB / 2;
    const int nt = (a.N + C::BN - 1) / C::BN, mt = (a.x.T + C::BM - 1) / C::BM;
    const int steps = a.x.nkb * (FP4_BLK / KS);
    const int lane = threadIdx.x & 63, wm = ng::wave_m<C>(), wn = ng::wave_n<C>();
    for (int64_t q = blockIdx.x; q < (int64_t)nt * mt; q += gridDim.x) {
        const int m0 = (int)(q % mt) * C::BM, n0 = (int)(q / mt) * C::BN;
        auto rowa = [&](int r) { return a.x.data + (int64_t)min(m0 + r, a.x.T - 1) * a.x.pitch; };
        auto rowb = [&](int r) {
            return LB == ng::KC ? a.w + (int64_t)min(n0 + r, a.NW - 1) * a.wpitch
                                : a.w + (int64_t)r * a.wpitch + (int64_t)n0 * 2;
        };
        auto off = [&](int kt) {
            const int p = kt / steps, k = kt % steps;
            return ng::StepOff{(size_t)(p * a.x.plane + (int64_t)k * C::ROWB),
                               (size_t)(LB == ng::KC ? (int64_t)k * C::ROWB
                                                     : (int64_t)k * KS * a.wpitch)};
        };
        ng::Acc<C> acc;
        if constexpr (LB == ng::KC)
            ng::mainloop<C, TWELL_BF16>(L, rowa, rowb, off, 0, steps * a.x.planes, acc);
        else
            ng::mainloop_mixed<C, TWELL_BF16, ng::KC, ng::KM>(L, rowa, rowb, off, 0,
                                                             steps * a.x.planes, acc, 1 << 30,
                                                             a.NW - n0);
#pragma unroll
        for (int mi = 0; mi < C::MI; ++mi)
#pragma unroll
            for (int ni = 0; ni < C::NI; ++ni)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int m = m0 + ng::acc_row<C>(wm, mi, e, lane);
                    const int n = n0 + ng::acc_col<C>(wn, ni, lane);
                    if (m < a.x.T && n < a.N) {
                        const float v = acc.v[mi][ni][e];
                        if (a.dto == TWELL_BF16)
                            ((uint16_t *)a.out)[m * a.ldo + n] = (uint16_t)f32x2_to_bf16x2(v, 0.f);
                        else
                            ((float *)a.out)[m * a.ldo + n] = v;
                    }
                }
    }
}

using C64 = ng::Cfg<64, 128, 2, 4, 4, 64>;
using C256 = ng::Cfg<256, 256, 2, 4, 2, 128>;

template <class C, int LB> void gemm_one(const GemmArgs &a, hipStream_t s)
{
    const int64_t tiles = (int64_t)((a.N + C::BN - 1) / C::BN) * ((a.x.T + C::BM - 1) / C::BM);
    const uint32_t grid = (uint32_t)(tiles < 1 << 20 ? tiles : 1 << 20);
    fp4_gemm_kernel<C, LB><<<grid, C::NT, 0, s>>>(a);
}
template <int LB> void gemm(const GemmArgs &a, hipStream_t s)
{
    const int64_t big = (int64_t)((a.N + 255) / 256) * ((a.x.T + 255) / 256);
    if (big >= 128)
        gemm_one<C256, LB>(a, s);
    else
        gemm_one<C64, LB>(a, s);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }
bool few(int T, int planes) { return T * (int64_t)planes <= 64; }

} // namespace

void fp4_dequant(const Fp4 &w, void *out, int64_t ld, int dt, int rows, int cols, hipStream_t s);

void fp4_rows(const Acts &x, const Fp4 &w, void *out, int64_t ldo, int dto, hipStream_t s)
{
    const RowsArgs a = {x.data, x.planes == 3 ? x.plane : x.pitch, x.T, x.planes, x.T * x.planes,
                        w, out, ldo, dto, 0, 0};
    if (w.group == 32)
        rows_group<32>(a, s);
    else if (w.group == 64)
        rows_group<64>(a, s);
    else
        rows_group<128>(a, s);
}

// Workspace: the packed activations, then the weights' values. dx: of dY W.
size_t fp4_mm_workspace(const twell_mat_t *x, int rows, int cols, bool dx)
{
    const size_t pack = fp4_pack_bytes(x);
    if (!dx && few(x->rows, x->dtype == TWELL_BF16 ? 1 : 3))
        return pack;
    const size_t r = dx ? (size_t)fp4_blocks(rows) * FP4_BLK : rows;
    return up256(pack) + r * fp4_blocks(cols) * FP4_BLK * 2;
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
    if (!dx && few(a.T, a.planes)) {
        fp4_rows(a, w, out->data, out->ld, out->dtype, s);
        tm.mark("fp4_rows");
    } else {
        uint8_t *wv = (uint8_t *)ws + up256(fp4_pack_bytes(x));
        const int cols = w.nkb * FP4_BLK, rows = dx ? fp4_blocks(w.rows) * FP4_BLK : w.rows;
        fp4_dequant(w, wv, cols, TWELL_BF16, rows, cols, s);
        tm.mark("fp4_dequant");
        const GemmArgs g = {a, wv, (int64_t)cols * 2, dx ? w.cols : w.rows, dx ? cols : rows,
                            out->data, out->ld, (int)out->dtype};
        dx ? gemm<ng::KM>(g, s) : gemm<ng::KC>(g, s);
        tm.mark("fp4_gemm");
    }
    return hipGetLastError() == hipSuccess ? TWELL_OK : TWELL_E_HIP;
}
