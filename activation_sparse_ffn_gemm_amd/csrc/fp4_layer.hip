// The sparse layer y = (ReLU(x Wg^T) * (x Wu^T)) Wd for few tokens with its
// matrices in 4 bits (the layer of decode.hip, whose weights' bytes are the
// time, at a quarter of them).
//  1. g = x Wg^T and u = x Wu^T in one kernel, the product of few tokens, whose
//     results are a = g u where g's gate is open. u is formed of every neuron:
//     up to 2^26 weights that is sooner done than a second launch that waits for
//     the gates and gathers rows (one token, 1% open, 2304 x 6144: 11.6 against
//     18.1 us of the layer; 4096 x 8192: 14.5 against 25.2, 20% open 21 against 94). Past that
//     the gates go first and a second kernel reads wu's rows of the open ones
//     (4096 x 32768, 1% open: 43 against 47). More than one tile of tokens takes
//     the product of many tokens, its contraction in parts, and a small kernel
//     that adds the parts and forms a.
//  2. down: a workgroup takes a slice of a token's columns; its waves share the
//     neurons, gather the slice of wd's row for the open gates, and their sums
//     meet in LDS in a fixed order.
#include "fp4.hpp"

namespace {

struct LayerArgs {
    int T, d, f;
    Fp4 wd;
    float *a; // [T][f]
    float *y;
};

constexpr int LW = 8; // waves of a workgroup

// a of the parts' sums of gates and up products, [parts][T][2 f]; four a thread.
__global__ __launch_bounds__(64) void fp4_act_kernel(const float *gu, int parts, int T, int f, float *a)
{
    const int64_t q = ((int64_t)blockIdx.x * 64 + threadIdx.x) * 4;
    if (q >= (int64_t)T * f)
        return;
    const int64_t t = q / f, n = q % f, stride = (int64_t)T * 2 * f;
    const float *p = gu + t * 2 * f + n;
    floatx4_t g = {0.f, 0.f, 0.f, 0.f}, u = g;
    for (int k = 0; k < parts; k += 4) { // in order, four in flight
        floatx4_t v[4], w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float *s = p + min(k + i, parts - 1) * stride;
            v[i] = *(const floatx4_t *)s, w[i] = *(const floatx4_t *)(s + f);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (k + i < parts)
                g += v[i], u += w[i];
    }
    *(floatx4_t *)(a + q) = floatx4_t{fp4_act(g[0], u[0]), fp4_act(g[1], u[1]),
                                      fp4_act(g[2], u[2]), fp4_act(g[3], u[3])};
}

// A wave takes 64 neurons of a token, whose gates are in a: it goes through the
// open ones, all lanes on a row of wu.
struct UpArgs {
    const void *x;
    int64_t ldx;
    int dt, T, d, f;
    Fp4 w;
    float *a;
};
__global__ __launch_bounds__(64 * LW) void fp4_up_kernel(UpArgs p)
{
    constexpr int DEEP = 4; // pieces of 512 columns in flight
    const int lane = threadIdx.x & 63, nc = p.f / 64, shift = 31 - __builtin_clz(p.w.group);
    const int item = (int)blockIdx.x * LW + wave_id();
    if (item >= p.T * nc)
        return;
    const int t = item / nc, n = item % nc * 64;
    float *ap = p.a + (int64_t)t * p.f + n + lane;
    const float g = *ap;
    const void *x = row_ptr(p.x, p.dt, p.ldx, t);
    float a = __uint_as_float(FP4_CLOSED);
    for (uint64_t open = __ballot(!(g <= 0.f)); open; open &= open - 1) {
        const int i = __builtin_ctzll(open);
        const uint8_t *row = p.w.q + (int64_t)(n + i) * p.w.pitch;
        float u = 0.f;
        for (int j0 = 8 * lane; j0 < p.d + 8 * lane; j0 += 512 * DEEP) {
            uint32_t q[DEEP];
            uint16_t s[DEEP];
            uint4 lo[DEEP], hi[DEEP];
#pragma unroll
            for (int k = 0; k < DEEP; ++k) { // (d is a multiple of 64; past it: not counted)
                const int j = min(j0 + 512 * k, p.d - 8);
                q[k] = *(const uint32_t *)(row + j / 2);
                s[k] = p.w.scale[(int64_t)(j >> shift) * p.f + n + i];
                if (p.dt == TWELL_BF16) {
                    lo[k] = ldg16u((const uint16_t *)x + j);
                } else {
                    lo[k] = ldg16u((const float *)x + j);
                    hi[k] = ldg16u((const float *)x + j + 4);
                }
            }
#pragma unroll
            for (int k = 0; k < DEEP; ++k) {
                float c[8], xv[8], v = 0.f;
                fp4x8_to_f32(q[k], c);
                if (p.dt == TWELL_BF16) {
                    elem<TWELL_BF16>::widen(lo[k], xv);
                } else {
                    elem<TWELL_F32>::widen(lo[k], xv);
                    elem<TWELL_F32>::widen(hi[k], xv + 4);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v = fmaf(c[e], xv[e], v);
                if (j0 + 512 * k < p.d)
                    u = fmaf(v, bf16_to_f32(s[k]), u);
            }
        }
        u = wave_sum(u);
        if (lane == i)
            a = fp4_act(g, u);
    }
    *ap = a;
}

// LPR: lanes of a row, eight columns each (a slice is 8 LPR columns)
constexpr int UB = 16; // sets of 64 neurons that a wave lists at a time
template <int LPR> __global__ __launch_bounds__(64 * LW) void fp4_down_kernel(LayerArgs p)
{
    constexpr int RPW = 64 / LPR, COLS = 8 * LPR, DEEP = 8; // rows of a load, loads in flight
    __shared__ int li[LW][64 * UB];
    __shared__ float la[LW][64 * UB];
    __shared__ float red[LW * RPW][COLS];
    const int lane = threadIdx.x & 63, w = wave_id(), sub = lane / LPR;
    const int nsl = (p.d + COLS - 1) / COLS, t = (int)blockIdx.x / nsl, sl = (int)blockIdx.x % nsl;
    const int word = sl * LPR + lane % LPR;
    const bool in = word * 8 < p.d;
    const float *ap = p.a + (int64_t)t * p.f;
    const uint8_t *wq = p.wd.q + (in ? word * 4 : 0);
    const uint16_t *ws = p.wd.scale + (int64_t)(in ? word * 8 / p.wd.group : 0) * p.f;
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        acc[e] = 0.f;
    const int nu = p.f / 64;
    for (int u0 = w; u0 < nu; u0 += LW * UB) {
        uint32_t a[UB];
#pragma unroll
        for (int u = 0; u < UB; ++u)
            a[u] = u0 + LW * u < nu ? __float_as_uint(ap[(u0 + LW * u) * 64 + lane]) : FP4_CLOSED;
        int n = 0;
#pragma unroll
        for (int u = 0; u < UB; ++u) {
            const uint64_t m = __ballot(a[u] != FP4_CLOSED);
            if (a[u] != FP4_CLOSED) {
                const int at = n + __popcll(m & ((1ull << lane) - 1));
                li[w][at] = (u0 + LW * u) * 64 + lane;
                la[w][at] = __uint_as_float(a[u]);
            }
            n += __popcll(m);
        }
        __builtin_amdgcn_wave_barrier();
        for (int i = 0; i < n; i += DEEP * RPW) {
            uint32_t q[DEEP];
            float s[DEEP], v[DEEP];
#pragma unroll
            for (int k = 0; k < DEEP; ++k) {
                const int e = i + k * RPW + sub, r = li[w][min(e, n - 1)];
                q[k] = *(const uint32_t *)(wq + (int64_t)r * p.wd.pitch);
                s[k] = bf16_to_f32(ws[r]);
                v[k] = la[w][min(e, n - 1)];
            }
#pragma unroll
            for (int k = 0; k < DEEP; ++k)
                if (i + k * RPW + sub < n) {
                    float c[8];
                    fp4x8_to_f32(q[k], c);
                    const float f = v[k] * s[k];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        acc[e] = fmaf(f, c[e], acc[e]);
                }
        }
        __builtin_amdgcn_wave_barrier();
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        red[w * RPW + sub][lane % LPR * 8 + e] = acc[e];
    __syncthreads();
    const int c = sl * COLS + threadIdx.x;
    if (threadIdx.x < COLS && c < p.d) {
        float v = red[0][threadIdx.x];
#pragma unroll
        for (int u = 1; u < LW * RPW; ++u)
            v += red[u][threadIdx.x];
        p.y[(int64_t)t * p.d + c] = v;
    }
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

} // namespace

// Workspace: the packed activations, a, the parts of the gates and up products.
size_t fp4_layer_workspace(const twell_mat_t *x, int d_ff)
{
    const size_t a = up256((size_t)x->rows * d_ff * 4);
    return up256(fp4_pack_bytes(x)) + a * (1 + 2 * fp4_gates_parts(x, d_ff));
}

hipError_t launch_fp4_layer(const twell_mat_t *x, const twell_fp4_t *wg, const twell_fp4_t *wu,
                            const twell_fp4_t *wd, float *y, void *ws, twell_timing_t *timing,
                            hipStream_t s)
{
    Timer tm(timing, s);
    bool packed;
    const Acts acts = fp4_pack(x, ws, s, &packed);
    if (packed)
        tm.mark("fp4_pack");
    const int T = x->rows, d = x->cols, f = wg->rows, parts = fp4_gates_parts(x, f);
    float *a = (float *)((uint8_t *)ws + up256(fp4_pack_bytes(x)));
    const Fp4 g = fp4_arg(wg), u = fp4_arg(wu);
    if (parts > 0) {
        float *gu = a + up256((size_t)T * f * 4) / 4;
        fp4_gates(acts, g, u, gu, s);
        tm.mark("fp4_gates");
        fp4_act_kernel<<<(uint32_t)(((int64_t)T * f / 4 + 63) / 64), 64, 0, s>>>(gu, parts, T, f, a);
        tm.mark("fp4_act");
    } else if ((int64_t)f * d <= 1 << 26) { // (see the top)
        fp4_rows(acts, g, &u, a, f, TWELL_F32, s);
        tm.mark("fp4_gate_up");
    } else {
        fp4_rows(acts, g, nullptr, a, f, TWELL_F32, s);
        tm.mark("fp4_gate");
        const UpArgs p = {x->data, x->ld, (int)x->dtype, T, d, f, u, a};
        fp4_up_kernel<<<(uint32_t)((T * (f / 64) + LW - 1) / LW), 64 * LW, 0, s>>>(p);
        tm.mark("fp4_up");
    }
    const LayerArgs p = {T, d, f, fp4_arg(wd), a, y};
    // a slice of 512 columns reads the gates' list least often, one of 128 fills the
    // chip for few tokens
    const int64_t wide = T * ((d + 511) / 512), slices = T * ((d + 127) / 128);
    if (wide >= 256)
        fp4_down_kernel<64><<<(uint32_t)wide, 64 * LW, 0, s>>>(p);
    else
        fp4_down_kernel<16><<<(uint32_t)slices, 64 * LW, 0, s>>>(p);
    tm.mark("fp4_down");
    return hipGetLastError();
}
