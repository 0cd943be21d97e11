// The sparse layer y = (ReLU(x Wg^T) * (x Wu^T)) Wd for few tokens with its
// matrices in 4 bits (the layer of decode.hip, whose weights' bytes are the
// time, at a quarter of them).
//  1. g = x Wg^T, the product of few tokens, and, in the same kernel, where a
//     neuron's gate is open, wu's row and a = g u. More than one tile of tokens
//     takes the product of many tokens, its contraction in parts, and a second
//     kernel that adds the parts and goes on to a.
//  2. down: a workgroup takes a slice of a token's columns; its waves share the
//     neurons, gather the slice of wd's row for the open gates, and their sums
//     meet in LDS in a fixed order.
#include "fp4.hpp"

namespace {

struct LayerArgs {
    int T, d, f, parts;
    Fp4Up up;
    Fp4 wd;
    const float *g; // [parts][T][f]
    float *a;       // [T][f]
    float *y;
};

// A wave takes 64 neurons of a token.
constexpr int LW = 8; // waves of a workgroup
__global__ __launch_bounds__(64 * LW) void fp4_up_kernel(LayerArgs p)
{
    const int lane = threadIdx.x & 63, nc = p.f / 64;
    const int item = (int)blockIdx.x * LW + wave_id();
    if (item >= p.T * nc)
        return;
    const int t = item / nc, n = item % nc * 64 + lane;
    const int64_t at = (int64_t)t * p.f + n;
    float g = 0.f;
    for (int k = 0; k < p.parts; k += 8) { // in order, eight in flight
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = p.g[at + (int64_t)min(k + i, p.parts - 1) * p.T * p.f];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k + i < p.parts)
                g += v[i];
    }
    p.a[at] = fp4_up(p.up, g, t, n);
}

// LPR: lanes of a row, eight columns each (a slice is 8 LPR columns)
constexpr int UB = 8; // sets of 64 neurons that a wave lists at a time
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

// Workspace: the packed activations, a, the parts of g.
size_t fp4_layer_workspace(const twell_mat_t *x, int d_ff)
{
    const size_t a = up256((size_t)x->rows * d_ff * 4);
    const int parts = fp4_gate_parts(x, d_ff);
    return up256(fp4_pack_bytes(x)) + a * (1 + parts);
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
    float *a = (float *)((uint8_t *)ws + up256(fp4_pack_bytes(x)));
    float *g = a + up256((size_t)x->rows * wg->rows * 4) / 4;
    const LayerArgs p = {x->rows, x->cols, wg->rows, fp4_gate_parts(x, wg->rows),
                         {x->data, x->ld, (int)x->dtype, x->cols, fp4_arg(wu)},
                         fp4_arg(wd), g, a, y};
    if (p.parts == 0) {
        fp4_rows(acts, fp4_arg(wg), a, p.f, TWELL_F32, &p.up, s);
        tm.mark("fp4_gate_up");
    } else {
        fp4_gate(acts, fp4_arg(wg), g, s);
        tm.mark("fp4_gate");
        fp4_up_kernel<<<(uint32_t)((p.T * (p.f / 64) + LW - 1) / LW), 64 * LW, 0, s>>>(p);
        tm.mark("fp4_up");
    }
    // a slice of 512 columns reads the gates' list least often, one of 128 fills
    // the chip for few tokens
    if (p.T * ((p.d + 511) / 512) >= 256)
        fp4_down_kernel<64><<<(uint32_t)(p.T * ((p.d + 511) / 512)), 64 * LW, 0, s>>>(p);
    else
        fp4_down_kernel<16><<<(uint32_t)(p.T * ((p.d + 127) / 128)), 64 * LW, 0, s>>>(p);
    tm.mark("fp4_down");
    return hipGetLastError();
}
