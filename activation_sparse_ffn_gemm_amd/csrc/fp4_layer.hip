// The sparse layer y = (ReLU(x Wg^T) * (x Wu^T)) Wd for few tokens with its
// matrices in 4 bits (the layer of decode.hip, whose weights' bytes are the
// time, at a quarter of them).
//  1. g = x Wg^T and u = x Wu^T in one kernel, the product of few tokens, whose
//     results are a = g u where g's gate is open. u is formed of every neuron:
//     a second launch that waits for the gates and gathers wu's rows of the open
//     ones reads fewer bytes and takes longer (one token, 1% open, 2304 x 6144: 15.4
//     against 10.3 us of the layer; 4096 x 8192 22.4 against 13.4; 20% open 90 against
//     21; only at 4096 x 32768 38.7 against 44.5, with 10% open 93 against 60). More
//     than few tokens take the product of many tokens, its contraction in one or two
//     parts, and a small kernel that adds the parts and forms a (4.2 us at 64 x
//     6144, a launch and a trip; forming it where it is read, once for each slice of
//     columns, takes 5.8 more there).
//  2. down: a workgroup takes a slice of a token's columns; its waves share the
//     neurons, gather the slice of wd's row for the open gates, and their sums
//     meet in LDS in a fixed order. Two trips to memory, the gates' and the rows':
//     one token 4.6 us (18 workgroups), 64 tokens 8.4 (320).
// The layer of 2304 x 6144, 1% open: one token 9.9 us, 64 tokens 23.6.
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
    } else {
        fp4_rows(acts, g, &u, a, f, TWELL_F32, s);
        tm.mark("fp4_gate_up");
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
