// The sparse layer y = (ReLU(x Wg^T) * (x Wu^T)) Wd for few tokens with its
// matrices in 4 bits (the layer of decode.hip, whose weights' bytes are the
// time, at a quarter of them). Three launches:
//  1. g = x Wg^T, the product of few tokens.
//  2. up: a wave takes 64 neurons of a token; for each open gate it reads wu's
//     row, a = g u takes g's place in the workspace.
//  3. down: a workgroup takes 512 columns of a token; its waves share the
//     neurons, each gathers the piece of wd's row for its open gates, and their
//     sums meet in LDS in a fixed order.
#include "fp4.hpp"

namespace {

constexpr int LW = 8; // waves of a workgroup
// a of a closed gate: the one float that an open gate's a, a sum with +0, is not
constexpr uint32_t CLOSED = 0x80000000u;

struct LayerArgs {
    const void *x;
    int64_t ldx;
    int dt, T, d, f;
    Fp4 wu, wd;
    float *a; // [T][f]: g, then a
    float *y;
};

// NW: dwords (eight columns) of a row in a lane
template <int NW> __global__ __launch_bounds__(64 * LW) void fp4_up_kernel(LayerArgs p)
{
    const int lane = threadIdx.x & 63, nc = p.f / 64;
    const int item = (int)blockIdx.x * LW + wave_id();
    if (item >= p.T * nc)
        return;
    const int t = item / nc, n0 = item % nc * 64;
    float *ap = p.a + (int64_t)t * p.f + n0 + lane;
    const float g = *ap;
    uint64_t open = __ballot(!(g <= 0.f));
    float a = __uint_as_float(CLOSED);
    if (open) {
        float x[NW][8];
#pragma unroll
        for (int w = 0; w < NW; ++w)
            load8(row_ptr(p.x, p.dt, p.ldx, t), p.dt, 8 * (lane + 64 * w), p.d, x[w]);
        while (open) {
            const int i = __builtin_ctzll(open);
            open &= open - 1;
            const uint8_t *row = p.wu.q + (int64_t)(n0 + i) * p.wu.pitch;
            float u = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const int word = lane + 64 * w;
                if (word * 8 < p.d) {
                    float c[8], v = 0.f;
                    fp4x8_to_f32(*(const uint32_t *)(row + word * 4), c);
                    const float s = bf16_to_f32(
                        p.wu.scale[(int64_t)(word * 8 / p.wu.group) * p.f + n0 + i]);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v = fmaf(c[e], x[w][e], v);
                    u = fmaf(v, s, u);
                }
            }
            u = wave_sum(u);
            if (lane == i)
                a = g * u + 0.f;
        }
    }
    *ap = a;
}

constexpr int UB = 8; // sets of 64 neurons that a wave lists at a time
__global__ __launch_bounds__(64 * LW) void fp4_down_kernel(LayerArgs p)
{
    __shared__ int li[LW][64 * UB];
    __shared__ float la[LW][64 * UB];
    __shared__ float red[LW][64 * 8];
    const int lane = threadIdx.x & 63, w = wave_id();
    const int nsl = (p.d + 511) / 512, t = (int)blockIdx.x / nsl;
    const int word = (int)blockIdx.x % nsl * 64 + lane;
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
            a[u] = u0 + LW * u < nu ? __float_as_uint(ap[(u0 + LW * u) * 64 + lane]) : CLOSED;
        int n = 0;
#pragma unroll
        for (int u = 0; u < UB; ++u) {
            const uint64_t m = __ballot(a[u] != CLOSED);
            if (a[u] != CLOSED) {
                const int at = n + __popcll(m & ((1ull << lane) - 1));
                li[w][at] = (u0 + LW * u) * 64 + lane;
                la[w][at] = __uint_as_float(a[u]);
            }
            n += __popcll(m);
        }
        __builtin_amdgcn_wave_barrier();
        for (int i = 0; i < n; i += 8) {
            uint32_t q[8];
            float s[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int r = li[w][min(i + k, n - 1)];
                q[k] = *(const uint32_t *)(wq + (int64_t)r * p.wd.pitch);
                s[k] = bf16_to_f32(ws[r]);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (i + k < n) {
                    float c[8];
                    fp4x8_to_f32(q[k], c);
                    const float v = la[w][i + k] * s[k];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        acc[e] = fmaf(v, c[e], acc[e]);
                }
        }
        __builtin_amdgcn_wave_barrier();
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        red[w][lane * 8 + e] = acc[e];
    __syncthreads();
    const int c = (int)blockIdx.x % nsl * 512 + threadIdx.x;
    if (c < p.d) {
        float v = red[0][threadIdx.x];
#pragma unroll
        for (int u = 1; u < LW; ++u)
            v += red[u][threadIdx.x];
        p.y[(int64_t)t * p.d + c] = v;
    }
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

void launch_up(const LayerArgs &p, hipStream_t s)
{
    const uint32_t grid = (uint32_t)((p.T * (p.f / 64) + LW - 1) / LW);
    switch ((p.d + 511) / 512) {
    case 1: fp4_up_kernel<1><<<grid, 64 * LW, 0, s>>>(p); break;
    case 2: fp4_up_kernel<2><<<grid, 64 * LW, 0, s>>>(p); break;
    case 3: fp4_up_kernel<3><<<grid, 64 * LW, 0, s>>>(p); break;
    case 4: fp4_up_kernel<4><<<grid, 64 * LW, 0, s>>>(p); break;
    case 5: fp4_up_kernel<5><<<grid, 64 * LW, 0, s>>>(p); break;
    case 6: fp4_up_kernel<6><<<grid, 64 * LW, 0, s>>>(p); break;
    case 7: fp4_up_kernel<7><<<grid, 64 * LW, 0, s>>>(p); break;
    default: fp4_up_kernel<8><<<grid, 64 * LW, 0, s>>>(p); break; // d <= 4096
    }
}

} // namespace

size_t fp4_layer_workspace(const twell_mat_t *x, int d_ff)
{
    return up256(fp4_pack_bytes(x)) + (size_t)x->rows * d_ff * 4;
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
    const LayerArgs p = {x->data, x->ld, (int)x->dtype, x->rows, x->cols, wg->rows,
                         fp4_arg(wu), fp4_arg(wd), a, y};
    fp4_rows(acts, fp4_arg(wg), a, p.f, TWELL_F32, s);
    tm.mark("fp4_rows");
    launch_up(p, s);
    tm.mark("fp4_up");
    fp4_down_kernel<<<(uint32_t)(p.T * ((p.d + 511) / 512)), 64 * LW, 0, s>>>(p);
    tm.mark("fp4_down");
    return hipGetLastError();
}
