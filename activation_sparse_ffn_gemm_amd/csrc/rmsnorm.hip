// Root-mean-square norm of a residual stream, forward and backward.
//
// Forward, per row: h = residual + x (float32), r = 1 / sqrt(mean(h^2) + eps),
// n = h r gain. Everything is one pass: a row stays in registers between the
// sum of squares and the output, in float32; h and n are each rounded once,
// when they are stored (the norm is of the unrounded h). 8-bit output: the
// lanes of a 16-lane group hold 128 consecutive columns (eight each), so a
// block's amax is four DPP moves away and q is written from registers.
//
// Backward, per row, with xh = h r and dg = dn gain:
//   dh = r (dg - xh mean(dg xh)) + dres,   dgain = sum over rows of dn xh.
// r is formed again from h: the two sums the row needs anyway (h^2, dg h) are
// taken in the same pass, and nothing has to be kept from the forward.
// dgain: every workgroup sums its rows in registers, in row order, writes one
// partial row of float32, and a second kernel adds the partial rows in
// workgroup order: results repeat bit for bit (no atomics).
//
// Both are bound by HBM: each array is read or written once.
#include "fp8.hpp"

namespace {

constexpr int NT = 256; // threads of a workgroup

// Sum over the LPR lanes that share a row: a wave, or the whole workgroup
// (through buf, NT / 64 floats; the caller gives a buffer of its own to each
// sum, so no barrier is needed before the write).
template <int LPR> DEVI float row_sum(float v, float *buf)
{
    v = wave_sum(v);
    if constexpr (LPR == 64)
        return v;
    const int w = wave_id();
    if ((threadIdx.x & 63) == 0)
        buf[w] = v;
    __syncthreads();
    return (buf[0] + buf[1]) + (buf[2] + buf[3]);
}

struct FwdArgs {
    const void *x, *res, *gain;
    void *h, *n;
    uint8_t *q;
    float *scale;
    int64_t ldx, ldr, ldh, ldn;
    int T, d, dtx, dtr, dtg, dtn;
    float eps;
};

template <int LPR, int C> __global__ __launch_bounds__(NT) void rmsnorm_fwd_kernel(FwdArgs a)
{
    constexpr int RPB = NT / LPR; // rows per workgroup
    __shared__ float buf[NT / 64];
    const int lane = LPR == 64 ? threadIdx.x & 63 : threadIdx.x;
    const int64_t t = (int64_t)blockIdx.x * RPB + (LPR == 64 ? wave_id() : 0);
    if (t >= a.T)
        return; // LPR == 64 only: a whole wave, and no barrier follows
    const int d = a.d;
    Row<LPR, C> h;
    {
        const void *px = row_ptr(a.x, a.dtx, a.ldx, t);
        h.load(px, a.dtx, d, lane);
        if (a.res) {
            Row<LPR, C> r;
            const void *pr = row_ptr(a.res, a.dtr, a.ldr, t);
            r.load(pr, a.dtr, d, lane);
            h.widen(px, a.dtx, d, lane);
            r.widen(pr, a.dtr, d, lane);
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    h.v[c][i] += r.v[c][i];
            h.store(row_ptr(a.h, a.dtr, a.ldh, t), a.dtr, d, lane);
        } else {
            h.widen(px, a.dtx, d, lane);
        }
    }
    Row<LPR, C> g;
    g.load(a.gain, a.dtg, d, lane);
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            ss = fmaf(h.v[c][i], h.v[c][i], ss);
    ss = row_sum<LPR>(ss, buf);
    const float r = 1.f / sqrtf(ss / (float)d + a.eps);
    g.widen(a.gain, a.dtg, d, lane);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            h.v[c][i] = h.v[c][i] * r * g.v[c][i];
    if (!a.q) {
        h.store(row_ptr(a.n, a.dtn, a.ldn, t), a.dtn, d, lane);
        return;
    }
    const int64_t pitch = fp8_pitch(d);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int j = 8 * (lane + LPR * c);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = abs_bits(h.v[c][i]);
            m = b > m ? b : m;
        }
        const float s = fp8_scale(row16_umax(m));
        if (j < pitch) {
            *(uint2 *)(a.q + t * pitch + j) = quant8(h.v[c], s, 1.f / s);
            if ((lane & 15) == 0)
                a.scale[(int64_t)(j / FP8_BLK) * a.T + t] = s;
        }
    }
}

struct BwdArgs {
    const void *dn, *h, *gain, *dres;
    void *dh;
    float *part; // [workgroups][d]
    int64_t lddn, ldh, lddres, lddh;
    int T, d, dtdn, dth, dtg, dtdres, dtdh;
    float eps;
};

template <int LPR, int C> __global__ __launch_bounds__(NT) void rmsnorm_bwd_kernel(BwdArgs a)
{
    constexpr int RPB = NT / LPR;
    extern __shared__ float lds[]; // LPR == 64: d floats (the waves' dgain sums)
    __shared__ float buf[2][2][NT / 64];
    const int lane = LPR == 64 ? threadIdx.x & 63 : threadIdx.x;
    const int w = LPR == 64 ? wave_id() : 0;
    const int d = a.d;
    float acc[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc[c][i] = 0.f;
    int it = 0;
    for (int64_t t = (int64_t)blockIdx.x * RPB + w; t < a.T; t += (int64_t)gridDim.x * RPB, ++it) {
        Row<LPR, C> h, dn, g;
        const void *ph = row_ptr(a.h, a.dth, a.ldh, t), *pd = row_ptr(a.dn, a.dtdn, a.lddn, t);
        h.load(ph, a.dth, d, lane);
        dn.load(pd, a.dtdn, d, lane);
        g.load(a.gain, a.dtg, d, lane);
        h.widen(ph, a.dth, d, lane);
        dn.widen(pd, a.dtdn, d, lane);
        g.widen(a.gain, a.dtg, d, lane);
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ss = fmaf(h.v[c][i], h.v[c][i], ss);
                g.v[c][i] *= dn.v[c][i];
                dot = fmaf(g.v[c][i], h.v[c][i], dot);
            }
        // two buffers in turn: a wave may still read the last row's sums
        ss = row_sum<LPR>(ss, buf[it & 1][0]);
        dot = row_sum<LPR>(dot, buf[it & 1][1]);
        const float r = 1.f / sqrtf(ss / (float)d + a.eps);
        const float m = dot * r / (float)d; // mean(dg xh)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float xh = h.v[c][i] * r;
                acc[c][i] = fmaf(dn.v[c][i], xh, acc[c][i]);
                h.v[c][i] = r * fmaf(-xh, m, g.v[c][i]);
            }
        if (a.dres) {
            const void *pr = row_ptr(a.dres, a.dtdres, a.lddres, t);
            dn.load(pr, a.dtdres, d, lane);
            dn.widen(pr, a.dtdres, d, lane);
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    h.v[c][i] += dn.v[c][i];
        }
        h.store(row_ptr(a.dh, a.dtdh, a.lddh, t), a.dtdh, d, lane);
    }
    float *part = a.part + (int64_t)blockIdx.x * d;
    if constexpr (LPR == 64) { // the waves' sums, added in wave order
        for (int q = 0; q < NT / 64; ++q) {
            if (w == q) {
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int j = 8 * (lane + LPR * c) + i;
                        if (j < d)
                            lds[j] = q ? lds[j] + acc[c][i] : acc[c][i];
                    }
            }
            __syncthreads();
        }
        for (int j = threadIdx.x; j < d; j += NT)
            part[j] = lds[j];
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int j = 8 * (lane + LPR * c) + i;
                if (j < d)
                    part[j] = acc[c][i];
            }
    }
}

// dgain[j] = sum of the G partial rows, in row order: 64 columns per
// workgroup, SL slices of consecutive rows, joined in slice order.
constexpr int SL = 16;
__global__ __launch_bounds__(64 * SL) void rmsnorm_dgain_kernel(const float *part, int G, int d,
                                                              float *dgain)
{
    __shared__ float s[SL][64];
    const int lane = threadIdx.x & 63, w = wave_id();
    const int j = blockIdx.x * 64 + lane;
    const int per = (G + SL - 1) / SL, g0 = min(G, w * per), g1 = min(G, g0 + per);
    float v = 0.f;
    if (j < d)
        for (int g = g0; g < g1; ++g)
            v += part[(int64_t)g * d + j];
    s[w][lane] = v;
    __syncthreads();
    if (w == 0 && j < d) {
        for (int q = 1; q < SL; ++q)
            v += s[q][lane];
        dgain[j] = v;
    }
}

// Rows one wave each once there are enough of them to give every SIMD two
// waves; fewer, or longer, rows take a whole workgroup.
constexpr int WAVE_ROWS = 2048;

int bwd_groups(int T, int d)
{
    const int rpb = T >= WAVE_ROWS && d <= 2048 ? 4 : 1;
    const int g = (T + rpb - 1) / rpb;
    return g < 512 ? g : 512;
}

} // namespace

hipError_t launch_rmsnorm_fwd(const twell_mat_t *x, const twell_mat_t *res, const void *gain,
                              int dtg, float eps, const twell_mat_t *h, const twell_mat_t *n,
                              const twell_fp8_t *n8, twell_timing_t *timing, hipStream_t s)
{
    FwdArgs a = {};
    a.x = x->data, a.ldx = x->ld, a.dtx = x->dtype, a.T = x->rows, a.d = x->cols;
    a.gain = gain, a.dtg = dtg, a.eps = eps;
    if (res) {
        a.res = res->data, a.ldr = res->ld, a.dtr = res->dtype;
        a.h = h->data, a.ldh = h->ld;
    }
    if (n8)
        a.q = n8->q, a.scale = n8->scale;
    else
        a.n = n->data, a.ldn = n->ld, a.dtn = n->dtype;
    Timer tm(timing, s);
    const int T = a.T, d = a.d;
    if (T >= WAVE_ROWS && d <= 4096) {
        const dim3 grid((T + 3) / 4);
        if (d <= 512)
            rmsnorm_fwd_kernel<64, 1><<<grid, NT, 0, s>>>(a);
        else if (d <= 1024)
            rmsnorm_fwd_kernel<64, 2><<<grid, NT, 0, s>>>(a);
        else if (d <= 2048)
            rmsnorm_fwd_kernel<64, 4><<<grid, NT, 0, s>>>(a);
        else
            rmsnorm_fwd_kernel<64, 8><<<grid, NT, 0, s>>>(a);
    } else if (d <= 2048) {
        rmsnorm_fwd_kernel<NT, 1><<<T, NT, 0, s>>>(a);
    } else if (d <= 4096) {
        rmsnorm_fwd_kernel<NT, 2><<<T, NT, 0, s>>>(a);
    } else if (d <= 8192) {
        rmsnorm_fwd_kernel<NT, 4><<<T, NT, 0, s>>>(a);
    } else {
        rmsnorm_fwd_kernel<NT, 8><<<T, NT, 0, s>>>(a);
    }
    tm.mark("rmsnorm_fwd");
    return hipGetLastError();
}

size_t rmsnorm_bwd_workspace(int T, int d) { return (size_t)bwd_groups(T, d) * d * 4; }

hipError_t launch_rmsnorm_bwd(const twell_mat_t *dn, const twell_mat_t *h, const void *gain,
                              int dtg, float eps, const twell_mat_t *dres, const twell_mat_t *dh,
                              float *dgain, void *ws, twell_timing_t *timing, hipStream_t s)
{
    BwdArgs a = {};
    a.dn = dn->data, a.lddn = dn->ld, a.dtdn = dn->dtype, a.T = dn->rows, a.d = dn->cols;
    a.h = h->data, a.ldh = h->ld, a.dth = h->dtype;
    a.gain = gain, a.dtg = dtg, a.eps = eps;
    if (dres)
        a.dres = dres->data, a.lddres = dres->ld, a.dtdres = dres->dtype;
    a.dh = dh->data, a.lddh = dh->ld, a.dtdh = dh->dtype;
    a.part = (float *)ws;
    Timer tm(timing, s);
    const int T = a.T, d = a.d, G = bwd_groups(T, d);
    if (T >= WAVE_ROWS && d <= 2048) {
        const size_t lds = (size_t)d * 4;
        if (d <= 512)
            rmsnorm_bwd_kernel<64, 1><<<G, NT, lds, s>>>(a);
        else if (d <= 1024)
            rmsnorm_bwd_kernel<64, 2><<<G, NT, lds, s>>>(a);
        else
            rmsnorm_bwd_kernel<64, 4><<<G, NT, lds, s>>>(a);
    } else if (T > 0) {
        if (d <= 2048)
            rmsnorm_bwd_kernel<NT, 1><<<G, NT, 0, s>>>(a);
        else if (d <= 4096)
            rmsnorm_bwd_kernel<NT, 2><<<G, NT, 0, s>>>(a);
        else if (d <= 8192)
            rmsnorm_bwd_kernel<NT, 4><<<G, NT, 0, s>>>(a);
        else
            rmsnorm_bwd_kernel<NT, 8><<<G, NT, 0, s>>>(a);
    }
    tm.mark("rmsnorm_bwd");
    rmsnorm_dgain_kernel<<<(d + 63) / 64, 64 * SL, 0, s>>>(a.part, G, d, dgain);
    tm.mark("rmsnorm_dgain");
    return hipGetLastError();
}
