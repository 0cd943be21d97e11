// Root-mean-square norm of a residual stream, forward and backward.
//
// Forward, per row: h = residual + x (float32), r = 1 / sqrt(mean(h^2) + eps),
// n = h r gain. Everything is one pass: a row stays in registers between the
// sum of squares and the output, in float32; h and n are each rounded once,
// when they are stored (the norm is of the unrounded h).
//
// 8-bit output: the lanes of a 16-lane group hold 128 consecutive columns
// (eight each), so a block's amax is four DPP moves away and q is written from
// registers. The row is taken in 64 bits there, so that q is the e4m3 value
// nearest to n / scale: in 32 bits the roundings of h, h r, h r gain, the scale
// and the quotient put one value in a million on the wrong side of a tie
// between two e4m3 values, a sixteenth off. Beside a residual's memory traffic
// the arithmetic is hidden (8192 x 2048: 28.4 us, bf16 out 29.2); of a bf16 x
// alone, 50 MB, it is the bound (16.2 us).
//
// Backward, per row, with xh = h r and dg = dn gain:
//   dh = r (dg - xh mean(dg xh)) + dres,   dgain = sum over rows of dn xh.
// r is formed again from h: the two sums the row needs anyway (h^2, dg h) are
// taken in the same pass, and nothing has to be kept from the forward.
// dgain: every workgroup sums its rows in registers, in row order, writes one
// partial row of float32, and a second kernel adds the partial rows in
// workgroup order: results repeat bit for bit (no atomics).
//
// Both are bound by HBM: each array is read or written once (8192 x 2048,
// float32 x or dn, bf16 stream: forward 5.2 to 5.7 TB/s, backward 4.8). What is left
// to save beside the traffic is instructions: rows that fill their lanes are
// kernels of their own, without zeroed registers and tests (36 -> 31 us).
#include "fp8.hpp"

namespace {

// Lanes that share a row: every lane holds eight elements, sixteen in rows
// past 8192. Registers stay few (32), so the chip is full of rows in flight;
// rows of 2048 as one wave's 32 elements a lane ran at 3.3 TB/s, as four
// waves' eight at 5.0.
template <int LPR> DEVI int row_lane() { return (int)threadIdx.x % LPR; }

template <int CTRL> DEVI double dpp_mov(double v)
{
    const int2 q = __builtin_bit_cast(int2, v);
    return __builtin_bit_cast(double,
                              make_int2(__builtin_amdgcn_mov_dpp(q.x, CTRL, 0xF, 0xF, false),
                                        __builtin_amdgcn_mov_dpp(q.y, CTRL, 0xF, 0xF, false)));
}
// Maximum over each group of 16 lanes (values that are not negative).
DEVI double row16_max(double v)
{
    v = fmax(v, dpp_mov<0xB1>(v));
    v = fmax(v, dpp_mov<0x4E>(v));
    v = fmax(v, dpp_mov<0x141>(v));
    return fmax(v, dpp_mov<0x140>(v));
}
DEVI float upper_word(double v)
{
    return __uint_as_float((uint32_t)(__builtin_bit_cast(uint64_t, v) >> 32));
}
// 1 / v and 1 / sqrt(v), from the hardware's estimates by a Newton step: within
// 2^-40 or so, where the e4m3 quotient needs 2^-30. 1 / sqrt(infinity) is 0 and
// 1 / sqrt(0) infinity, as the estimate says.
DEVI double rcp64(double v)
{
    const double y = __builtin_amdgcn_rcp(v);
    return fma(fma(-v, y, 1.), y, y);
}
DEVI double rsqrt64(double v)
{
    const double y = __builtin_amdgcn_rsq(v);
    const double z = fma(0.5 * y, fma(-v * y, y, 1.), y);
    return v > 0. && v < __builtin_inf() ? z : y;
}

// Sum over the LPR lanes that share a row, in every one of them. Past a wave
// it goes through buf (a float for each wave of the workgroup); each sum of a
// kernel has a buf of its own, so no barrier is needed before it is written.
DEVI double wave_sum64(double v)
{
    v += dpp_mov<0xB1>(v);
    v += dpp_mov<0x4E>(v);
    v += dpp_mov<0x141>(v);
    v += dpp_mov<0x140>(v);
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}
template <int LPR, class F> DEVI F row_sum(F v, F *buf)
{
    if constexpr (LPR < 64) {
        v += dpp_mov<0xB1>(v);
        v += dpp_mov<0x4E>(v);
        v += dpp_mov<0x141>(v);
        v += dpp_mov<0x140>(v);
        if constexpr (LPR == 32)
            v += __shfl_xor(v, 16, 64);
        return v;
    } else {
        if constexpr (sizeof(F) == 8)
            v = wave_sum64(v);
        else
            v = wave_sum(v);
        if constexpr (LPR > 64) {
            constexpr int W = LPR / 64; // waves of a row
            const int w = wave_id();
            if ((threadIdx.x & 63) == 0)
                buf[w] = v;
            __syncthreads();
            const F *b = buf + w / W * W;
            v = b[0];
#pragma unroll
            for (int i = 1; i < W; ++i)
                v += b[i];
        }
        return v;
    }
}

// Sum of N values by halves: short chains of additions, small errors.
template <int N> DEVI float tree_sum(const float *p)
{
    if constexpr (N == 1)
        return p[0];
    else
        return tree_sum<N / 2>(p) + tree_sum<N / 2>(p + N / 2);
}

// The same of W <= 16 values in LDS, a lane of each W taking one of them.
template <int W> DEVI float tree_sum_lanes(const float *p)
{
    float v = p[threadIdx.x & (W - 1)];
    if constexpr (W > 1)
        v += dpp_mov<0xB1>(v);
    if constexpr (W > 2)
        v += dpp_mov<0x4E>(v);
    if constexpr (W > 4)
        v += dpp_mov<0x141>(v);
    if constexpr (W > 8)
        v += dpp_mov<0x140>(v);
    return v;
}

// Two float sums over a row's lanes with one barrier. FEW: without the 32
// registers that a row's sixteen pairs take in every lane, which rows of two
// chunks a lane do not have (in scratch 2000 x 16384 took 105 us, so 102; 2000 x
// 16383 124 and 112; rows of one chunk lose 1%).
template <int LPR, bool FEW> DEVI void row_sum2(float &u, float &v, float *bu, float *bv)
{
    if constexpr (LPR <= 64) {
        u = row_sum<LPR>(u, bu), v = row_sum<LPR>(v, bv);
    } else {
        constexpr int W = LPR / 64;
        const int w = wave_id();
        u = wave_sum(u), v = wave_sum(v);
        if ((threadIdx.x & 63) == 0)
            bu[w] = u, bv[w] = v;
        __syncthreads();
        const int w0 = w / W * W;
        if constexpr (FEW)
            u = tree_sum_lanes<W>(bu + w0), v = tree_sum_lanes<W>(bv + w0);
        else
            u = tree_sum<W>(bu + w0), v = tree_sum<W>(bv + w0);
    }
}

struct FwdArgs {
    const void *x, *res, *gain;
    void *h, *n;
    uint8_t *q;
    float *scale;
    int64_t ldx, ldr, ldh, ldn;
    int T, d, dtx, dtr, dtg, dtn;
    int t0; // the launch's first row
    float eps;
    double inv_d; // 1 / d
};

constexpr int fwd_threads(int lpr) { return lpr < 256 ? 256 : lpr; }

template <int LPR, int C, RowKind KIND>
__global__ __launch_bounds__(fwd_threads(LPR)) void rmsnorm_fwd_kernel(FwdArgs a)
{
    constexpr int RPB = fwd_threads(LPR) / LPR; // rows per workgroup
    __shared__ float buf[fwd_threads(LPR) / 64];
    const int lane = row_lane<LPR>();
    const int64_t t = a.t0 + (int64_t)blockIdx.x * RPB + (LPR >= 64 ? wave_id() * 64 : (int)threadIdx.x) / LPR;
    // a workgroup's rows past T store nothing; they read the last row
    const int d = t < a.T ? a.d : 0;
    const int64_t tl = t < a.T ? t : a.T - 1;
    Row<LPR, C, KIND> h, g;
    h.load(row_ptr(a.x, a.dtx, a.ldx, tl), a.dtx, a.d, lane);
    if (a.res) {
        Row<LPR, C, KIND> r;
        r.load(row_ptr(a.res, a.dtr, a.ldr, tl), a.dtr, a.d, lane);
        g.load(a.gain, a.dtg, a.d, lane);
        h.widen(a.dtx);
        r.widen(a.dtr);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h.v[c][i] += r.v[c][i];
        h.template store<true>(row_ptr(a.h, a.dtr, a.ldh, t), a.dtr, d, lane);
    } else {
        g.load(a.gain, a.dtg, a.d, lane);
        h.widen(a.dtx);
    }
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            ss = fmaf(h.v[c][i], h.v[c][i], ss);
    ss = row_sum<LPR>(ss, buf);
    const float r = 1.f / sqrtf(ss / (float)a.d + a.eps);
    g.widen(a.dtg);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            h.v[c][i] = h.v[c][i] * r * g.v[c][i];
    h.template store<true>(row_ptr(a.n, a.dtn, a.ldn, t), a.dtn, d, lane);
}

// The same with n in 8 bits.
template <int LPR, int C, RowKind KIND>
__global__ __launch_bounds__(fwd_threads(LPR)) void rmsnorm_fwd8_kernel(FwdArgs a)
{
    constexpr int RPB = fwd_threads(LPR) / LPR;
    __shared__ double buf[fwd_threads(LPR) / 64];
    const int lane = row_lane<LPR>();
    const int64_t t = a.t0 + (int64_t)blockIdx.x * RPB + (LPR >= 64 ? wave_id() * 64 : (int)threadIdx.x) / LPR;
    const int d = t < a.T ? a.d : 0;
    const int64_t tl = t < a.T ? t : a.T - 1;
    double p[C][8]; // h, then h gain
    double ss = 0.;
    Row<LPR, C, KIND> h, g;
    h.load(row_ptr(a.x, a.dtx, a.ldx, tl), a.dtx, a.d, lane);
    if (a.res) {
        Row<LPR, C, KIND> r;
        r.load(row_ptr(a.res, a.dtr, a.ldr, tl), a.dtr, a.d, lane);
        g.load(a.gain, a.dtg, a.d, lane);
        h.widen(a.dtx);
        r.widen(a.dtr);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[c][i] = (double)h.v[c][i] + (double)r.v[c][i];
                h.v[c][i] += r.v[c][i];
            }
        h.template store<true>(row_ptr(a.h, a.dtr, a.ldh, t), a.dtr, d, lane);
    } else {
        g.load(a.gain, a.dtg, a.d, lane);
        h.widen(a.dtx);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                p[c][i] = (double)h.v[c][i];
    }
    g.widen(a.dtg);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            ss = fma(p[c][i], p[c][i], ss);
            p[c][i] *= (double)g.v[c][i];
        }
    // Amax of this lane's block of h gain: before the row's sum, beside whose
    // barrier it costs less, but not in rows that fill their lanes, which have
    // others in flight to hide the barrier and want the registers (2000 x 8192:
    // 31.5 us, behind the sum 31.9; 8192 x 2048 of bf16 x alone: 17.3 and 16.2).
    constexpr bool EARLY = KIND != FULL;
    double m[C];
    // The 64-bit maximum passes over NaN. The upper words, read as floats, are
    // NaN where p is NaN or infinite (no finite p comes near 2^1017), and the
    // 32-bit maximum keeps it: such a block's amax and scale are infinite.
    auto amax = [&](int c) {
        float top = 0.f;
        m[c] = 0.;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            m[c] = fmax(m[c], fabs(p[c][i]));
            top = __builtin_elementwise_maximum(top, fabsf(upper_word(p[c][i])));
        }
        m[c] = row16_max(top == top ? m[c] : __builtin_inf());
    };
#pragma unroll
    for (int c = 0; c < C; ++c)
        if (EARLY)
            amax(c);
    ss = row_sum<LPR>(ss, buf);
    const double r = rsqrt64(ss * a.inv_d + (double)a.eps);
    const int64_t pitch = fp8_pitch(a.d);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int j = 8 * (lane + LPR * c);
        if (!EARLY)
            amax(c);
        // scale = max(amax, 2^-64) / 448; a NaN of r stays
        const double y = m[c] * r;
        const float s = (float)((y <= (double)FP8_AMAX_MIN ? (double)FP8_AMAX_MIN : y) * (1. / FP8_MAX));
        // p k = n / scale; zeros (and NaN, where p is) in a block of no finite scale
        const double k = s < __builtin_inff() ? r * rcp64((double)s) : 0.;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            p[c][i] *= k;
        if (j < pitch && t < a.T) {
            stg8_nt(a.q + t * pitch + j, quant8(p[c]));
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

// Eight waves a workgroup, so that there are few partial rows for the waves in
// flight; sixteen for the widest rows, and for narrow ones, which are many a
// workgroup then (8192 x 512: 13.7 us, with eight 14.4; 4096 x 1024: 15.6, with
// eight 15.0).
constexpr int bwd_threads(int lpr) { return lpr <= 64 ? 1024 : lpr < 512 ? 512 : lpr; }

template <int LPR, int C, RowKind KIND>
__global__ __launch_bounds__(bwd_threads(LPR)) void rmsnorm_bwd_kernel(BwdArgs a)
{
    constexpr int NT = bwd_threads(LPR), RPB = NT / LPR, NW = NT / 64;
    constexpr int COLS = 8 * LPR * C;
    __shared__ float buf[2][2][NW];
    __shared__ __attribute__((aligned(16))) float lds[RPB > 1 ? RPB : 1][RPB > 1 ? COLS : 4];
    const int lane = row_lane<LPR>();
    const int row = (LPR >= 64 ? wave_id() * 64 : (int)threadIdx.x) / LPR;
    float acc[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc[c][i] = 0.f;
    Row<LPR, C, KIND> g;
    g.load(a.gain, a.dtg, a.d, lane);
    g.widen(a.dtg);
    int it = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * RPB; t0 < a.T; t0 += (int64_t)gridDim.x * RPB, ++it) {
        const int64_t t = t0 + row;
        // rows past T store nothing and add nothing; they read the last row
        const bool in = RPB == 1 || t < a.T;
        const int d = in ? a.d : 0;
        const int64_t tl = in ? t : a.T - 1;
        Row<LPR, C, KIND> h, dn, rs;
        h.load(row_ptr(a.h, a.dth, a.ldh, tl), a.dth, a.d, lane);
        dn.load(row_ptr(a.dn, a.dtdn, a.lddn, tl), a.dtdn, a.d, lane);
        if (a.dres)
            rs.load(row_ptr(a.dres, a.dtdres, a.lddres, tl), a.dtdres, a.d, lane);
        h.widen(a.dth);
        dn.widen(a.dtdn);
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ss = fmaf(h.v[c][i], h.v[c][i], ss);
                dot = fmaf(g.v[c][i] * dn.v[c][i], h.v[c][i], dot);
            }
        // two buffers in turn: a wave may still read the last row's sums
        row_sum2<LPR, (C > 1)>(ss, dot, buf[it & 1][0], buf[it & 1][1]);
        const float r = 1.f / sqrtf(ss / (float)a.d + a.eps);
        const float m = dot * r / (float)a.d; // mean(dg xh)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float xh = h.v[c][i] * r;
                acc[c][i] = in ? fmaf(dn.v[c][i], xh, acc[c][i]) : acc[c][i];
                h.v[c][i] = r * fmaf(-xh, m, g.v[c][i] * dn.v[c][i]);
            }
        if (a.dres) {
            rs.widen(a.dtdres);
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    h.v[c][i] += rs.v[c][i];
        }
        h.template store<false>(row_ptr(a.dh, a.dtdh, a.lddh, t), a.dtdh, d, lane);
    }
    // the row slots' sums, added by halves
    float *part = a.part + (int64_t)blockIdx.x * a.d;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int j = 8 * (lane + LPR * c);
        if constexpr (RPB > 1) {
            *(floatx4_t *)&lds[row][j] = floatx4_t{acc[c][0], acc[c][1], acc[c][2], acc[c][3]};
            *(floatx4_t *)&lds[row][j + 4] = floatx4_t{acc[c][4], acc[c][5], acc[c][6], acc[c][7]};
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (j + i < a.d)
                    part[j + i] = acc[c][i];
        }
    }
    if constexpr (RPB > 1) {
        __syncthreads();
        for (int j = threadIdx.x; j < a.d; j += NT) {
            float p[RPB];
#pragma unroll
            for (int q = 0; q < RPB; ++q)
                p[q] = lds[q][j];
            part[j] = tree_sum<RPB>(p);
        }
    }
}

// dgain[j] = sum of the G partial rows, in a fixed order: 64 columns per
// workgroup, SL slices of consecutive rows; a lane has eight rows' loads in
// flight and adds them by halves, and so the slices (512 rows added one by one
// were most of dgain's error: 2.1e-7 of its norm, so 1.2e-7).
constexpr int SL = 16;
__global__ __launch_bounds__(64 * SL) void rmsnorm_dgain_kernel(const float *part, int G, int d,
                                                              float *dgain)
{
    __shared__ float s[SL][64];
    const int lane = threadIdx.x & 63, w = wave_id();
    const int j = blockIdx.x * 64 + lane, jc = min(j, d - 1);
    const int per = (G + SL - 1) / SL, g0 = min(G, w * per), g1 = min(G, g0 + per);
    float v = 0.f;
    for (int g = g0; g < g1; g += 8) {
        float p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            p[i] = part[(int64_t)min(g + i, g1 - 1) * d + jc];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            p[i] = g + i < g1 ? p[i] : 0.f;
        v += tree_sum<8>(p);
    }
    s[w][lane] = v;
    __syncthreads();
    if (w == 0 && j < d) {
        float p[SL];
#pragma unroll
        for (int q = 0; q < SL; ++q)
            p[q] = s[q][lane];
        dgain[j] = tree_sum<SL>(p);
    }
}

// Lanes of a row of d elements: eight each, as many as it needs.
int row_lanes(int d)
{
    int l = 16;
    while (l < 1024 && 8 * l < d)
        l *= 2;
    return l;
}

// Rows that fill their lanes leave out the tests; not those of sixteen waves:
// without tests the compiler holds more loads at once, and past 64 registers a
// CU has one such row instead of two (2000 x 8192 to 8 bits: 36 and 31 us).
RowKind row_kind(int d)
{
    const int l = row_lanes(d);
    return d & 7 ? RAGGED : d == 8 * l && l < 1024 ? FULL : EIGHTS;
}

// Workgroups (and partial rows of dgain) of the backward, of the g turns that
// all the rows make.
// Up to two turns: one workgroup, which writes dgain itself (two turns of 1024
// columns 4.4 us, as two workgroups and a second launch 5.4; three 5.5 and 5.4,
// four of 64 columns 8.5 and 5.7).
// Workgroups of sixteen waves: one a CU. Of eight: two a CU, unless their
// partial rows weigh more than they gain, one for each 3/8 columns' turns (one
// and two a CU, us: 4096 columns, 1000 turns 17.4 and 19.9, 8192 turns 96.7 and
// 93.0; 2304 columns, 600 turns 12.2 and 12.7, 8192 turns 80.7 and 59.5; 1500
// columns, 513 turns 14.6 and 12.7, 1200 turns 20.6 and 18.2).
// All have the same number of turns or one less (4096 columns, 300 turns: 11.5
// with 150, 13.7 with 300; 8192 columns, 513 turns: 20.8 with 171, 22.9 with 256).
// With two a CU and more than two turns they are 512 even so: fewer no longer
// fill the memory's queues (2048 columns, 2049 turns: 28.1, with 410 30.5).
int bwd_groups(int T, int d)
{
    constexpr int CUS = 256;
    const int lpr = row_lanes(d), nt = bwd_threads(lpr), rpb = nt / lpr;
    const int64_t g = ((int64_t)T + rpb - 1) / rpb;
    if (g <= 2)
        return g > 0;
    const int most = nt == 512 && 8 * g > 3 * (int64_t)d ? 2 * CUS : CUS;
    const int64_t turns = (g + most - 1) / most;
    if (most > CUS && turns > 2)
        return most;
    return (int)((g + turns - 1) / turns);
}

// A launch has fewer than 2^32 threads: at most 2^31 here, further rows in
// launches of their own.
template <int LPR, int C, RowKind KIND> void fwd_one(FwdArgs a, hipStream_t s)
{
    constexpr int NT = fwd_threads(LPR), RPB = NT / LPR, MOST = (int)((1u << 31) / LPR);
    for (a.t0 = 0; a.t0 < a.T; a.t0 += MOST) {
        const int rows = a.T - a.t0 < MOST ? a.T - a.t0 : MOST;
        const dim3 grid((rows + RPB - 1) / RPB);
        if (a.q)
            rmsnorm_fwd8_kernel<LPR, C, KIND><<<grid, NT, 0, s>>>(a);
        else
            rmsnorm_fwd_kernel<LPR, C, KIND><<<grid, NT, 0, s>>>(a);
    }
}

template <RowKind KIND> void fwd_sizes(const FwdArgs &a, hipStream_t s)
{
    switch (row_lanes(a.d)) {
    case 16: return fwd_one<16, 1, KIND>(a, s);
    case 32: return fwd_one<32, 1, KIND>(a, s);
    case 64: return fwd_one<64, 1, KIND>(a, s);
    case 128: return fwd_one<128, 1, KIND>(a, s);
    case 256: return fwd_one<256, 1, KIND>(a, s);
    case 512: return fwd_one<512, 1, KIND>(a, s);
    }
    if constexpr (KIND != FULL)
        a.d <= 8192 ? fwd_one<1024, 1, KIND>(a, s) : fwd_one<1024, 2, KIND>(a, s);
}

template <int LPR, int C, RowKind KIND> void bwd_one(const BwdArgs &a, int G, hipStream_t s)
{
    rmsnorm_bwd_kernel<LPR, C, KIND><<<G, bwd_threads(LPR), 0, s>>>(a);
}

template <RowKind KIND> void bwd_sizes(const BwdArgs &a, int G, hipStream_t s)
{
    switch (row_lanes(a.d)) {
    case 16: return bwd_one<16, 1, KIND>(a, G, s);
    case 32: return bwd_one<32, 1, KIND>(a, G, s);
    case 64: return bwd_one<64, 1, KIND>(a, G, s);
    case 128: return bwd_one<128, 1, KIND>(a, G, s);
    case 256: return bwd_one<256, 1, KIND>(a, G, s);
    case 512: return bwd_one<512, 1, KIND>(a, G, s);
    }
    if constexpr (KIND != FULL)
        a.d <= 8192 ? bwd_one<1024, 1, KIND>(a, G, s) : bwd_one<1024, 2, KIND>(a, G, s);
}

} // namespace

hipError_t launch_rmsnorm_fwd(const twell_mat_t *x, const twell_mat_t *res, const void *gain,
                              int dtg, float eps, const twell_mat_t *h, const twell_mat_t *n,
                              const twell_fp8_t *n8, twell_timing_t *timing, hipStream_t s)
{
    FwdArgs a = {};
    a.x = x->data, a.ldx = x->ld, a.dtx = x->dtype, a.T = x->rows, a.d = x->cols;
    a.gain = gain, a.dtg = dtg, a.eps = eps, a.inv_d = 1. / x->cols;
    if (res) {
        a.res = res->data, a.ldr = res->ld, a.dtr = res->dtype;
        a.h = h->data, a.ldh = h->ld;
    }
    if (n8)
        a.q = n8->q, a.scale = n8->scale;
    else
        a.n = n->data, a.ldn = n->ld, a.dtn = n->dtype;
    Timer tm(timing, s);
    switch (row_kind(a.d)) {
    case FULL: fwd_sizes<FULL>(a, s); break;
    case EIGHTS: fwd_sizes<EIGHTS>(a, s); break;
    case RAGGED: fwd_sizes<RAGGED>(a, s); break;
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
    const int G = bwd_groups(a.T, a.d);
    a.part = G == 1 ? dgain : (float *)ws;
    Timer tm(timing, s);
    if (a.T > 0) {
        switch (row_kind(a.d)) {
        case FULL: bwd_sizes<FULL>(a, G, s); break;
        case EIGHTS: bwd_sizes<EIGHTS>(a, G, s); break;
        case RAGGED: bwd_sizes<RAGGED>(a, G, s); break;
        }
    }
    tm.mark("rmsnorm_bwd");
    if (G != 1) {
        rmsnorm_dgain_kernel<<<(a.d + 63) / 64, 64 * SL, 0, s>>>(a.part, G, a.d, dgain);
        tm.mark("rmsnorm_dgain");
    }
    return hipGetLastError();
}
