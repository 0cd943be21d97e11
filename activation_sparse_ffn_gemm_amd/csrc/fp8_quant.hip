// A matrix in 8 bits with block scales, of itself and of its transpose.
//
//   s = max(amax(block), 2^-64) / 448,  q = e4m3(x / s)
//
// over blocks of 1 x 128 or 128 x 128 elements. One workgroup takes a 128 x
// 128 tile of x into registers, 64 elements per thread (eight rows of eight
// consecutive columns), so the tile holds whole blocks of every kind asked
// for: x is read once whatever is written. Row amaxes are DPP moves inside
// the 16 lanes that share a row, column amaxes go over the thread's own rows,
// the wave's other lanes and the workgroup's waves (LDS). The transpose is
// turned in LDS as bytes. Bound by HBM: x in, q (and q_t) out.
#include "fp8.hpp"

namespace {

constexpr int NT = 256, TS = FP8_BLK;
static_assert(TS == 128, "a tile is one block of each kind");

struct QuantArgs {
    const void *x;
    uint8_t *q, *qt;
    float *s, *st;
    int64_t ld;
    int R, C, dt, tiles_c;
    int block; // scales of the whole tile (128 x 128) instead of its rows' / columns'
};

__global__ __launch_bounds__(NT) void fp8_quant_kernel(QuantArgs a)
{
    __shared__ uint32_t cmax[4][TS]; // column amaxes of each wave's 32 rows
    __shared__ uint32_t wmax[4];
    __shared__ uint2 turn[TS][TS / 8]; // [column][eight rows], chunks swizzled
    const int tid = threadIdx.x, lane = tid & 63, w = wave_id();
    const int tr = blockIdx.x / a.tiles_c, tc = blockIdx.x % a.tiles_c;
    const int cc = tid & 15, rr = tid >> 4; // this thread's column chunk and row group
    const int r0 = tr * TS + rr * 8, c0 = tc * TS + cc * 8;
    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + i;
        const uint8_t *p = (const uint8_t *)row_ptr(a.x, a.dt, a.ld, r < a.R ? r : 0);
        if (r < a.R && c0 + 8 <= a.C) {
            if (a.dt == TWELL_BF16) {
                elem<TWELL_BF16>::widen(ldg16u(p + 2 * (int64_t)c0), v[i]);
            } else {
                elem<TWELL_F32>::widen(ldg16u(p + 4 * (int64_t)c0), v[i]);
                elem<TWELL_F32>::widen(ldg16u(p + 4 * (int64_t)c0 + 16), v[i] + 4);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[i][k] = r >= a.R || c0 + k >= a.C ? 0.f
                          : a.dt == TWELL_BF16     ? elem<TWELL_BF16>::load1(p, c0 + k)
                                                   : elem<TWELL_F32>::load1(p, c0 + k);
        }
    }
    uint32_t m = 0;
    if (a.block) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t b = abs_bits(v[i][k]);
                m = b > m ? b : m;
            }
        m = row16_umax(m);
#pragma unroll
        for (int o = 16; o < 64; o <<= 1) {
            const uint32_t b = (uint32_t)__shfl_xor((int)m, o, 64);
            m = b > m ? b : m;
        }
        if (lane == 0)
            wmax[w] = m;
        __syncthreads();
        m = max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3]));
    }
    const float sb = a.block ? fp8_scale(m) : 0.f;
    const float ib = a.block ? 1.f / sb : 0.f;
    if (a.block && tid == 0) {
        // [column block][row block], and the same number for the transpose
        if (a.q)
            a.s[(int64_t)tc * fp8_blocks(a.R) + tr] = sb;
        if (a.qt)
            a.st[(int64_t)tr * fp8_blocks(a.C) + tc] = sb;
    }
    if (a.q) {
        const int64_t pitch = fp8_pitch(a.C);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float s = sb, inv = ib;
            if (!a.block) {
                uint32_t rm = 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t b = abs_bits(v[i][k]);
                    rm = b > rm ? b : rm;
                }
                s = fp8_scale(row16_umax(rm));
                inv = 1.f / s;
            }
            const int r = r0 + i;
            if (r < a.R) {
                *(uint2 *)(a.q + (int64_t)r * pitch + c0) = quant8(v[i], s, inv);
                if (!a.block && cc == 0)
                    a.s[(int64_t)tc * a.R + r] = s;
            }
        }
    }
    if (!a.qt)
        return;
    if (!a.block) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint32_t km = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t b = abs_bits(v[i][k]);
                km = b > km ? b : km;
            }
#pragma unroll
            for (int o = 16; o < 64; o <<= 1) {
                const uint32_t b = (uint32_t)__shfl_xor((int)km, o, 64);
                km = b > km ? b : km;
            }
            if (lane < 16)
                cmax[w][cc * 8 + k] = km;
        }
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int c = cc * 8 + k;
        float s = sb, inv = ib;
        if (!a.block) {
            s = fp8_scale(max(max(cmax[0][c], cmax[1][c]), max(cmax[2][c], cmax[3][c])));
            inv = 1.f / s;
            if (rr == 0 && tc * TS + c < a.C)
                a.st[(int64_t)tr * a.C + tc * TS + c] = s;
        }
        float u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            u[i] = v[i][k];
        turn[c][rr ^ cc] = quant8(u, s, inv);
    }
    __syncthreads();
    const int64_t pitch = fp8_pitch(a.R);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int c = k * 16 + (tid >> 4), ch = tid & 15;
        if (tc * TS + c < a.C)
            *(uint2 *)(a.qt + (int64_t)(tc * TS + c) * pitch + tr * TS + ch * 8) =
                turn[c][ch ^ (c >> 3)];
    }
}

} // namespace

hipError_t launch_fp8_quant(const twell_mat_t *x, const twell_fp8_t *o, const twell_fp8_t *ot,
                            twell_timing_t *timing, hipStream_t s)
{
    QuantArgs a = {};
    a.x = x->data, a.ld = x->ld, a.dt = x->dtype, a.R = x->rows, a.C = x->cols;
    if (o)
        a.q = o->q, a.s = o->scale;
    if (ot)
        a.qt = ot->q, a.st = ot->scale;
    a.block = (o ? o : ot)->block_rows == TS;
    a.tiles_c = fp8_blocks(a.C);
    Timer tm(timing, s);
    fp8_quant_kernel<<<dim3((uint32_t)(fp8_blocks(a.R) * (int64_t)a.tiles_c)), NT, 0, s>>>(a);
    tm.mark("fp8_quant");
    return hipGetLastError();
}
