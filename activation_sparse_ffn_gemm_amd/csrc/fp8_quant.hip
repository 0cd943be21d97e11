// A matrix in 8 bits with block scales, of itself and of its transpose.
//
//   s = max(amax(block), 2^-64) / 448,  q = e4m3(x / s)
//
// over blocks of 1 x 128 or 128 x 128 elements. One workgroup takes a 128 x
// 128 tile of x into registers, 32 elements per thread (four rows of eight
// consecutive columns), so the tile holds whole blocks of every kind asked
// for: x is read once whatever is written. Row amaxes are DPP moves inside
// the 16 lanes that share a row; column amaxes go over the thread's own rows,
// the wave's other lanes and the workgroup's waves (LDS). The transpose is
// turned in LDS as bytes. Bound by HBM: x in, q (and q_t) out; a thread holds
// few elements so that several tiles are on a CU, one loading while another
// stores (64 elements a thread took 19.1 us for 8192 x 2048 bf16 and its
// transpose).
#include "fp8.hpp"

namespace {

constexpr int NT = 512, NW = NT / 64, TS = FP8_BLK;
constexpr int RPT = TS * 16 / NT; // rows of a thread
static_assert(TS == 128 && RPT == 4, "a tile is one block of each kind; four rows a thread");

struct QuantArgs {
    const void *x;
    uint8_t *q, *qt;
    float *s, *st;
    int64_t ld;
    int R, C, dt, tiles_c;
};

DEVI uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// LDS word of rows 4 rr .. 4 rr + 3 of column c of the turned tile: 32 words a
// column, its 16-byte chunks XOR-ed with the column's eights so that the 16
// columns and four row groups a wave writes at once lie on distinct banks
// (the columns' upper half one column further, on the other 32 banks).
DEVI int turn_word(int c, int rr)
{
    return (c + (c >> 6)) * 32 + (rr ^ (((c >> 3) & 7) << 2));
}

// ROWS: q of x, COLS: q of its transpose, BLOCK: 128 x 128 blocks.
template <bool ROWS, bool COLS, bool BLOCK>
__global__ __launch_bounds__(NT, 6) void fp8_quant_kernel(QuantArgs a)
{
    __shared__ uint32_t cmax[NW][TS]; // column amaxes of each wave's rows
    __shared__ __attribute__((aligned(16))) float cs[2][TS]; // the columns' scales and 1 / scales
    __shared__ __attribute__((aligned(16))) uint32_t turn[COLS ? (TS + 1) * 32 : 1];
    const int tid = threadIdx.x, lane = tid & 63, w = wave_id();
    const int tr = blockIdx.x / a.tiles_c, tc = blockIdx.x % a.tiles_c;
    const int cc = tid & 15, rr = tid >> 4; // this thread's column chunk and row group
    const int r0 = tr * TS + rr * RPT, c0 = tc * TS + cc * 8;
    float v[RPT][8];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
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
    BlockScale sb = {};
    if constexpr (BLOCK) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                m = umax(m, abs_bits(v[i][k]));
        m = row16_umax(m);
#pragma unroll
        for (int o = 16; o < 64; o <<= 1)
            m = umax(m, (uint32_t)__shfl_xor((int)m, o, 64));
        if (lane == 0)
            cmax[w][0] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NW; ++i)
            m = umax(m, cmax[i][0]);
        sb = fp8_scale(m);
        if (tid == 0) {
            // [column block][row block], and the same number for the transpose
            if (ROWS)
                a.s[(int64_t)tc * fp8_blocks(a.R) + tr] = sb.s;
            if (COLS)
                a.st[(int64_t)tr * fp8_blocks(a.C) + tc] = sb.s;
        }
    } else if constexpr (COLS) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < RPT; ++i)
                m = umax(m, abs_bits(v[i][k]));
#pragma unroll
            for (int o = 16; o < 64; o <<= 1)
                m = umax(m, (uint32_t)__shfl_xor((int)m, o, 64));
            if (lane < 16)
                cmax[w][cc * 8 + k] = m;
        }
        __syncthreads();
        if (tid < TS) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < NW; ++i)
                m = umax(m, cmax[i][tid]);
            const BlockScale b = fp8_scale(m);
            cs[0][tid] = b.s;
            cs[1][tid] = b.inv;
            if (tc * TS + tid < a.C)
                a.st[(int64_t)tr * a.C + tc * TS + tid] = b.s;
        }
    }
    if constexpr (ROWS) {
        const int64_t pitch = fp8_pitch(a.C);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            BlockScale b = sb;
            if (!BLOCK) {
                uint32_t m = 0;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    m = umax(m, abs_bits(v[i][k]));
                b = fp8_scale(row16_umax(m));
            }
            const int r = r0 + i;
            if (r < a.R) {
                *(uint2 *)(a.q + (int64_t)r * pitch + c0) = quant8(v[i], b);
                if (!BLOCK && cc == 0)
                    a.s[(int64_t)tc * a.R + r] = b.s;
            }
        }
    }
    if constexpr (COLS) {
        if (!BLOCK)
            __syncthreads(); // cs
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float s = BLOCK ? sb.s : cs[0][cc * 8 + k];
            const float inv = BLOCK ? sb.inv : cs[1][cc * 8 + k];
            turn[turn_word(cc * 8 + k, rr)] = f32x4_to_e4m3x4(
                div_by(v[0][k], s, inv), div_by(v[1][k], s, inv),
                div_by(v[2][k], s, inv), div_by(v[3][k], s, inv));
        }
        __syncthreads();
        const int64_t pitch = fp8_pitch(a.R);
#pragma unroll
        for (int i = 0; i < TS * 8 / NT; ++i) { // 16 bytes: column c, rows 16 ch ..
            const int q = tid + i * NT, c = q >> 3, ch = q & 7;
            if (tc * TS + c < a.C)
                *(uint4 *)(a.qt + (int64_t)(tc * TS + c) * pitch + tr * TS + ch * 16) =
                    *(const uint4 *)&turn[turn_word(c, 4 * ch)];
        }
    }
}

template <bool ROWS, bool COLS> void launch_layout(const QuantArgs &a, bool block, hipStream_t s)
{
    const dim3 grid((uint32_t)(fp8_blocks(a.R) * (int64_t)a.tiles_c));
    if (block)
        fp8_quant_kernel<ROWS, COLS, true><<<grid, NT, 0, s>>>(a);
    else
        fp8_quant_kernel<ROWS, COLS, false><<<grid, NT, 0, s>>>(a);
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
    const bool block = (o ? o : ot)->block_rows == TS;
    a.tiles_c = fp8_blocks(a.C);
    Timer tm(timing, s);
    if (o && ot)
        launch_layout<true, true>(a, block, s);
    else if (o)
        launch_layout<true, false>(a, block, s);
    else
        launch_layout<false, true>(a, block, s);
    tm.mark("fp8_quant");
    return hipGetLastError();
}
