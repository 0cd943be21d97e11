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
// turned in LDS as bytes. bf16 stays two to a word until it is quantised, and
// its maxima are taken two at a time.
//
// Bound by HBM (x in, q and q_t out) with the arithmetic close behind: 8192 x
// 2048 bf16 and its transpose 14.0 us, 4.9 TB/s; a thread holds few elements so
// that several tiles are on a CU, one loading while another stores (64 elements
// a thread 19.1, half as many workgroups a CU 16.1 where this was 15.9).
#include <type_traits>

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
    int R, C, tiles_c;
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

// The value of lane I of each four.
template <int I> DEVI float quad_lane(float v)
{
    return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), I * 0x55,
                                                              0xF, 0xF, false));
}

// Bytes of four rows by four columns (a row a word, first column lowest) turned:
// a column a word.
DEVI void turn4(uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3, uint32_t *c)
{
    // perm(a, b, sel): byte n is byte sel_n of b (0-3) and a (4-7)
    const uint32_t a = __builtin_amdgcn_perm(r1, r0, 0x05010400), b = __builtin_amdgcn_perm(r1, r0, 0x07030602);
    const uint32_t d = __builtin_amdgcn_perm(r3, r2, 0x05010400), e = __builtin_amdgcn_perm(r3, r2, 0x07030602);
    c[0] = __builtin_amdgcn_perm(d, a, 0x05040100), c[1] = __builtin_amdgcn_perm(d, a, 0x07060302);
    c[2] = __builtin_amdgcn_perm(e, b, 0x05040100), c[3] = __builtin_amdgcn_perm(e, b, 0x07060302);
}

// Eight consecutive elements of a row in 32-bit words, as they are stored, and
// the running maximum of absolute values: as integers these order like the
// floats (infinity above all, NaN above infinity). bf16 goes two to a word.
template <int DT> struct Eight;
template <> struct Eight<TWELL_BF16> {
    static constexpr int W = 4;
    typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
    uint32_t w[W];
    DEVI void load(const void *row, int c, int C)
    {
        const uint16_t *p = (const uint16_t *)row + c;
        uint4 q = make_uint4(0, 0, 0, 0);
        if (c + 8 <= C)
            q = ldg16u(p);
        w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
        if (c < C && c + 8 > C) {
#pragma unroll
            for (int k = 0; k < 7; ++k)
                if (c + k < C)
                    w[k / 2] |= (uint32_t)p[k] << (16 * (k & 1));
        }
    }
    DEVI float operator[](int k) const { return k & 1 ? bf16_hi(w[k / 2]) : bf16_lo(w[k / 2]); }
    DEVI uint32_t abs(int k) const { return w[k] & 0x7fff7fffu; }
    // word by word, and over a word's elements (the bits of a float)
    DEVI static uint32_t max2(uint32_t a, uint32_t b)
    {
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a),
                                                                      __builtin_bit_cast(u16x2_t, b)));
    }
    DEVI static uint32_t top(uint32_t a) { return umax(a << 16, a & 0xffff0000u); }
    DEVI static uint32_t elem_bits(uint32_t word, int k) { return k & 1 ? word & 0xffff0000u : word << 16; }
};
template <> struct Eight<TWELL_F32> {
    static constexpr int W = 8;
    uint32_t w[W];
    DEVI void load(const void *row, int c, int C)
    {
        const float *p = (const float *)row + c;
        uint4 q = make_uint4(0, 0, 0, 0), r = q;
        if (c + 8 <= C)
            q = ldg16u(p), r = ldg16u(p + 4);
        w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
        w[4] = r.x, w[5] = r.y, w[6] = r.z, w[7] = r.w;
        if (c < C && c + 8 > C) {
#pragma unroll
            for (int k = 0; k < 7; ++k)
                if (c + k < C)
                    w[k] = __float_as_uint(p[k]);
        }
    }
    DEVI float operator[](int k) const { return __uint_as_float(w[k]); }
    DEVI uint32_t abs(int k) const { return w[k] & 0x7fffffffu; }
    DEVI static uint32_t max2(uint32_t a, uint32_t b) { return umax(a, b); }
    DEVI static uint32_t top(uint32_t a) { return a; }
    DEVI static uint32_t elem_bits(uint32_t word, int) { return word; }
};

// ROWS: q of x, COLS: q of its transpose, BLOCK: 128 x 128 blocks.
template <int DT, bool ROWS, bool COLS, bool BLOCK>
__global__ __launch_bounds__(NT) void fp8_quant_kernel(QuantArgs a)
{
    using E = Eight<DT>;
    constexpr int W = E::W, EPW = 8 / W; // words of a thread's row, elements of a word
    __shared__ uint32_t cmax[NW][TS / EPW]; // column amaxes of each wave's rows
    __shared__ __attribute__((aligned(16))) float cs[2][TS]; // the columns' scales and 1 / scales
    __shared__ __attribute__((aligned(16))) uint32_t turn[COLS ? (TS + 1) * 32 : 1];
    const int tid = threadIdx.x, lane = tid & 63, w = wave_id();
    const int tr = blockIdx.x / a.tiles_c, tc = blockIdx.x % a.tiles_c;
    const int cc = tid & 15, rr = tid >> 4; // this thread's column chunk and row group
    const int r0 = tr * TS + rr * RPT, c0 = tc * TS + cc * 8;
    E v[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) { // rows past x are empty
        const int r = r0 + i;
        v[i].load(row_ptr(a.x, DT, a.ld, r < a.R ? r : 0), c0, r < a.R ? a.C : 0);
    }
    BlockScale sb = {};
    if constexpr (BLOCK) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
            for (int k = 0; k < W; ++k)
                m = E::max2(m, v[i].abs(k));
        m = row16_umax(E::top(m));
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
                a.s[(int64_t)tc * fp8_blocks(a.R) + tr] = sb.held;
            if (COLS)
                a.st[(int64_t)tr * fp8_blocks(a.C) + tc] = sb.held;
        }
    } else if constexpr (COLS) {
#pragma unroll
        for (int k = 0; k < W; ++k) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < RPT; ++i)
                m = E::max2(m, v[i].abs(k));
#pragma unroll
            for (int o = 16; o < 64; o <<= 1)
                m = E::max2(m, (uint32_t)__shfl_xor((int)m, o, 64));
            if (lane < 16)
                cmax[w][cc * W + k] = m;
        }
        __syncthreads();
        if (tid < TS) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < NW; ++i)
                m = E::max2(m, cmax[i][tid / EPW]);
            const BlockScale b = fp8_scale(E::elem_bits(m, tid % EPW));
            cs[0][tid] = b.s;
            cs[1][tid] = b.inv;
            if (tc * TS + tid < a.C)
                a.st[(int64_t)tr * a.C + tc * TS + tid] = b.held;
        }
    }
    uint2 q[RPT]; // this thread's rows in 8 bits
    if constexpr (ROWS || BLOCK) {
        BlockScale b = sb;
        if constexpr (!BLOCK) { // each of four lanes makes one row's scale
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                uint32_t t = 0;
#pragma unroll
                for (int k = 0; k < W; ++k)
                    t = E::max2(t, v[i].abs(k));
                t = row16_umax(E::top(t));
                m = (cc & 3) == i ? t : m;
            }
            b = fp8_scale(m);
            if (cc < RPT && r0 + cc < a.R)
                a.s[(int64_t)tc * a.R + r0 + cc] = b.held;
        }
        auto row = [&](auto I) {
            constexpr int i = decltype(I)::value;
            const BlockScale br = BLOCK ? b : BlockScale{quad_lane<i>(b.s), quad_lane<i>(b.inv), 0.f};
            float u[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                u[k] = v[i][k];
            q[i] = quant8(u, br);
        };
        row(std::integral_constant<int, 0>());
        row(std::integral_constant<int, 1>());
        row(std::integral_constant<int, 2>());
        row(std::integral_constant<int, 3>());
    }
    if constexpr (ROWS) {
        const int64_t pitch = fp8_pitch(a.C);
#pragma unroll
        for (int i = 0; i < RPT; ++i)
            if (r0 + i < a.R)
                stg8_nt(a.q + (int64_t)(r0 + i) * pitch + c0, q[i]);
    }
    if constexpr (COLS) {
        if constexpr (BLOCK) { // one scale: the rows' bytes, turned
            uint32_t c[8];
            turn4(q[0].x, q[1].x, q[2].x, q[3].x, c);
            turn4(q[0].y, q[1].y, q[2].y, q[3].y, c + 4);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                turn[turn_word(cc * 8 + k, rr)] = c[k];
        } else {
            __syncthreads(); // cs
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const BlockScale b = {cs[0][cc * 8 + k], cs[1][cc * 8 + k], 0.f};
                const float u[RPT] = {v[0][k], v[1][k], v[2][k], v[3][k]};
                turn[turn_word(cc * 8 + k, rr)] = quant4(u, b);
            }
        }
        __syncthreads();
        const int64_t pitch = fp8_pitch(a.R);
#pragma unroll
        for (int i = 0; i < TS * 8 / NT; ++i) { // 16 bytes: column c, rows 16 ch ..
            const int q = tid + i * NT, c = q >> 3, ch = q & 7;
            if (tc * TS + c < a.C)
                stg16u_nt(a.qt + (int64_t)(tc * TS + c) * pitch + tr * TS + ch * 16,
                          *(const uint4 *)&turn[turn_word(c, 4 * ch)]);
        }
    }
}

template <int DT, bool ROWS, bool COLS>
void launch_layout(const QuantArgs &a, bool block, hipStream_t s)
{
    const dim3 grid((uint32_t)(fp8_blocks(a.R) * (int64_t)a.tiles_c));
    if (block)
        fp8_quant_kernel<DT, ROWS, COLS, true><<<grid, NT, 0, s>>>(a);
    else
        fp8_quant_kernel<DT, ROWS, COLS, false><<<grid, NT, 0, s>>>(a);
}

template <int DT>
void launch_type(const QuantArgs &a, bool rows, bool cols, bool block, hipStream_t s)
{
    if (rows && cols)
        launch_layout<DT, true, true>(a, block, s);
    else if (rows)
        launch_layout<DT, true, false>(a, block, s);
    else
        launch_layout<DT, false, true>(a, block, s);
}

} // namespace

hipError_t launch_fp8_quant(const twell_mat_t *x, const twell_fp8_t *o, const twell_fp8_t *ot,
                            twell_timing_t *timing, hipStream_t s)
{
    QuantArgs a = {};
    a.x = x->data, a.ld = x->ld, a.R = x->rows, a.C = x->cols;
    if (o)
        a.q = o->q, a.s = o->scale;
    if (ot)
        a.qt = ot->q, a.st = ot->scale;
    const bool block = (o ? o : ot)->block_rows == TS;
    a.tiles_c = fp8_blocks(a.C);
    Timer tm(timing, s);
    if (x->dtype == TWELL_BF16)
        launch_type<TWELL_BF16>(a, o, ot, block, s);
    else
        launch_type<TWELL_F32>(a, o, ot, block, s);
    tm.mark("fp8_quant");
    return hipGetLastError();
}
