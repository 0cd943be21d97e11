// out = A B^T of two 8-bit matrices with block scales:
//   out[m][n] = sum over blocks kb of 128 k of
//               sa[kb][m] sb[kb][n] sum_{k in kb} qa[m][k] qb[n][k].
// The inner sum starts from zero; its result joins the output's float32
// accumulator scaled. It is taken either
//   by one 16x16x128 instruction on the 8-bit values (TWELL_SUMS_FP8). That
//   instruction does not add in full 32 bits: measured on the part, products
//   of k 8i .. 8i + 7 are aligned to the largest of the eight and keep 13 bits
//   below it (2^16 + 2^3 is exact, 2^16 + 2^2 is not; products of different
//   eights, and the accumulator, meet in float32). On random operands the
//   result is off by 1.4e-5 of its norm, a hundredth of bfloat16's rounding,
//   so it serves results that are rounded to bfloat16; or
//   by four 16x16x32 instructions on the values widened to bfloat16
//   (TWELL_SUMS_F32): widening is exact and those instructions add in float32
//   (off by 1e-8), at half the rate.
//
// The B rows go to the instruction's first operand and the A rows (tokens) to
// its second: a lane's four results then belong to one token and four
// consecutive n. Which k a lane's 32 bytes are does not matter as long as
// both operands agree, so each lane takes 32 consecutive bytes of its row.
#include "fp8.hpp"

namespace {

typedef int intx8_t __attribute__((ext_vector_type(8)));

struct MmArgs {
    const uint8_t *qa, *qb;
    const float *sa, *sb;
    void *out;
    int64_t ldo, pitch;
    int M, N, nkb, dto;
    int ra, rb;   // rows of a scale block (1 or 128) of A and of B
    int nsa, nsb; // scales per block of k
};

DEVI intx8_t frag32(const uint8_t *p)
{
    const uint4 a = ldg16(p), b = ldg16(p + 16);
    return intx8_t{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}
DEVI floatx4_t mfma_e4m3(intx8_t a, intx8_t b)
{
    const floatx4_t zero = {0.f, 0.f, 0.f, 0.f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}

// the same sum over the operands widened to bfloat16, eight k of a lane's 32
// at a time
DEVI bf16x8_t widen8(int lo, int hi)
{
    bf16x2_t p[4];
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, 1.f, false);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, 1.f, true);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, 1.f, false);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, 1.f, true);
    return bf16x8_t{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
}
DEVI floatx4_t mfma_wide(intx8_t a, intx8_t b)
{
    floatx4_t c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 8; i += 2)
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(a[i], a[i + 1]), widen8(b[i], b[i + 1]),
                                                    c, 0, 0, 0);
    return c;
}
template <int SUMS> DEVI floatx4_t block_sum(intx8_t a, intx8_t b)
{
    return SUMS == TWELL_SUMS_FP8 ? mfma_e4m3(a, b) : mfma_wide(a, b);
}

constexpr int WV = 8; // waves of a workgroup: each takes every eighth block of k

// TB tiles of 16 tokens by 16 n per workgroup.
template <int TB, int SUMS>
__global__ __launch_bounds__(64 * WV) void fp8_mm_rows_kernel(MmArgs a)
{
    __shared__ floatx4_t part[WV][TB][64];
    const int lane = threadIdx.x & 63, w = wave_id();
    const int l16 = lane & 15, q4 = lane >> 4;
    const int tiles_n = (a.N + 15) / 16;
    const int n0 = (int)(blockIdx.x % tiles_n) * 16;
    const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * (16 * TB);
    const uint8_t *pb = a.qb + (int64_t)min(n0 + l16, a.N - 1) * a.pitch + q4 * 32;
    const uint8_t *pa[TB];
    int am[TB];
    floatx4_t acc[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) {
        am[t] = (int)min(m0 + t * 16 + l16, (int64_t)a.M - 1);
        pa[t] = a.qa + (int64_t)am[t] * a.pitch + q4 * 32;
        acc[t] = floatx4_t{0.f, 0.f, 0.f, 0.f};
    }
    int nb[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        nb[e] = min(n0 + q4 * 4 + e, a.N - 1) / a.rb;
    for (int kb = w; kb < a.nkb; kb += WV) {
        const intx8_t fb = frag32(pb + (int64_t)kb * FP8_BLK);
        float sb[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            sb[e] = a.sb[(int64_t)kb * a.nsb + nb[e]];
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            const intx8_t fa = frag32(pa[t] + (int64_t)kb * FP8_BLK);
            const float sa = a.sa[(int64_t)kb * a.nsa + am[t] / a.ra];
            const floatx4_t p = block_sum<SUMS>(fb, fa);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[t][e] = fmaf(p[e], sa * sb[e], acc[t][e]);
        }
    }
#pragma unroll
    for (int t = 0; t < TB; ++t)
        part[w][t][lane] = acc[t];
    __syncthreads();
    // wave w joins tile w's partial sums, in wave order
    if (w >= TB)
        return;
    floatx4_t o = part[0][w][lane];
#pragma unroll
    for (int q = 1; q < WV; ++q)
        o += part[q][w][lane];
    const int64_t m = m0 + w * 16 + l16;
    if (m >= a.M)
        return;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int n = n0 + q4 * 4 + e;
        if (n < a.N) {
            if (a.dto == TWELL_BF16)
                ((uint16_t *)a.out)[m * a.ldo + n] = (uint16_t)f32x2_to_bf16x2(o[e], 0.f);
            else
                ((float *)a.out)[m * a.ldo + n] = o[e];
        }
    }
}

template <int SUMS> void launch_rows(const MmArgs &a, hipStream_t s)
{
    const int64_t tn = (a.N + 15) / 16;
    const int tb = a.M <= 16 ? 1 : a.M <= 32 ? 2 : 4;
    const dim3 grid((uint32_t)(tn * ((a.M + 16 * tb - 1) / (16 * tb))));
    if (tb == 1)
        fp8_mm_rows_kernel<1, SUMS><<<grid, 64 * WV, 0, s>>>(a);
    else if (tb == 2)
        fp8_mm_rows_kernel<2, SUMS><<<grid, 64 * WV, 0, s>>>(a);
    else
        fp8_mm_rows_kernel<4, SUMS><<<grid, 64 * WV, 0, s>>>(a);
}

} // namespace

size_t fp8_mm_workspace(int M, int N, int K) { return 0; }

hipError_t launch_fp8_mm(const twell_fp8_t *A, const twell_fp8_t *B, const twell_mat_t *out,
                         int sums, void *ws, twell_timing_t *timing, hipStream_t s)
{
    MmArgs a = {};
    a.qa = A->q, a.sa = A->scale, a.qb = B->q, a.sb = B->scale;
    a.out = out->data, a.ldo = out->ld, a.dto = out->dtype;
    a.pitch = fp8_pitch(A->cols);
    a.M = A->rows, a.N = B->rows, a.nkb = fp8_blocks(A->cols);
    a.ra = A->block_rows, a.rb = B->block_rows;
    a.nsa = (a.M + a.ra - 1) / a.ra, a.nsb = (a.N + a.rb - 1) / a.rb;
    Timer tm(timing, s);
    if (sums == TWELL_SUMS_FP8)
        launch_rows<TWELL_SUMS_FP8>(a, s);
    else
        launch_rows<TWELL_SUMS_F32>(a, s);
    tm.mark("fp8_mm_rows");
    return hipGetLastError();
}
