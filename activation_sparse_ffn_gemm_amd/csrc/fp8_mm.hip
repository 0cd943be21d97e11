// out = A B^T of two 8-bit matrices with block scales:
//   out[m][n] = sum over blocks kb of 128 k of
//               sa[kb][m] sb[kb][n] sum_{k in kb} qa[m][k] qb[n][k].
// The product of two scales may be denormal or infinite where a result is
// neither: they are applied one after the other, or with such cases set apart.
// The inner sum starts from zero; its result joins the output's float32
// accumulator scaled. It is taken either
//   by one 16x16x128 instruction on the 8-bit values (TWELL_SUMS_FP8). That
//   instruction does not add in full 32 bits: measured on the part, products
//   of k 8i .. 8i + 7 are aligned to the largest of the eight and keep 13 bits
//   below it (2^16 + 2^3 is exact, 2^16 + 2^2 is not; products of different
//   eights, and the accumulator, meet in float32). A sum is off by less than
//   8 * 2^-13 of its terms' sizes, and one large product beside seven small ones
//   in every eight comes close to that; on normal values by 1.4e-5 of the
//   results' norm, on a normed stream with a few large channels by 3e-5, where
//   bfloat16's rounding is 1.7e-3. So it serves results that are rounded to
//   bfloat16 and whose large terms do not cancel; or
//   by four 16x16x32 instructions on the values widened to bfloat16
//   (TWELL_SUMS_F32): widening is exact and those instructions add in float32
//   (off by 1e-8), at half the rate.
//
// The B rows go to the instruction's first operand and the A rows (tokens) to
// its second: a lane's four results then belong to one token and four
// consecutive n. Which k a lane's 32 bytes are does not matter as long as
// both operands agree, so each lane takes 32 consecutive bytes of its row.
#include <cmath>
#include <type_traits>

#include "fp8.hpp"
#include "ntgemm.hpp"

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
    float *part;  // split contraction: [parts][M][N] float32 partial sums
    int parts, per; // parts, blocks of k in each
};

DEVI floatx4_t mfma_e4m3(intx8_t a, intx8_t b)
{
    const floatx4_t zero = {0.f, 0.f, 0.f, 0.f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}
// the first operand times 2^(ea - 127)
DEVI floatx4_t mfma_e4m3(intx8_t a, intx8_t b, int ea)
{
    const floatx4_t zero = {0.f, 0.f, 0.f, 0.f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, ea, 0, 127);
}

// the same sum over the operands widened to bfloat16, eight k of a lane's 32
// at a time, times two, a power of two
DEVI bf16x8_t widen8(int lo, int hi, float two)
{
    bf16x2_t p[4];
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, two, false);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, two, true);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, two, false);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, two, true);
    return bf16x8_t{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
}

// Two scales' product may be denormal or infinite where the result is neither.
// Where rows of B share a scale, its power of two (as far as 2^100) can go to
// B's operand instead, and the rest, in [1, 2), to A's scale.
struct Power {
    int e; // of the float 2^(e - 127)
    DEVI static Power of(float s) // zeros, denormals, infinities and NaN too
    {
        return {min(max((int)(__float_as_uint(s) >> 23 & 255), 27), 227)};
    }
    DEVI float two() const { return __uint_as_float((uint32_t)e << 23); }
    DEVI float rest(float s) const { return ldexpf(s, 127 - e); }
};
// A 16-row fragment of one block of k, and the block's sums of two of them.
template <int SUMS> struct Frag;
template <> struct Frag<TWELL_SUMS_FP8> {
    intx8_t v;
    DEVI void set(intx8_t x) { v = x; }
    DEVI void set(intx8_t x, Power) { v = x; }
    DEVI static floatx4_t mul(const Frag &a, const Frag &b) { return mfma_e4m3(a.v, b.v); }
    DEVI static floatx4_t mul(const Frag &a, const Frag &b, Power p) { return mfma_e4m3(a.v, b.v, p.e); }
};
template <> struct Frag<TWELL_SUMS_F32> {
    bf16x8_t v[4];
    DEVI void set(intx8_t x, Power p = {127})
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = widen8(x[2 * i], x[2 * i + 1], p.two());
    }
    DEVI static floatx4_t mul(const Frag &a, const Frag &b, Power) { return mul(a, b); }
    DEVI static floatx4_t mul(const Frag &a, const Frag &b)
    {
        floatx4_t c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], c, 0, 0, 0);
        return c;
    }
};

// ---------------------------------------------------------------- large products
// One workgroup computes BM tokens x BN n. A block of 128 k is one step: its
// 128-byte rows of both operands, and their scales, go straight from global
// memory to LDS, NST steps resident, each row's 16-byte chunks XOR-swizzled so
// that the 16 rows a fragment read touches lie on distinct banks. A wave owns
// WN x WM of the tile: NI fragments of B rows by MI of A rows, 32 bytes a lane.
//
// The order within a step is written out (a scheduling barrier after every
// matrix product), because the two waves of a SIMD have little else to hide
// behind each other:
// - A fragment of B is read one row of products before its own.
// - A product's four results are scaled into the accumulators three products
//   later, when they have left the matrix unit.
// - The loads of step + NST - 1 go out one by one beside the step's first
//   products, into the stage that the step before has left.
// - The step's one barrier stands before its last row of products. By then
//   every read of its stage is done and the next stage's loads are in, so the
//   next step's first fragments are read beside that last row.
//
// Of the two large tiles a CU holds one workgroup, so there is nobody to work
// while it begins and ends. There the workgroups stay and take further tiles:
// the next tile's first loads go out before this one's results are stored, and
// the stores drain beside its first steps (8192 x 5632 over 2048: 93 -> 88 us; 90
// with the scales' test). Stores write whole 128-byte lines, through LDS: float32
// results stored from the accumulators, 64 bytes of a row at a time, took 173 us
// there, so 165 (168 with the test).
//
// What bounds a step: fast sums, the matrix unit with the scales' steps beside
// it (a loop of registers alone runs at 3463 TF, 1.24 us a step of 256 x 256)
// and the loads from L2 (11 TB/s; 1.5 us with them). Full sums, vector
// instructions: widening a wave's 11 fragments (176 instructions for 24
// products of 192 x 256) and the scales take turns with the matrix unit; a loop
// of registers alone with this mix takes 2.56 us a step, the kernel 2.5,
// whatever the order of the instructions.
template <int BM_, int BN_, int WGM_, int WGN_, int NST_> struct TileCfg {
    static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, NST = NST_;
    static constexpr int NWV = WGM * WGN, NT = 64 * NWV;
    static constexpr int WM = BM / WGM, WN = BN / WGN, MI = WM / 16, NI = WN / 16;
    static constexpr int ROWS = BM + BN;                 // B rows first, then A rows
    static constexpr int WBB = BN / 8 / NWV, WBA = BM / 8 / NWV; // 1 KB loads (eight rows) a wave
    static constexpr int WB = WBB + WBA;
    static constexpr int NSC = ROWS / 64;                // 64-scale loads: wave w load w % NSC
    static constexpr int SYNC = (NI - 1) * MI;           // product at which a step's barrier is
    static constexpr int LPS = (WB + 1 + SYNC - 1) / SYNC; // loads beside a product before it
    static constexpr int SCALES = ROWS * FP8_BLK;        // byte offset of a stage's scales
    static constexpr int STAGE = SCALES + ROWS * 4;
    // the epilogue's rows, 16 tokens a wave at a time: WE n in bf16, 32 in
    // float32, padded so that 16 rows start on 16 distinct banks
    static constexpr int WE = WN < 64 ? WN : 64, OROW = 128 + 16, OUTB = 16 * OROW * NWV;
    static constexpr bool STAY = NST == 2; // workgroups go on to further tiles
    static constexpr int LDS = NST * STAGE + (STAY ? OUTB : 0);
    static_assert(BN % (8 * NWV) == 0 && BM % (8 * NWV) == 0 && BN % 64 == 0 && BM % 64 == 0 &&
                      NSC <= NWV, "whole loads");
    static_assert(WN % 32 == 0 && WN <= FP8_BLK && FP8_BLK % WN == 0,
                  "a wave's n share one 128-row scale block");
    static_assert(NI % 2 == 0, "two fragments of B in turn");
    static_assert(NST >= 2 && (NST - 2) * (WB + 1) < 64, "loads in flight must fit vmcnt");
    static_assert(OUTB <= NST * STAGE && LDS <= 160 * 1024, "LDS");
};

using ng::dma16;
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// ng::dma16 for four bytes a lane
DEVI void dma4(const float *base, uint32_t off, uint32_t lds, int kb, int kb1)
{
    asm volatile("s_cmp_ge_i32 %3, %4\n\ts_cbranch_scc1 .Lskip%=\n\t"
                 "s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1\n.Lskip%=:"
                 :
                 : "v"(off), "s"(base), "s"(lds), "s"(kb), "s"(kb1)
                 : "m0", "scc");
}
#pragma clang diagnostic pop

// Waits until at most N of this wave's loads are in flight, or, where fewer
// than `full` steps are left (fewer are in flight than N allows for), until
// none is.
template <int N> DEVI void wait_oldest(int left, int full)
{
    if constexpr (N == 0)
        ng::wait_vm<0>();
    else
        asm volatile("s_cmp_lt_i32 %0, %1\n\ts_cbranch_scc1 .Lall%=\n\ts_waitcnt vmcnt(%2)\n\t"
                     "s_branch .Ldone%=\n.Lall%=:\n\ts_waitcnt vmcnt(0)\n.Ldone%=:"
                     :
                     : "s"(left), "s"(full), "n"(N)
                     : "scc");
}

// v, as if it were new here: what is formed of it is not kept in registers
// through the loop over the tiles, where there are none to spare.
DEVI int here(int v)
{
    asm volatile("" : "+v"(v));
    return v;
}

// BLKB: B's scale block is 128 rows, so a wave's n share one scale per step.
template <class C, int SUMS, bool BLKB>
__global__ __launch_bounds__(C::NT, C::NWV / 4) void fp8_mm_tile_kernel(MmArgs a)
{
    __shared__ __attribute__((aligned(16))) uint8_t L[C::LDS];
    // XCD-aware order: XCD k takes the k-th contiguous run of a grouped tile
    // order (GM token tiles x all n tiles per group, token tile fastest)
    constexpr int GM = 8;
    const int n_nt = (a.N + C::BN - 1) / C::BN, n_mt = (a.M + C::BM - 1) / C::BM;
    const int64_t total = (int64_t)n_nt * n_mt * a.parts;
    const int64_t per = (total + NXCD - 1) / NXCD;
    const int64_t run0 = blockIdx.x % NXCD * per;
    const int64_t run1 = run0 + per < total ? run0 + per : total;
    int64_t q0 = run0 + blockIdx.x / NXCD;
    if (q0 >= run1)
        return;
    const int lane = threadIdx.x & 63, w = wave_id();
    const int wm = w / C::WGN, wn = w % C::WGN, l16 = lane & 15, q4 = lane >> 4;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(ng::lds_u8 *)L;
    const int ws = w % C::NSC;
    const bool sisb = ws * 64 < C::BN;
    const float *ssrc = sisb ? a.sb : a.sa;
    const int ns = sisb ? a.nsb : a.nsa;

    // The tile and this wave's loads of it: eight rows of one operand each,
    // lane l byte 16 l of the 1 KB, i.e. the chunk that the swizzle puts
    // there. Rows past an operand read its last row (their outputs are dropped).
    int m0, n0, part, kb0, kb1;
    const uint8_t *srcb, *srca;
    uint32_t off[C::WB], soff;
    auto place = [&] {
        const int lane = here((int)threadIdx.x) & 63;
        part = (int)(q0 / ((int64_t)n_nt * n_mt));
        const int q = (int)(q0 % ((int64_t)n_nt * n_mt));
        const int64_t gsz = (int64_t)GM * n_nt;
        const int grp = (int)(q / gsz), grows = min(GM, n_mt - grp * GM), gr = (int)(q % gsz);
        m0 = (grp * GM + gr % grows) * C::BM, n0 = gr / grows * C::BN;
        kb0 = part * a.per, kb1 = min(a.nkb, kb0 + a.per);
        srcb = a.qb + (int64_t)n0 * a.pitch, srca = a.qa + (int64_t)m0 * a.pitch;
#pragma unroll
        for (int g = 0; g < C::WB; ++g) {
            const int r = (g < C::WBB ? w * C::WBB + g : w * C::WBA + g - C::WBB) * 8 + lane / 8;
            const int last = g < C::WBB ? a.N - 1 - n0 : a.M - 1 - m0;
            off[g] = (uint32_t)min(r, last) * (uint32_t)a.pitch +
                     (((lane & 7) ^ ((r >> 1) & 7)) << 4);
        }
        const int srow = sisb ? min(n0 + ws * 64 + lane, a.N - 1)
                              : min(m0 + ws * 64 - C::BN + lane, a.M - 1);
        soff = (uint32_t)(srow / (sisb ? a.rb : a.ra)) * 4u;
    };
    // load g of this wave (g == WB: its scales) for step kb into stage st
    auto load = [&](int g, int kb, int st) {
        const uint32_t dst = lds0 + (uint32_t)st * C::STAGE;
        if (g < C::WBB)
            dma16(srcb + (int64_t)kb * FP8_BLK, off[g], dst + (w * C::WBB + g) * 1024, kb, kb1);
        else if (g < C::WB)
            dma16(srca + (int64_t)kb * FP8_BLK, off[g],
                  dst + C::BN * FP8_BLK + (w * C::WBA + g - C::WBB) * 1024, kb, kb1);
        else
            dma4(ssrc + (int64_t)kb * ns, soff, dst + C::SCALES + ws * 256, kb, kb1);
    };
    auto first_loads = [&] {
#pragma unroll
        for (int k = 0; k < C::NST - 1; ++k)
#pragma unroll
            for (int g = 0; g <= C::WB; ++g)
                load(g, kb0 + k, k);
    };

    // byte of this lane's two chunks (q4 and q4 + 4) in a 16-row fragment
    const int f0 = l16 * FP8_BLK + ((q4 ^ ((l16 >> 1) & 7)) << 4), f1 = f0 ^ 64;
    auto frag = [&](const uint8_t *p) {
        const uint4 u = *(const uint4 *)(p + f0), v = *(const uint4 *)(p + f1);
        return intx8_t{(int)u.x, (int)u.y, (int)u.z, (int)u.w,
                       (int)v.x, (int)v.y, (int)v.z, (int)v.w};
    };
    const uint8_t *Bw = L + wn * C::WN * FP8_BLK, *Aw = L + (C::BN + wm * C::WM) * FP8_BLK;
    const float *sbw = (const float *)(L + C::SCALES) + wn * C::WN;
    const float *saw = (const float *)(L + C::SCALES) + C::BN + wm * C::WM;
    auto fence = [] { // LDS reads stay on their side (their targets are written by the loads)
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
    };
    // the loads of the oldest step in flight are in, and every wave is here;
    // left: steps from that one to the end
    auto sync = [&](int left) {
        fence();
        wait_oldest<(C::NST - 2) * (C::WB + 1)>(left, C::NST - 1);
        __builtin_amdgcn_s_waitcnt(0xC07F); // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        fence();
    };

    // the next products' fragments as they lie in LDS: of B two in turn where
    // products take them as they are
    constexpr int RB = SUMS == TWELL_SUMS_FP8 ? 2 : 1;
    // A 128-row scale of B and one of A make one factor a token. Where that is no
    // normal float the results still have to be right: the small tiles split B's
    // scale (2% of their time at most; one scale after the other costs 6%, the
    // test below 12%, their steps are short). The large tiles test the factor
    // once a step, and where it is not normal, seldom, add those tokens' products
    // apart, one scale after the other (1 to 2%; splitting 3%).
    constexpr bool SPLIT = BLKB && !C::STAY;
    intx8_t rb[RB], ra[C::MI];
    float sa[C::MI], sb = 1.f;
    floatx4_t sb4[2]; // B's scales of this and the next row of products
    place();
    first_loads();
    sync(kb1 - kb0);
    for (;;) { // tiles
        floatx4_t acc[C::NI][C::MI];
#pragma unroll
        for (int i = 0; i < C::NI; ++i)
#pragma unroll
            for (int j = 0; j < C::MI; ++j)
                acc[i][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
        rb[0] = frag(Bw);
        sb4[0] = *(const floatx4_t *)(sbw + q4 * 4);
#pragma unroll
        for (int j = 0; j < C::MI; ++j) {
            ra[j] = frag(Aw + j * 16 * FP8_BLK);
            sa[j] = saw[j * 16 + l16];
        }
        if (BLKB)
            sb = sbw[0];
        for (int kb = kb0, st = 0; kb < kb1; ++kb) {
            const int free = st == 0 ? C::NST - 1 : st - 1; // the last step's stage
            const int cur = st * C::STAGE;
            st = st == C::NST - 1 ? 0 : st + 1;
            const int nxt = st * C::STAGE;
            Frag<SUMS> fa[C::MI], fb;
            float s[C::MI];
            const Power two = Power::of(sb);
#pragma unroll
            for (int j = 0; j < C::MI; ++j) {
                fa[j].set(ra[j]);
                s[j] = BLKB ? sa[j] * (SPLIT ? two.rest(sb) : sb) : sa[j];
            }
            if constexpr (BLKB && !SPLIT) {
                bool odd = false;
#pragma unroll
                for (int j = 0; j < C::MI; ++j)
                    odd |= !__builtin_isnormal(s[j]);
                if (__builtin_expect(__any(odd), 0)) {
#pragma unroll
                    for (int i = 0; i < C::NI; ++i) {
                        fb.set(frag(Bw + cur + i * 16 * FP8_BLK));
#pragma unroll
                        for (int j = 0; j < C::MI; ++j) {
                            const floatx4_t p = Frag<SUMS>::mul(fb, fa[j]);
                            const float t = __builtin_isnormal(s[j]) ? 0.f : sa[j];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                acc[i][j][e] = fmaf(p[e] * t, sb, acc[i][j][e]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < C::MI; ++j)
                        s[j] = __builtin_isnormal(s[j]) ? s[j] : 0.f;
                }
            }
            constexpr int NP = C::NI * C::MI;
            constexpr int LAG = SUMS == TWELL_SUMS_FP8 && C::MI > 2 ? 3 : 2;
            floatx4_t v[LAG + 1];
            auto scale = [&](int t) { // product t into its accumulator
                const int i = t / C::MI, j = t % C::MI;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[i][j][e] = BLKB ? fmaf(v[t % (LAG + 1)][e], s[j], acc[i][j][e])
                                        : fmaf(v[t % (LAG + 1)][e] * s[j], sb4[i & 1][e], acc[i][j][e]);
            };
#pragma unroll
            for (int t = 0; t < NP; ++t) {
                const int i = t / C::MI, j = t % C::MI;
                if (j == 0) {
                    if (i == C::NI - 1)
                        sync(kb1 - kb - 1);
                    if constexpr (SPLIT)
                        fb.set(rb[i % RB], two);
                    else
                        fb.set(rb[i % RB]);
                    if (i < C::NI - 1) {
                        rb[(i + 1) % RB] = frag(Bw + cur + (i + 1) * 16 * FP8_BLK);
                    } else {
                        rb[0] = frag(Bw + nxt);
                        if (BLKB)
                            sb = *(const float *)((const uint8_t *)sbw + nxt);
                    }
                }
                if constexpr (SPLIT)
                    v[t % (LAG + 1)] = Frag<SUMS>::mul(fb, fa[j], two);
                else
                    v[t % (LAG + 1)] = Frag<SUMS>::mul(fb, fa[j]);
                if (t >= LAG)
                    scale(t - LAG);
                static_assert(LAG <= C::MI, "the last row's scales are used by then");
                if (!BLKB && j == LAG - 1) // the row before is scaled: its place is free
                    sb4[(i + 1) & 1] = *(const floatx4_t *)((const uint8_t *)(
                        sbw + (i < C::NI - 1 ? (i + 1) * 16 : 0) + q4 * 4) + (i < C::NI - 1 ? cur : nxt));
                if (i == C::NI - 1) {
                    ra[j] = frag(Aw + nxt + j * 16 * FP8_BLK);
                    sa[j] = *(const float *)((const uint8_t *)(saw + j * 16 + l16) + nxt);
                }
#pragma unroll
                for (int g = t * C::LPS; g < (t + 1) * C::LPS && g <= C::WB; ++g)
                    load(g, kb + C::NST - 1, free);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int t = NP - LAG; t < NP; ++t)
                scale(t);
        }
        // ---- the next tile's first loads, into stages that every wave has left
        // (what it read of them beside its last products is not used)
        const int mw = m0 + wm * C::WM, nw = n0 + wn * C::WN, pt = part;
        const bool whole = m0 + C::BM <= a.M && n0 + C::BN <= a.N;
        // A whole tile's S stores all follow those loads, so the loads are in when
        // at most S of this wave's accesses are on their way (they end in order).
        auto arrive = [&](auto S) {
            fence();
            if (whole)
                ng::wait_vm<decltype(S)::value>();
            else
                ng::wait_vm<0>();
            __builtin_amdgcn_s_barrier();
            fence();
        };
        q0 += gridDim.x / NXCD;
        const bool more = C::STAY && q0 < run1;
        if (more) {
            place();
            first_loads();
        } else if (!C::STAY) {
            __syncthreads(); // the rows below lie in the stages
        }
        fence(); // no store before the loads
        // ---- epilogue: lane's element e of tile (i, j) is token j * 16 + l16,
        // n i * 16 + q4 * 4 + e of the wave's part. The values pass through the
        // wave's own piece of LDS, 16 tokens x WE n at a time, so that a store
        // instruction writes whole runs of WE values.
        auto store = [&](auto type, void *out, int64_t ld) {
            using T = decltype(type);
            constexpr int ES = sizeof(T), WE = ES == 4 ? 32 : C::WE;
            constexpr int VPL = 16 / ES, LPR = WE / VPL; // values a lane, lanes of a run
            const int lane = here((int)threadIdx.x) & 63, l16 = lane & 15, q4 = lane >> 4;
            const int c8 = lane % LPR, rr = lane / LPR;
            uint8_t *buf = L + (C::STAY ? C::NST * C::STAGE : 0) + w * 16 * C::OROW;
#pragma unroll
            for (int j = 0; j < C::MI; ++j)
#pragma unroll
                for (int h = 0; h < C::WN / WE; ++h) {
#pragma unroll
                    for (int i = 0; i < WE / 16; ++i) {
                        const floatx4_t v = acc[h * (WE / 16) + i][j];
                        uint8_t *p = buf + l16 * C::OROW + (i * 16 + q4 * 4) * ES;
                        if constexpr (ES == 4)
                            *(floatx4_t *)p = v;
                        else
                            *(uint2 *)p = make_uint2(f32x2_to_bf16x2(v[0], v[1]),
                                                     f32x2_to_bf16x2(v[2], v[3]));
                    }
                    const int n = nw + h * WE + c8 * VPL;
#pragma unroll
                    for (int r0 = 0; r0 < 16; r0 += 64 / LPR) {
                        const int m = mw + j * 16 + r0 + rr;
                        const uint4 v = *(const uint4 *)(buf + (r0 + rr) * C::OROW + c8 * 16);
                        T *row = (T *)out + m * ld;
                        if (whole || (m < a.M && n + VPL <= a.N)) {
                            stg16u_nt(row + n, v);
                        } else if (m < a.M) {
                            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int e = 0; e < VPL; ++e)
                                if (n + e < a.N)
                                    row[n + e] = (T)(u[e * ES / 4] >> (8 * ES * e % 32));
                        }
                    }
                }
            if (more)
                arrive(std::integral_constant<int, C::MI * (C::WN / WE) * (16 * LPR / 64)>());
        };
        if (a.parts > 1 || a.dto == TWELL_F32)
            store(uint32_t(), a.parts > 1 ? a.part + (int64_t)pt * a.M * a.N : (float *)a.out,
                  a.parts > 1 ? a.N : a.ldo);
        else
            store(uint16_t(), a.out, a.ldo);
        if (!more)
            return;
    }
}

// out = the sum of the parts, in order; four n a thread.
__global__ __launch_bounds__(256) void fp8_mm_join_kernel(MmArgs a)
{
    const int64_t n4 = (a.N + 3) / 4, q = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (q >= n4 * a.M)
        return;
    const int64_t m = q / n4;
    const int n = (int)(q % n4) * 4;
    const float *p = a.part + m * a.N + n;
    const int64_t stride = (int64_t)a.M * a.N;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (n + 4 <= a.N) {
        for (int i = 0; i < a.parts; ++i) {
            const uint4 u = ldg16u(p + i * stride);
            v[0] += __uint_as_float(u.x), v[1] += __uint_as_float(u.y);
            v[2] += __uint_as_float(u.z), v[3] += __uint_as_float(u.w);
        }
    } else {
        for (int i = 0; i < a.parts; ++i)
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (n + e < a.N)
                    v[e] += p[i * stride + e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (n + e < a.N) {
            if (a.dto == TWELL_BF16)
                ((uint16_t *)a.out)[m * a.ldo + n + e] = (uint16_t)f32x2_to_bf16x2(v[e], 0.f);
            else
                ((float *)a.out)[m * a.ldo + n + e] = v[e];
        }
}

// ---------------------------------------------------------------- few tokens
// A workgroup computes 16 NB n for 16 TB tokens, its WV waves taking every
// WV-th block of k; their sums meet in LDS. A wave's rows of a block go to its
// own piece of LDS, two blocks in turn, as whole 128-byte lines (eight adjacent
// lanes a row): loaded straight into the fragments' registers, where adjacent
// lanes are different rows, every lane is a request of its own, and 16 tokens
// by 2304 n over 6144 took 8.1 us in place of 4.6. No barrier: a wave waits for
// its own loads. The scales are staged SCB blocks of k at a time.
template <int TB, int NB, int WV, int SCB, int SUMS>
__global__ __launch_bounds__(64 * WV) void fp8_mm_rows_kernel(MmArgs a)
{
    constexpr int NF = NB + TB, STG = NF * 2048; // fragments of a block, B's first
    constexpr int BUF = WV * 2 * STG;
    static_assert(BUF >= WV * NB * TB * 1024, "the sums reuse the blocks' space");
    __shared__ __attribute__((aligned(16))) uint8_t L[BUF];
    __shared__ float ssa[SCB][16 * TB];
    __shared__ __attribute__((aligned(16))) float ssb[SCB][16 * NB];
    const int lane = threadIdx.x & 63, w = wave_id();
    const int l16 = lane & 15, q4 = lane >> 4;
    const int tiles_n = (a.N + 16 * NB - 1) / (16 * NB);
    const int n0 = (int)(blockIdx.x % tiles_n) * (16 * NB);
    const int m0 = (int)(blockIdx.x / tiles_n) * (16 * TB);
    // load i of a block: eight rows of fragment i / 2, lane l the chunk of row
    // l / 8 that the swizzle puts at byte 16 l. Rows past an operand read its
    // last row; their outputs are dropped.
    const uint8_t *srcb = a.qb + (int64_t)n0 * a.pitch, *srca = a.qa + (int64_t)m0 * a.pitch;
    uint32_t off[2 * NF];
#pragma unroll
    for (int i = 0; i < 2 * NF; ++i) {
        const int r = (i < 2 * NB ? i : i - 2 * NB) * 8 + lane / 8;
        const int last = i < 2 * NB ? a.N - 1 - n0 : a.M - 1 - m0;
        off[i] = (uint32_t)min(r, last) * (uint32_t)a.pitch + (((lane & 7) ^ ((r >> 1) & 7)) << 4);
    }
    uint8_t *Lw = L + w * 2 * STG;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(ng::lds_u8 *)Lw;
    auto fetch = [&](int kb, int st) {
#pragma unroll
        for (int i = 0; i < 2 * NF; ++i)
            dma16((i < 2 * NB ? srcb : srca) + (int64_t)kb * FP8_BLK, off[i],
                  lds0 + (uint32_t)(st * STG + i * 1024), kb, a.nkb);
    };
    floatx4_t acc[NB][TB];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int t = 0; t < TB; ++t)
            acc[i][t] = floatx4_t{0.f, 0.f, 0.f, 0.f};
    const int f0 = l16 * FP8_BLK + ((q4 ^ ((l16 >> 1) & 7)) << 4), f1 = f0 ^ 64;
    auto frag = [&](const uint8_t *p) {
        const uint4 u = *(const uint4 *)(p + f0), v = *(const uint4 *)(p + f1);
        return intx8_t{(int)u.x, (int)u.y, (int)u.z, (int)u.w,
                       (int)v.x, (int)v.y, (int)v.z, (int)v.w};
    };
    // The i-th block of this wave among the SCB from k0, nkb when there is none.
    // Workgroups begin an eighth of the way apart: rows whose pitch is a large
    // power of two would otherwise be read from the same few memory channels by
    // all workgroups at once (one token by 8192 over 8192: 16.8 -> 13.8 us,
    // 16 by 4096 over 4096: 6.8 -> 6.3). It goes by their n, so that within one
    // kernel a token's sums do not depend on the tokens beside it; how many these
    // are chooses the kernel, and so the order of its additions.
    const uint32_t turn = (uint32_t)n0 / (128 * NB) & 7;
    auto steps = [&](int k0) {
        return (int)((uint32_t)(min(SCB, a.nkb - k0) - w + WV - 1) / WV);
    };
    auto block = [&](int k0, int i) {
        const int n = steps(k0), q = i + (int)(turn * (uint32_t)n >> 3);
        return i < n ? k0 + w + WV * (q < n ? q : q - n) : a.nkb;
    };
    int kb = block(0, 0);
    fetch(kb, 0);
    int st = 0;
    for (int k0 = 0; k0 < a.nkb; k0 += SCB) {
        const int nk = min(SCB, a.nkb - k0);
        if (k0)
            __syncthreads(); // the last scales are used
        for (int q = threadIdx.x; q < nk * 16 * TB; q += 64 * WV)
            ssa[q / (16 * TB)][q % (16 * TB)] =
                a.sa[(int64_t)(k0 + q / (16 * TB)) * a.nsa +
                     min(m0 + q % (16 * TB), a.M - 1) / a.ra];
        for (int q = threadIdx.x; q < nk * 16 * NB; q += 64 * WV)
            ssb[q / (16 * NB)][q % (16 * NB)] =
                a.sb[(int64_t)(k0 + q / (16 * NB)) * a.nsb +
                     min(n0 + q % (16 * NB), a.N - 1) / a.rb];
        __syncthreads();
        const int n = steps(k0);
        for (int i = 0; i < n; ++i, st ^= 1) {
            const int kc = kb - k0;
            kb = i + 1 < n ? block(k0, i + 1) : k0 + SCB < a.nkb ? block(k0 + SCB, 0) : a.nkb;
            // the other piece was read a block ago; its loads, then this one's wait
            fetch(kb, st ^ 1);
            if (kb < a.nkb)
                ng::wait_vm<2 * NF>();
            else
                ng::wait_vm<0>();
            asm volatile("" ::: "memory");
            const uint8_t *S = Lw + st * STG;
            Frag<SUMS> fb[NB];
            floatx4_t sb[NB];
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                fb[i].set(frag(S + i * 2048));
                sb[i] = *(const floatx4_t *)&ssb[kc][i * 16 + q4 * 4];
            }
#pragma unroll
            for (int t = 0; t < TB; ++t) {
                Frag<SUMS> fa;
                fa.set(frag(S + (NB + t) * 2048));
                const float sa = ssa[kc][t * 16 + l16];
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    const floatx4_t p = Frag<SUMS>::mul(fb[i], fa);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[i][t][e] = fmaf(p[e] * sa, sb[i][e], acc[i][t][e]);
                }
            }
            // the reads are done before the piece is loaded again
            __builtin_amdgcn_s_waitcnt(0xC07F);
            asm volatile("" ::: "memory");
        }
    }
    __syncthreads();
    floatx4_t(*part)[NB * TB][64] = (floatx4_t(*)[NB * TB][64])L;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int t = 0; t < TB; ++t)
            part[w][i * TB + t][lane] = acc[i][t];
    __syncthreads();
    // tile q's partial sums are joined by wave q % WV, in wave order
    for (int q = w; q < NB * TB; q += WV) {
        floatx4_t o = part[0][q][lane];
#pragma unroll
        for (int u = 1; u < WV; ++u)
            o += part[u][q][lane];
        const int m = m0 + q % TB * 16 + l16;
        if (m >= a.M)
            continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int n = n0 + q / TB * 16 + q4 * 4 + e;
            if (n < a.N) {
                if (a.dto == TWELL_BF16)
                    ((uint16_t *)a.out)[m * a.ldo + n] = (uint16_t)f32x2_to_bf16x2(o[e], 0.f);
                else
                    ((float *)a.out)[m * a.ldo + n] = o[e];
            }
        }
    }
}

template <int TB, int NB, int WV, int SCB, int SUMS> void rows_one(const MmArgs &a, hipStream_t s)
{
    const int64_t tn = (a.N + 16 * NB - 1) / (16 * NB);
    const dim3 grid((uint32_t)(tn * ((a.M + 16 * TB - 1) / (16 * TB))));
    fp8_mm_rows_kernel<TB, NB, WV, SCB, SUMS><<<grid, 64 * WV, 0, s>>>(a);
}
using T256 = TileCfg<256, 256, 4, 2, 2>; // waves of 64 tokens x 128 n
using T192 = TileCfg<192, 256, 4, 2, 2>; // waves of 48 x 128
using T128 = TileCfg<128, 128, 2, 4, 3>; // waves of 64 x 32
using T64 = TileCfg<64, 128, 2, 4, 3>;   // waves of 32 x 32

template <class C, int SUMS, bool BLKB> void launch_tile(const MmArgs &a, hipStream_t s)
{
    const int64_t total = (int64_t)((a.N + C::BN - 1) / C::BN) * ((a.M + C::BM - 1) / C::BM) *
                          a.parts;
    int64_t wgs = (total + NXCD - 1) / NXCD * NXCD;
    if (C::STAY && wgs > 256)
        wgs = 256; // one for each CU
    const dim3 grid((uint32_t)wgs);
    fp8_mm_tile_kernel<C, SUMS, BLKB><<<grid, C::NT, 0, s>>>(a);
}

// Which kernel takes a product, and in how many parts of the contraction: the
// least of the times that these measured figures give (us; they order the
// kernels, no more). A tile kernel is counted as a tile per CU at a time, a step
// of 128 k at `step` and `tile` for its beginning and end; full sums cost what
// widening and the bfloat16 instruction do. (Two tiles of 64 x 128 fit a CU and
// share it: a second round of them is counted 10 to 20% dearer than it is, and
// rounds that leave CUs idle run faster than counted, at higher clocks. Of 27
// sizes from 130 to 4096 tokens, each in three modes, the choice was the fastest
// or within 5% in 73 of 81, and at worst 19% behind: 2000 x 4100 over 700.) Parts
// add a second launch and the partial sums' way through memory. A rows kernel's
// wave takes 0.15 for each fragment of a block of k (its loads' issue), unless all
// the workgroups' reads together pass what the L2s serve (12 MB a us).
enum Kernel { ROWS_1_1, ROWS_1_2, ROWS_2_2, ROWS_2_2_8, TILE_64, TILE_128, TILE_192, TILE_256 };
struct Plan {
    Kernel k;
    int parts, per; // parts of the contraction, blocks of k in each
};

Plan plan(int M, int N, int nkb, int sums, int rb)
{
    const bool full = sums == TWELL_SUMS_F32, blkb = rb == FP8_BLK;
    Plan best = {TILE_64, 1, nkb};
    double least = 1e300;
    auto up = [](double a, double b) { return ceil(a / b); };
    auto offer = [&](Kernel k, int parts, double t) {
        if (t < least)
            least = t, best = {k, parts, (nkb + parts - 1) / parts};
    };
    const struct {
        Kernel k;
        int tb, nb, wv, occ; // occ: workgroups that a CU runs in the time of one
    } rows[] = {{ROWS_1_1, 1, 1, 8, 1}, {ROWS_1_2, 1, 2, 8, 1}, {ROWS_2_2, 2, 2, 4, 2},
                {ROWS_2_2_8, 2, 2, 8, 1}};
    for (const auto &r : rows) {
        const double wg = up(M, 16 * r.tb) * up(N, 16 * r.nb);
        if (wg * 64 * r.wv > 4294967295.) // threads of a launch
            continue;
        const double lat = up(wg, 256 * r.occ) * (up(nkb, r.wv) * 0.15 * (r.tb + r.nb) + 0.8);
        const double mem = wg * 16 * (r.tb + r.nb) * nkb * FP8_BLK / 12e6;
        offer(r.k, 1, 2.0 + (lat > mem ? lat : mem));
    }
    const struct {
        Kernel k;
        int bm, bn;
        double step, tile;
    } tiles[] = {{TILE_64, 64, 128, full ? 0.62 : 0.37, 1.5},
                 {TILE_128, 128, 128, full ? 1.3 : 0.5, full ? 1.8 : 2.5},
                 {TILE_192, 192, 256, !full ? 1.35 : blkb ? 2.2 : 2.4, full ? 5.0 : 4.2},
                 {TILE_256, 256, 256, full ? 3.2 : 1.52, full ? 5.0 : 4.2}};
    for (const auto &c : tiles) {
        // full sums hold their operands widened: with a scale for each row of B
        // as well, 256 x 256 does not fit the registers (4.0 a step, 192 x 256
        // 2.4); with 128-row scales it keeps five lane constants of a tile, none
        // of a step, in scratch
        if (c.k == TILE_256 && full && !blkb)
            continue;
        for (int parts = 1; parts <= 32 && parts <= nkb; parts *= 2) {
            const double wg = up(M, c.bm) * up(N, c.bn) * parts;
            const double join = parts == 1 ? 0. : 3.0 + (double)parts * M * N * 8 / 4e6;
            offer(c.k, parts, 2.6 + up(wg, 256) * (up(nkb, parts) * c.step + c.tile) + join);
        }
    }
    best.parts = best.per ? (nkb + best.per - 1) / best.per : 1;
    return best;
}

template <int SUMS, bool BLKB> void launch_sums(const MmArgs &a, Kernel k, hipStream_t s)
{
    switch (k) {
    case ROWS_1_1: return rows_one<1, 1, 8, 64, SUMS>(a, s);
    case ROWS_1_2: return rows_one<1, 2, 8, 64, SUMS>(a, s);
    case ROWS_2_2: return rows_one<2, 2, 4, 64, SUMS>(a, s);
    case ROWS_2_2_8: return rows_one<2, 2, 8, 32, SUMS>(a, s);
    case TILE_64: return launch_tile<T64, SUMS, BLKB>(a, s);
    case TILE_128: return launch_tile<T128, SUMS, BLKB>(a, s);
    case TILE_192:
        return launch_tile<T192, SUMS, BLKB>(a, s);
    case TILE_256:
        if constexpr (SUMS == TWELL_SUMS_FP8 || BLKB)
            launch_tile<T256, SUMS, BLKB>(a, s);
        return;
    }
}

} // namespace

size_t fp8_mm_workspace(int M, int N, int K)
{
    const int nkb = fp8_blocks(K);
    int parts = 1; // the most that any call of these sizes takes
    for (int sums : {TWELL_SUMS_F32, TWELL_SUMS_FP8})
        for (int rb : {1, FP8_BLK}) {
            const int p = plan(M, N, nkb, sums, rb).parts;
            parts = p > parts ? p : parts;
        }
    return parts > 1 ? (size_t)parts * M * N * 4 : 0;
}

int launch_fp8_mm(const twell_fp8_t *A, const twell_fp8_t *B, const twell_mat_t *out, int sums,
                  void *ws, size_t ws_bytes, twell_timing_t *timing, hipStream_t s)
{
    MmArgs a = {};
    a.qa = A->q, a.sa = A->scale, a.qb = B->q, a.sb = B->scale;
    a.out = out->data, a.ldo = out->ld, a.dto = out->dtype;
    a.pitch = fp8_pitch(A->cols);
    a.M = A->rows, a.N = B->rows, a.nkb = fp8_blocks(A->cols);
    a.ra = A->block_rows, a.rb = B->block_rows;
    a.nsa = (a.M + a.ra - 1) / a.ra, a.nsb = (a.N + a.rb - 1) / a.rb;
    const Plan p = plan(a.M, a.N, a.nkb, sums, a.rb);
    if (p.parts > 1 && (!ws || ws_bytes < (size_t)p.parts * a.M * a.N * 4))
        return TWELL_E_WORKSPACE;
    a.parts = p.parts, a.per = p.per, a.part = (float *)ws;
    Timer tm(timing, s);
    const bool blkb = a.rb == FP8_BLK;
    if (sums == TWELL_SUMS_FP8)
        blkb ? launch_sums<TWELL_SUMS_FP8, true>(a, p.k, s)
             : launch_sums<TWELL_SUMS_FP8, false>(a, p.k, s);
    else
        blkb ? launch_sums<TWELL_SUMS_F32, true>(a, p.k, s)
             : launch_sums<TWELL_SUMS_F32, false>(a, p.k, s);
    static const char *const names[] = {"fp8_mm_rows_1x1", "fp8_mm_rows_1x2", "fp8_mm_rows_2x2",
                                        "fp8_mm_rows_2x2_8", "fp8_mm_tile64", "fp8_mm_tile128",
                                        "fp8_mm_tile192", "fp8_mm_tile256"};
    tm.mark(names[p.k]);
    if (a.parts > 1) {
        const int64_t q = (int64_t)((a.N + 3) / 4) * a.M;
        fp8_mm_join_kernel<<<(uint32_t)((q + 255) / 256), 256, 0, s>>>(a);
        tm.mark("fp8_mm_join");
    }
    return hipGetLastError() == hipSuccess ? TWELL_OK : TWELL_E_HIP;
}
