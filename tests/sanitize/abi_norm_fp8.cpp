// Host-side checks of the norm, quantisation and 8-bit product calls, built
// without device code and run under AddressSanitizer and
// UndefinedBehaviorSanitizer (no GPU is touched):
//   - each entry point, fed the edges of its arguments' ranges one by one and
//     in pairs, refuses what its documentation refuses before it reaches the
//     HIP runtime, or has no rows and nothing to do;
//   - each workspace sizer, fed sizes up to INT32_MAX, returns without
//     undefined behaviour, 0 for what its call refuses, and enough for the
//     partial sums that its call keeps there.
// Every call either has one argument that must be refused or a workspace of
// no bytes, so none is launched. Prints "abi_norm_fp8 ok" and exits 0; a
// failed expectation exits 1, a sanitizer report aborts the program.
#include <climits>
#include <cmath>
#include <cstdio>
#include <cstring>

#include "twell.h"

static int failures = 0;

#define EXPECT(cond)                                                                       \
    do {                                                                                   \
        if (!(cond)) {                                                                     \
            std::fprintf(stderr, "%s:%d: expectation failed: %s\n", __FILE__, __LINE__,    \
                         #cond);                                                           \
            ++failures;                                                                    \
        }                                                                                  \
    } while (0)

// addresses that are never dereferenced: aligned to 16, to 4, to nothing
static void *const FAKE = (void *)(uintptr_t)0x100000;
static void *const BY4 = (void *)(uintptr_t)0x100004;
static void *const ODD = (void *)(uintptr_t)0x100001;

static const int32_t EDGES[] = {INT_MIN, INT_MIN + 1, -129, -1, 0, 1, 2, 127, 128, 129, 1000,
                                16383, 16384, 16385, (1 << 24) - 1, 1 << 24, (1 << 24) + 1,
                                1 << 28, (1 << 28) + 1, INT_MAX - 128, INT_MAX - 1, INT_MAX};
static const int64_t LDS[] = {INT64_MIN, -1, 0, 255, (int64_t)INT_MAX, ((int64_t)1 << 31) + 1,
                              ((int64_t)1 << 40), INT64_MAX};

static twell_mat_t mat(int32_t rows = 4, int32_t cols = 256, int64_t ld = -7,
                       twell_dtype dt = TWELL_BF16, void *p = FAKE)
{
    twell_mat_t m;
    std::memset(&m, 0, sizeof m);
    m.rows = rows;
    m.cols = cols;
    m.ld = ld == -7 ? (int64_t)cols : ld;
    m.dtype = dt;
    m.data = p;
    return m;
}

static twell_fp8_t fp8(int32_t rows = 4, int32_t cols = 256, int32_t br = 1, void *q = FAKE,
                       void *s = FAKE)
{
    twell_fp8_t m;
    std::memset(&m, 0, sizeof m);
    m.rows = rows;
    m.cols = cols;
    m.block_rows = br;
    m.q = (uint8_t *)q;
    m.scale = (float *)s;
    return m;
}

static bool refused(int rc) { return rc < 0 && std::strlen(twell_status_str(rc)) > 0; }

static void check_norm_fwd()
{
    const twell_mat_t ok = mat(), f32 = mat(4, 256, -7, TWELL_F32);
    auto f = [](const twell_mat_t *x, const twell_mat_t *r, const twell_mat_t *h,
                const twell_mat_t *n, const twell_fp8_t *n8, float eps, const void *g = FAKE) {
        return twell_rmsnorm_fwd(x, r, g, TWELL_F32, eps, h, n, n8, nullptr, nullptr);
    };
    const twell_fp8_t ok8 = fp8();
    EXPECT(refused(f(nullptr, &ok, &ok, &ok, nullptr, 1e-6f)));
    EXPECT(refused(f(&ok, &ok, &ok, nullptr, nullptr, 1e-6f)));
    EXPECT(refused(f(&ok, &ok, &ok, &ok, &ok8, 1e-6f)));
    EXPECT(refused(f(&ok, nullptr, &ok, &ok, nullptr, 1e-6f)));
    EXPECT(refused(f(&ok, &ok, &f32, &ok, nullptr, 1e-6f)));
    EXPECT(refused(f(&ok, &ok, &ok, &ok, nullptr, 1e-6f, nullptr)));
    EXPECT(refused(f(&ok, &ok, &ok, &ok, nullptr, 1e-6f, ODD)));
    for (float eps : {NAN, INFINITY, -INFINITY, -1e-30f})
        EXPECT(refused(f(&ok, &ok, &ok, &ok, nullptr, eps)));
    for (int32_t r : EDGES)
        for (int32_t c : EDGES) {
            const twell_mat_t m = mat(r, c);
            const twell_fp8_t e = fp8(r, c, 2);
            EXPECT(refused(f(&m, nullptr, nullptr, &ok, nullptr, 0.f)) || (r == 4 && c == 256));
            EXPECT(refused(f(&m, nullptr, nullptr, nullptr, &e, 0.f)));
        }
    for (int64_t ld : LDS) {
        const twell_mat_t m = mat(4, 256, ld), bad = mat(4, 256, -7, TWELL_BF16, ODD);
        EXPECT(refused(f(&m, &bad, nullptr, &ok, nullptr, 0.f)));
        EXPECT(refused(f(&bad, &ok, nullptr, &m, nullptr, 0.f)));
    }
    for (int dt : {INT_MIN, -1, 2, 9, INT_MAX}) {
        const twell_mat_t m = mat(4, 256, -7, (twell_dtype)dt);
        EXPECT(refused(f(&m, nullptr, nullptr, &ok, nullptr, 0.f)));
        EXPECT(refused(f(&ok, nullptr, nullptr, &m, nullptr, 0.f)));
        EXPECT(refused(twell_rmsnorm_fwd(&ok, nullptr, FAKE, (twell_dtype)dt, 0.f, nullptr, &ok,
                                         nullptr, nullptr, nullptr)));
    }
    const twell_fp8_t by4 = fp8(4, 256, 1, BY4), odd = fp8(4, 256, 1, FAKE, ODD);
    EXPECT(refused(f(&ok, nullptr, nullptr, nullptr, &by4, 0.f)));
    EXPECT(refused(f(&ok, nullptr, nullptr, nullptr, &odd, 0.f)));
    const twell_mat_t none = mat(0, 256, -7, TWELL_BF16, nullptr);
    EXPECT(f(&none, &none, &none, &none, nullptr, 0.f) == TWELL_OK);
}

static void check_norm_bwd()
{
    for (int32_t r : EDGES)
        for (int32_t c : EDGES) {
            const size_t need = twell_rmsnorm_bwd_workspace_bytes(r, c);
            const bool valid = r >= 1 && r <= (1 << 28) && c >= 1 && c <= TWELL_NORM_COLS;
            // at least one row of partial sums, at most one for each workgroup
            EXPECT(valid ? need >= (size_t)c * 4 && need <= (size_t)c * 4 * 4096 : need == 0);
            const twell_mat_t m = mat(r, c);
            if (r != 0) {
                EXPECT(refused(twell_rmsnorm_bwd(&m, &m, FAKE, TWELL_F32, 0.f, nullptr, &m,
                                                 (float *)FAKE, FAKE, need ? need - 1 : 0,
                                                 nullptr, nullptr)));
                EXPECT(refused(twell_rmsnorm_bwd(&m, &m, FAKE, TWELL_F32, 0.f, nullptr, &m,
                                                 (float *)FAKE, nullptr, need, nullptr,
                                                 nullptr)));
            }
        }
    const twell_mat_t ok = mat();
    for (int64_t ld : LDS) {
        const twell_mat_t m = mat(4, 256, ld);
        EXPECT(refused(twell_rmsnorm_bwd(&m, &ok, FAKE, TWELL_F32, 0.f, &ok, &ok, (float *)FAKE,
                                         FAKE, 0, nullptr, nullptr)));
    }
    EXPECT(refused(twell_rmsnorm_bwd(&ok, &ok, FAKE, TWELL_F32, 0.f, &ok, &ok, (float *)FAKE,
                                     BY4, (size_t)1 << 40, nullptr, nullptr)));
    EXPECT(refused(twell_rmsnorm_bwd(&ok, &ok, FAKE, TWELL_F32, 0.f, &ok, &ok, nullptr, FAKE,
                                     (size_t)1 << 40, nullptr, nullptr)));
}

static void check_quant()
{
    const twell_mat_t ok = mat();
    for (int32_t r : EDGES)
        for (int32_t c : EDGES) {
            const twell_mat_t m = mat(r, c);
            // an odd address for the codes: refused whatever the sizes, unless
            // there is nothing to do
            const twell_fp8_t o = fp8(r, c, 1, ODD), t = fp8(c, r, 128, ODD);
            const bool empty = r == 0 || c == 0;
            const int rc = twell_fp8_quant(&m, &o, nullptr, nullptr, nullptr);
            const int rt = twell_fp8_quant(&m, nullptr, &t, nullptr, nullptr);
            EXPECT(refused(rc) || (empty && rc == TWELL_OK));
            EXPECT(refused(rt) || (empty && rt == TWELL_OK));
            EXPECT(refused(twell_fp8_quant(&m, &o, &t, nullptr, nullptr)) || empty);
        }
    for (int32_t b : EDGES)
        if (b != 1 && b != 128) {
            const twell_fp8_t o = fp8(4, 256, b);
            EXPECT(refused(twell_fp8_quant(&ok, &o, nullptr, nullptr, nullptr)));
        }
    EXPECT(refused(twell_fp8_quant(nullptr, nullptr, nullptr, nullptr, nullptr)));
    EXPECT(refused(twell_fp8_quant(&ok, nullptr, nullptr, nullptr, nullptr)));
}

static void check_matmul()
{
    const twell_fp8_t a = fp8(), b = fp8(8, 256, 128);
    for (int32_t M : EDGES)
        for (int32_t N : EDGES)
            for (int32_t K : EDGES) {
                const size_t need = twell_fp8_matmul_workspace_bytes(M, N, K);
                if (M < 0 || N < 0 || K < 0 || K > TWELL_MAX_K)
                    EXPECT(need == 0);
                else
                    EXPECT(need == 0 || need >= (size_t)M * (size_t)N * 8); // two parts or more
            }
    for (int32_t r : EDGES)
        for (int32_t c : EDGES) {
            const twell_fp8_t x = fp8(r, c), odd = fp8(8, c, 1, ODD);
            const twell_mat_t o = mat(r, 8), bad = mat(r, 7);
            if (r == 0)
                continue;
            EXPECT(refused(twell_fp8_matmul(&x, &b, &bad, TWELL_SUMS_F32, nullptr, 0, nullptr,
                                            nullptr)));
            EXPECT(refused(twell_fp8_matmul(&x, &odd, &o, TWELL_SUMS_FP8, nullptr, 0, nullptr,
                                            nullptr)) ||
                   c == 0);
        }
    for (int64_t ld : LDS) {
        const twell_mat_t o = mat(4, 8, ld, TWELL_F32, ODD);
        EXPECT(refused(twell_fp8_matmul(&a, &b, &o, TWELL_SUMS_F32, nullptr, 0, nullptr,
                                        nullptr)));
    }
    const twell_mat_t o = mat(4, 8);
    for (int32_t s : EDGES)
        if (s != TWELL_SUMS_F32 && s != TWELL_SUMS_FP8)
            EXPECT(refused(twell_fp8_matmul(&a, &b, &o, s, nullptr, 0, nullptr, nullptr)));
    EXPECT(refused(twell_fp8_matmul(&a, &b, &o, 0, BY4, (size_t)1 << 40, nullptr, nullptr)));
    EXPECT(refused(twell_fp8_matmul(nullptr, &b, &o, 0, nullptr, 0, nullptr, nullptr)));
    EXPECT(refused(twell_fp8_matmul(&a, nullptr, &o, 0, nullptr, 0, nullptr, nullptr)));
    EXPECT(refused(twell_fp8_matmul(&a, &b, nullptr, 0, nullptr, 0, nullptr, nullptr)));
    // a product split over its contraction refuses a workspace too small
    const size_t need = twell_fp8_matmul_workspace_bytes(300, 256, 8192);
    const twell_fp8_t sa = fp8(300, 8192), sb = fp8(256, 8192);
    const twell_mat_t so = mat(300, 256);
    if (need)
        EXPECT(twell_fp8_matmul(&sa, &sb, &so, 0, FAKE, need - 1, nullptr, nullptr) ==
               TWELL_E_WORKSPACE);
}

int main()
{
    check_norm_fwd();
    check_norm_bwd();
    check_quant();
    check_matmul();
    if (failures)
        return 1;
    std::puts("abi_norm_fp8 ok");
    return 0;
}
