// Host-side checks of the calls on weights in 4 bits, built without device code
// and run under AddressSanitizer and UndefinedBehaviorSanitizer (no GPU is
// touched): each entry point, fed the edges of its arguments' ranges, refuses
// what its documentation refuses, and each workspace sizer returns without
// undefined behaviour, 0 for what its call refuses. Every call has one argument
// that must be refused, a workspace of no bytes where one is needed, or nothing to
// do, so none is launched. Prints "abi_fp4 ok" and exits 0; a failed expectation
// exits 1, a sanitizer report aborts the program.
#include <climits>
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

static void *const FAKE = (void *)(uintptr_t)0x100000;
static void *const ODD = (void *)(uintptr_t)0x100001;
static const int32_t EDGES[] = {INT_MIN, -129, -1, 0, 1, 2, 16, 17, 64, 65, 127, 128, 129, 4096,
                                (1 << 21) - 1, 1 << 21, (1 << 21) + 1, 1 << 27, 1 << 28,
                                (1 << 28) + 1, INT_MAX - 128, INT_MAX};
static const int64_t LDS[] = {INT64_MIN, -1, 0, 255, ((int64_t)1 << 31) + 1, INT64_MAX};

static twell_mat_t mat(int32_t rows, int32_t cols, int64_t ld = -7, twell_dtype dt = TWELL_BF16,
                       void *p = FAKE)
{
    twell_mat_t m;
    std::memset(&m, 0, sizeof m);
    m.rows = rows, m.cols = cols, m.ld = ld == -7 ? (int64_t)cols : ld, m.dtype = dt, m.data = p;
    return m;
}
static twell_fp4_t fp4(int32_t rows, int32_t cols, int32_t group = 64, void *q = FAKE,
                       void *s = FAKE)
{
    twell_fp4_t m;
    std::memset(&m, 0, sizeof m);
    m.rows = rows, m.cols = cols, m.group = group, m.q = (uint8_t *)q, m.scale = (uint16_t *)s;
    return m;
}
static bool refused(int rc) { return rc < 0 && std::strlen(twell_status_str(rc)) > 0; }

int main()
{
    for (int32_t r : EDGES)
        for (int32_t c : EDGES) {
            const bool empty = r == 0 || c == 0;
            const twell_mat_t m = mat(r, c);
            const twell_fp4_t odd = fp4(r, c, 64, ODD), group = fp4(r, c, 65);
            const int rc = twell_fp4_quant(&m, &odd, nullptr, nullptr);
            const int rd = twell_fp4_dequant(&odd, &m, nullptr, nullptr);
            EXPECT(refused(rc));
            EXPECT(refused(rd));
            EXPECT(refused(twell_fp4_quant(&m, &group, nullptr, nullptr)));
            const twell_fp4_t w = fp4(r, c);
            if (empty && r >= 0 && c >= 0 && r <= 1 << 28 && c <= 1 << 28)
                EXPECT(twell_fp4_quant(&m, &w, nullptr, nullptr) == TWELL_OK);
            for (int32_t T : EDGES) {
                for (twell_dtype dt : {TWELL_BF16, TWELL_F32}) {
                    const size_t need = twell_fp4_matmul_workspace_bytes(dt, T, r, c);
                    const size_t back = twell_fp4_matmul_dx_workspace_bytes(dt, T, r, c);
                    if (T <= 0 || r < 0 || c < 0 || c > 1 << 21)
                        EXPECT(need == 0);
                    if (T <= 0 || r < 0 || c < 0 || r > 1 << 21)
                        EXPECT(back == 0);
                    // float32 and a column too many for any alignment: a workspace
                    const twell_mat_t x = mat(T, c, -7, TWELL_F32), o = mat(T, r);
                    const twell_mat_t dy = mat(T, r, -7, TWELL_F32), dx = mat(T, c);
                    if (T != 0 && r != 0 && c != 0) {
                        EXPECT(refused(twell_fp4_matmul(&x, &w, &o, nullptr, 0, nullptr, nullptr)));
                        EXPECT(refused(twell_fp4_matmul_dx(&dy, &w, &dx, nullptr, 0, nullptr, nullptr)));
                    }
                    const size_t lay = twell_fp4_decode_workspace_bytes(dt, T, r, c);
                    EXPECT(lay == 0 || (T >= 0 && T <= TWELL_DECODE_T && r % 64 == 0 && c % 128 == 0));
                }
                const twell_mat_t x = mat(T, c);
                if (T != 0)
                    EXPECT(refused(twell_fp4_decode_fwd(&x, &w, &w, &w, (float *)FAKE, nullptr, 0,
                                                        nullptr, nullptr)));
            }
        }
    const twell_fp4_t w = fp4(128, 256);
    const twell_mat_t x = mat(4, 256), y = mat(4, 128);
    for (int64_t ld : LDS) {
        const twell_mat_t m = mat(4, 256, ld, TWELL_F32, ODD), n = mat(4, 128, ld, TWELL_F32, ODD);
        EXPECT(refused(twell_fp4_matmul(&m, &w, &y, FAKE, 1 << 30, nullptr, nullptr)));
        EXPECT(refused(twell_fp4_matmul(&x, &w, &n, FAKE, 1 << 30, nullptr, nullptr)));
        EXPECT(refused(twell_fp4_matmul_dx(&n, &w, &x, FAKE, 1 << 30, nullptr, nullptr)));
        EXPECT(refused(twell_fp4_decode_fwd(&m, &w, &w, &w, (float *)FAKE, FAKE, 1 << 30, nullptr,
                                            nullptr)));
    }
    for (int dt : {INT_MIN, -1, 2, INT_MAX}) {
        const twell_mat_t m = mat(4, 256, -7, (twell_dtype)dt);
        EXPECT(refused(twell_fp4_matmul(&m, &w, &y, FAKE, 1 << 30, nullptr, nullptr)));
        EXPECT(refused(twell_fp4_matmul_dx(&y, &w, &m, FAKE, 1 << 30, nullptr, nullptr)));
        EXPECT(twell_fp4_matmul_workspace_bytes((twell_dtype)dt, 4, 8, 8) == 0);
        EXPECT(twell_fp4_decode_workspace_bytes((twell_dtype)dt, 4, 256, 128) == 0);
    }
    EXPECT(refused(twell_fp4_matmul(nullptr, &w, &y, FAKE, 1, nullptr, nullptr)));
    EXPECT(refused(twell_fp4_matmul(&x, nullptr, &y, FAKE, 1, nullptr, nullptr)));
    EXPECT(refused(twell_fp4_matmul_dx(&y, &w, nullptr, FAKE, 1, nullptr, nullptr)));
    EXPECT(refused(twell_fp4_quant(nullptr, nullptr, nullptr, nullptr)));
    EXPECT(refused(twell_fp4_dequant(nullptr, nullptr, nullptr, nullptr)));
    EXPECT(refused(twell_fp4_decode_fwd(&x, &w, nullptr, &w, (float *)FAKE, FAKE, 1, nullptr, nullptr)));
    if (failures)
        return 1;
    std::puts("abi_fp4 ok");
    return 0;
}
