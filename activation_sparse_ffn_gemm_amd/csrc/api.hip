// C-ABI entry points: argument validation, then launches on the caller's
// stream. Nothing here allocates, synchronises or keeps state.
#include "common.hpp"

hipError_t launch_gate_pack(twell_dtype dt, const void *x, const void *wg_t, int T, int dm,
                            const twell_t *o, void *ws, int32_t *status, twell_timing_t *timing,
                            hipStream_t s);
size_t dec_gate_workspace(int dt, int T, int dm, int dff);
hipError_t launch_ffn_fwd(twell_dtype dt, const void *x, const twell_t *h, const void *wu_t,
                          const void *wd, int dm, float *y, void *ws, int32_t *status,
                          twell_timing_t *timing, hipStream_t s);
size_t fwd_workspace(int dt, int T, int dm, int dff, int W);
hipError_t launch_to_hybrid(const twell_t *h, const hybrid_t *o, int32_t *status,
                            twell_timing_t *timing, hipStream_t s);
hipError_t launch_bwd(twell_dtype dt, const void *x, const void *dy, const hybrid_t *h,
                      const void *wg_t, const void *wu_t, const void *wd, int dm, float l1,
                      float *dx,
                      float *dwg_t, float *dwu_t, float *dwd, void *ws, int32_t *status,
                      twell_timing_t *timing, hipStream_t s);
size_t bwd_workspace_layout(int dt, int T, int dm, int dff, int K, int max_ovf);
hipError_t launch_hyb_fwd(twell_dtype dt, const void *x, const hybrid_t *h, const void *wu_t,
                          const void *wd, int dm, float *y, void *ws, int32_t *status,
                          twell_timing_t *timing, hipStream_t s);
size_t hyb_fwd_workspace(int dt, int T, int dm, int max_ovf, int dff, int K);
size_t dec_layer_workspace(int dt, int T, int dm, int dff, int W);
hipError_t launch_dec_layer(twell_dtype dt, const void *x, const void *wg_t, const void *wu_t,
                            const void *wd, int dm, const twell_t *o, float *y, void *ws,
                            int32_t *status, twell_timing_t *timing, hipStream_t s);

hipError_t launch_rmsnorm_fwd(const twell_mat_t *x, const twell_mat_t *res, const void *gain,
                              int dtg, float eps, const twell_mat_t *h, const twell_mat_t *n,
                              const twell_fp8_t *n8, twell_timing_t *timing, hipStream_t s);
size_t rmsnorm_bwd_workspace(int T, int d);
hipError_t launch_rmsnorm_bwd(const twell_mat_t *dn, const twell_mat_t *h, const void *gain,
                              int dtg, float eps, const twell_mat_t *dres, const twell_mat_t *dh,
                              float *dgain, void *ws, twell_timing_t *timing, hipStream_t s);
hipError_t launch_fp8_quant(const twell_mat_t *x, const twell_fp8_t *o, const twell_fp8_t *ot,
                            twell_timing_t *timing, hipStream_t s);
size_t fp8_mm_workspace(int M, int N, int K);
int launch_fp8_mm(const twell_fp8_t *A, const twell_fp8_t *B, const twell_mat_t *out, int sums,
                  void *ws, size_t ws_bytes, twell_timing_t *timing, hipStream_t s);

hipError_t launch_fp4_quant(const twell_mat_t *x, const twell_fp4_t *o, twell_timing_t *timing,
                            hipStream_t s);
hipError_t launch_fp4_dequant(const twell_fp4_t *w, const twell_mat_t *out, twell_timing_t *timing,
                              hipStream_t s);
size_t fp4_mm_workspace(const twell_mat_t *x, int rows, int cols, bool dx);
int launch_fp4_mm(const twell_mat_t *x, const twell_fp4_t *w, const twell_mat_t *out, bool dx,
                  void *ws, size_t ws_bytes, twell_timing_t *timing, hipStream_t s);
size_t fp4_layer_workspace(const twell_mat_t *x, int d_ff);
hipError_t launch_fp4_layer(const twell_mat_t *x, const twell_fp4_t *wg, const twell_fp4_t *wu,
                            const twell_fp4_t *wd, float *y, void *ws, twell_timing_t *timing,
                            hipStream_t s);

namespace {

bool a16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

bool dtype_ok(int dt) { return dt == TWELL_BF16 || dt == TWELL_F32; }

int check_dm(twell_dtype dt, int32_t dm)
{
    const int max_dm = dt == TWELL_BF16 ? 4096 : 2048;
    return (dm >= 64 && dm <= max_dm && dm % 64 == 0) ? TWELL_OK : TWELL_E_SHAPE;
}

int check_dff(int32_t dff)
{
    return (dff >= TWELL_TILE_C && dff <= 32768 && dff % TWELL_TILE_C == 0) ? TWELL_OK
                                                                              : TWELL_E_SHAPE;
}

// dtype, token count, d_model and d_ff within the documented limits
bool sizes_ok(int dt, int32_t T, int32_t dm, int32_t dff)
{
    return dtype_ok(dt) && T >= 0 && T <= TWELL_MAX_ROWS && !check_dm((twell_dtype)dt, dm) &&
           !check_dff(dff);
}

// a hybrid's K and backup capacity for T rows of d_ff columns; ELL slots are
// numbered t * K + s in 32-bit integers (the backward's transpose)
bool hybrid_sizes_ok(int32_t T, int32_t dff, int32_t K, int32_t max_ovf)
{
    return K >= 1 && K <= dff && K <= 32767 && max_ovf >= 0 && max_ovf <= TWELL_MAX_ROWS &&
           (int64_t)T * K <= INT32_MAX;
}

int check_twell(const twell_t *h, twell_dtype dt)
{
    if (!h)
        return TWELL_E_NULL;
    if (!dtype_ok(h->dtype) || h->dtype != dt)
        return TWELL_E_DTYPE;
    if (h->T < 0 || h->T > TWELL_MAX_ROWS || h->width < 1 || h->width > TWELL_TILE_C)
        return TWELL_E_SHAPE;
    if (int rc = check_dff(h->d_ff))
        return rc;
    if (h->T > 0 && (!h->count || !h->col || !h->val))
        return TWELL_E_NULL;
    return TWELL_OK;
}

int check_hybrid(const hybrid_t *h, twell_dtype dt)
{
    if (!h)
        return TWELL_E_NULL;
    if (!dtype_ok(h->dtype) || h->dtype != dt)
        return TWELL_E_DTYPE;
    if (h->T < 0 || h->T > TWELL_MAX_ROWS || !hybrid_sizes_ok(h->T, h->d_ff, h->K, h->max_ovf))
        return TWELL_E_SHAPE;
    if (int rc = check_dff(h->d_ff))
        return rc;
    if (!h->n_ovf)
        return TWELL_E_NULL;
    if (h->T > 0 && (!h->row_nnz || !h->row_slot || !h->ell_col || !h->ell_val))
        return TWELL_E_NULL;
    if (h->max_ovf > 0 && (!h->ovf_rows || !h->dense))
        return TWELL_E_NULL;
    return TWELL_OK;
}

int hip_rc(hipError_t e) { return e == hipSuccess ? TWELL_OK : TWELL_E_HIP; }

bool aligned(const void *p, uintptr_t n) { return (uintptr_t)p % n == 0; }
bool aligned_dt(const void *p, int dt) { return aligned(p, dt == TWELL_BF16 ? 2 : 4); }

// a matrix of rows x cols
int check_mat(const twell_mat_t *m, int32_t rows, int32_t cols)
{
    if (!dtype_ok(m->dtype))
        return TWELL_E_DTYPE;
    if (m->rows != rows || m->cols != cols || (rows > 1 && m->ld < cols) || m->ld < 0 ||
        m->ld > ((int64_t)1 << 31))
        return TWELL_E_SHAPE;
    if (rows > 0 && cols > 0 && !m->data)
        return TWELL_E_NULL;
    return aligned_dt(m->data, m->dtype) ? TWELL_OK : TWELL_E_ALIGN;
}

int check_fp8(const twell_fp8_t *m)
{
    if (m->rows < 0 || m->rows > TWELL_MAX_ROWS || m->cols < 0 || m->cols > TWELL_MAX_ROWS ||
        (m->block_rows != 1 && m->block_rows != TWELL_FP8_BLOCK))
        return TWELL_E_SHAPE;
    if (m->rows > 0 && m->cols > 0 && (!m->q || !m->scale))
        return TWELL_E_NULL;
    return a16(m->q) && aligned(m->scale, 4) ? TWELL_OK : TWELL_E_ALIGN;
}

int check_fp4(const twell_fp4_t *m)
{
    if (m->rows < 0 || m->rows > TWELL_MAX_ROWS || m->cols < 0 || m->cols > TWELL_MAX_ROWS ||
        (m->group != 32 && m->group != 64 && m->group != 128))
        return TWELL_E_SHAPE;
    if (m->rows > 0 && m->cols > 0 && (!m->q || !m->scale))
        return TWELL_E_NULL;
    return a16(m->q) && aligned(m->scale, 2) ? TWELL_OK : TWELL_E_ALIGN;
}

bool eps_ok(float eps) { return eps >= 0.f && eps <= 3.4e38f; }

// rows and columns of the norm
bool norm_sizes_ok(int32_t rows, int32_t cols)
{
    return rows >= 0 && rows <= TWELL_MAX_ROWS && cols >= 1 && cols <= TWELL_NORM_COLS;
}

// 128 x 128 (or finer) tiles of a launch are numbered in 31 bits
bool tiles_ok(int64_t rows, int64_t cols, int64_t tr, int64_t tc)
{
    return ((rows + tr - 1) / tr) * ((cols + tc - 1) / tc) <= INT32_MAX;
}

// sizes of a 4-bit product (dx: of its gradient): T tokens, w [N][K]
bool fp4_sizes_ok(int32_t T, int32_t N, int32_t K, bool dx)
{
    return T >= 0 && T <= TWELL_MAX_ROWS && N >= 0 && N <= TWELL_MAX_ROWS && K >= 0 &&
           K <= TWELL_MAX_ROWS && (dx ? N : K) <= TWELL_FP4_MAX_K &&
           ((int64_t)T + 15) / 16 * (((int64_t)(dx ? K : N) + 127) / 128) <= 1 << 23;
}

// a matrix whose rows take the most workspace that any strides make them take
twell_mat_t worst_mat(twell_dtype dt, int32_t rows, int32_t cols)
{
    return {rows, cols, cols, dt, (void *)(uintptr_t)2};
}

int fp4_mm(const twell_mat_t *x, const twell_fp4_t *w, const twell_mat_t *out, bool dx,
           void *workspace, size_t workspace_bytes, twell_timing_t *timing, void *stream)
{
    if (!x || !w || !out)
        return TWELL_E_NULL;
    if (int rc = check_fp4(w))
        return rc;
    if (!fp4_sizes_ok(x->rows, w->rows, w->cols, dx))
        return TWELL_E_SHAPE;
    if (int rc = check_mat(x, x->rows, dx ? w->rows : w->cols))
        return rc;
    if (int rc = check_mat(out, x->rows, dx ? w->cols : w->rows))
        return rc;
    if (!a16(workspace))
        return TWELL_E_ALIGN;
    if (out->rows == 0 || out->cols == 0)
        return TWELL_OK;
    return launch_fp4_mm(x, w, out, dx, workspace, workspace_bytes, timing, (hipStream_t)stream);
}

} // namespace

// Every argument check of twell_decode_fwd except the workspace's (shared
// with twell_decode_fwd_noalloc, whose scratch is the library's own).
int check_decode_args(twell_dtype dt, const void *x, const void *wg_t, const void *wu_t,
                      const void *wd, int32_t d_model, const twell_t *out, const float *y)
{
    if (!dtype_ok(dt))
        return TWELL_E_DTYPE;
    if (!wg_t || !wu_t || !wd || !out)
        return TWELL_E_NULL;
    if (int rc = check_twell(out, dt))
        return rc;
    if (out->T > 0 && (!x || !y))
        return TWELL_E_NULL;
    if (int rc = check_dm(dt, d_model))
        return rc;
    if (out->T > TWELL_DECODE_T)
        return TWELL_E_SHAPE;
    if (!a16(x) || !a16(wg_t) || !a16(wu_t) || !a16(wd) || !a16(y))
        return TWELL_E_ALIGN;
    return TWELL_OK;
}

extern "C" {

const char *twell_status_str(int code)
{
    switch (code) {
    case TWELL_OK: return "ok";
    case TWELL_E_NULL: return "a required pointer is NULL";
    case TWELL_E_SHAPE: return "a size is out of range or inconsistent";
    case TWELL_E_DTYPE: return "unsupported or mismatched element type";
    case TWELL_E_ALIGN: return "a pointer is not 16-byte aligned";
    case TWELL_E_WORKSPACE: return "workspace too small";
    case TWELL_E_HIP: return "HIP launch failed";
    case TWELL_E_SCRATCH: return "the call needs more scratch than the static buffer holds";
    default: return "unknown status";
    }
}

size_t twell_gate_workspace_bytes(twell_dtype dt, int32_t T, int32_t d_model, int32_t d_ff)
{
    if (!sizes_ok(dt, T, d_model, d_ff))
        return 0;
    return T <= TWELL_DECODE_T ? dec_gate_workspace(dt, T, d_model, d_ff) : 0;
}

int twell_gate_pack(twell_dtype dt, const void *x, const void *wg_t, int32_t T, int32_t d_model,
                    const twell_t *out, void *workspace, size_t workspace_bytes,
                    int32_t *dev_status, twell_timing_t *timing, void *stream)
{
    if (!dtype_ok(dt))
        return TWELL_E_DTYPE;
    if ((!x && T != 0) || !wg_t || !out)
        return TWELL_E_NULL;
    if (int rc = check_twell(out, dt))
        return rc;
    if (int rc = check_dm(dt, d_model))
        return rc;
    if (T < 0 || T > TWELL_MAX_ROWS || out->T != T)
        return TWELL_E_SHAPE;
    if (!a16(x) || !a16(wg_t))
        return TWELL_E_ALIGN;
    const size_t need = twell_gate_workspace_bytes(dt, T, d_model, out->d_ff);
    if (workspace_bytes < need || (need && !workspace))
        return TWELL_E_WORKSPACE;
    if (!a16(workspace))
        return TWELL_E_ALIGN;
    if (T == 0)
        return TWELL_OK;
    return hip_rc(launch_gate_pack(dt, x, wg_t, T, d_model, out, workspace, dev_status, timing,
                                   (hipStream_t)stream));
}

size_t twell_fwd_workspace_bytes(twell_dtype dt, int32_t T, int32_t d_model, int32_t d_ff,
                                 int32_t width)
{
    if (!sizes_ok(dt, T, d_model, d_ff) || width < 1 || width > TWELL_TILE_C)
        return 0;
    return fwd_workspace(dt, T, d_model, d_ff, width);
}

int twell_ffn_fwd(twell_dtype dt, const void *x, const twell_t *h, const void *wu_t,
                  const void *wd, int32_t d_model, float *y, void *workspace,
                  size_t workspace_bytes, int32_t *dev_status, twell_timing_t *timing,
                  void *stream)
{
    if (!dtype_ok(dt))
        return TWELL_E_DTYPE;
    if (!h || !wu_t || !wd)
        return TWELL_E_NULL;
    if (int rc = check_twell(h, dt))
        return rc;
    if (h->T > 0 && (!x || !y))
        return TWELL_E_NULL;
    if (int rc = check_dm(dt, d_model))
        return rc;
    if (!a16(x) || !a16(wu_t) || !a16(wd) || !a16(y))
        return TWELL_E_ALIGN;
    const size_t need = twell_fwd_workspace_bytes(dt, h->T, d_model, h->d_ff, h->width);
    if (workspace_bytes < need || (need && !workspace))
        return TWELL_E_WORKSPACE;
    if (!a16(workspace))
        return TWELL_E_ALIGN;
    if (h->T == 0)
        return TWELL_OK;
    return hip_rc(launch_ffn_fwd(dt, x, h, wu_t, wd, d_model, y, workspace, dev_status, timing,
                                 (hipStream_t)stream));
}

size_t twell_decode_workspace_bytes(twell_dtype dt, int32_t T, int32_t d_model, int32_t d_ff,
                                    int32_t width)
{
    if (!sizes_ok(dt, T, d_model, d_ff) || T > TWELL_DECODE_T || width < 1 ||
        width > TWELL_TILE_C)
        return 0;
    return dec_layer_workspace(dt, T, d_model, d_ff, width);
}

int twell_decode_fwd(twell_dtype dt, const void *x, const void *wg_t, const void *wu_t,
                     const void *wd, int32_t d_model, const twell_t *out, float *y,
                     void *workspace, size_t workspace_bytes, int32_t *dev_status,
                     twell_timing_t *timing, void *stream)
{
    if (int rc = check_decode_args(dt, x, wg_t, wu_t, wd, d_model, out, y))
        return rc;
    const size_t need =
        twell_decode_workspace_bytes(dt, out->T, d_model, out->d_ff, out->width);
    if (workspace_bytes < need || (need && !workspace))
        return TWELL_E_WORKSPACE;
    if (!a16(workspace))
        return TWELL_E_ALIGN;
    if (out->T == 0)
        return TWELL_OK;
    return hip_rc(launch_dec_layer(dt, x, wg_t, wu_t, wd, d_model, out, y, workspace,
                                   dev_status, timing, (hipStream_t)stream));
}

int twell_to_hybrid(const twell_t *h, const hybrid_t *out, int32_t *dev_status,
                    twell_timing_t *timing, void *stream)
{
    if (!h || !out)
        return TWELL_E_NULL;
    if (!dtype_ok(h->dtype))
        return TWELL_E_DTYPE;
    if (int rc = check_twell(h, h->dtype))
        return rc;
    if (int rc = check_hybrid(out, h->dtype))
        return rc;
    if (out->T != h->T || out->d_ff != h->d_ff)
        return TWELL_E_SHAPE;
    return hip_rc(launch_to_hybrid(h, out, dev_status, timing, (hipStream_t)stream));
}

size_t hybrid_fwd_workspace_bytes(twell_dtype dt, int32_t T, int32_t d_model, int32_t d_ff,
                                  int32_t K, int32_t max_ovf)
{
    if (!sizes_ok(dt, T, d_model, d_ff) || !hybrid_sizes_ok(T, d_ff, K, max_ovf))
        return 0;
    return hyb_fwd_workspace(dt, T, d_model, max_ovf, d_ff, K);
}

int hybrid_ffn_fwd(twell_dtype dt, const void *x, const hybrid_t *h, const void *wu_t,
                   const void *wd, int32_t d_model, float *y, void *workspace,
                   size_t workspace_bytes, int32_t *dev_status, twell_timing_t *timing,
                   void *stream)
{
    if (!dtype_ok(dt))
        return TWELL_E_DTYPE;
    if (!h || !wu_t || !wd)
        return TWELL_E_NULL;
    if (int rc = check_hybrid(h, dt))
        return rc;
    if (h->T > 0 && (!x || !y))
        return TWELL_E_NULL;
    if (int rc = check_dm(dt, d_model))
        return rc;
    if (!a16(x) || !a16(wu_t) || !a16(wd) || !a16(y) || !a16(workspace))
        return TWELL_E_ALIGN;
    const size_t need = hybrid_fwd_workspace_bytes(dt, h->T, d_model, h->d_ff, h->K, h->max_ovf);
    if (workspace_bytes < need || (need && !workspace))
        return TWELL_E_WORKSPACE;
    if (h->T == 0)
        return TWELL_OK;
    return hip_rc(launch_hyb_fwd(dt, x, h, wu_t, wd, d_model, y, workspace, dev_status, timing,
                                 (hipStream_t)stream));
}

size_t hybrid_bwd_workspace_bytes(twell_dtype dt, int32_t T, int32_t d_model, int32_t d_ff,
                                  int32_t K, int32_t max_ovf)
{
    if (!sizes_ok(dt, T, d_model, d_ff) || !hybrid_sizes_ok(T, d_ff, K, max_ovf))
        return 0;
    return bwd_workspace_layout(dt, T, d_model, d_ff, K, max_ovf);
}

int hybrid_ffn_bwd(twell_dtype dt, const void *x, const void *dy, const hybrid_t *h,
                   const void *wg_t, const void *wu_t, const void *wd, int32_t d_model,
                   float l1, float *dx, float *dwg_t, float *dwu_t, float *dwd, void *workspace,
                   size_t workspace_bytes, int32_t *dev_status, twell_timing_t *timing,
                   void *stream)
{
    if (!dtype_ok(dt))
        return TWELL_E_DTYPE;
    if (!h || !wg_t || !wu_t || !wd || !dwg_t || !dwu_t || !dwd)
        return TWELL_E_NULL;
    if (int rc = check_hybrid(h, dt))
        return rc;
    if (h->T > 0 && (!x || !dy || !dx))
        return TWELL_E_NULL;
    if (int rc = check_dm(dt, d_model))
        return rc;
    if (!a16(x) || !a16(dy) || !a16(wg_t) || !a16(wu_t) || !a16(wd) || !a16(dx) || !a16(dwg_t) ||
        !a16(dwu_t) || !a16(dwd) || !a16(workspace))
        return TWELL_E_ALIGN;
    const size_t need = hybrid_bwd_workspace_bytes(dt, h->T, d_model, h->d_ff, h->K, h->max_ovf);
    if (workspace_bytes < need || (need && !workspace))
        return TWELL_E_WORKSPACE;
    if (!(l1 == l1) || l1 > 3.4e38f || l1 < -3.4e38f) // NaN or infinite
        return TWELL_E_SHAPE;
    return hip_rc(launch_bwd(dt, x, dy, h, wg_t, wu_t, wd, d_model, l1, dx, dwg_t, dwu_t, dwd,
                             workspace, dev_status, timing, (hipStream_t)stream));
}

int twell_rmsnorm_fwd(const twell_mat_t *x, const twell_mat_t *residual, const void *gain,
                      twell_dtype gain_dtype, float eps, const twell_mat_t *h,
                      const twell_mat_t *n, const twell_fp8_t *n8, twell_timing_t *timing,
                      void *stream)
{
    if (!x || !gain || (residual && !h) || (!n && !n8))
        return TWELL_E_NULL;
    if (!dtype_ok(gain_dtype))
        return TWELL_E_DTYPE;
    if (!norm_sizes_ok(x->rows, x->cols) || (h && !residual) || (n && n8) || !eps_ok(eps))
        return TWELL_E_SHAPE;
    const int32_t T = x->rows, d = x->cols;
    for (const twell_mat_t *m : {x, residual, h, n})
        if (m)
            if (int rc = check_mat(m, T, d))
                return rc;
    if (residual && h->dtype != residual->dtype)
        return TWELL_E_DTYPE;
    if (n8) {
        if (n8->rows != T || n8->cols != d || n8->block_rows != 1)
            return TWELL_E_SHAPE;
        if (int rc = check_fp8(n8))
            return rc;
    }
    if (!aligned_dt(gain, gain_dtype))
        return TWELL_E_ALIGN;
    if (T == 0)
        return TWELL_OK;
    return hip_rc(launch_rmsnorm_fwd(x, residual, gain, gain_dtype, eps, h, n, n8, timing,
                                     (hipStream_t)stream));
}

size_t twell_rmsnorm_bwd_workspace_bytes(int32_t rows, int32_t cols)
{
    return norm_sizes_ok(rows, cols) ? rmsnorm_bwd_workspace(rows, cols) : 0;
}

int twell_rmsnorm_bwd(const twell_mat_t *dn, const twell_mat_t *h, const void *gain,
                      twell_dtype gain_dtype, float eps, const twell_mat_t *dres,
                      const twell_mat_t *dh, float *dgain, void *workspace,
                      size_t workspace_bytes, twell_timing_t *timing, void *stream)
{
    if (!dn || !h || !gain || !dh || !dgain)
        return TWELL_E_NULL;
    if (!dtype_ok(gain_dtype))
        return TWELL_E_DTYPE;
    if (!norm_sizes_ok(dn->rows, dn->cols) || !eps_ok(eps))
        return TWELL_E_SHAPE;
    const int32_t T = dn->rows, d = dn->cols;
    for (const twell_mat_t *m : {dn, h, dres, dh})
        if (m)
            if (int rc = check_mat(m, T, d))
                return rc;
    if (!aligned_dt(gain, gain_dtype) || !aligned(dgain, 4) || !a16(workspace))
        return TWELL_E_ALIGN;
    const size_t need = twell_rmsnorm_bwd_workspace_bytes(T, d);
    if (workspace_bytes < need || (need && !workspace))
        return TWELL_E_WORKSPACE;
    return hip_rc(launch_rmsnorm_bwd(dn, h, gain, gain_dtype, eps, dres, dh, dgain, workspace,
                                     timing, (hipStream_t)stream));
}

int twell_fp8_quant(const twell_mat_t *x, const twell_fp8_t *out, const twell_fp8_t *out_t,
                    twell_timing_t *timing, void *stream)
{
    if (!x || (!out && !out_t))
        return TWELL_E_NULL;
    if (x->rows < 0 || x->rows > TWELL_MAX_ROWS || x->cols < 0 || x->cols > TWELL_MAX_ROWS)
        return TWELL_E_SHAPE;
    const int32_t R = x->rows, C = x->cols;
    if (int rc = check_mat(x, R, C))
        return rc;
    if ((out && (out->rows != R || out->cols != C)) ||
        (out_t && (out_t->rows != C || out_t->cols != R)) ||
        (out && out_t && out->block_rows != out_t->block_rows) ||
        !tiles_ok(R, C, TWELL_FP8_BLOCK, TWELL_FP8_BLOCK))
        return TWELL_E_SHAPE;
    for (const twell_fp8_t *m : {out, out_t})
        if (m)
            if (int rc = check_fp8(m))
                return rc;
    if (R == 0 || C == 0)
        return TWELL_OK;
    return hip_rc(launch_fp8_quant(x, out, out_t, timing, (hipStream_t)stream));
}

size_t twell_fp8_matmul_workspace_bytes(int32_t M, int32_t N, int32_t K)
{
    if (M < 0 || M > TWELL_MAX_ROWS || N < 0 || N > TWELL_MAX_ROWS || K < 0 || K > TWELL_MAX_K ||
        !tiles_ok(M, N, 16, 16))
        return 0;
    return fp8_mm_workspace(M, N, K);
}

int twell_fp8_matmul(const twell_fp8_t *a, const twell_fp8_t *b, const twell_mat_t *out,
                     int32_t sums, void *workspace, size_t workspace_bytes, twell_timing_t *timing,
                     void *stream)
{
    if (!a || !b || !out)
        return TWELL_E_NULL;
    for (const twell_fp8_t *m : {a, b})
        if (int rc = check_fp8(m))
            return rc;
    if (a->cols != b->cols || a->cols > TWELL_MAX_K || !tiles_ok(a->rows, b->rows, 16, 16) ||
        (sums != TWELL_SUMS_F32 && sums != TWELL_SUMS_FP8))
        return TWELL_E_SHAPE;
    if (int rc = check_mat(out, a->rows, b->rows))
        return rc;
    if (!a16(workspace))
        return TWELL_E_ALIGN;
    if (a->rows == 0 || b->rows == 0)
        return TWELL_OK;
    return launch_fp8_mm(a, b, out, sums, workspace, workspace_bytes, timing, (hipStream_t)stream);
}

int twell_fp4_quant(const twell_mat_t *x, const twell_fp4_t *out, twell_timing_t *timing,
                    void *stream)
{
    if (!x || !out)
        return TWELL_E_NULL;
    if (int rc = check_fp4(out))
        return rc;
    if (int rc = check_mat(x, out->rows, out->cols))
        return rc;
    if (x->rows == 0 || x->cols == 0)
        return TWELL_OK;
    return hip_rc(launch_fp4_quant(x, out, timing, (hipStream_t)stream));
}

int twell_fp4_dequant(const twell_fp4_t *w, const twell_mat_t *out, twell_timing_t *timing,
                      void *stream)
{
    if (!w || !out)
        return TWELL_E_NULL;
    if (int rc = check_fp4(w))
        return rc;
    if (int rc = check_mat(out, w->rows, w->cols))
        return rc;
    if (w->rows == 0 || w->cols == 0)
        return TWELL_OK;
    return hip_rc(launch_fp4_dequant(w, out, timing, (hipStream_t)stream));
}

size_t twell_fp4_matmul_workspace_bytes(twell_dtype x_dtype, int32_t T, int32_t N, int32_t K)
{
    if (!dtype_ok(x_dtype) || !fp4_sizes_ok(T, N, K, false) || T == 0 || N == 0)
        return 0;
    const twell_mat_t x = worst_mat(x_dtype, T, K);
    return fp4_mm_workspace(&x, N, K, false);
}

int twell_fp4_matmul(const twell_mat_t *x, const twell_fp4_t *w, const twell_mat_t *out,
                     void *workspace, size_t workspace_bytes, twell_timing_t *timing,
                     void *stream)
{
    return fp4_mm(x, w, out, false, workspace, workspace_bytes, timing, stream);
}

size_t twell_fp4_matmul_dx_workspace_bytes(twell_dtype dy_dtype, int32_t T, int32_t N, int32_t K)
{
    if (!dtype_ok(dy_dtype) || !fp4_sizes_ok(T, N, K, true) || T == 0 || K == 0)
        return 0;
    const twell_mat_t dy = worst_mat(dy_dtype, T, N);
    return fp4_mm_workspace(&dy, N, K, true);
}

int twell_fp4_matmul_dx(const twell_mat_t *dy, const twell_fp4_t *w, const twell_mat_t *dx,
                        void *workspace, size_t workspace_bytes, twell_timing_t *timing,
                        void *stream)
{
    return fp4_mm(dy, w, dx, true, workspace, workspace_bytes, timing, stream);
}

size_t twell_fp4_decode_workspace_bytes(twell_dtype x_dtype, int32_t T, int32_t d_model,
                                        int32_t d_ff)
{
    if (!dtype_ok(x_dtype) || T < 0 || T > TWELL_DECODE_T || check_dm(TWELL_BF16, d_model) ||
        check_dff(d_ff))
        return 0;
    const twell_mat_t x = worst_mat(x_dtype, T, d_model);
    return fp4_layer_workspace(&x, d_ff);
}

int twell_fp4_decode_fwd(const twell_mat_t *x, const twell_fp4_t *wg_t, const twell_fp4_t *wu_t,
                         const twell_fp4_t *wd, float *y, void *workspace, size_t workspace_bytes,
                         twell_timing_t *timing, void *stream)
{
    if (!x || !wg_t || !wu_t || !wd || (x->rows > 0 && !y))
        return TWELL_E_NULL;
    if (x->rows < 0 || x->rows > TWELL_DECODE_T)
        return TWELL_E_SHAPE;
    if (int rc = check_dm(TWELL_BF16, x->cols))
        return rc;
    if (int rc = check_dff(wg_t->rows))
        return rc;
    for (const twell_fp4_t *m : {wg_t, wu_t, wd}) {
        if (int rc = check_fp4(m))
            return rc;
        if (m->rows != wg_t->rows || m->cols != x->cols || m->group != wg_t->group)
            return TWELL_E_SHAPE;
    }
    if (int rc = check_mat(x, x->rows, x->cols))
        return rc;
    if (!a16(y) || !a16(workspace))
        return TWELL_E_ALIGN;
    if (x->rows == 0)
        return TWELL_OK;
    const size_t need = fp4_layer_workspace(x, wg_t->rows);
    if (workspace_bytes < need || !workspace)
        return TWELL_E_WORKSPACE;
    return hip_rc(launch_fp4_layer(x, wg_t, wu_t, wd, y, workspace, timing, (hipStream_t)stream));
}

} // extern "C"
