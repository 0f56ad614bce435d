// C ABI of the NVFP4 GPTQ / Schur Replay quantizer: argument validation,
// workspace carving and kernel sequencing.  See include/nvq.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <string>
#include <thread>
#include <vector>

#include "../../include/nvq.h"
#include "common.h"
#include "kernels.h"

using namespace nvq;

namespace {

thread_local std::string g_last_error;

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return code;
}

int hip_status(hipError_t e, const char* where) {
  if (e == hipSuccess) return NVQ_OK;
  return fail(NVQ_ERR_HIP, "%s: %s", where, hipGetErrorString(e));
}

constexpr size_t kAlign = 256;
size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

struct QuantWs {
  size_t wp, w0, eslab, invd, mb, part, total;
};

// chol: the Cholesky-factor form also keeps the input weights in the working
// precision (w0) and the diagonal blocks' M - I (mb, k * 16 floats).
QuantWs quant_ws(int64_t m, int64_t k, bool f64, bool chol = false) {
  QuantWs w;
  const size_t es = f64 ? sizeof(double) : sizeof(float);
  size_t off = 0;
  w.wp = off;   off += align_up((size_t)m * k * es);
  w.w0 = off;   if (chol) off += align_up((size_t)m * k * es);
  w.eslab = off; off += align_up((size_t)m * kSuperBatch * es);
  w.invd = off;  off += align_up((size_t)k * sizeof(float));
  w.mb = off;    if (chol) off += align_up((size_t)k * kBlock * sizeof(float));
  w.part = off;  off += align_up((size_t)m * ((k + kGemmTile - 1) / kGemmTile) * sizeof(float));
  w.total = off;
  return w;
}

bool dtype_ok(int d) { return d == NVQ_DTYPE_F32 || d == NVQ_DTYPE_BF16; }

hipError_t hessian_run(const void* X, int x_dtype, int64_t n, int64_t k, int64_t ldx, float* H, void* ws,
                       hipStream_t s) {
  if (x_dtype == NVQ_DTYPE_BF16) return syrk_bf16((const uint16_t*)X, n, k, ldx, H, ws, s);
  hipError_t e = symmetrize_from_upper(H, k, s);
  if (e == hipSuccess) {
    GemmArgs a{};
    a.A = (const float*)X; a.lda = ldx;   // stored [n x k] = op(A)^T
    a.B = (const float*)X; a.ldb = ldx;
    a.C = H; a.ldc = k;
    a.M = k; a.N = k; a.K = n; a.batch = 1; a.alpha = 1.0f; a.beta = 1.0f;
    e = gemm_f32(a, true, false, false, kEpiAxpby, s);
  }
  if (e == hipSuccess) e = symmetrize_from_upper(H, k, s);
  return e;
}

// fail() with the entry point's name in front of the message.
int failp(int code, const char* fn, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = std::string(fn) + ": " + buf;
  return code;
}

int quant_check(const char* fn, const void* W, int w_dtype, int64_t m, int64_t k, int64_t ldw, const float* U,
                const float* H, const float* g, int n_cand, unsigned flags, const uint8_t* codes,
                const uint8_t* scales, const float* row_err, const void* ws, size_t ws_bytes) {
  const bool rtn = flags & NVQ_FLAG_RTN;
  const bool want_err = !(flags & NVQ_FLAG_NO_ERR);
  if (flags & ~(NVQ_FLAG_RTN | NVQ_FLAG_NO_ERR | NVQ_FLAG_FP64 | NVQ_FLAG_INDEP | NVQ_FLAG_CHECK_FINITE |
                NVQ_FLAG_CHOL_FACTOR))
    return failp(NVQ_ERR_VALUE, fn, "unknown flags 0x%x", flags);
  if (!W || !g || !codes || !scales) return failp(NVQ_ERR_NULL, fn, "W, g, codes and scales are required");
  if (!rtn && !U) return failp(NVQ_ERR_NULL, fn, "U is required without NVQ_FLAG_RTN");
  if (want_err && (!H || !row_err)) return failp(NVQ_ERR_NULL, fn, "H and row_err are required unless NVQ_FLAG_NO_ERR");
  if (!dtype_ok(w_dtype)) return failp(NVQ_ERR_DTYPE, fn, "w_dtype %d", w_dtype);
  if (m <= 0 || k <= 0 || k % 16 != 0 || ldw < k || ldw % 4 != 0)
    return failp(NVQ_ERR_SHAPE, fn, "m=%lld k=%lld ldw=%lld (need m>0, k>0, k%%16==0, ldw>=k, ldw%%4==0)",
                 (long long)m, (long long)k, (long long)ldw);
  if (n_cand < 1 || n_cand > 16) return failp(NVQ_ERR_NCAND, fn, "n_cand=%d", n_cand);
  if (!aligned(codes, 8)) return failp(NVQ_ERR_ALIGN, fn, "codes must be 8-byte aligned");
  if ((U && !aligned(U, 16)) || (H && !aligned(H, 16))) return failp(NVQ_ERR_ALIGN, fn, "U and H must be 16-byte aligned");
  QuantWs L = quant_ws(m, k, (flags & NVQ_FLAG_FP64) && !rtn, (flags & NVQ_FLAG_CHOL_FACTOR) && !rtn);
  if (!ws || ws_bytes < L.total || !aligned(ws, kAlign))
    return failp(NVQ_ERR_WORKSPACE, fn, "workspace needs %zu bytes (256-aligned), got %zu", L.total, ws_bytes);
  return NVQ_OK;
}

// A batch of nb equal-shape matrices for the quantizer: matrix e reads W + e
// * stride_w (elements of its dtype), U + e * stride_u, H + e * stride_h,
// g[e], writes codes + e*m*k/2, scales + e*m*k/16, row_err + e*m,
// row_loss + e*m, and uses its own workspace block at base + e * ws_stride
// bytes (the QuantWs layout).  Every launch covers all nb matrices.
struct QBatch {
  int64_t nb = 1, stride_w = 0, stride_u = 0, stride_h = 0;
  size_t ws_stride = 0;
};

// Weighted error dW H' dW^T, H' = 2 triu(H, 1) + diag(H), into the
// per-column-tile partial sums, then summed per row.
hipError_t weighted_error_all(const void* W, int bf, int64_t m, int64_t k, int64_t ldw, const float* H,
                              const float* g, const uint8_t* codes, const uint8_t* scales, float* row_err, float* dW,
                              float* part, const QBatch& qb, hipStream_t s) {
  const int64_t wsf = (int64_t)(qb.ws_stride / sizeof(float));
  const int64_t np = (k + kGemmTile - 1) / kGemmTile;
  hipError_t e = delta_w_launch(W, bf, m, k, ldw, codes, scales, g, dW, s, 0, -1, qb.nb, qb.stride_w, wsf);
  if (e == hipSuccess) {
    GemmArgs a{};
    a.A = dW; a.lda = k;
    a.B = H; a.ldb = k;
    a.D = dW; a.ldd = k;
    a.P = part; a.ldp = np;
    a.M = m; a.N = k; a.K = k; a.batch = (int)qb.nb; a.bi = 1; a.alpha = 1.0f; a.beta = 0.0f;
    a.sA2 = wsf; a.sB2 = qb.stride_h; a.sD2 = wsf; a.sP2 = wsf;
    a.kmode = kGemmKSymUpperB; a.noff = 0;
    e = gemm_f32(a, false, false, false, kEpiRowDot, s);
  }
  if (e == hipSuccess) e = row_sum_launch(part, m, np, row_err, s, qb.nb, wsf);
  return e;
}

// The fp32 sweep with two-level lazy updates (the same sums as eager GPTQ
// updates, in another order): a batch's errors update the rest of its
// 512-column block at once, and a finished block's error slab updates every
// later column.
hipError_t sweep_f32(int64_t m, int64_t k, const float* U, const float* g, int n_cand, bool indep, uint8_t* codes,
                     uint8_t* scales, float* row_loss, float* Wp, float* Eslab, const float* invd, const QBatch& qb,
                     hipStream_t s, const float* W0, const float* Mb) {
  const int64_t wsf = (int64_t)(qb.ws_stride / sizeof(float));
  SweepStrides bs;
  bs.wp = wsf; bs.u = qb.stride_u; bs.invd = wsf; bs.e = wsf; bs.mb = wsf;
  auto rank_update = [&](const float* Eb, int64_t r0, int64_t c0, int64_t kk, int64_t ncol) {
    GemmArgs a{};
    a.A = Eb; a.lda = kSuperBatch;
    a.B = U + r0 * k + c0; a.ldb = k;
    a.C = Wp + c0; a.ldc = k;
    a.M = m; a.N = ncol; a.K = kk; a.batch = (int)qb.nb; a.bi = 1; a.alpha = -1.0f; a.beta = 1.0f;
    a.sA2 = wsf; a.sB2 = qb.stride_u; a.sC2 = wsf;
    return gemm_f32(a, false, false, false, kEpiAxpby, s);
  };
  // With larger candidate groups the sweep launch itself applies the earlier
  // batches' errors of the block to its rows (pre columns); else a GEMM after
  // each batch updates the rest of the block.
  const bool inblock = sweep_applies_inblock(n_cand);
  hipError_t e = hipSuccess;
  for (int64_t s0 = 0; e == hipSuccess && s0 < k; s0 += kSuperBatch) {
    const int64_t s1 = std::min<int64_t>(k, s0 + kSuperBatch);
    for (int64_t i1 = s0; e == hipSuccess && i1 < s1; i1 += kBatch) {
      const int ncols = (int)std::min<int64_t>(kBatch, s1 - i1);
      e = sweep_batch_launch(Wp, U, invd, g, m, k, (int)i1, ncols, n_cand, indep, codes, scales, Eslab + (i1 - s0),
                             kSuperBatch, row_loss, s, qb.nb, bs, inblock ? (int)(i1 - s0) : 0, W0, Mb);
      const int64_t i2 = i1 + ncols;
      if (e == hipSuccess && !inblock && i2 < s1) e = rank_update(Eslab + (i1 - s0), i1, i2, ncols, s1 - i2);
    }
    if (e == hipSuccess && s1 < k) e = rank_update(Eslab, s0, s1, s1 - s0, k - s1);
  }
  return e;
}

// The quantization of nb matrices (arguments already checked).
hipError_t quant_run(const void* W, int w_dtype, int64_t m, int64_t k, int64_t ldw, const float* U, const float* H,
                     const float* g, int n_cand, unsigned flags, uint8_t* codes, uint8_t* scales, float* row_err,
                     float* row_loss, char* base, hipStream_t s, QBatch qb = QBatch()) {
  const bool rtn = flags & NVQ_FLAG_RTN;
  const bool want_err = !(flags & NVQ_FLAG_NO_ERR);
  const bool f64 = (flags & NVQ_FLAG_FP64) && !rtn;
  const bool indep = flags & NVQ_FLAG_INDEP;
  const bool chol = (flags & NVQ_FLAG_CHOL_FACTOR) && !rtn;
  QuantWs L = quant_ws(m, k, f64, chol);
  if (qb.ws_stride == 0) qb.ws_stride = L.total;
  float* Wp = (float*)(base + L.wp);
  float* Eslab = (float*)(base + L.eslab);
  float* invd = (float*)(base + L.invd);
  float* Mb = chol ? (float*)(base + L.mb) : nullptr;
  float* part = (float*)(base + L.part);
  const int bf = w_dtype == NVQ_DTYPE_BF16;
  hipError_t e = hipSuccess;

  if (rtn) {
    e = rtn_launch(W, bf, m, k, ldw, g, n_cand, codes, scales, row_loss, s, qb.nb, qb.stride_w);
  } else if (f64) {
    // The same sweep and two-level lazy updates with fp64 working weights and errors.
    double* Wd = (double*)(base + L.wp);
    double* W0d = chol ? (double*)(base + L.w0) : nullptr;
    double* Ed = (double*)(base + L.eslab);
    const int64_t wsd = (int64_t)(qb.ws_stride / sizeof(double));
    SweepStrides bs;
    bs.wp = wsd; bs.u = qb.stride_u; bs.e = wsd; bs.mb = (int64_t)(qb.ws_stride / sizeof(float));
    e = load_working_copy_f64(W, bf, m, k, ldw, Wd, s, qb.nb, qb.stride_w, wsd);
    if (e == hipSuccess && chol) e = chol_block_m_launch(U, k, Mb, s, qb.nb, qb.stride_u, bs.mb);
    if (e == hipSuccess && chol) e = load_working_copy_f64(W, bf, m, k, ldw, W0d, s, qb.nb, qb.stride_w, wsd);
    if (e == hipSuccess && row_loss) e = fill_f32(row_loss, qb.nb * m, 0.0f, s);
    for (int64_t s0 = 0; e == hipSuccess && s0 < k; s0 += kSuperBatch) {
      const int64_t s1 = std::min<int64_t>(k, s0 + kSuperBatch);
      for (int64_t i1 = s0; e == hipSuccess && i1 < s1; i1 += kBatch) {
        const int ncols = (int)std::min<int64_t>(kBatch, s1 - i1);
        e = sweep_batch_launch_f64(Wd, U, g, m, k, (int)i1, ncols, n_cand, indep, codes, scales, Ed + (i1 - s0),
                                   kSuperBatch, row_loss, s, qb.nb, bs, W0d, Mb);
        const int64_t i2 = i1 + ncols;
        if (e == hipSuccess && i2 < s1)
          e = rank_update_f64(Ed + (i1 - s0), kSuperBatch, U + i1 * k + i2, k, Wd + i2, k, m, s1 - i2, ncols, s,
                              qb.nb, wsd, qb.stride_u, wsd);
      }
      if (e == hipSuccess && s1 < k)
        e = rank_update_f64(Ed, kSuperBatch, U + s0 * k + s1, k, Wd + s1, k, m, k - s1, s1 - s0, s, qb.nb, wsd,
                            qb.stride_u, wsd);
    }
  } else {
    const int64_t wsf = (int64_t)(qb.ws_stride / sizeof(float));
    float* W0 = chol ? (float*)(base + L.w0) : nullptr;
    e = inv_diag_launch(U, k, invd, s, qb.nb, qb.stride_u, wsf, chol);
    if (e == hipSuccess && chol) e = chol_block_m_launch(U, k, Mb, s, qb.nb, qb.stride_u, wsf);
    if (e == hipSuccess) e = load_working_copy(W, bf, m, k, ldw, Wp, s, qb.nb, qb.stride_w, wsf);
    if (e == hipSuccess && chol) e = load_working_copy(W, bf, m, k, ldw, W0, s, qb.nb, qb.stride_w, wsf);
    if (e == hipSuccess && row_loss) e = fill_f32(row_loss, qb.nb * m, 0.0f, s);
    if (e == hipSuccess)
      e = sweep_f32(m, k, U, g, n_cand, indep, codes, scales, row_loss, Wp, Eslab, invd, qb, s, W0, Mb);
  }
  if (e == hipSuccess && want_err)
    e = weighted_error_all(W, bf, m, k, ldw, H, g, codes, scales, row_err, Wp, part, qb, s);
  if (e == hipSuccess && (flags & NVQ_FLAG_CHECK_FINITE))
    e = reject_nonfinite_rows_launch(W, bf, m, k, ldw, g, codes, scales, want_err ? row_err : nullptr, row_loss, s,
                                     qb.nb, qb.stride_w);
  return e;
}

}  // namespace

extern "C" {

const char* nvq_status_string(int status) {
  switch (status) {
    case NVQ_OK: return "ok";
    case NVQ_ERR_NULL: return "null pointer";
    case NVQ_ERR_SHAPE: return "invalid shape";
    case NVQ_ERR_DTYPE: return "unsupported dtype";
    case NVQ_ERR_NCAND: return "candidate count outside [1, 16]";
    case NVQ_ERR_WORKSPACE: return "workspace too small or misaligned";
    case NVQ_ERR_VALUE: return "invalid scalar argument";
    case NVQ_ERR_HIP: return "HIP runtime error";
    case NVQ_ERR_ALIGN: return "misaligned pointer";
    default: return "unknown status";
  }
}

const char* nvq_last_error(void) { return g_last_error.c_str(); }

// ---------------------------------------------------------------------------
size_t hessian_workspace_size(int64_t n, int64_t k, int x_dtype) {
  if (n <= 0 || k <= 0) return 0;
  if (x_dtype == NVQ_DTYPE_BF16) return align_up(syrk_bf16_workspace(n, k));
  return 0;
}

int hessian_accumulate(const void* X, int x_dtype, int64_t n, int64_t k, int64_t ldx, float* H, void* ws,
                       size_t ws_bytes, void* stream) {
  if (!H) return fail(NVQ_ERR_NULL, "hessian_accumulate: H is NULL");
  if (!dtype_ok(x_dtype)) return fail(NVQ_ERR_DTYPE, "hessian_accumulate: x_dtype %d", x_dtype);
  if (n < 0 || k <= 0 || k % 16 != 0 || ldx < k || ldx % 4 != 0)
    return fail(NVQ_ERR_SHAPE, "hessian_accumulate: n=%lld k=%lld ldx=%lld (need n>=0, k>0, k%%16==0, ldx>=k, ldx%%4==0)",
                (long long)n, (long long)k, (long long)ldx);
  if (n == 0) return NVQ_OK;
  if (!X) return fail(NVQ_ERR_NULL, "hessian_accumulate: X is NULL");
  if (!aligned(H, 16)) return fail(NVQ_ERR_ALIGN, "hessian_accumulate: H must be 16-byte aligned");
  if (!aligned(X, 16)) return fail(NVQ_ERR_ALIGN, "hessian_accumulate: X must be 16-byte aligned");
  if (x_dtype == NVQ_DTYPE_BF16 && ldx % 8 != 0)
    return fail(NVQ_ERR_SHAPE, "hessian_accumulate: bf16 rows must be 16-byte aligned (ldx %% 8 == 0)");
  size_t need = hessian_workspace_size(n, k, x_dtype);
  if (need && (!ws || ws_bytes < need || !aligned(ws, kAlign)))
    return fail(NVQ_ERR_WORKSPACE, "hessian_accumulate: workspace needs %zu bytes (256-aligned), got %zu", need,
                ws_bytes);
  return hip_status(hessian_run(X, x_dtype, n, k, ldx, H, ws, (hipStream_t)stream), "hessian_accumulate");
}

// ---- Hessian over host-resident activations ---------------------------------
namespace {
size_t host_chunk_bytes(int64_t chunk, int64_t k, int x_dtype) {
  return align_up((size_t)chunk * k * (x_dtype == NVQ_DTYPE_BF16 ? 2 : 4));
}
// Rows [r0, r0 + rows) of a host matrix with row stride ld into a dense buffer.
void copy_rows_host(char* dst, const char* src, int64_t rows, int64_t row_bytes, int64_t ld_bytes) {
  auto part = [&](int64_t a, int64_t b) {
    if (ld_bytes == row_bytes) {
      std::memcpy(dst + a * row_bytes, src + a * ld_bytes, (size_t)((b - a) * row_bytes));
    } else {
      for (int64_t r = a; r < b; ++r) std::memcpy(dst + r * row_bytes, src + r * ld_bytes, (size_t)row_bytes);
    }
  };
  const int64_t bytes = rows * row_bytes;
  const int nt = bytes >= (64ll << 20) ? 8 : (bytes >= (8ll << 20) ? 4 : 1);
  if (nt == 1) { part(0, rows); return; }
  std::vector<std::thread> th;
  for (int t = 0; t < nt; ++t) th.emplace_back(part, rows * t / nt, rows * (t + 1) / nt);
  for (auto& x : th) x.join();
}
}  // namespace

size_t hessian_host_workspace_size(int64_t chunk, int64_t k, int x_dtype) {
  if (chunk <= 0 || k <= 0 || !dtype_ok(x_dtype)) return 0;
  return 2 * host_chunk_bytes(chunk, k, x_dtype) + hessian_workspace_size(chunk, k, x_dtype);
}
size_t hessian_host_staging_size(int64_t chunk, int64_t k, int x_dtype) {
  if (chunk <= 0 || k <= 0 || !dtype_ok(x_dtype)) return 0;
  return 2 * host_chunk_bytes(chunk, k, x_dtype);
}

int hessian_accumulate_host(const void* X_host, int x_dtype, int64_t n, int64_t k, int64_t ldx, float* H,
                            int64_t chunk, void* ws, size_t ws_bytes, void* staging, size_t staging_bytes,
                            void* stream, void* copy_stream) {
  const char* fn = "hessian_accumulate_host";
  if (!H) return failp(NVQ_ERR_NULL, fn, "H is NULL");
  if (!dtype_ok(x_dtype)) return failp(NVQ_ERR_DTYPE, fn, "x_dtype %d", x_dtype);
  if (n < 0 || k <= 0 || k % 16 != 0 || ldx < k)
    return failp(NVQ_ERR_SHAPE, fn, "n=%lld k=%lld ldx=%lld (need n>=0, k>0, k%%16==0, ldx>=k)", (long long)n,
                 (long long)k, (long long)ldx);
  if (chunk <= 0) return failp(NVQ_ERR_SHAPE, fn, "chunk=%lld (need > 0)", (long long)chunk);
  if (n == 0) return NVQ_OK;
  if (!X_host) return failp(NVQ_ERR_NULL, fn, "X_host is NULL");
  if (!aligned(H, 16)) return failp(NVQ_ERR_ALIGN, fn, "H must be 16-byte aligned");
  const size_t need = hessian_host_workspace_size(chunk, k, x_dtype);
  if (!ws || ws_bytes < need || !aligned(ws, kAlign))
    return failp(NVQ_ERR_WORKSPACE, fn, "workspace needs %zu bytes (256-aligned), got %zu", need, ws_bytes);
  const size_t sneed = hessian_host_staging_size(chunk, k, x_dtype);
  if (staging && staging_bytes < sneed)
    return failp(NVQ_ERR_WORKSPACE, fn, "staging needs %zu bytes, got %zu", sneed, staging_bytes);

  const int64_t es = x_dtype == NVQ_DTYPE_BF16 ? 2 : 4;
  const size_t cb = host_chunk_bytes(chunk, k, x_dtype);
  char* dev[2] = {(char*)ws, (char*)ws + cb};
  void* hws = (char*)ws + 2 * cb;
  char* stg[2] = {(char*)staging, staging ? (char*)staging + cb : nullptr};
  hipStream_t s = (hipStream_t)stream, cs = copy_stream ? (hipStream_t)copy_stream : s;
  hipEvent_t copied[2] = {nullptr, nullptr}, used[2] = {nullptr, nullptr};
  hipError_t e = hipSuccess;
  for (int b = 0; b < 2 && e == hipSuccess; ++b) {
    e = hipEventCreateWithFlags(&copied[b], hipEventDisableTiming);
    if (e == hipSuccess) e = hipEventCreateWithFlags(&used[b], hipEventDisableTiming);
  }
  const char* src = (const char*)X_host;
  for (int64_t t0 = 0, i = 0; e == hipSuccess && t0 < n; t0 += chunk, ++i) {
    const int b = (int)(i & 1);
    const int64_t rows = std::min<int64_t>(chunk, n - t0);
    const char* from = src + t0 * ldx * es;
    int64_t from_ld = ldx * es;
    if (stg[0]) {
      // The copy out of this staging buffer two chunks ago must be done.
      if (i >= 2) e = hipEventSynchronize(copied[b]);
      if (e != hipSuccess) break;
      copy_rows_host(stg[b], from, rows, k * es, ldx * es);
      from = stg[b];
      from_ld = k * es;
    }
    // The device buffer's previous chunk must have been consumed.
    if (i >= 2) e = hipStreamWaitEvent(cs, used[b], 0);
    if (e == hipSuccess)
      e = hipMemcpy2DAsync(dev[b], (size_t)(k * es), from, (size_t)from_ld, (size_t)(k * es), (size_t)rows,
                           hipMemcpyHostToDevice, cs);
    if (e == hipSuccess) e = hipEventRecord(copied[b], cs);
    if (e == hipSuccess) e = hipStreamWaitEvent(s, copied[b], 0);
    if (e == hipSuccess) e = hessian_run(dev[b], x_dtype, rows, k, k, H, hws, s);
    if (e == hipSuccess) e = hipEventRecord(used[b], s);
  }
  // With staging, return only once the staging buffers have been read, so the
  // caller may reuse them at once.
  for (int b = 0; b < 2 && stg[0] && e == hipSuccess; ++b) e = hipEventSynchronize(copied[b]);
  for (int b = 0; b < 2; ++b) {
    if (copied[b]) (void)hipEventDestroy(copied[b]);
    if (used[b]) (void)hipEventDestroy(used[b]);
  }
  return hip_status(e, fn);
}

// ---- consumer: NVFP4 weight-only GEMM ------------------------------------------
size_t nvfp4_gemm_workspace_size(int64_t T, int64_t k, int64_t m) { return align_up(nvfp4_gemm_workspace(T, k, m)); }

namespace {
// Arguments of nvfp4_gemm and its no-allocation variant; *empty is set when
// there is nothing to compute.
int gemm_check(const char* fn, const void* X, int x_dtype, int64_t T, int64_t k, int64_t ldx, const uint8_t* codes,
               const uint8_t* scales, const float* g, int64_t m, const void* Y, int y_dtype, int64_t ldy, bool* empty) {
  *empty = false;
  if (x_dtype != NVQ_DTYPE_BF16) return failp(NVQ_ERR_DTYPE, fn, "x_dtype %d (activations must be bf16)", x_dtype);
  if (!dtype_ok(y_dtype)) return failp(NVQ_ERR_DTYPE, fn, "y_dtype %d", y_dtype);
  if (T < 0 || m < 0 || k <= 0 || k % 16 != 0 || ldx < k || ldx % 8 != 0 || ldy < m)
    return failp(NVQ_ERR_SHAPE, fn, "T=%lld m=%lld k=%lld ldx=%lld ldy=%lld (need k%%16==0, ldx>=k, ldx%%8==0, ldy>=m)",
                 (long long)T, (long long)m, (long long)k, (long long)ldx, (long long)ldy);
  if (T == 0 || m == 0) {
    *empty = true;
    return NVQ_OK;
  }
  if (!X || !codes || !scales || !g || !Y) return failp(NVQ_ERR_NULL, fn, "X, codes, scales, g and Y are required");
  if (!aligned(X, 16)) return failp(NVQ_ERR_ALIGN, fn, "X must be 16-byte aligned");
  if (!aligned(codes, 8)) return failp(NVQ_ERR_ALIGN, fn, "codes must be 8-byte aligned");
  return NVQ_OK;
}
}  // namespace

int nvfp4_gemm(const void* X, int x_dtype, int64_t T, int64_t k, int64_t ldx, const uint8_t* codes,
               const uint8_t* scales, const float* g, int64_t m, void* Y, int y_dtype, int64_t ldy, void* ws,
               size_t ws_bytes, void* stream) {
  const char* fn = "nvfp4_gemm";
  bool empty = false;
  const int rc = gemm_check(fn, X, x_dtype, T, k, ldx, codes, scales, g, m, Y, y_dtype, ldy, &empty);
  if (rc != NVQ_OK || empty) return rc;
  const size_t need = nvfp4_gemm_workspace(T, k, m);
  if (need && (!ws || ws_bytes < need || !aligned(ws, kAlign)))
    return failp(NVQ_ERR_WORKSPACE, fn, "workspace needs %zu bytes (256-aligned), got %zu", need, ws_bytes);
  return hip_status(nvfp4_gemm_launch((const uint16_t*)X, T, k, ldx, codes, scales, g, m, Y,
                                      y_dtype == NVQ_DTYPE_BF16, ldy, (float*)ws, (hipStream_t)stream), fn);
}

int nvfp4_gemm_noalloc(const void* X, int x_dtype, int64_t T, int64_t k, int64_t ldx, const uint8_t* codes,
                       const uint8_t* scales, const float* g, int64_t m, void* Y, int y_dtype, int64_t ldy,
                       void* stream) {
  const char* fn = "nvfp4_gemm_noalloc";
  bool empty = false;
  const int rc = gemm_check(fn, X, x_dtype, T, k, ldx, codes, scales, g, m, Y, y_dtype, ldy, &empty);
  if (rc != NVQ_OK || empty) return rc;
  const size_t need = nvfp4_gemm_workspace(T, k, m);
  if (need > kNoAllocScratchBytes)
    return failp(NVQ_ERR_WORKSPACE, fn,
                 "T=%lld k=%lld m=%lld needs %zu bytes of partial sums; this variant holds at most %zu "
                 "(use nvfp4_gemm with a workspace)",
                 (long long)T, (long long)k, (long long)m, need, kNoAllocScratchBytes);
  float* scr = nullptr;
  hipError_t e = noalloc_scratch(&scr);
  if (e != hipSuccess) return hip_status(e, fn);
  return hip_status(nvfp4_gemm_launch((const uint16_t*)X, T, k, ldx, codes, scales, g, m, Y,
                                      y_dtype == NVQ_DTYPE_BF16, ldy, scr, (hipStream_t)stream), fn);
}

// Grouped Hessians: experts of at least kGroupedLarge tokens (or every expert
// when the grouped k = 4096 launch does not apply) are gathered and
// accumulated one at a time; the others are gathered one after another into
// the same row buffer and accumulated K4G_EXP at a time by one grouped launch
// each (a launch also ends when the buffer is full).  The buffer holds the
// largest expert's rows, and at least min(the small experts' rows, 2 GiB).
constexpr int64_t kGroupedLarge = 16384;
constexpr size_t kGroupedRowBytes = (size_t)2 << 30;

static bool grouped_launch_applies(int64_t k, int x_dtype) {
  return x_dtype == NVQ_DTYPE_BF16 && syrk_k4_grouped_applies(k);
}

static int64_t grouped_rows_cap(const int64_t* grp_off, int64_t G, int64_t k, int x_dtype, int64_t* nmax_out) {
  int64_t nmax = 0, small = 0;
  const bool grouped = grouped_launch_applies(k, x_dtype);
  for (int64_t e = 0; e < G; ++e) {
    const int64_t ne = grp_off[e + 1] - grp_off[e];
    nmax = std::max<int64_t>(nmax, ne);
    if (grouped && ne < kGroupedLarge) small += ne;
  }
  *nmax_out = nmax;
  const size_t esize = x_dtype == NVQ_DTYPE_BF16 ? 2 : 4;
  const int64_t cap = (int64_t)(kGroupedRowBytes / ((size_t)k * esize));
  return std::max<int64_t>(nmax, std::min<int64_t>(small, cap));
}

size_t hessian_grouped_workspace_size(const int64_t* grp_off, int64_t G, int64_t k, int x_dtype) {
  if (!grp_off || G <= 0 || k <= 0 || !dtype_ok(x_dtype)) return 0;
  int64_t nmax = 0;
  const int64_t rows = grouped_rows_cap(grp_off, G, k, x_dtype, &nmax);
  if (nmax <= 0) return 0;
  const size_t esize = x_dtype == NVQ_DTYPE_BF16 ? 2 : 4;
  return align_up((size_t)rows * k * esize) + hessian_workspace_size(nmax, k, x_dtype);
}

int hessian_accumulate_grouped(const void* X, int x_dtype, int64_t n, int64_t k, int64_t ldx, const int32_t* tok_idx,
                               const int64_t* grp_off, int64_t G, float* H, void* ws, size_t ws_bytes, void* stream) {
  if (!H || !grp_off) return fail(NVQ_ERR_NULL, "hessian_accumulate_grouped: H and grp_off are required");
  if (!dtype_ok(x_dtype)) return fail(NVQ_ERR_DTYPE, "hessian_accumulate_grouped: x_dtype %d", x_dtype);
  if (G <= 0 || n < 0 || k <= 0 || k % 16 != 0 || ldx < k || ldx % (x_dtype == NVQ_DTYPE_BF16 ? 8 : 4) != 0)
    return fail(NVQ_ERR_SHAPE, "hessian_accumulate_grouped: G=%lld n=%lld k=%lld ldx=%lld", (long long)G,
                (long long)n, (long long)k, (long long)ldx);
  if (grp_off[0] != 0) return fail(NVQ_ERR_VALUE, "hessian_accumulate_grouped: grp_off[0] must be 0");
  for (int64_t e = 0; e < G; ++e)
    if (grp_off[e + 1] < grp_off[e])
      return fail(NVQ_ERR_VALUE, "hessian_accumulate_grouped: grp_off must be non-decreasing (group %lld)", (long long)e);
  if (grp_off[G] == 0) return NVQ_OK;
  if (n == 0) return fail(NVQ_ERR_SHAPE, "hessian_accumulate_grouped: assignments given but n = 0");
  if (!X || !tok_idx) return fail(NVQ_ERR_NULL, "hessian_accumulate_grouped: X and tok_idx are required");
  if (!aligned(H, 16) || !aligned(X, 16)) return fail(NVQ_ERR_ALIGN, "hessian_accumulate_grouped: X and H must be 16-byte aligned");
  const size_t need = hessian_grouped_workspace_size(grp_off, G, k, x_dtype);
  if (!ws || ws_bytes < need || !aligned(ws, kAlign))
    return fail(NVQ_ERR_WORKSPACE, "hessian_accumulate_grouped: workspace needs %zu bytes (256-aligned), got %zu", need,
                ws_bytes);
  hipStream_t s = (hipStream_t)stream;
  const int esize = x_dtype == NVQ_DTYPE_BF16 ? 2 : 4;
  int64_t nmax = 0;
  const int64_t cap = grouped_rows_cap(grp_off, G, k, x_dtype, &nmax);
  const bool grouped = grouped_launch_applies(k, x_dtype);
  char* rows = (char*)ws;
  void* hws = rows + align_up((size_t)cap * k * esize);
  hipError_t err = hipSuccess;
  for (int64_t e = 0; err == hipSuccess && e < G; ++e) {
    const int64_t ne = grp_off[e + 1] - grp_off[e];
    if (ne == 0 || (grouped && ne < kGroupedLarge)) continue;
    err = gather_rows(X, esize, ldx, tok_idx + grp_off[e], n, ne, k, rows, s);
    if (err == hipSuccess) err = hessian_run(rows, x_dtype, ne, k, k, H + (size_t)e * k * k, hws, s);
  }
  if (grouped) {
    K4Grouped g{};
    int nexp = 0;
    int64_t used = 0;
    for (int64_t e = 0; err == hipSuccess && e <= G; ++e) {
      const int64_t ne = e < G ? grp_off[e + 1] - grp_off[e] : 0;
      if (e < G && (ne == 0 || ne >= kGroupedLarge)) continue;
      if (nexp > 0 && (e == G || nexp == K4G_EXP || used + ne > cap)) {
        err = syrk_bf16_grouped((const uint16_t*)rows, k, g, nexp, H, s);
        nexp = 0;
        used = 0;
      }
      if (e == G || err != hipSuccess) break;
      err = gather_rows(X, esize, ldx, tok_idx + grp_off[e], n, ne, k, rows + (size_t)used * k * esize, s);
      g.beg[nexp] = (int32_t)used;
      g.cnt[nexp] = (int32_t)ne;
      g.hexp[nexp] = (int32_t)e;
      ++nexp;
      used += ne;
    }
  }
  return hip_status(err, "hessian_accumulate_grouped");
}

// ---------------------------------------------------------------------------
size_t factor_hinv_workspace_size(int64_t k) { return k > 0 ? align_up(factor_workspace(k)) : 0; }

int factor_hinv(const float* H, int64_t k, float damp_rel, float* U, float* lambda_out, int32_t* info, void* ws,
                size_t ws_bytes, void* stream) {
  if (!H || !U || !lambda_out || !info) return fail(NVQ_ERR_NULL, "factor_hinv: H, U, lambda_out and info are required");
  if (k <= 0 || k % 16 != 0) return fail(NVQ_ERR_SHAPE, "factor_hinv: k=%lld (need k>0, k%%16==0)", (long long)k);
  if (!(damp_rel >= 0.0f) || !std::isfinite(damp_rel))
    return fail(NVQ_ERR_VALUE, "factor_hinv: damp_rel must be finite and >= 0");
  if (H == U) return fail(NVQ_ERR_VALUE, "factor_hinv: U must not overlap H");
  if (!aligned(H, 16) || !aligned(U, 16)) return fail(NVQ_ERR_ALIGN, "factor_hinv: H and U must be 16-byte aligned");
  size_t need = factor_hinv_workspace_size(k);
  if (!ws || ws_bytes < need || !aligned(ws, kAlign))
    return fail(NVQ_ERR_WORKSPACE, "factor_hinv: workspace needs %zu bytes (256-aligned), got %zu", need, ws_bytes);
  return hip_status(factor_hinv_launch(H, k, 1, k * k, damp_rel, U, k * k, lambda_out, info, ws, 1,
                                       (hipStream_t)stream), "factor_hinv");
}

// factor_hinv_batched and factor_chol_batched: the same checks, the U form or
// the Cholesky-factor form over passes of as many matrices as the workspace
// holds.
static int factor_batched(const char* fn, bool chol, const float* H, int64_t k, int64_t batch, int64_t stride_h,
                          float damp_rel, float* U, int64_t stride_u, float* lambda_out, int32_t* info, void* ws,
                          size_t ws_bytes, void* stream) {
  if (batch < 0) return failp(NVQ_ERR_SHAPE, fn, "batch=%lld", (long long)batch);
  if (batch == 0) return NVQ_OK;
  if (!H || !U || !lambda_out || !info) return failp(NVQ_ERR_NULL, fn, "H, the output, lambda_out and info are required");
  if (k <= 0 || k % 16 != 0) return failp(NVQ_ERR_SHAPE, fn, "k=%lld (need k>0, k%%16==0)", (long long)k);
  if (stride_h < k * k || stride_u < k * k || stride_h % 4 != 0 || stride_u % 4 != 0)
    return failp(NVQ_ERR_SHAPE, fn, "strides must be >= k*k and multiples of 4");
  if (!(damp_rel >= 0.0f) || !std::isfinite(damp_rel)) return failp(NVQ_ERR_VALUE, fn, "damp_rel must be finite and >= 0");
  if ((const float*)U < H + (size_t)stride_h * batch && H < (const float*)U + (size_t)stride_u * batch)
    return failp(NVQ_ERR_VALUE, fn, "the output must not overlap H");
  if (!aligned(H, 16) || !aligned(U, 16)) return failp(NVQ_ERR_ALIGN, fn, "H and the output must be 16-byte aligned");
  const size_t one = factor_hinv_workspace_size(k);
  if (!ws || ws_bytes < one || !aligned(ws, kAlign))
    return failp(NVQ_ERR_WORKSPACE, fn, "workspace needs at least %zu bytes (256-aligned), got %zu", one, ws_bytes);
  const int64_t chunk = std::min<int64_t>((int64_t)(ws_bytes / one), batch);
  return hip_status(factor_hinv_launch(H, k, batch, stride_h, damp_rel, U, stride_u, lambda_out, info, ws, chunk,
                                       (hipStream_t)stream, chol), fn);
}

int factor_hinv_batched(const float* H, int64_t k, int64_t batch, int64_t stride_h, float damp_rel, float* U,
                        int64_t stride_u, float* lambda_out, int32_t* info, void* ws, size_t ws_bytes, void* stream) {
  return factor_batched("factor_hinv_batched", false, H, k, batch, stride_h, damp_rel, U, stride_u, lambda_out, info,
                        ws, ws_bytes, stream);
}

int factor_chol_batched(const float* H, int64_t k, int64_t batch, int64_t stride_h, float damp_rel, float* V,
                        int64_t stride_v, float* lambda_out, int32_t* info, void* ws, size_t ws_bytes, void* stream) {
  return factor_batched("factor_chol_batched", true, H, k, batch, stride_h, damp_rel, V, stride_v, lambda_out, info,
                        ws, ws_bytes, stream);
}

size_t factor_chol_workspace_size(int64_t k) { return factor_hinv_workspace_size(k); }

int factor_chol(const float* H, int64_t k, float damp_rel, float* V, float* lambda_out, int32_t* info, void* ws,
                size_t ws_bytes, void* stream) {
  const char* fn = "factor_chol";
  if (!H || !V || !lambda_out || !info) return failp(NVQ_ERR_NULL, fn, "H, V, lambda_out and info are required");
  if (k <= 0 || k % 16 != 0) return failp(NVQ_ERR_SHAPE, fn, "k=%lld (need k>0, k%%16==0)", (long long)k);
  if (!(damp_rel >= 0.0f) || !std::isfinite(damp_rel)) return failp(NVQ_ERR_VALUE, fn, "damp_rel must be finite and >= 0");
  if (H == V) return failp(NVQ_ERR_VALUE, fn, "V must not overlap H");
  if (!aligned(H, 16) || !aligned(V, 16)) return failp(NVQ_ERR_ALIGN, fn, "H and V must be 16-byte aligned");
  const size_t need = factor_chol_workspace_size(k);
  if (!ws || ws_bytes < need || !aligned(ws, kAlign))
    return failp(NVQ_ERR_WORKSPACE, fn, "workspace needs %zu bytes (256-aligned), got %zu", need, ws_bytes);
  return hip_status(factor_hinv_launch(H, k, 1, k * k, damp_rel, V, k * k, lambda_out, info, ws, 1,
                                       (hipStream_t)stream, true), fn);
}

// ---------------------------------------------------------------------------
size_t nvfp4_global_scale_workspace_size(int64_t m, int64_t k) {
  return (m > 0 && k > 0) ? align_up((size_t)global_scale_parts(m, k) * sizeof(float)) : 0;
}

int nvfp4_global_scale(const void* W, int w_dtype, int64_t m, int64_t k, int64_t ldw, float* g_out, void* ws,
                       size_t ws_bytes, void* stream) {
  if (!W || !g_out) return fail(NVQ_ERR_NULL, "nvfp4_global_scale: W and g_out are required");
  if (!dtype_ok(w_dtype)) return fail(NVQ_ERR_DTYPE, "nvfp4_global_scale: w_dtype %d", w_dtype);
  if (m <= 0 || k <= 0 || ldw < k) return fail(NVQ_ERR_SHAPE, "nvfp4_global_scale: m=%lld k=%lld ldw=%lld",
                                               (long long)m, (long long)k, (long long)ldw);
  size_t need = nvfp4_global_scale_workspace_size(m, k);
  if (!ws || ws_bytes < need || !aligned(ws, kAlign))
    return fail(NVQ_ERR_WORKSPACE, "nvfp4_global_scale: workspace needs %zu bytes, got %zu", need, ws_bytes);
  return hip_status(global_scale_launch(W, w_dtype == NVQ_DTYPE_BF16, m, k, ldw, g_out, (float*)ws,
                                        global_scale_parts(m, k), (hipStream_t)stream),
                    "nvfp4_global_scale");
}

// ---------------------------------------------------------------------------
size_t gptq_nvfp4_workspace_size(int64_t m, int64_t k, unsigned flags) {
  if (m <= 0 || k <= 0) return 0;
  const bool rtn = flags & NVQ_FLAG_RTN;
  return quant_ws(m, k, (flags & NVQ_FLAG_FP64) && !rtn, (flags & NVQ_FLAG_CHOL_FACTOR) && !rtn).total;
}

int gptq_nvfp4_quantize(const void* W, int w_dtype, int64_t m, int64_t k, int64_t ldw, const float* U,
                        const float* H, const float* g, int n_cand, unsigned flags, uint8_t* codes, uint8_t* scales,
                        float* row_err, float* row_loss, void* ws, size_t ws_bytes, void* stream) {
  const int rc = quant_check("gptq_nvfp4_quantize", W, w_dtype, m, k, ldw, U, H, g, n_cand, flags, codes, scales,
                             row_err, ws, ws_bytes);
  if (rc != NVQ_OK) return rc;
  return hip_status(quant_run(W, w_dtype, m, k, ldw, U, H, g, n_cand, flags, codes, scales, row_err, row_loss,
                              (char*)ws, (hipStream_t)stream),
                    "gptq_nvfp4_quantize");
}

int gptq_nvfp4_quantize_batched(const void* W, int w_dtype, int64_t batch, int64_t m, int64_t k, int64_t ldw,
                                int64_t stride_w, const float* U, int64_t stride_u, const float* H, int64_t stride_h,
                                const float* g, int n_cand, unsigned flags, uint8_t* codes, uint8_t* scales,
                                float* row_err, float* row_loss, void* ws, size_t ws_bytes, void* stream) {
  if (batch < 0) return fail(NVQ_ERR_SHAPE, "gptq_nvfp4_quantize_batched: batch=%lld", (long long)batch);
  if (batch == 0) return NVQ_OK;
  const int rc = quant_check("gptq_nvfp4_quantize_batched", W, w_dtype, m, k, ldw, U, H, g, n_cand, flags, codes,
                             scales, row_err, ws, ws_bytes);
  if (rc != NVQ_OK) return rc;
  const bool rtn = flags & NVQ_FLAG_RTN, want_err = !(flags & NVQ_FLAG_NO_ERR);
  if (stride_w < m * ldw || (!rtn && (stride_u < k * k || stride_u % 4 != 0)) ||
      (want_err && (stride_h < k * k || stride_h % 4 != 0)))
    return fail(NVQ_ERR_SHAPE, "gptq_nvfp4_quantize_batched: strides must cover one element (W: m*ldw, U and H: k*k, "
                               "multiples of 4)");
  // As many matrices per pass as the workspace holds (each launch covers all of them).
  const QuantWs L = quant_ws(m, k, (flags & NVQ_FLAG_FP64) && !rtn, (flags & NVQ_FLAG_CHOL_FACTOR) && !rtn);
  const int64_t chunk = std::max<int64_t>(1, std::min<int64_t>({batch, (int64_t)(ws_bytes / L.total), 65535}));
  const size_t es = w_dtype == NVQ_DTYPE_BF16 ? 2 : 4;
  QBatch qb;
  qb.stride_w = stride_w; qb.stride_u = stride_u; qb.stride_h = stride_h; qb.ws_stride = L.total;
  hipError_t err = hipSuccess;
  for (int64_t e = 0; err == hipSuccess && e < batch; e += chunk) {
    qb.nb = std::min<int64_t>(chunk, batch - e);
    err = quant_run((const char*)W + (size_t)e * stride_w * es, w_dtype, m, k, ldw,
                    U ? U + (size_t)e * stride_u : nullptr, H ? H + (size_t)e * stride_h : nullptr, g + e, n_cand,
                    flags, codes + (size_t)e * m * (k / 2), scales + (size_t)e * m * (k / kBlock),
                    row_err ? row_err + (size_t)e * m : nullptr, row_loss ? row_loss + (size_t)e * m : nullptr,
                    (char*)ws, (hipStream_t)stream, qb);
  }
  return hip_status(err, "gptq_nvfp4_quantize_batched");
}

// ---------------------------------------------------------------------------
int nvq_check_finite(const void* A, int dtype, int64_t rows, int64_t cols, int64_t ld, int32_t* status,
                     void* stream) {
  const char* fn = "nvq_check_finite";
  if (!status) return failp(NVQ_ERR_NULL, fn, "status is NULL");
  if (!dtype_ok(dtype)) return failp(NVQ_ERR_DTYPE, fn, "dtype %d", dtype);
  if (rows < 0 || cols <= 0 || ld < cols || rows > 0x7FFFFFFE)
    return failp(NVQ_ERR_SHAPE, fn, "rows=%lld cols=%lld ld=%lld (need 0<=rows<2^31-1, cols>0, ld>=cols)",
                 (long long)rows, (long long)cols, (long long)ld);
  if (rows > 0 && !A) return failp(NVQ_ERR_NULL, fn, "A is NULL");
  if (!aligned(status, 4)) return failp(NVQ_ERR_ALIGN, fn, "status must be 4-byte aligned");
  return hip_status(nonfinite_scan_launch(A, dtype == NVQ_DTYPE_BF16, rows, cols, ld, status, (hipStream_t)stream), fn);
}

// ---------------------------------------------------------------------------
int nvfp4_dequantize(const uint8_t* codes, const uint8_t* scales, const float* g, int64_t m, int64_t k, void* out,
                     int out_dtype, void* stream) {
  if (m < 0 || k <= 0 || k % 16 != 0) return fail(NVQ_ERR_SHAPE, "nvfp4_dequantize: m=%lld k=%lld", (long long)m,
                                                  (long long)k);
  if (!dtype_ok(out_dtype)) return fail(NVQ_ERR_DTYPE, "nvfp4_dequantize: out_dtype %d", out_dtype);
  if (m == 0) return NVQ_OK;
  if (!codes || !scales || !g || !out) return fail(NVQ_ERR_NULL, "nvfp4_dequantize: null argument");
  if (!aligned(codes, 8) || !aligned(out, 16)) return fail(NVQ_ERR_ALIGN, "nvfp4_dequantize: codes need 8-byte and out 16-byte alignment");
  return hip_status(dequant_launch(codes, scales, g, m, k, out, out_dtype == NVQ_DTYPE_BF16, (hipStream_t)stream),
                    "nvfp4_dequantize");
}

// ---- mixture of experts: router, sort by expert, experts' products, weighted sum ----
namespace {
// [T x top_k] slots of E experts, for the router and its gradient.
int topk_check(const char* fn, int dtype, int64_t T, int64_t E, int64_t ld, int top_k) {
  if (!dtype_ok(dtype)) return failp(NVQ_ERR_DTYPE, fn, "dtype %d", dtype);
  if (T < 0 || T > 0x7FFFFFFF || E < 1 || E > kMoeMaxExperts || ld < E)
    return failp(NVQ_ERR_SHAPE, fn, "T=%lld E=%lld ld=%lld (need 0<=T<2^31, 1<=E<=%lld, ld>=E)", (long long)T,
                 (long long)E, (long long)ld, (long long)kMoeMaxExperts);
  if (top_k < 1 || top_k > E || top_k > kMoeMaxTopK)
    return failp(NVQ_ERR_VALUE, fn, "top_k=%d (need 1 <= top_k <= min(E, %d))", top_k, kMoeMaxTopK);
  return NVQ_OK;
}
// T top_k, or -1 if it is not a row count that int32 positions can hold.
int64_t slots(int64_t T, int64_t top_k) {
  if (T < 0 || top_k < 1 || top_k > 0x7FFFFFFF || T > 0x7FFFFFFF || T * top_k > 0x7FFFFFFF) return -1;
  return T * top_k;
}
// The shared arguments of the experts' products: rows in groups, NVFP4 experts [m x k], one output row per row.
int experts_check(const char* fn, int64_t rows, const int64_t* grp_off, int64_t G, const uint8_t* codes,
                  const uint8_t* scales, const float* g, int64_t m, int64_t k, const void* out, int out_dtype,
                  int64_t ldo, int64_t width) {
  if (!dtype_ok(out_dtype)) return failp(NVQ_ERR_DTYPE, fn, "output dtype %d", out_dtype);
  if (rows < 0 || rows > 0x7FFFFFFF || G < 1 || G > 0x7FFFFF || m < 1 || k < 16 || k % 16 != 0 || m > 4000000 ||
      k > 4000000 || ldo < width)
    return failp(NVQ_ERR_SHAPE, fn,
                 "rows=%lld G=%lld m=%lld k=%lld ldo=%lld (need 0<=rows<2^31, 1<=G<2^23, m>0, k>0, k%%16==0, m and k "
                 "at most 4000000, ldo>=%lld)",
                 (long long)rows, (long long)G, (long long)m, (long long)k, (long long)ldo, (long long)width);
  if (rows == 0) return NVQ_OK;
  if (!grp_off || !codes || !scales || !g || !out)
    return failp(NVQ_ERR_NULL, fn, "grp_off, codes, scales, g and the output are required");
  if (!aligned(grp_off, 8) || !aligned(codes, 8) || !aligned(g, 4) || !aligned(out, out_dtype == NVQ_DTYPE_BF16 ? 2 : 4))
    return failp(NVQ_ERR_ALIGN, fn, "grp_off and codes must be 8-byte aligned, g and the output by their elements");
  return NVQ_OK;
}
int experts_status(hipError_t e, const char* fn, int64_t rows, int64_t G, int64_t width) {
  if (e == kTooManyTiles)
    return failp(NVQ_ERR_SHAPE, fn, "rows=%lld, G=%lld and %lld columns make more tiles than one launch holds", (long long)rows,
                 (long long)G, (long long)width);
  return hip_status(e, fn);
}
size_t elem_size(int dtype) { return dtype == NVQ_DTYPE_BF16 ? 2 : 4; }
}  // namespace

int moe_topk(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld, int top_k, int renorm, int32_t* ids,
             float* weights, void* stream) {
  const char* fn = "moe_topk";
  const int rc = topk_check(fn, dtype, T, E, ld, top_k);
  if (rc != NVQ_OK || T == 0) return rc;
  if (!logits || !ids || !weights) return failp(NVQ_ERR_NULL, fn, "logits, ids and weights are required");
  if (!aligned(logits, elem_size(dtype)) || !aligned(ids, 4) || !aligned(weights, 4))
    return failp(NVQ_ERR_ALIGN, fn, "logits, ids and weights must be aligned by their elements");
  return hip_status(moe_topk_launch(logits, dtype == NVQ_DTYPE_BF16, T, E, ld, top_k, renorm != 0, ids, weights,
                                    (hipStream_t)stream), fn);
}

int moe_topk_backward(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld, const int32_t* ids,
                      const float* weights, const float* dweights, int top_k, int renorm, void* dlogits, int64_t ldd,
                      void* stream) {
  const char* fn = "moe_topk_backward";
  const int rc = topk_check(fn, dtype, T, E, ld, top_k);
  if (rc != NVQ_OK) return rc;
  if (ldd < E) return failp(NVQ_ERR_SHAPE, fn, "ldd=%lld (need >= E=%lld)", (long long)ldd, (long long)E);
  if (T == 0) return NVQ_OK;
  if (!logits || !ids || !weights || !dweights || !dlogits)
    return failp(NVQ_ERR_NULL, fn, "logits, ids, weights, dweights and dlogits are required");
  const size_t es = elem_size(dtype);
  if (!aligned(logits, es) || !aligned(dlogits, es) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(dweights, 4))
    return failp(NVQ_ERR_ALIGN, fn, "pointers must be aligned by their elements");
  if (dlogits == logits) return failp(NVQ_ERR_VALUE, fn, "dlogits may not be logits");
  return hip_status(moe_topk_backward_launch(logits, dtype == NVQ_DTYPE_BF16, T, E, ld, ids, weights, dweights, top_k,
                                             renorm != 0, dlogits, ldd, (hipStream_t)stream), fn);
}

size_t moe_sort_workspace_size(int64_t T, int64_t top_k, int64_t E) {
  const int64_t n = slots(T, top_k);
  return n > 0 && E >= 1 && E <= kMoeMaxExperts ? align_up(moe_sort_workspace(n, E)) : 0;
}

int moe_sort(const int32_t* ids, int64_t T, int64_t top_k, int64_t E, int32_t* tok_idx, int64_t* grp_off, int32_t* pos,
             void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "moe_sort";
  const int64_t n = slots(T, top_k);
  if (n < 0 || E < 1 || E > kMoeMaxExperts)
    return failp(NVQ_ERR_SHAPE, fn, "T=%lld top_k=%lld E=%lld (need T>=0, top_k>0, T*top_k<2^31, 1<=E<=%lld)",
                 (long long)T, (long long)top_k, (long long)E, (long long)kMoeMaxExperts);
  if (!grp_off || (n > 0 && (!ids || !tok_idx || !pos)))
    return failp(NVQ_ERR_NULL, fn, "ids, tok_idx, grp_off and pos are required");
  if (!aligned(grp_off, 8) || !aligned(ids, 4) || !aligned(tok_idx, 4) || !aligned(pos, 4))
    return failp(NVQ_ERR_ALIGN, fn, "grp_off must be 8-byte aligned, ids, tok_idx and pos 4-byte");
  const size_t need = moe_sort_workspace(n, E);
  if (need && (!ws || ws_bytes < need || !aligned(ws, kAlign)))
    return failp(NVQ_ERR_WORKSPACE, fn, "workspace needs %zu bytes (256-aligned), got %zu", need, ws_bytes);
  return hip_status(moe_sort_launch(ids, n, (int)top_k, E, tok_idx, grp_off, pos, ws, (hipStream_t)stream), fn);
}

int nvfp4_gemm_grouped(const void* X, int x_dtype, int64_t n, int64_t k, int64_t ldx, const int32_t* tok_idx,
                       int64_t rows, const int64_t* grp_off, int64_t G, const uint8_t* codes, const uint8_t* scales,
                       const float* g, int64_t m, void* Y, int y_dtype, int64_t ldy, void* stream) {
  const char* fn = "nvfp4_gemm_grouped";
  if (x_dtype != NVQ_DTYPE_BF16) return failp(NVQ_ERR_DTYPE, fn, "x_dtype %d (activations must be bf16)", x_dtype);
  const int rc = experts_check(fn, rows, grp_off, G, codes, scales, g, m, k, Y, y_dtype, ldy, m);
  if (rc != NVQ_OK) return rc;
  if (n < 0 || n > 0x7FFFFFFF || ldx < k || ldx % 8 != 0 || ldx > (1ll << 35) / std::max<int64_t>(n, 1) ||
      (!tok_idx && rows > n) || (rows > 0 && n == 0))
    return failp(NVQ_ERR_SHAPE, fn,
                 "n=%lld rows=%lld ldx=%lld k=%lld (need 0<=n<2^31, ldx>=k, ldx%%8==0, n*ldx<=2^35, rows<=n without "
                 "tok_idx, and tokens if there are rows)",
                 (long long)n, (long long)rows, (long long)ldx, (long long)k);
  if (rows == 0) return NVQ_OK;
  if (!X) return failp(NVQ_ERR_NULL, fn, "X is NULL");
  if (!aligned(X, 16)) return failp(NVQ_ERR_ALIGN, fn, "X must be 16-byte aligned");
  if (!aligned(tok_idx, 4)) return failp(NVQ_ERR_ALIGN, fn, "tok_idx must be 4-byte aligned");
  if (Y == X) return failp(NVQ_ERR_VALUE, fn, "Y may not be X");
  return experts_status(nvfp4_gemm_grouped_launch((const uint16_t*)X, n, k, ldx, tok_idx, rows, grp_off, G, codes, scales,
                                                  g, m, Y, y_dtype == NVQ_DTYPE_BF16, ldy, (hipStream_t)stream),
                        fn, rows, G, m);
}

int nvfp4_gemm_grouped_dx(const void* dY, int dy_dtype, int64_t rows, int64_t m, int64_t lddy, const int64_t* grp_off,
                          int64_t G, const uint8_t* codes, const uint8_t* scales, const float* g, int64_t k, void* dX,
                          int dx_dtype, int64_t lddx, void* stream) {
  const char* fn = "nvfp4_gemm_grouped_dx";
  if (dy_dtype != NVQ_DTYPE_BF16) return failp(NVQ_ERR_DTYPE, fn, "dy_dtype %d (gradients must be bf16)", dy_dtype);
  const int rc = experts_check(fn, rows, grp_off, G, codes, scales, g, m, k, dX, dx_dtype, lddx, k);
  if (rc != NVQ_OK) return rc;
  if (lddy < m) return failp(NVQ_ERR_SHAPE, fn, "lddy=%lld (need >= m=%lld)", (long long)lddy, (long long)m);
  if (rows == 0) return NVQ_OK;
  if (!dY) return failp(NVQ_ERR_NULL, fn, "dY is NULL");
  if (!aligned(dY, 2)) return failp(NVQ_ERR_ALIGN, fn, "dY must be 2-byte aligned");
  if (dX == dY) return failp(NVQ_ERR_VALUE, fn, "dX may not be dY");
  return experts_status(nvfp4_gemm_grouped_dx_launch((const uint16_t*)dY, rows, m, lddy, grp_off, G, codes, scales, g, k,
                                                     dX, dx_dtype == NVQ_DTYPE_BF16, lddx, (hipStream_t)stream),
                        fn, rows, G, k);
}

int moe_combine(const void* Y, int y_dtype, int64_t rows, int64_t d, int64_t ldy, const int32_t* pos,
                const float* weights, int64_t T, int64_t top_k, void* out, int out_dtype, int64_t ldo, void* stream) {
  const char* fn = "moe_combine";
  if (!dtype_ok(y_dtype) || !dtype_ok(out_dtype)) return failp(NVQ_ERR_DTYPE, fn, "y_dtype %d, out_dtype %d", y_dtype, out_dtype);
  if (slots(T, top_k) < 0 || rows < 0 || rows > 0x7FFFFFFF || d < 1 || d > (1ll << 33) || ldy < d || ldo < d)
    return failp(NVQ_ERR_SHAPE, fn,
                 "T=%lld top_k=%lld rows=%lld d=%lld ldy=%lld ldo=%lld (need T>=0, top_k>0, T*top_k<2^31, "
                 "0<=rows<2^31, 0<d<=2^33, ldy>=d, ldo>=d)",
                 (long long)T, (long long)top_k, (long long)rows, (long long)d, (long long)ldy, (long long)ldo);
  if (T == 0) return NVQ_OK;
  if ((rows > 0 && !Y) || !pos || !out) return failp(NVQ_ERR_NULL, fn, "Y, pos and out are required");
  if (!aligned(Y, elem_size(y_dtype)) || !aligned(out, elem_size(out_dtype)) || !aligned(pos, 4) || !aligned(weights, 4))
    return failp(NVQ_ERR_ALIGN, fn, "pointers must be aligned by their elements");
  if (out == Y) return failp(NVQ_ERR_VALUE, fn, "out may not be Y");
  return hip_status(moe_combine_launch(Y, y_dtype == NVQ_DTYPE_BF16, rows, d, ldy, pos, weights, T, (int)top_k, out,
                                       out_dtype == NVQ_DTYPE_BF16, ldo, (hipStream_t)stream), fn);
}

int moe_combine_backward(const void* dout, int dout_dtype, int64_t T, int64_t d, int64_t ldd, const void* Y, int y_dtype,
                         int64_t rows, int64_t ldy, const int32_t* pos, const float* weights, int64_t top_k, void* dY,
                         int64_t lddy, float* dweights, void* stream) {
  const char* fn = "moe_combine_backward";
  if (!dtype_ok(y_dtype) || !dtype_ok(dout_dtype)) return failp(NVQ_ERR_DTYPE, fn, "dout_dtype %d, y_dtype %d", dout_dtype, y_dtype);
  if (slots(T, top_k) < 0 || rows < 0 || rows > 0x7FFFFFFF || d < 1 || ldd < d || (dweights && ldy < d) || (dY && lddy < d))
    return failp(NVQ_ERR_SHAPE, fn,
                 "T=%lld top_k=%lld rows=%lld d=%lld ldd=%lld ldy=%lld lddy=%lld (need T>=0, top_k>0, T*top_k<2^31, "
                 "0<=rows<2^31, d>0, leading dimensions >= d)",
                 (long long)T, (long long)top_k, (long long)rows, (long long)d, (long long)ldd, (long long)ldy,
                 (long long)lddy);
  if (!dY && !dweights) return failp(NVQ_ERR_NULL, fn, "dY or dweights is required");
  if (T == 0) return NVQ_OK;
  if (!dout || !pos || (rows > 0 && dweights && !Y)) return failp(NVQ_ERR_NULL, fn, "dout and pos are required, and Y for dweights");
  const size_t es = elem_size(y_dtype);
  if (!aligned(dout, elem_size(dout_dtype)) || !aligned(Y, es) || !aligned(dY, es) || !aligned(pos, 4) ||
      !aligned(weights, 4) || !aligned(dweights, 4))
    return failp(NVQ_ERR_ALIGN, fn, "pointers must be aligned by their elements");
  if (dY && (dY == Y || dY == dout)) return failp(NVQ_ERR_VALUE, fn, "dY may not be Y or dout");
  return hip_status(moe_combine_backward_launch(dout, dout_dtype == NVQ_DTYPE_BF16, T, d, ldd, Y,
                                                y_dtype == NVQ_DTYPE_BF16, rows, ldy, pos, weights, (int)top_k, dY, lddy,
                                                dweights, (hipStream_t)stream), fn);
}

// ---- MXFP4: quantization, product, gradient; the gated activation -------------------------
namespace {
constexpr int64_t kMaxWidth = 4000000;   // of one row, as for the experts' products
// n rows of k values in blocks of 32.
int mx_shape(const char* fn, int64_t n, int64_t k) {
  if (n < 0 || n > 0x7FFFFFFF || k < 32 || k % 32 != 0 || k > kMaxWidth)
    return failp(NVQ_ERR_SHAPE, fn, "rows=%lld k=%lld (need 0<=rows<2^31, k>0, k%%32==0, k at most %lld)", (long long)n, (long long)k,
                 (long long)kMaxWidth);
  return NVQ_OK;
}
int mx_weights(const char* fn, int64_t m, const uint8_t* codes, const uint8_t* scales) {
  if (!codes || !scales) return failp(NVQ_ERR_NULL, fn, "codes and scales are required");
  if (!aligned(codes, 16)) return failp(NVQ_ERR_ALIGN, fn, "codes must be 16-byte aligned");
  return NVQ_OK;
}
int tiles_status(hipError_t e, const char* fn, int64_t n, int64_t width) {
  if (e == kTooManyTiles)
    return failp(NVQ_ERR_SHAPE, fn, "rows=%lld and %lld columns make more tiles than one launch holds", (long long)n, (long long)width);
  return hip_status(e, fn);
}
}  // namespace

int mxfp4_quantize(const void* X, int x_dtype, int64_t n, int64_t k, int64_t ldx, uint8_t* codes, uint8_t* scales, void* stream) {
  const char* fn = "mxfp4_quantize";
  if (!dtype_ok(x_dtype)) return failp(NVQ_ERR_DTYPE, fn, "x_dtype %d", x_dtype);
  const int rc = mx_shape(fn, n, k);
  if (rc != NVQ_OK) return rc;
  if (ldx < k) return failp(NVQ_ERR_SHAPE, fn, "ldx=%lld (need >= k=%lld)", (long long)ldx, (long long)k);
  if (n == 0) return NVQ_OK;
  if (!X || !codes || !scales) return failp(NVQ_ERR_NULL, fn, "X, codes and scales are required");
  if (!aligned(X, elem_size(x_dtype)) || !aligned(codes, 16))
    return failp(NVQ_ERR_ALIGN, fn, "X must be aligned by its elements, codes 16-byte");
  return hip_status(mxfp4_quantize_launch(X, x_dtype == NVQ_DTYPE_BF16, n, k, ldx, codes, scales, (hipStream_t)stream), fn);
}

int mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t n, int64_t k, void* out, int out_dtype, void* stream) {
  const char* fn = "mxfp4_dequantize";
  if (!dtype_ok(out_dtype)) return failp(NVQ_ERR_DTYPE, fn, "out_dtype %d", out_dtype);
  int rc = mx_shape(fn, n, k);
  if (rc != NVQ_OK || n == 0) return rc;
  rc = mx_weights(fn, n, codes, scales);
  if (rc != NVQ_OK) return rc;
  if (!out) return failp(NVQ_ERR_NULL, fn, "out is required");
  if (!aligned(out, 16)) return failp(NVQ_ERR_ALIGN, fn, "out must be 16-byte aligned");
  return hip_status(mxfp4_dequantize_launch(codes, scales, n, k, out, out_dtype == NVQ_DTYPE_BF16, (hipStream_t)stream), fn);
}

size_t mxfp4_gemm_workspace_size(int x_dtype, int64_t n, int64_t k, int64_t m) {
  if (n <= 0 || k <= 0 || m <= 0 || (!dtype_ok(x_dtype) && x_dtype != NVQ_DTYPE_MXFP4)) return 0;
  return align_up(mxfp4_gemm_workspace(x_dtype == NVQ_DTYPE_MXFP4, x_dtype == NVQ_DTYPE_BF16, n, k, m));
}

int mxfp4_gemm(const void* X, int x_dtype, const uint8_t* x_scales, int64_t n, int64_t k, int64_t ldx, const uint8_t* codes,
               const uint8_t* scales, int64_t m, void* Y, int y_dtype, int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "mxfp4_gemm";
  const bool packed = x_dtype == NVQ_DTYPE_MXFP4;
  if ((!packed && !dtype_ok(x_dtype)) || !dtype_ok(y_dtype)) return failp(NVQ_ERR_DTYPE, fn, "x_dtype %d, y_dtype %d", x_dtype, y_dtype);
  int rc = mx_shape(fn, n, k);
  if (rc != NVQ_OK) return rc;
  if (m < 1 || m > kMaxWidth || (packed ? ldx != k : ldx < k) || ldy < m)
    return failp(NVQ_ERR_SHAPE, fn, "m=%lld k=%lld ldx=%lld ldy=%lld (need 0<m<=%lld, ldx>=k, ldx==k for MXFP4, ldy>=m)", (long long)m,
                 (long long)k, (long long)ldx, (long long)ldy, (long long)kMaxWidth);
  if (n == 0) return NVQ_OK;
  rc = mx_weights(fn, m, codes, scales);
  if (rc != NVQ_OK) return rc;
  if (!X || !Y || (packed && !x_scales)) return failp(NVQ_ERR_NULL, fn, "X, Y and with MXFP4 x_scales are required");
  if (!aligned(X, packed ? 16 : elem_size(x_dtype)) || !aligned(Y, elem_size(y_dtype)))
    return failp(NVQ_ERR_ALIGN, fn, "X and Y must be aligned by their elements, MXFP4 codes 16-byte");
  if (Y == X) return failp(NVQ_ERR_VALUE, fn, "Y may not be X");
  const size_t need = mxfp4_gemm_workspace(packed, x_dtype == NVQ_DTYPE_BF16, n, k, m);
  if (need && (!ws || ws_bytes < need || !aligned(ws, kAlign)))
    return failp(NVQ_ERR_WORKSPACE, fn, "workspace needs %zu bytes (256-aligned), got %zu", need, ws_bytes);
  return tiles_status(mxfp4_gemm_launch(X, packed, x_dtype == NVQ_DTYPE_BF16, x_scales, n, k, ldx, codes, scales, m, Y,
                                        y_dtype == NVQ_DTYPE_BF16, ldy, ws, (hipStream_t)stream), fn, n, m);
}

// The first rows on expanded weights, the rest after them in the same workspace; or
// none on expanded weights, if dY's alignment asks for it.
static size_t dx_rest_workspace(int64_t n, int64_t m, int64_t k) {
  return n == 0 ? 0 : mxfp4_gemm_dx_few(n) ? mxfp4_gemm_dx_few_workspace(n, m, k) : mxfp4_gemm_dx_split_workspace(n, m, k);
}
static size_t dx_workspace(int64_t n, int64_t m, int64_t k) {
  const int64_t rows = mxfp4_gemm_dx_expanded_rows(n, m, k);
  return std::max({rows ? (size_t)m * k * 2 : 0, dx_rest_workspace(n - rows, m, k), dx_rest_workspace(n, m, k)});
}

size_t mxfp4_gemm_dx_workspace_size(int64_t n, int64_t m, int64_t k) {
  return n > 0 && n <= 0x7FFFFFFF && m > 0 && m <= kMaxWidth && k > 0 && k <= kMaxWidth ? align_up(dx_workspace(n, m, k)) : 0;
}

int mxfp4_gemm_dx(const void* dY, int dy_dtype, int64_t n, int64_t m, int64_t lddy, const uint8_t* codes, const uint8_t* scales,
                  int64_t k, void* dX, int dx_dtype, int64_t lddx, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "mxfp4_gemm_dx";
  if (dy_dtype != NVQ_DTYPE_BF16) return failp(NVQ_ERR_DTYPE, fn, "dy_dtype %d (gradients must be bf16)", dy_dtype);
  if (!dtype_ok(dx_dtype)) return failp(NVQ_ERR_DTYPE, fn, "dx_dtype %d", dx_dtype);
  int rc = mx_shape(fn, n, k);
  if (rc != NVQ_OK) return rc;
  if (m < 1 || m > kMaxWidth || lddy < m || lddx < k)
    return failp(NVQ_ERR_SHAPE, fn, "m=%lld k=%lld lddy=%lld lddx=%lld (need 0<m<=%lld, lddy>=m, lddx>=k)", (long long)m, (long long)k,
                 (long long)lddy, (long long)lddx, (long long)kMaxWidth);
  if (n == 0) return NVQ_OK;
  rc = mx_weights(fn, m, codes, scales);
  if (rc != NVQ_OK) return rc;
  if (!dY || !dX) return failp(NVQ_ERR_NULL, fn, "dY and dX are required");
  if (!aligned(dY, 2) || !aligned(dX, elem_size(dx_dtype))) return failp(NVQ_ERR_ALIGN, fn, "dY and dX must be aligned by their elements");
  if (dX == dY) return failp(NVQ_ERR_VALUE, fn, "dX may not be dY");
  const size_t need = dx_workspace(n, m, k);
  if (need && (!ws || ws_bytes < need || !aligned(ws, kAlign)))
    return failp(NVQ_ERR_WORKSPACE, fn, "workspace needs %zu bytes (256-aligned), got %zu", need, ws_bytes);
  const uint16_t* d = (const uint16_t*)dY;
  const int bf16 = dx_dtype == NVQ_DTYPE_BF16;
  int64_t rows = lddy % 8 == 0 && aligned(d, 16) && lddy < 1 << 22 ? mxfp4_gemm_dx_expanded_rows(n, m, k) : 0;
  if (rows) {
    const int rc =
        tiles_status(mxfp4_gemm_dx_expanded_launch(d, rows, m, lddy, codes, scales, k, dX, bf16, lddx, ws, (hipStream_t)stream), fn, n, k);
    if (rc != NVQ_OK || rows == n) return rc;
  }
  const auto rest = mxfp4_gemm_dx_few(n - rows) ? mxfp4_gemm_dx_few_launch : mxfp4_gemm_dx_launch;
  return tiles_status(rest(d + rows * lddy, n - rows, m, lddy, codes, scales, k, (char*)dX + rows * lddx * (bf16 ? 2 : 4), bf16, lddx, ws,
                           (hipStream_t)stream), fn, n, k);
}

int swiglu(const void* X, int x_dtype, int64_t n, int64_t h, int64_t ldx, void* out, int out_dtype, int64_t ldo, void* stream) {
  const char* fn = "swiglu";
  if (!dtype_ok(x_dtype) || !dtype_ok(out_dtype)) return failp(NVQ_ERR_DTYPE, fn, "x_dtype %d, out_dtype %d", x_dtype, out_dtype);
  if (n < 0 || n > 0x7FFFFFFF || h < 1 || h > kMaxWidth || ldx < 2 * h || ldo < h)
    return failp(NVQ_ERR_SHAPE, fn, "n=%lld h=%lld ldx=%lld ldo=%lld (need 0<=n<2^31, 0<h<=%lld, ldx>=2h, ldo>=h)", (long long)n,
                 (long long)h, (long long)ldx, (long long)ldo, (long long)kMaxWidth);
  if (n == 0) return NVQ_OK;
  if (!X || !out) return failp(NVQ_ERR_NULL, fn, "X and out are required");
  if (!aligned(X, elem_size(x_dtype)) || !aligned(out, elem_size(out_dtype)))
    return failp(NVQ_ERR_ALIGN, fn, "X and out must be aligned by their elements");
  if (out == X) return failp(NVQ_ERR_VALUE, fn, "out may not be X");
  return hip_status(swiglu_launch(X, x_dtype == NVQ_DTYPE_BF16, n, h, ldx, out, out_dtype == NVQ_DTYPE_BF16, ldo, (hipStream_t)stream), fn);
}

int swiglu_backward(const void* dout, int64_t ldd, const void* X, int dtype, int64_t n, int64_t h, int64_t ldx, void* dX, int64_t lddx,
                    void* stream) {
  const char* fn = "swiglu_backward";
  if (!dtype_ok(dtype)) return failp(NVQ_ERR_DTYPE, fn, "dtype %d", dtype);
  if (n < 0 || n > 0x7FFFFFFF || h < 1 || h > kMaxWidth || ldx < 2 * h || ldd < h || lddx < 2 * h)
    return failp(NVQ_ERR_SHAPE, fn, "n=%lld h=%lld ldx=%lld ldd=%lld lddx=%lld (need 0<=n<2^31, 0<h<=%lld, ldx and lddx>=2h, ldd>=h)",
                 (long long)n, (long long)h, (long long)ldx, (long long)ldd, (long long)lddx, (long long)kMaxWidth);
  if (n == 0) return NVQ_OK;
  if (!dout || !X || !dX) return failp(NVQ_ERR_NULL, fn, "dout, X and dX are required");
  const size_t es = elem_size(dtype);
  if (!aligned(dout, es) || !aligned(X, es) || !aligned(dX, es))
    return failp(NVQ_ERR_ALIGN, fn, "pointers must be aligned by their elements");
  if (dX == X || dX == dout) return failp(NVQ_ERR_VALUE, fn, "dX may not be X or dout");
  return hip_status(swiglu_backward_launch(dout, ldd, X, dtype == NVQ_DTYPE_BF16, n, h, ldx, dX, lddx, (hipStream_t)stream), fn);
}

// ---- a whole mixture-of-experts MLP for a few tokens ------------------------------------
namespace {
bool moe_mlp_sizes(int64_t T, int64_t E, int64_t top_k, int64_t h) {
  return T >= 0 && T <= kMoeMlpTokens && E >= 1 && E <= kMoeMaxExperts && top_k >= 1 && top_k <= kMoeMaxTopK && h >= 32 && h % 16 == 0 &&
         h <= kMaxWidth;
}
}  // namespace

size_t nvfp4_moe_mlp_workspace_size(int64_t T, int64_t E, int64_t top_k, int64_t h) {
  return T > 0 && moe_mlp_sizes(T, E, top_k, h) ? align_up(nvfp4_moe_mlp_workspace(T, E, top_k, h)) : 0;
}

int nvfp4_moe_mlp(const void* X, int x_dtype, int64_t T, int64_t d, int64_t ldx, const void* logits, int logits_dtype, int64_t E,
                  int64_t ldl, int64_t top_k, int renorm, int32_t* ids, float* weights, const uint8_t* gate_up_codes,
                  const uint8_t* gate_up_scales, const float* gate_up_g, int64_t h, const uint8_t* down_codes,
                  const uint8_t* down_scales, const float* down_g, int64_t m, void* out, int out_dtype, int64_t ldo, void* ws,
                  size_t ws_bytes, void* stream) {
  const char* fn = "nvfp4_moe_mlp";
  if (x_dtype != NVQ_DTYPE_BF16) return failp(NVQ_ERR_DTYPE, fn, "x_dtype %d (activations must be bf16)", x_dtype);
  if (!dtype_ok(out_dtype) || (logits && !dtype_ok(logits_dtype)))
    return failp(NVQ_ERR_DTYPE, fn, "logits_dtype %d, out_dtype %d", logits_dtype, out_dtype);
  if (!moe_mlp_sizes(T, E, std::max<int64_t>(1, std::min<int64_t>(top_k, kMoeMaxTopK)), h) || d < 32 || d % 16 != 0 || d > kMaxWidth ||
      ldx < d || ldx % 8 != 0 || m < 1 || m > kMaxWidth || ldo < m || (logits && ldl < E) ||
      ldx > ((1ll << 30) - d) / std::max<int64_t>(1, T - 1))
    return failp(NVQ_ERR_SHAPE, fn,
                 "T=%lld d=%lld ldx=%lld E=%lld ldl=%lld h=%lld m=%lld ldo=%lld (need 0<=T<=%lld, 1<=E<=%lld, d and h at least 32 and "
                 "multiples of 16, m>0, each at most %lld, ldx>=d, ldx%%8==0, (T-1)*ldx+d<=2^30, ldl>=E, ldo>=m)",
                 (long long)T, (long long)d, (long long)ldx, (long long)E, (long long)ldl, (long long)h, (long long)m, (long long)ldo,
                 (long long)kMoeMlpTokens, (long long)kMoeMaxExperts, (long long)kMaxWidth);
  if (top_k < 1 || top_k > kMoeMaxTopK || (logits && top_k > E))
    return failp(NVQ_ERR_VALUE, fn, "top_k=%lld (need 1 <= top_k <= %d, and with logits <= E)", (long long)top_k, kMoeMaxTopK);
  if (T == 0) return NVQ_OK;
  if (!X || !ids || !weights || !gate_up_codes || !gate_up_scales || !gate_up_g || !down_codes || !down_scales || !down_g || !out)
    return failp(NVQ_ERR_NULL, fn, "X, ids, weights, both products' codes, scales and g, and out are required");
  if (!aligned(X, 16) || !aligned(gate_up_codes, 8) || !aligned(down_codes, 8) || !aligned(gate_up_g, 4) || !aligned(down_g, 4) ||
      !aligned(ids, 4) || !aligned(weights, 4) || !aligned(out, elem_size(out_dtype)) || (logits && !aligned(logits, elem_size(logits_dtype))))
    return failp(NVQ_ERR_ALIGN, fn, "X must be 16-byte aligned, codes 8-byte, the others by their elements");
  if (out == X || out == logits) return failp(NVQ_ERR_VALUE, fn, "out may not be X or logits");
  const size_t need = nvfp4_moe_mlp_workspace_size(T, E, top_k, h);
  if (!ws || ws_bytes < need || !aligned(ws, kAlign))
    return failp(NVQ_ERR_WORKSPACE, fn, "workspace needs %zu bytes (256-aligned), got %zu", need, ws_bytes);
  return hip_status(nvfp4_moe_mlp_launch((const uint16_t*)X, T, d, ldx, logits, logits && logits_dtype == NVQ_DTYPE_BF16, E, ldl, (int)top_k,
                                         renorm != 0, ids, weights, gate_up_codes, gate_up_scales, gate_up_g, h, down_codes, down_scales,
                                         down_g, m, out, out_dtype == NVQ_DTYPE_BF16, ldo, ws, (hipStream_t)stream), fn);
}

}  // extern "C"
