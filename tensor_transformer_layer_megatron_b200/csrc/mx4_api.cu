// C ABI of the microscaled 4-bit operators: validation only, the work is in mx4.cu and
// gemm_mx4.cu.
#include "../../include/mgt_layer.h"
#include "mgt_internal.h"
#include "mx4_internal.h"

using namespace mgt;

namespace {

mgt_status status_of(cudaError_t e) { return e == cudaSuccess ? MGT_OK : MGT_ECUDA; }

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int64_t up128(int64_t n) { return (n + 127) / 128 * 128; }

// Launches take 1-D grids of at most 2^31 - 1 blocks, one per 128 x 32 elements at least.
constexpr int64_t kMostElements = (int64_t)1 << 42;

mgt_status check(const mgt_mx4* q) {
  if (!q->codes || !q->scales || q->rows < 1 || q->cols < 1) return MGT_EINVAL;
  if (q->format != MGT_MXFP4 && q->format != MGT_NVFP4) return MGT_EUNSUPPORTED;
  if (q->format == MGT_NVFP4 && !q->factor) return MGT_EINVAL;
  if (q->ld % 128 || q->ld < up128(q->cols)) return MGT_EINVAL;
  if (!aligned(q->codes, 16) || !aligned(q->scales, 16) || !aligned(q->factor, 4))
    return MGT_EUNSUPPORTED;
  if (q->rows > (1 << 30) || q->cols > (1 << 30) || up128(q->rows) * q->ld > kMostElements)
    return MGT_EUNSUPPORTED;
  return MGT_OK;
}

// Two results in one place (parts of one buffer are fine).
bool same_place(const mgt_mx4* a, const mgt_mx4* b) {
  return a && b && (a->codes == b->codes || a->scales == b->scales);
}

bool dtype_ok(int32_t d) { return d == MGT_F32 || d == MGT_BF16; }
unsigned esz(int32_t d) { return d == MGT_F32 ? 4 : 2; }

Mx4Out view(const mgt_mx4* q, int64_t row = 0, int64_t col = 0) {
  if (!q) return Mx4Out{nullptr, nullptr, 0};
  const int64_t tile_cols = q->format == MGT_MXFP4 ? 128 : 64;
  return Mx4Out{q->codes + (row * q->ld + col) / 2,
                q->scales + ((row / 128) * (q->ld / tile_cols) + col / tile_cols) * 512, q->ld};
}

const float* factor_of(const mgt_mx4* q) {
  return q && q->format == MGT_NVFP4 ? q->factor : nullptr;
}

// SMs of the current device; 0 where it is not a Blackwell part, -1 on an error. Asked once per
// device (the answer cannot change).
int sms() {
  static std::atomic<int> known[64];  // SMs + 1
  int dev = 0, nsm = 0, major = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  if (dev < 64) {
    const int k = known[dev].load(std::memory_order_relaxed);
    if (k) return k - 1;
  }
  if (cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess)
    return -1;
  if (major != 10) nsm = 0;
  if (dev < 64) known[dev].store(nsm + 1, std::memory_order_relaxed);
  return nsm;
}
#define MX4_SMS(n)             \
  const int n = sms();         \
  if (n < 0) return MGT_ECUDA; \
  if (n == 0) return MGT_EUNSUPPORTED

}  // namespace

extern "C" {

mgt_status mgt_mx4_sizes(int32_t format, int32_t rows, int32_t cols, int64_t* ld,
                         size_t* code_bytes, size_t* scale_bytes) {
  if (rows < 1 || cols < 1 || !ld || !code_bytes || !scale_bytes) return MGT_EINVAL;
  if (format != MGT_MXFP4 && format != MGT_NVFP4) return MGT_EUNSUPPORTED;
  *ld = up128(cols);
  *code_bytes = (size_t)rows * (size_t)(*ld / 2);
  *scale_bytes = (size_t)up128(rows) * (size_t)(*ld / (format == MGT_MXFP4 ? 32 : 16));
  return MGT_OK;
}

mgt_status mgt_mx4_tensor_factor(int32_t dtype, int32_t rows, int32_t cols, const void* x,
                                 int64_t ldx, float* factor, void* stream) {
  if (rows < 1 || cols < 1 || !x || !factor || ldx < cols) return MGT_EINVAL;
  if (!dtype_ok(dtype) || !aligned(x, esz(dtype)) || !aligned(factor, 4)) return MGT_EUNSUPPORTED;
  MX4_SMS(n);
  return status_of(launch_mx4_factor(dtype == MGT_BF16, rows, cols, x, ldx, factor, n,
                                     static_cast<cudaStream_t>(stream)));
}

mgt_status mgt_mx4_quantize(int32_t dtype, const void* x, int64_t ldx, const mgt_mx4* q,
                            const mgt_mx4* qt, void* stream) {
  if (!x || (!q && !qt)) return MGT_EINVAL;
  mgt_status e;
  if ((q && (e = check(q)) != MGT_OK) || (qt && (e = check(qt)) != MGT_OK)) return e;
  if (q && qt && (q->format != qt->format || q->rows != qt->cols || q->cols != qt->rows))
    return MGT_EINVAL;
  // one read of x serves both layouts, with one factor
  if (q && qt && q->format == MGT_NVFP4 && q->factor != qt->factor) return MGT_EINVAL;
  const int rows = q ? q->rows : qt->cols, cols = q ? q->cols : qt->rows;
  if (ldx < cols) return MGT_EINVAL;
  if (!dtype_ok(dtype) || !aligned(x, esz(dtype))) return MGT_EUNSUPPORTED;
  if (same_place(q, qt)) return MGT_EINVAL;
  MX4_SMS(n);
  (void)n;
  return status_of(launch_mx4_quantize(q ? q->format : qt->format, dtype == MGT_BF16, rows, cols,
                                       x, ldx, factor_of(q ? q : qt), view(q), view(qt),
                                       static_cast<cudaStream_t>(stream)));
}

mgt_status mgt_mx4_dequantize(const mgt_mx4* q, int32_t dtype, void* y, int64_t ldy,
                              void* stream) {
  if (!q || !y) return MGT_EINVAL;
  const mgt_status e = check(q);
  if (e != MGT_OK) return e;
  if (ldy < q->cols) return MGT_EINVAL;
  if (!dtype_ok(dtype) || !aligned(y, esz(dtype))) return MGT_EUNSUPPORTED;
  MX4_SMS(n);
  (void)n;
  return status_of(launch_mx4_dequantize(q->format, dtype == MGT_BF16, q->rows, q->cols, view(q),
                                         factor_of(q), y, ldy,
                                         static_cast<cudaStream_t>(stream)));
}

mgt_status mgt_gemm_mx4(const mgt_mx4* A, const mgt_mx4* B, void* C, int32_t c_dtype, int64_t ldc,
                        int32_t* status, void* stream) {
  if (!A || !B || !C || !status) return MGT_EINVAL;
  mgt_status e;
  if ((e = check(A)) != MGT_OK || (e = check(B)) != MGT_OK) return e;
  if (A->format != B->format || A->cols != B->cols || ldc < B->rows) return MGT_EINVAL;
  if (!dtype_ok(c_dtype) || !aligned(C, esz(c_dtype)) || !aligned(status, 4))
    return MGT_EUNSUPPORTED;
  MX4_SMS(n);
  Mx4Gemm g = {};
  g.fmt = A->format;
  g.M = A->rows; g.N = B->rows; g.K = A->cols;
  g.A = view(A); g.B = view(B);
  g.a_factor = factor_of(A); g.b_factor = factor_of(B);
  g.C = C; g.c_f32 = c_dtype == MGT_F32; g.ldc = ldc;
  g.err = status;
  return status_of(launch_gemm_mx4(g, n, static_cast<cudaStream_t>(stream)));
}

mgt_status mgt_gemm_mx4_gated(const mgt_mx4* X, const mgt_mx4* W, int32_t act, const mgt_mx4* a,
                              void* u, int64_t ldu, int32_t* status, void* stream) {
  if (!X || !W || !a || !status) return MGT_EINVAL;
  mgt_status e;
  if ((e = check(X)) != MGT_OK || (e = check(W)) != MGT_OK || (e = check(a)) != MGT_OK) return e;
  if (act < MGT_ACT_SILU || act > MGT_ACT_GELU_TANH) return MGT_EUNSUPPORTED;
  if (X->format != W->format || X->format != a->format || X->cols != W->cols ||
      X->rows != a->rows || W->rows != 2 * up128(a->cols) || (u && ldu < 2 * (int64_t)a->cols))
    return MGT_EINVAL;
  if (!aligned(u, 2) || !aligned(status, 4)) return MGT_EUNSUPPORTED;
  if (same_place(a, X) || same_place(a, W)) return MGT_EINVAL;
  MX4_SMS(n);
  Mx4Gemm g = {};
  g.fmt = X->format;
  g.M = X->rows; g.N = a->cols; g.K = X->cols;
  g.A = view(X); g.B = view(W);
  g.a_factor = factor_of(X); g.b_factor = factor_of(W);
  g.gated = 1; g.act = act;
  g.a = view(a); g.out_factor = factor_of(a);
  g.u = u; g.ldu = ldu;
  g.err = status;
  return status_of(launch_gemm_mx4(g, n, static_cast<cudaStream_t>(stream)));
}

mgt_status mgt_mx4_gated_bwd(int32_t act, int32_t rows, int32_t ffn, const void* da, int64_t ldda,
                             const void* u, int64_t ldu, const mgt_mx4* du, const mgt_mx4* dut,
                             const mgt_mx4* at, void* stream) {
  if (rows < 1 || ffn < 1 || ffn > (1 << 29) || !da || !u || (!du && !dut && !at))
    return MGT_EINVAL;
  mgt_status e;
  if ((du && (e = check(du)) != MGT_OK) || (dut && (e = check(dut)) != MGT_OK) ||
      (at && (e = check(at)) != MGT_OK))
    return e;
  const int64_t half = up128(ffn);
  if ((du && (du->rows != rows || du->cols != 2 * half)) ||
      (dut && (dut->rows != 2 * half || dut->cols != rows)) ||
      (at && (at->rows != ffn || at->cols != rows)) || ldda < ffn || ldu < 2 * (int64_t)ffn)
    return MGT_EINVAL;
  const mgt_mx4* some = du ? du : dut ? dut : at;
  if ((du && du->format != some->format) || (dut && dut->format != some->format) ||
      (at && at->format != some->format))
    return MGT_EINVAL;
  if (act < MGT_ACT_SILU || act > MGT_ACT_GELU_TANH) return MGT_EUNSUPPORTED;
  if (!aligned(da, 2) || !aligned(u, 2)) return MGT_EUNSUPPORTED;
  if (same_place(du, dut) || same_place(du, at) || same_place(dut, at)) return MGT_EINVAL;
  MX4_SMS(n);
  (void)n;
  return status_of(launch_mx4_gated_bwd(
      some->format, act, rows, ffn, da, ldda, u, ldu, factor_of(du), factor_of(dut),
      factor_of(at), view(du), du ? view(du, 0, half) : view(nullptr), view(dut),
      dut ? view(dut, half, 0) : view(nullptr), view(at), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
