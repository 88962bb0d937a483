// Declarations shared by the microscaled 4-bit kernels and their C ABI.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace mgt {

// Allow `kern` on the current device `bytes` of dynamic shared memory, once per device (the
// attribute belongs to a device's copy of the kernel). One object per kernel.
struct SmemLimit {
  std::atomic<uint64_t> done{0};
  template <typename K>
  cudaError_t allow(K kern, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
  }
};

// How many clusters of a launch shape are resident at once, asked for once per device (devices may
// differ in SMs and in how these are grouped). shape < kShapes, size (CTAs of a cluster) at most 8.
struct ResidentClusters {
  static constexpr int kDevices = 64, kShapes = 17;
  std::atomic<int> known[kDevices][kShapes][9];  // + 1
  // *n = the answer of ask(&n), a cudaError_t
  template <typename Ask>
  cudaError_t get(int dev, int shape, int size, int* n, Ask ask) {
    std::atomic<int>* k = dev < kDevices ? &known[dev][shape][size] : nullptr;
    *n = k ? k->load(std::memory_order_relaxed) - 1 : -1;
    if (*n >= 0) return cudaSuccess;
    const cudaError_t e = ask(n);
    if (e == cudaSuccess && k) k->store(*n + 1, std::memory_order_relaxed);
    return e;
  }
};

// A 4-bit operand: packed codes (rows of ld / 2 bytes), scale tiles, leading dimension.
struct Mx4Out {
  uint8_t* codes;
  uint8_t* scales;
  long long ld;
};

// C[m, n] = f_a f_b sum_k A(m, k) B(n, k): A [M][K] activations, B [N][K] weights. Gated: B holds
// gate rows 0 .. N-1 and up rows from N rounded up to 128; the result act(gate) * up leaves
// quantised in `a` (and gate, up in bf16 in u, where given) instead of in C.
struct Mx4Gemm {
  int fmt, M, N, K;
  Mx4Out A, B;
  const float* a_factor;  // {amax, factor} of the tensor; null: 1
  const float* b_factor;
  void* C;
  int c_f32;
  long long ldc;
  int gated, act;
  Mx4Out a;
  const float* out_factor;
  void* u;
  long long ldu;
  int* err;
};
cudaError_t launch_gemm_mx4(const Mx4Gemm& g, int num_sms, cudaStream_t s);

// fmt: 0 mxfp4, 1 nvfp4; dtype: 0 fp32, 1 bf16. factor (nvfp4): {amax, f}.
cudaError_t launch_mx4_factor(int dtype, int rows, int cols, const void* x, long long ldx,
                              float* out, int num_sms, cudaStream_t s);
cudaError_t launch_mx4_quantize(int fmt, int dtype, int rows, int cols, const void* x,
                                long long ldx, const float* factor, const Mx4Out& out,
                                const Mx4Out& out_t, cudaStream_t s);
cudaError_t launch_mx4_dequantize(int fmt, int dtype, int rows, int cols, const Mx4Out& q,
                                  const float* factor, void* y, long long ldy, cudaStream_t s);
cudaError_t launch_mx4_gated_bwd(int fmt, int act, int rows, int F, const void* da,
                                 long long ldda, const void* u, long long ldu, const float* f_du,
                                 const float* f_dut, const float* f_at, const Mx4Out& dg,
                                 const Mx4Out& dup, const Mx4Out& dgt, const Mx4Out& dupt,
                                 const Mx4Out& at, cudaStream_t s);

}  // namespace mgt
