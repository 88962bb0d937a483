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

// Launch shape of the few-row product (mx4_skinny_kernel in gemm_mx4.cu) for M tokens.
constexpr int kSkinnyRows = 128;        // weight rows of a CTA's tile (per matrix)
constexpr int kSkinnyTokens = 256;      // most tokens of a tile
constexpr int kSkinnyGatedTokens = 64;  // the same for a gated product, and its most tokens at all
struct SkinnyShape {
  int tokens;       // of a tile: a multiple of 16
  int stages;       // 256 elements of the summed axis each; 0: no shape fits
  int stage_bytes;  // operands and scales
  int tmem_cols;    // allocated tensor-memory columns
  int smem;         // dynamic shared memory
  bool two;         // two CTAs per SM
};
constexpr SkinnyShape skinny_shape(bool nvfp4, bool gated, int M) {
  SkinnyShape r = {};
  const int most = gated ? kSkinnyGatedTokens : kSkinnyTokens;
  const int matrices = gated ? 2 : 1, scale_tiles = nvfp4 ? 4 : 2;  // of a stage and 128 rows
  r.tokens = M < most ? (M + 15) & ~15 : most;
  const int groups = r.tokens > 128 ? 2 : 1;  // 128-row groups of the tokens' scales
  const int operand_bytes = (matrices * kSkinnyRows + r.tokens) * 128;
  const int scales = (matrices + groups) * scale_tiles;
  r.stage_bytes = operand_bytes + scales * 512;
  const int acc = matrices * ((r.tokens + 31) & ~31);
  // Two CTAs per SM where each gets two stages at least, and as many stages as shared and tensor
  // memory hold. The partial tile, which takes the stages' place, has to fit into their operands.
  for (int per_sm = 2; per_sm > 0 && !r.stages; --per_sm) {
    const int bytes = (per_sm == 2 ? 113 : 227) * 1024 - 2048, columns = 512 / per_sm;
    int n = bytes / r.stage_bytes;
    while (n > 0 && acc + n * scales * 4 > columns) --n;
    if (n >= 2 && matrices * r.tokens * kSkinnyRows * 4 <= n * operand_bytes) r.stages = n;
    r.two = per_sm == 2;
  }
  r.tmem_cols = 32;
  while (r.tmem_cols < acc + r.stages * scales * 4) r.tmem_cols *= 2;
  r.smem = 1024 + r.stages * (r.stage_bytes + 16) + 64;
  return r;
}
// Every number of tokens has a shape, and a gated product shares its SM (its kernel has no other form).
constexpr bool skinny_shapes_fit() {
  for (int M = 1; M <= kSkinnyTokens; ++M)
    for (int k = 0; k < 4; ++k) {
      if ((k & 1) && M > kSkinnyGatedTokens) continue;
      const SkinnyShape s = skinny_shape(k & 2, k & 1, M);
      if (!s.stages || ((k & 1) && !s.two)) return false;
    }
  return true;
}
static_assert(skinny_shapes_fit(), "a token count without a launch shape");

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
