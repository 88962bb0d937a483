// Quantisers of the microscaled 4-bit formats (mx4_device.cuh): tensor factor, quantisation
// along the rows and, from the same read, along the columns (the transposed operand that the
// backward products sum over), the gated block's backward fused with both quantisations, and
// the way back to bf16 or fp32. All are bound by HBM: each element is read once.
#include "../../include/mgt_layer.h"
#include "mx4_device.cuh"
#include "mx4_internal.h"

namespace mgt {
namespace {

template <typename T>
struct Vec8;  // eight consecutive elements as loaded
template <>
struct Vec8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    a = __ldg(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void load_n(const __nv_bfloat16* p, int n) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = 2 * i < n ? __bfloat16_as_ushort(p[2 * i]) : 0;
      const uint32_t hi = 2 * i + 1 < n ? __bfloat16_as_ushort(p[2 * i + 1]) : 0;
      w[i] = lo | (hi << 16);
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ float at(int j) const {
    const uint32_t w = j < 2 ? a.x : j < 4 ? a.y : j < 6 ? a.z : a.w;
    return j & 1 ? bf16_hi(w) : bf16_lo(w);
  }
  // Largest |x| as fp32 bits: bf16 magnitudes order like their bits, two to a word.
  __device__ __forceinline__ uint32_t amax() const {
    const uint32_t k = 0x7fff7fffu;
    const uint32_t m = max_u16x2(max_u16x2(a.x & k, a.y & k), max_u16x2(a.z & k, a.w & k));
    return max(m << 16, m & 0xffff0000u);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void load_n(const float* p, int n) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.f;
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ float at(int j) const {
    return j < 4 ? (j < 2 ? (j ? a.y : a.x) : (j == 2 ? a.z : a.w))
                 : (j < 6 ? (j == 4 ? b.x : b.y) : (j == 6 ? b.z : b.w));
  }
  __device__ __forceinline__ uint32_t amax() const {
    return max(max(max(abs_bits(a.x), abs_bits(a.y)), max(abs_bits(a.z), abs_bits(a.w))),
               max(max(abs_bits(b.x), abs_bits(b.y)), max(abs_bits(b.z), abs_bits(b.w))));
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

// Eight elements from column c of a row of `cols`; zeros behind the last column. vec: the row
// base is 16-byte aligned (c is a multiple of 8).
template <typename T>
__device__ __forceinline__ void load8(Vec8<T>& r, const T* row, int c, int cols, bool row_ok,
                                      bool vec) {
  if (!row_ok || c >= cols)
    r.zero();
  else if (vec && c + 8 <= cols)
    r.load(row + c);
  else
    r.load_n(row + c, cols - c);
}

// A walk over (row, group of columns) in row-major order, `stride` items a step, with one
// division at the start.
struct Walk {
  long long row, drow;
  int g, dg, groups;
  __device__ __forceinline__ Walk(unsigned long long first, unsigned long long stride, int n) {
    groups = n;
    row = (long long)(first / (unsigned)n);
    g = (int)(first - (unsigned long long)row * (unsigned)n);
    drow = (long long)(stride / (unsigned)n);
    dg = (int)(stride - (unsigned long long)drow * (unsigned)n);
  }
  __device__ __forceinline__ void step() {
    row += drow;
    g += dg;
    if (g >= groups) {
      g -= groups;
      ++row;
    }
  }
};

// ---------------------------------------------------------------------------- tensor factor
// out = {amax over the finite elements, f = 2^ceil(log2(amax / 2688)), 1 for amax = 0}: 2688 =
// 6 * 448 is the largest product of an element and a block scale. Block maxima meet in an
// atomic maximum on the bits of out[0] (order free); the last block to arrive, counted in
// out[1], writes f over the count. Both words are zeroed before the launch.
template <typename T>
__global__ void __launch_bounds__(256) mx4_factor_kernel(int rows, int cols, const T* __restrict__ x,
                                                         long long ldx, bool vec, float* out) {
  __shared__ uint32_t red[8];
  uint32_t m = 0;
  constexpr int U = 4;
  Walk at(blockIdx.x * 256ull + threadIdx.x, gridDim.x * 256ull, (cols + 7) / 8);
  while (at.row < rows) {
    Vec8<T> w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      load8(w[u], x + at.row * ldx, at.g * 8, cols, at.row < rows, vec);
      at.step();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t all = w[u].amax();
      if (all < 0x7f800000u) {
        m = max(m, all);
      } else {  // infinities and NaNs do not count
        float v[8];
        w[u].get(v);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t b = abs_bits(v[k]);
          m = max(m, b < 0x7f800000u ? b : 0u);
        }
      }
    }
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < 8; ++w) m = max(m, red[w]);
    uint32_t* words = reinterpret_cast<uint32_t*>(out);
    atomicMax(words, m);
    __threadfence();
    if (atomicAdd(words + 1, 1u) == gridDim.x - 1) {
      __threadfence();
      m = atomicMax(words, 0u);
      // amax = 2^e * 1.frac; 2688 = 2^11 * 1.3125 (fraction bits 0x280000)
      int e = (int)(m >> 23) - 127 - 11 + ((m & 0x7fffffu) > 0x280000u ? 1 : 0);
      e = max(e, -126);
      out[1] = m ? __uint_as_float((uint32_t)(e + 127) << 23) : 1.f;
    }
  }
}

// ---------------------------------------------------------------------------- rows and columns
// A lane holds a patch of 8 rows by PC columns, a warp 4 x 8 patches (32 rows by 8 PC columns), a
// CTA four warps below one another (128 rows). A patch gives whole 32-bit words of codes along its
// rows and along its columns, and the largest magnitude of a block is a shuffle over the two or
// four (gated: four or eight) lanes that share it, along either direction: the transposed operand
// needs no trip through shared memory, and a lane has eight loads in flight.
constexpr int kTileRows = 128;
constexpr int kTileThreads = 128;

struct Patch {
  long long r;  // first row
  int c;        // first column
  template <int PC>
  __device__ __forceinline__ static Patch of(int cols) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tiles_c = (((cols + 127) & ~127) + 8 * PC - 1) / (8 * PC);
    const unsigned tr = blockIdx.x / (unsigned)tiles_c, tc = blockIdx.x - tr * (unsigned)tiles_c;
    return Patch{(long long)tr * kTileRows + warp * 32 + (lane >> 3) * 8,
                 (int)tc * 8 * PC + (lane & 7) * PC};
  }
};

// Largest magnitude over the N lanes, a power of two, that share a block; `step` lanes apart.
template <int N>
__device__ __forceinline__ uint32_t lanes_max(uint32_t m, int step) {
#pragma unroll
  for (int o = 1; o < N; o *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, o * step));
  return m;
}

// Codes of PC = 8 or 4 consecutive elements.
template <int FMT, int PC>
__device__ __forceinline__ uint32_t codes_of(const float (&v)[PC], const Mx4Block& q,
                                             const Mx4Factor& f) {
  if constexpr (PC == 8) {
    return mx4_codes8<FMT>(v, q, f);
  } else {
    const float w[8] = {v[0], v[1], v[2], v[3], 0.f, 0.f, 0.f, 0.f};
    return mx4_codes8<FMT>(w, q, f);
  }
}

// Row-wise operand: row i of the patch, v its PC elements, m their largest magnitude's bits.
template <int FMT, int PC>
__device__ __forceinline__ void put_row(const float (&v)[PC], uint32_t m, uint8_t* codes,
                                        uint8_t* scale, bool ok, bool first, const Mx4Factor& f) {
  const Mx4Block q = mx4_block<FMT>(lanes_max<Mx4Fmt<FMT>::kBlock / PC>(m, 1), f);
  const uint32_t w = codes_of<FMT, PC>(v, q, f);
  if (ok) {
    if constexpr (PC == 8)
      *reinterpret_cast<uint32_t*>(codes) = w;
    else
      *reinterpret_cast<uint16_t*>(codes) = (uint16_t)w;
    if (first) *scale = (uint8_t)q.byte;
  }
}
// Transposed operand: column j of the patch, v its eight elements.
template <int FMT>
__device__ __forceinline__ void put_col(const float (&v)[8], uint32_t m, uint8_t* codes,
                                        uint8_t* scale, bool ok, bool first, const Mx4Factor& f) {
  const Mx4Block q = mx4_block<FMT>(lanes_max<Mx4Fmt<FMT>::kBlock / 8>(m, 8), f);
  const uint32_t w = mx4_codes8<FMT>(v, q, f);
  if (ok) {
    *reinterpret_cast<uint32_t*>(codes) = w;
    if (first) *scale = (uint8_t)q.byte;
  }
}

// Addresses of a patch in one operand: rows (columns) i of the patch follow each other by `ld / 2`
// bytes of codes and 16 bytes of scales (the eight lie in one group of 32).
struct PatchOut {
  uint8_t *codes, *scale;
  long long step;
  bool first;  // this lane writes the block's scale
  template <int FMT>
  __device__ __forceinline__ static PatchOut of(const Mx4Out& o, long long row, long long col) {
    return PatchOut{o.codes + (row * o.ld + col) / 2,
                    o.scales + mx4_scale_off<FMT>(row, (int)(col / Mx4Fmt<FMT>::kBlock), o.ld),
                    o.ld / 2, col % Mx4Fmt<FMT>::kBlock == 0};
  }
};

template <int FMT, typename T, bool ROWS, bool COLS>
__global__ void __launch_bounds__(kTileThreads)
    mx4_quantize_kernel(int rows, int cols, const T* __restrict__ x, long long ldx, bool vec,
                        const float* __restrict__ factor, Mx4Out out, Mx4Out out_t) {
  grid_dependency_wait();
  const Patch p = Patch::of<8>(cols);
  if (!COLS && p.r - (threadIdx.x & 24) >= rows) return;  // the whole warp is behind the last row
  const int kp = (cols + 127) & ~127;
  Vec8<T> w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) load8(w[i], x + (p.r + i) * ldx, p.c, cols, p.r + i < rows, vec);
  const Mx4Factor f = mx4_factor<FMT>(factor);
  if constexpr (ROWS) {
    const PatchOut o = PatchOut::of<FMT>(out, p.r, p.c);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v[8];
      w[i].get(v);
      put_row<FMT, 8>(v, w[i].amax(), o.codes + i * o.step, o.scale + 16 * i,
                      p.r + i < rows && p.c < kp, o.first, f);
    }
  }
  if constexpr (COLS) {
    const PatchOut o = PatchOut::of<FMT>(out_t, p.c, p.r);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float v[8];
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = w[i].at(j);
        m = max(m, abs_bits(v[i]));
      }
      put_col<FMT>(v, m, o.codes + j * o.step, o.scale + 16 * j, p.c + j < cols, o.first, f);
    }
  }
}

// ---------------------------------------------------------------------------- gated backward
// From da = dL/da and u = [gate | up]: dg = da * up * act'(gate), dup = da * act(gate), and
// a = act(gate) * up again. dg and dup leave quantised along the rows (for dX) and along the
// columns (for dW1), a along the columns (for dW2); none of them is written in 16 bits. Patches of
// 8 x 4: three results of 32 values stay in registers.
struct Quad {  // four consecutive bf16
  uint2 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int c, int cols, bool row_ok,
                                       bool vec) {
    a = make_uint2(0, 0);
    if (!row_ok || c >= cols) return;
    if (vec && c + 4 <= cols) {
      a = __ldg(reinterpret_cast<const uint2*>(row + c));
    } else {
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = c + i < cols ? __bfloat16_as_ushort(row[c + i]) : 0;
      a = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    }
  }
  __device__ __forceinline__ float at(int j) const {
    const uint32_t w = j < 2 ? a.x : a.y;
    return j & 1 ? bf16_hi(w) : bf16_lo(w);
  }
};

template <int FMT>
__device__ __forceinline__ void put_patch_rows(const float (&v)[8][4], const Mx4Out& out,
                                               const Patch& p, int rows, const Mx4Factor& f) {
  const PatchOut o = PatchOut::of<FMT>(out, p.r, p.c);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t m = max(max(abs_bits(v[i][0]), abs_bits(v[i][1])),
                           max(abs_bits(v[i][2]), abs_bits(v[i][3])));
    put_row<FMT, 4>(v[i], m, o.codes + i * o.step, o.scale + 16 * i, p.r + i < rows, o.first, f);
  }
}
template <int FMT>
__device__ __forceinline__ void put_patch_cols(const float (&v)[8][4], const Mx4Out& out,
                                               const Patch& p, int cols, const Mx4Factor& f) {
  const PatchOut o = PatchOut::of<FMT>(out, p.c, p.r);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float c[8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = v[i][j];
      m = max(m, abs_bits(c[i]));
    }
    put_col<FMT>(c, m, o.codes + j * o.step, o.scale + 16 * j, p.c + j < cols, o.first, f);
  }
}

template <int FMT>
__global__ void __launch_bounds__(kTileThreads)
    mx4_gated_bwd_kernel(int rows, int F, int act, const __nv_bfloat16* __restrict__ da,
                         long long ldda, bool vec_da, const __nv_bfloat16* __restrict__ u,
                         long long ldu, bool vec_g, bool vec_u, const float* __restrict__ f_du,
                         const float* __restrict__ f_dut, const float* __restrict__ f_at,
                         Mx4Out dg, Mx4Out dup, Mx4Out dgt, Mx4Out dupt, Mx4Out at) {
  grid_dependency_wait();
  const Patch p = Patch::of<4>(F);
  Quad wd[8], wg[8], wu[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const long long row = p.r + i;
    wd[i].load(da + row * ldda, p.c, F, row < rows, vec_da);
    wg[i].load(u + row * ldu, p.c, F, row < rows, vec_g);
    wu[i].load(u + row * ldu + F, p.c, F, row < rows, vec_u);
  }
  float g[8][4], q[8][4], a[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float h, dh;
      gate_and_grad(wg[i].at(j), act, h, dh);
      const float d = wd[i].at(j), up = wu[i].at(j);
      g[i][j] = d * up * dh;
      q[i][j] = d * h;
      a[i][j] = h * up;
    }
  if (dg.codes) {
    const Mx4Factor f = mx4_factor<FMT>(f_du);
    put_patch_rows<FMT>(g, dg, p, rows, f);
    put_patch_rows<FMT>(q, dup, p, rows, f);
  }
  if (dgt.codes) {
    const Mx4Factor f = mx4_factor<FMT>(f_dut);
    put_patch_cols<FMT>(g, dgt, p, F, f);
    put_patch_cols<FMT>(q, dupt, p, F, f);
  }
  if (at.codes) put_patch_cols<FMT>(a, at, p, F, mx4_factor<FMT>(f_at));
}

// ---------------------------------------------------------------------------- and back
// A lane decodes eight columns of eight rows, four rows apart, so that a warp's stores cover 128
// consecutive bytes (bf16) of four rows.
template <int FMT, typename T>
__global__ void __launch_bounds__(kTileThreads)
    mx4_dequantize_kernel(int rows, int cols, const uint8_t* __restrict__ codes,
                          const uint8_t* __restrict__ scales, long long ld,
                          const float* __restrict__ factor, T* __restrict__ y, long long ldy,
                          bool vec) {
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tiles_c = (cols + 63) / 64;
  const unsigned tr = blockIdx.x / (unsigned)tiles_c, tc = blockIdx.x - tr * (unsigned)tiles_c;
  const long long r0 = (long long)tr * kTileRows + warp * 32;
  const int c = (int)tc * 64 + (lane & 7) * 8;
  if (r0 >= rows || c >= cols) return;
  const float f = FMT == kNvfp4 ? factor[1] : 1.f;
  const int lr = lane >> 3;
  const uint8_t* cp = codes + ((r0 + lr) * ld + c) / 2;
  const uint8_t* sp = scales + mx4_scale_off<FMT>(r0 + lr, c / Mx4Fmt<FMT>::kBlock, ld);
  uint32_t w[8], sb[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool ok = r0 + lr + 4 * i < rows;
    w[i] = ok ? __ldg(reinterpret_cast<const uint32_t*>(cp + i * 2 * ld)) : 0;
    sb[i] = ok ? __ldg(sp + 64 * i) : 0;
  }
  T* o = y + (r0 + lr) * ldy + c;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (r0 + lr + 4 * i >= rows) break;
    const float s = mx4_scale_value<FMT>(sb[i]) * f;
    float v[8];
    e2m1x8_values(w[i], v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= s;
    T* e = o + (long long)(4 * i) * ldy;
    if (vec && c + 8 <= cols) {
      if constexpr (sizeof(T) == 2) {
        uint4 b;
        b.x = pack_bf16x2(v[0], v[1]);
        b.y = pack_bf16x2(v[2], v[3]);
        b.z = pack_bf16x2(v[4], v[5]);
        b.w = pack_bf16x2(v[6], v[7]);
        *reinterpret_cast<uint4*>(e) = b;
      } else {
        reinterpret_cast<float4*>(e)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(e)[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < cols) {
          if constexpr (sizeof(T) == 2)
            e[k] = __float2bfloat16_rn(v[k]);
          else
            e[k] = v[k];
        }
    }
  }
}

bool row_vec(const void* p, long long ld, int esz) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * esz) % 16 == 0;
}

unsigned grid_for(unsigned long long items, unsigned long long per_block, int num_sms,
                  int per_sm) {
  const unsigned long long want = (items + per_block - 1) / per_block;
  const unsigned long long most = (unsigned long long)num_sms * per_sm;
  return (unsigned)(want < most ? want : most);
}

// CTAs of a patch kernel: whole tiles of 128 rows, so that the transposed operand's padding is
// written, and columns up to the next multiple of 128.
unsigned tile_grid(int rows, int cols, int tile_cols) {
  const long long kp = ((long long)cols + 127) & ~127ll;
  return (unsigned)((((long long)rows + kTileRows - 1) / kTileRows) *
                    ((kp + tile_cols - 1) / tile_cols));
}

template <int FMT, typename T>
cudaError_t quantize_t(int rows, int cols, const T* x, long long ldx, const float* factor,
                       const Mx4Out& out, const Mx4Out& out_t, cudaStream_t s) {
  const bool vec = row_vec(x, ldx, sizeof(T));
  auto k = !out_t.codes ? mx4_quantize_kernel<FMT, T, true, false>
           : out.codes  ? mx4_quantize_kernel<FMT, T, true, true>
                        : mx4_quantize_kernel<FMT, T, false, true>;
  return launch_kernel(true, k, dim3(tile_grid(rows, cols, 64)), dim3(kTileThreads), 0, s, rows,
                       cols, x, ldx, vec, factor, out, out_t);
}

template <int FMT, typename T>
cudaError_t dequantize_t(int rows, int cols, const Mx4Out& q, const float* factor, T* y,
                         long long ldy, cudaStream_t s) {
  const long long tiles = (((long long)rows + kTileRows - 1) / kTileRows) * ((cols + 63) / 64);
  return launch_kernel(true, mx4_dequantize_kernel<FMT, T>, dim3((unsigned)tiles),
                       dim3(kTileThreads), 0, s, rows, cols, (const uint8_t*)q.codes,
                       (const uint8_t*)q.scales, q.ld, factor, y, ldy,
                       row_vec(y, ldy, sizeof(T)));
}

}  // namespace

cudaError_t launch_mx4_factor(int dtype, int rows, int cols, const void* x, long long ldx,
                              float* out, int num_sms, cudaStream_t s) {
  cudaError_t e = cudaMemsetAsync(out, 0, 2 * sizeof(float), s);
  if (e != cudaSuccess) return e;
  const unsigned long long n = (unsigned long long)rows * ((cols + 7) / 8);
  const dim3 grid(grid_for(n, 256 * 4, num_sms, 8));
  if (dtype)
    mx4_factor_kernel<<<grid, 256, 0, s>>>(rows, cols, (const __nv_bfloat16*)x, ldx,
                                           row_vec(x, ldx, 2), out);
  else
    mx4_factor_kernel<<<grid, 256, 0, s>>>(rows, cols, (const float*)x, ldx, row_vec(x, ldx, 4),
                                           out);
  return cudaGetLastError();
}

cudaError_t launch_mx4_quantize(int fmt, int dtype, int rows, int cols, const void* x,
                                long long ldx, const float* factor, const Mx4Out& out,
                                const Mx4Out& out_t, cudaStream_t s) {
  const __nv_bfloat16* b = (const __nv_bfloat16*)x;
  const float* f = (const float*)x;
  if (fmt == kMxfp4)
    return dtype ? quantize_t<kMxfp4>(rows, cols, b, ldx, factor, out, out_t, s)
                 : quantize_t<kMxfp4>(rows, cols, f, ldx, factor, out, out_t, s);
  return dtype ? quantize_t<kNvfp4>(rows, cols, b, ldx, factor, out, out_t, s)
               : quantize_t<kNvfp4>(rows, cols, f, ldx, factor, out, out_t, s);
}

cudaError_t launch_mx4_dequantize(int fmt, int dtype, int rows, int cols, const Mx4Out& q,
                                  const float* factor, void* y, long long ldy, cudaStream_t s) {
  __nv_bfloat16* b = (__nv_bfloat16*)y;
  float* f = (float*)y;
  if (fmt == kMxfp4)
    return dtype ? dequantize_t<kMxfp4>(rows, cols, q, factor, b, ldy, s)
                 : dequantize_t<kMxfp4>(rows, cols, q, factor, f, ldy, s);
  return dtype ? dequantize_t<kNvfp4>(rows, cols, q, factor, b, ldy, s)
               : dequantize_t<kNvfp4>(rows, cols, q, factor, f, ldy, s);
}

cudaError_t launch_mx4_gated_bwd(int fmt, int act, int rows, int F, const void* da,
                                 long long ldda, const void* u, long long ldu, const float* f_du,
                                 const float* f_dut, const float* f_at, const Mx4Out& dg,
                                 const Mx4Out& dup, const Mx4Out& dgt, const Mx4Out& dupt,
                                 const Mx4Out& at, cudaStream_t s) {
  const __nv_bfloat16* db = (const __nv_bfloat16*)da;
  const __nv_bfloat16* ub = (const __nv_bfloat16*)u;
  auto k = fmt == kMxfp4 ? mx4_gated_bwd_kernel<kMxfp4> : mx4_gated_bwd_kernel<kNvfp4>;
  auto vec = [](const void* p, long long ld) {  // loads of four bf16
    return (reinterpret_cast<uintptr_t>(p) & 7) == 0 && ld % 4 == 0;
  };
  return launch_kernel(true, k, dim3(tile_grid(rows, F, 32)), dim3(kTileThreads), 0, s, rows, F,
                       act, db, ldda, vec(db, ldda), ub, ldu, vec(ub, ldu), vec(ub + F, ldu), f_du,
                       f_dut, f_at, dg, dup, dgt, dupt, at);
}

}  // namespace mgt
