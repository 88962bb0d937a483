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

__device__ __forceinline__ uint32_t amax8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
  return m;
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

// Eight elements of a row (v: their values, m: the largest magnitude's bits) into the row-wise
// operand; a block's lanes are neighbours: 4 (mxfp4) or 2 (nvfp4).
template <int FMT>
__device__ __forceinline__ void store_row8(const float (&v)[8], uint32_t m, const Mx4Out& o,
                                           long long row, int col, bool ok, const Mx4Factor& f) {
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  if (FMT == kMxfp4) m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const Mx4Block q = mx4_block<FMT>(m, f);
  const uint32_t codes = mx4_codes8<FMT>(v, q, f);
  if (ok) {
    *reinterpret_cast<uint32_t*>(o.codes + (row * o.ld + col) / 2) = codes;
    if (col % Mx4Fmt<FMT>::kBlock == 0)
      o.scales[mx4_scale_off<FMT>(row, col / Mx4Fmt<FMT>::kBlock, o.ld)] = (uint8_t)q.byte;
  }
}
template <int FMT, typename T>
__device__ __forceinline__ void store_row8(const Vec8<T>& w, const Mx4Out& o, long long row,
                                           int col, bool ok, const Mx4Factor& f) {
  float v[8];
  w.get(v);
  store_row8<FMT>(v, w.amax(), o, row, col, ok, f);
}

// ---------------------------------------------------------------------------- rows only
// A warp takes 256 columns of a row, a lane eight of them (16 bytes of bf16); a block's maximum
// is a shuffle over 4 (mxfp4) or 2 (nvfp4) lanes. Four such items are loaded before the first
// is used, so a full grid keeps 64 KB of bf16 in flight per SM.
template <int FMT, typename T>
__global__ void __launch_bounds__(256)
    mx4_rows_kernel(int rows, int cols, const T* __restrict__ x, long long ldx, bool vec,
                    const float* __restrict__ factor, Mx4Out out) {
  constexpr int U = 4;
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int kp = (cols + 127) & ~127;
  const Mx4Factor f = mx4_factor<FMT>(factor);
  Walk at(blockIdx.x * 8ull + (threadIdx.x >> 5), gridDim.x * 8ull, (kp + 255) / 256);
  while (at.row < rows) {
    Vec8<T> w[U];
    long long row[U];
    int col[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      row[u] = at.row;
      col[u] = at.g * 256 + lane * 8;
      load8(w[u], x + row[u] * ldx, col[u], cols, row[u] < rows, vec);
      at.step();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) store_row8<FMT>(w[u], out, row[u], col[u], row[u] < rows && col[u] < kp, f);
  }
}

// ---------------------------------------------------------------------------- rows and columns
// A CTA takes 64 rows by 128 columns. Sixteen threads hold a row (eight columns each): they
// quantise along the row from registers and put the values into shared memory, from where a
// thread takes 16 rows of two neighbouring columns and quantises along the column; for mxfp4 two
// lanes 16 apart share a block of 32 rows. 64 rows are 32 bytes of a transposed row: one whole
// sector.
constexpr int kTR = 64, kTC = 128;

// Columns c, c + 1 (rows r .. r + 15, values in v[column][row]) into the transposed operand.
template <int FMT>
__device__ __forceinline__ void store_col16(float (&v)[2][16], const Mx4Out& o, long long r, int c,
                                            int cols, const uint32_t (&amax)[2],
                                            const Mx4Factor& f) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t m = amax[k];
    if (FMT == kMxfp4) m = max(m, __shfl_xor_sync(0xffffffffu, m, 16));
    const Mx4Block q = mx4_block<FMT>(m, f);
    float a[8], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] = v[k][i];
      b[i] = v[k][8 + i];
    }
    const uint2 w = make_uint2(mx4_codes8<FMT>(a, q, f), mx4_codes8<FMT>(b, q, f));
    if (c + k < cols) {
      *reinterpret_cast<uint2*>(o.codes + ((long long)(c + k) * o.ld + r) / 2) = w;
      if (r % Mx4Fmt<FMT>::kBlock == 0)
        o.scales[mx4_scale_off<FMT>(c + k, (int)(r / Mx4Fmt<FMT>::kBlock), o.ld)] =
            (uint8_t)q.byte;
    }
  }
}

// Shared-memory tile of one matrix. bf16: words of two columns, the halves of a 64-word row
// swapped on every other group of 16 rows, so that the two half-warps, 16 rows apart, read
// different banks. fp32: plain rows (a half-warp reads 128 bytes).
template <typename T>
__device__ __forceinline__ void tile_put(uint8_t* s, int r, int c8, const Vec8<T>& w) {
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(s + (r * 64 + ((c8 * 4) ^ ((r & 16)))) * 4) = w.a;
  } else {
    float4* d = reinterpret_cast<float4*>(s + (r * 128 + c8 * 8) * 4);
    d[0] = w.a;
    d[1] = w.b;
  }
}
template <typename T>
__device__ __forceinline__ void tile_get16(const uint8_t* s, int r, int cp, float (&v)[2][16],
                                           uint32_t (&amax)[2]) {
  uint32_t m = 0;
  amax[0] = amax[1] = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if constexpr (sizeof(T) == 2) {
      const uint32_t w =
          *reinterpret_cast<const uint32_t*>(s + ((r + i) * 64 + (cp ^ (r & 16))) * 4);
      v[0][i] = bf16_lo(w);
      v[1][i] = bf16_hi(w);
      m = max_u16x2(m, w & 0x7fff7fffu);
    } else {
      const float2 w = *reinterpret_cast<const float2*>(s + ((r + i) * 128 + 2 * cp) * 4);
      v[0][i] = w.x;
      v[1][i] = w.y;
      amax[0] = max(amax[0], abs_bits(w.x));
      amax[1] = max(amax[1], abs_bits(w.y));
    }
  }
  if constexpr (sizeof(T) == 2) {
    amax[0] = m << 16;
    amax[1] = m & 0xffff0000u;
  }
}

template <int FMT, typename T>
__global__ void __launch_bounds__(256)
    mx4_both_kernel(int rows, int cols, const T* __restrict__ x, long long ldx, bool vec,
                    const float* __restrict__ factor, Mx4Out out, Mx4Out out_t) {
  __shared__ __align__(16) uint8_t tile[kTR * kTC * sizeof(T)];
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tiles_c = (cols + kTC - 1) / kTC;
  const int c0 = (int)(blockIdx.x % tiles_c) * kTC;
  const long long r0 = (long long)(blockIdx.x / tiles_c) * kTR;
  const Mx4Factor f = mx4_factor<FMT>(factor);
  const int c8 = threadIdx.x & 15, rr = threadIdx.x >> 4;
  Vec8<T> w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const long long row = r0 + k * 16 + rr;
    load8(w[k], x + row * ldx, c0 + c8 * 8, cols, row < rows, vec);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const long long row = r0 + k * 16 + rr;
    tile_put(tile, k * 16 + rr, c8, w[k]);
    if (out.codes) store_row8<FMT>(w[k], out, row, c0 + c8 * 8, row < rows, f);
  }
  __syncthreads();
  const int cp = (warp & 3) * 16 + (lane & 15);
  const int r = (warp >> 2) * 32 + (lane >> 4) * 16;
  float v[2][16];
  uint32_t m[2];
  tile_get16<T>(tile, r, cp, v, m);
  store_col16<FMT>(v, out_t, r0 + r, c0 + 2 * cp, cols, m, f);
}

// ---------------------------------------------------------------------------- gated backward
// From da = dL/da and u = [gate | up]: dg = da * up * act'(gate), dup = da * act(gate), and
// a = act(gate) * up again. dg and dup leave quantised along the rows (for dX) and along the
// columns (for dW1), a along the columns (for dW2); none of them is written in 16 bits.
template <int FMT>
__global__ void __launch_bounds__(256)
    mx4_gated_bwd_kernel(int rows, int F, int act, const __nv_bfloat16* __restrict__ da,
                         long long ldda, bool vec_da, const __nv_bfloat16* __restrict__ u,
                         long long ldu, bool vec_g, bool vec_u, const float* __restrict__ f_du,
                         const float* __restrict__ f_dut, const float* __restrict__ f_at,
                         Mx4Out dg, Mx4Out dup, Mx4Out dgt, Mx4Out dupt, Mx4Out at) {
  extern __shared__ __align__(16) uint8_t tiles[];
  constexpr int kTile = kTR * kTC * 4;
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tiles_c = (F + kTC - 1) / kTC;
  const int c0 = (int)(blockIdx.x % tiles_c) * kTC;
  const long long r0 = (long long)(blockIdx.x / tiles_c) * kTR;
  const Mx4Factor if_du = mx4_factor<FMT>(dg.codes ? f_du : nullptr);
  const Mx4Factor if_dut = mx4_factor<FMT>(dgt.codes ? f_dut : nullptr);
  const Mx4Factor if_at = mx4_factor<FMT>(at.codes ? f_at : nullptr);
  const int c8 = threadIdx.x & 15, rr = threadIdx.x >> 4;
  const int col = c0 + c8 * 8;
  Vec8<__nv_bfloat16> wd[4], wg[4], wu[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const long long row = r0 + k * 16 + rr;
    load8(wd[k], da + row * ldda, col, F, row < rows, vec_da);
    load8(wg[k], u + row * ldu, col, F, row < rows, vec_g);
    load8(wu[k], u + row * ldu + F, col, F, row < rows, vec_u);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const long long row = r0 + k * 16 + rr;
    float d[8], g[8], p[8], a[8];
    wd[k].get(d);
    wg[k].get(g);
    wu[k].get(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float h, dh;
      gate_and_grad(g[i], act, h, dh);
      a[i] = h * p[i];
      g[i] = d[i] * p[i] * dh;
      p[i] = d[i] * h;
    }
    const int at_row = (k * 16 + rr) * 128 + c8 * 8;
    float4* s = reinterpret_cast<float4*>(tiles + at_row * 4);
    s[0] = make_float4(g[0], g[1], g[2], g[3]);
    s[1] = make_float4(g[4], g[5], g[6], g[7]);
    s = reinterpret_cast<float4*>(tiles + kTile + at_row * 4);
    s[0] = make_float4(p[0], p[1], p[2], p[3]);
    s[1] = make_float4(p[4], p[5], p[6], p[7]);
    s = reinterpret_cast<float4*>(tiles + 2 * kTile + at_row * 4);
    s[0] = make_float4(a[0], a[1], a[2], a[3]);
    s[1] = make_float4(a[4], a[5], a[6], a[7]);
    if (dg.codes) {
      store_row8<FMT>(g, amax8(g), dg, row, col, row < rows, if_du);
      store_row8<FMT>(p, amax8(p), dup, row, col, row < rows, if_du);
    }
  }
  __syncthreads();
  const int cp = (warp & 3) * 16 + (lane & 15);
  const int r = (warp >> 2) * 32 + (lane >> 4) * 16;
  float v[2][16];
  uint32_t m[2];
  if (dgt.codes) {
    tile_get16<float>(tiles, r, cp, v, m);
    store_col16<FMT>(v, dgt, r0 + r, c0 + 2 * cp, F, m, if_dut);
    tile_get16<float>(tiles + kTile, r, cp, v, m);
    store_col16<FMT>(v, dupt, r0 + r, c0 + 2 * cp, F, m, if_dut);
  }
  if (at.codes) {
    tile_get16<float>(tiles + 2 * kTile, r, cp, v, m);
    store_col16<FMT>(v, at, r0 + r, c0 + 2 * cp, F, m, if_at);
  }
}

// ---------------------------------------------------------------------------- and back
template <int FMT, typename T>
__global__ void __launch_bounds__(256)
    mx4_dequantize_kernel(int rows, int cols, const uint8_t* __restrict__ codes,
                          const uint8_t* __restrict__ scales, long long ld,
                          const float* __restrict__ factor, T* __restrict__ y, long long ldy,
                          bool vec) {
  grid_dependency_wait();
  const float f = FMT == kNvfp4 ? factor[1] : 1.f;
  for (Walk at(blockIdx.x * 256ull + threadIdx.x, gridDim.x * 256ull, (cols + 7) / 8);
       at.row < rows; at.step()) {
    const long long r = at.row;
    const int c = at.g * 8;
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(codes + (r * ld + c) / 2));
    const float s =
        mx4_scale_value<FMT>(__ldg(scales + mx4_scale_off<FMT>(r, c / Mx4Fmt<FMT>::kBlock, ld))) *
        f;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // magnitude code: 0, 0.5, then 1.m * 2^(e - 1)
      const uint32_t c4 = w >> (4 * k), mag = c4 & 7u;
      const float a = mag < 2 ? 0.5f * mag
                              : __uint_as_float((((mag >> 1) + 126u) << 23) | ((mag & 1u) << 22));
      v[k] = (c4 & 8u ? -a : a) * s;
    }
    T* o = y + r * ldy + c;
    if (vec && c + 8 <= cols) {
      if constexpr (sizeof(T) == 2) {
        uint4 p;
        p.x = pack_bf16x2(v[0], v[1]);
        p.y = pack_bf16x2(v[2], v[3]);
        p.z = pack_bf16x2(v[4], v[5]);
        p.w = pack_bf16x2(v[6], v[7]);
        *reinterpret_cast<uint4*>(o) = p;
      } else {
        reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < cols) {
          if constexpr (sizeof(T) == 2)
            o[k] = __float2bfloat16_rn(v[k]);
          else
            o[k] = v[k];
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

// Tiles of 64 rows by 128 columns; the rows are covered up to a multiple of 128, so that the
// transposed operand's padding is written.
unsigned tile_grid(int rows, int cols) {
  return (unsigned)((((long long)rows + 127) / 128) * (128 / kTR) * ((cols + kTC - 1) / kTC));
}

template <typename T>
cudaError_t quantize_t(int fmt, int rows, int cols, const T* x, long long ldx,
                       const float* factor, const Mx4Out& out, const Mx4Out& out_t, int num_sms,
                       cudaStream_t s) {
  const bool vec = row_vec(x, ldx, sizeof(T));
  if (out_t.codes) {
    const dim3 grid(tile_grid(rows, cols));
    auto k = fmt == kMxfp4 ? mx4_both_kernel<kMxfp4, T> : mx4_both_kernel<kNvfp4, T>;
    return launch_kernel(true, k, grid, dim3(256), 0, s, rows, cols, x, ldx, vec, factor, out,
                         out_t);
  }
  const unsigned long long items = (unsigned long long)rows * ((cols + 255) / 256);
  auto k = fmt == kMxfp4 ? mx4_rows_kernel<kMxfp4, T> : mx4_rows_kernel<kNvfp4, T>;
  return launch_kernel(true, k, dim3(grid_for(items, 8, num_sms, 8)), dim3(256), 0, s, rows, cols,
                       x, ldx, vec, factor, out);
}

template <typename T>
cudaError_t dequantize_t(int fmt, int rows, int cols, const Mx4Out& q, const float* factor, T* y,
                         long long ldy, int num_sms, cudaStream_t s) {
  const unsigned long long n = (unsigned long long)rows * ((cols + 7) / 8);
  auto k = fmt == kMxfp4 ? mx4_dequantize_kernel<kMxfp4, T> : mx4_dequantize_kernel<kNvfp4, T>;
  return launch_kernel(true, k, dim3(grid_for(n, 256, num_sms, 8)), dim3(256), 0, s, rows, cols,
                       (const uint8_t*)q.codes, (const uint8_t*)q.scales, q.ld, factor, y, ldy,
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
                                const Mx4Out& out_t, int num_sms, cudaStream_t s) {
  if (dtype)
    return quantize_t(fmt, rows, cols, (const __nv_bfloat16*)x, ldx, factor, out, out_t, num_sms,
                      s);
  return quantize_t(fmt, rows, cols, (const float*)x, ldx, factor, out, out_t, num_sms, s);
}

cudaError_t launch_mx4_dequantize(int fmt, int dtype, int rows, int cols, const Mx4Out& q,
                                  const float* factor, void* y, long long ldy, int num_sms,
                                  cudaStream_t s) {
  if (dtype) return dequantize_t(fmt, rows, cols, q, factor, (__nv_bfloat16*)y, ldy, num_sms, s);
  return dequantize_t(fmt, rows, cols, q, factor, (float*)y, ldy, num_sms, s);
}

cudaError_t launch_mx4_gated_bwd(int fmt, int act, int rows, int F, const void* da,
                                 long long ldda, const void* u, long long ldu, const float* f_du,
                                 const float* f_dut, const float* f_at, const Mx4Out& dg,
                                 const Mx4Out& dup, const Mx4Out& dgt, const Mx4Out& dupt,
                                 const Mx4Out& at, cudaStream_t s) {
  const __nv_bfloat16* ub = (const __nv_bfloat16*)u;
  auto k = fmt == kMxfp4 ? mx4_gated_bwd_kernel<kMxfp4> : mx4_gated_bwd_kernel<kNvfp4>;
  constexpr int smem = 3 * kTR * kTC * 4;
  static SmemLimit limit[2];
  cudaError_t e = limit[fmt].allow(k, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid(tile_grid(rows, F));
  return launch_kernel(true, k, grid, dim3(256), (size_t)smem, s, rows, F, act,
                       (const __nv_bfloat16*)da, ldda, row_vec(da, ldda, 2), ub, ldu,
                       row_vec(u, ldu, 2), row_vec(ub + F, ldu, 2), f_du, f_dut, f_at, dg, dup,
                       dgt, dupt, at);
}

}  // namespace mgt
