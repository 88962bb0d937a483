// Quantisers of the microscaled 4-bit formats (mx4_device.cuh): tensor factor, quantisation
// along the rows and, from the same read, along the columns (the transposed operand that the
// backward products sum over), the gated block's backward fused with both quantisations, and
// the way back to bf16 or fp32. All are bound by HBM: each element is read once.
#include "../../include/mgt_layer.h"
#include "mx4_device.cuh"
#include "mx4_internal.h"

namespace mgt {
namespace {

// Plain global loads, in program order with grid_dependency_wait(): the kernel before may still be
// writing these bytes while this one is already resident, so they are not read-only for its life
// and take neither the read-only path nor a place ahead of the wait.
__device__ __forceinline__ uint32_t ld4(const void* p) {
  uint32_t v;
  asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld8(const void* p) {
  uint2 v;
  asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld16(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ float4 as_float4(uint4 w) {
  return make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z),
                     __uint_as_float(w.w));
}

template <typename T>
struct Vec8;  // eight consecutive elements as loaded
template <>
struct Vec8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    a = ld16(p);
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
  // Rows of any alignment: the aligned words that hold the elements; one that starts at an odd
  // element takes a word more and is put together from neighbours. (Such a word holds an element
  // of its neighbours too, never anything but.)
  __device__ __forceinline__ void load_words(const __nv_bfloat16* p) {
    const uint32_t* w =
        reinterpret_cast<const uint32_t*>(reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)3);
    a = make_uint4(ld4(w), ld4(w + 1), ld4(w + 2), ld4(w + 3));
    if (reinterpret_cast<uintptr_t>(p) & 2) {
      const uint32_t e = ld4(w + 4);
      a.x = __byte_perm(a.x, a.y, 0x5432);
      a.y = __byte_perm(a.y, a.z, 0x5432);
      a.z = __byte_perm(a.z, a.w, 0x5432);
      a.w = __byte_perm(a.w, e, 0x5432);
    }
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
    a = as_float4(ld16(p));
    b = as_float4(ld16(p + 4));
  }
  __device__ __forceinline__ void load_words(const float* p) {
    a = as_float4(make_uint4(ld4(p), ld4(p + 1), ld4(p + 2), ld4(p + 3)));
    b = as_float4(make_uint4(ld4(p + 4), ld4(p + 5), ld4(p + 6), ld4(p + 7)));
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

// Groups of eight columns; cols may be any positive int (cols + 7 may not be one).
__host__ __device__ __forceinline__ int groups8(int cols) { return (cols - 1) / 8 + 1; }

// Eight elements from column c of a row of `cols`; zeros behind the last column. vec: the row
// base is 16-byte aligned (c is a multiple of 8). (c + 8 need not be an int.)
template <typename T>
__device__ __forceinline__ void load8(Vec8<T>& r, const T* row, int c, int cols, bool row_ok,
                                      bool vec) {
  if (!row_ok || c >= cols)
    r.zero();
  else if (vec && cols - c >= 8)
    r.load(row + c);
  else if (cols - c > 8)
    r.load_words(row + c);
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
// out[1], writes f over the count. Both words are zeroed by a launch before, of one thread:
// chained programmatically the two take 2.9 us for one row, with a memory set in its place 6.2.
// Bound by HBM: 4096 x 11008 fp32 29 us (6.2 TB/s), 8192 x 24576 bf16 61 us (6.6), 2048 x 4096
// bf16 6.4 us; rows that do not start on 16 bytes are read by words, 4096 x 11007 fp32 48 us, 8192
// x 24575 bf16 84, 2048 x 4095 bf16 9.9. 256 threads with
// four loads in flight, up to eight blocks per SM: no other shape tried was faster anywhere.
__global__ void mx4_zero2_kernel(float* out) {
  launch_dependents();
  grid_dependency_wait();
  out[0] = out[1] = 0.f;
}

template <typename T>
__global__ void __launch_bounds__(256) mx4_factor_kernel(int rows, int cols, const T* x,
                                                         long long ldx, bool vec, float* out) {
  __shared__ uint32_t red[8];
  launch_dependents();
  grid_dependency_wait();
  uint32_t m = 0;
  constexpr int U = 4;
  Walk at(blockIdx.x * 256ull + threadIdx.x, gridDim.x * 256ull, groups8(cols));
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
//
// Times (mxfp4 / nvfp4): bf16 along the rows 2048 x 4096 6.4 / 8.7 us, 8192 x 6144 26 / 34 us
// (4.8 TB/s / 3.7); bf16 both ways 2048 x 12288 22 / 27 us; fp32 both ways 4096 x 11008 48 / 49 us
// (4.8 TB/s). What bounds it is HBM for fp32 and, for bf16 and for nvfp4's quotients, the integer
// and fp32 instructions per element (both ways: 59 % of the ALU's peak, 2.4 instructions a clock
// and SM). Rows that do not start on 16 bytes are read by words: 2048 x 4095 bf16 9.4 / 13.9 us, with
// rows of 4101 in memory 2048 x 4096 10.0 / 14.2, fp32 both ways 4096 x 11007 64 / 65.
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

// Addresses of a patch in one operand: rows (columns) i of the patch follow each other by `step`
// bytes of codes and 16 bytes of scales (the eight lie in one group of 32).
struct PatchOut {
  uint8_t *codes, *scale;
  long long step;
  template <int FMT>
  __device__ __forceinline__ static PatchOut of(const Mx4Out& o, long long row, long long col,
                                                long long scale_col) {
    return PatchOut{o.codes + (row * o.ld + col) / 2,
                    o.scales + mx4_scale_off<FMT>(row, (int)(scale_col / Mx4Fmt<FMT>::kBlock), o.ld),
                    o.ld / 2};
  }
};

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  return __byte_perm(a, b, sel);
}

// Largest magnitudes (fp32 bits) of CNT rows or columns over the N lanes, `step` apart, that share
// a block. The upper halves of two of them travel in one word where they are enough: bf16 values
// have no more, and an mxfp4 scale is read from the exponent.
template <bool PACKED, int CNT, int N>
__device__ __forceinline__ void lanes_max(uint32_t (&m)[CNT], int step) {
  if constexpr (PACKED) {
#pragma unroll
    for (int i = 0; i < CNT; i += 2) {
      uint32_t k = prmt(m[i], m[i + 1], 0x7632);
#pragma unroll
      for (int o = 1; o < N; o *= 2) k = max_u16x2(k, __shfl_xor_sync(0xffffffffu, k, o * step));
      m[i] = k << 16;
      m[i + 1] = k & 0xffff0000u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < CNT; ++i)
#pragma unroll
      for (int o = 1; o < N; o *= 2)
        m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], o * step));
  }
}

// Patches: `pair` is elements (row i, columns 2 q and 2 q + 1), `each` replaces every element.
struct PatchBf16 {
  static constexpr int kCols = 8;
  Vec8<__nv_bfloat16> w[8];
  __device__ __forceinline__ uint32_t word(int i, int q) const {
    return q == 0 ? w[i].a.x : q == 1 ? w[i].a.y : q == 2 ? w[i].a.z : w[i].a.w;
  }
  __device__ __forceinline__ uint64_t pair(int i, int q) const {
    return f2_pack(bf16_lo(word(i, q)), bf16_hi(word(i, q)));
  }
  // Magnitudes two to a word: bf16 magnitudes order like their bits.
  __device__ __forceinline__ void max_bits(uint32_t (&rm)[8], uint32_t (&cm)[8]) const {
    uint32_t c[4] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t a[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        a[q] = word(i, q) & 0x7fff7fffu;
        c[q] = max_u16x2(c[q], a[q]);
      }
      const uint32_t m = max_u16x2(max_u16x2(a[0], a[1]), max_u16x2(a[2], a[3]));
      rm[i] = max(m << 16, m);  // only its upper half counts
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      cm[2 * q] = c[q] << 16;
      cm[2 * q + 1] = c[q];
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(F fn) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t* a[4] = {&w[i].a.x, &w[i].a.y, &w[i].a.z, &w[i].a.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) *a[q] = pack_bf16x2(fn(bf16_lo(*a[q])), fn(bf16_hi(*a[q])));
    }
  }
};
template <int PC>
struct PatchF32 {
  static constexpr int kCols = PC;
  float v[8][PC];
  __device__ __forceinline__ uint64_t pair(int i, int q) const {
    return f2_pack(v[i][2 * q], v[i][2 * q + 1]);
  }
  __device__ __forceinline__ void max_bits(uint32_t (&rm)[8], uint32_t (&cm)[PC]) const {
#pragma unroll
    for (int j = 0; j < PC; ++j) cm[j] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      rm[i] = 0;
#pragma unroll
      for (int j = 0; j < PC; ++j) {
        const uint32_t b = abs_bits(v[i][j]);
        rm[i] = max(rm[i], b);
        cm[j] = max(cm[j], b);
      }
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(F fn) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < PC; ++j) v[i][j] = fn(v[i][j]);
  }
};

// A pair scaled by a pair (mxfp4: exact; nvfp4: with the residual correction of mx4_scaled).
template <int FMT>
__device__ __forceinline__ void scaled2(uint64_t x, uint64_t inv, uint64_t neg_fs, float& a,
                                        float& b) {
  uint64_t y = f2_mul(x, inv);
  if constexpr (FMT == kNvfp4) y = f2_fma(f2_fma(y, neg_fs, x), inv, y);
  f2_unpack(y, a, b);
}

// Scale bytes of a warp's 32 rows (b: of this lane's eight rows, in its block): every lane writes one
// row's bytes, all NB blocks that the warp covers, as one store instead of eight by a few lanes
// each. Lane c of the eight along a row takes row c of the eight, and the other blocks' bytes of it
// from their lanes. `scale`: of the patch's first row, the warp's first block.
template <int NB>
__device__ __forceinline__ void put_row_scales(const uint32_t (&b)[8], uint8_t* scale, int nrows) {
  const int c = threadIdx.x & 7;
  const uint32_t lo = b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);
  const uint32_t hi = b[4] | (b[5] << 8) | (b[6] << 16) | (b[7] << 24);
  auto byte = [&](int row) { return ((row & 4 ? hi : lo) >> (8 * (row & 3))) & 255u; };
  const int mine = c / (8 / NB);
  uint32_t w = byte(c) << (8 * mine);
#pragma unroll
  for (int k = 1; k < NB; ++k) {
    const int x = k * (8 / NB);
    w |= __shfl_xor_sync(0xffffffffu, byte(c ^ x), x) << (8 * (mine ^ k));
  }
  if (c < nrows) {
    scale += 16 * c;
    if constexpr (NB == 4)
      *reinterpret_cast<uint32_t*>(scale) = w;
    else if constexpr (NB == 2)
      *reinterpret_cast<uint16_t*>(scale) = (uint16_t)w;
    else
      *scale = (uint8_t)w;
  }
}
// Scale bytes of this lane's PC columns (b): the G lanes that share the blocks write PC / G each.
template <int PC, int G>
__device__ __forceinline__ void put_col_scales(const uint32_t (&b)[PC], uint8_t* scale, int ncols) {
  constexpr int kEach = PC / G;
  const int g = (threadIdx.x >> 3) & (G - 1);
#pragma unroll
  for (int m = 0; m < kEach; ++m) {
    uint32_t v = b[m];
#pragma unroll
    for (int k = 1; k < G; ++k) v = g == k ? b[k * kEach + m] : v;
    const int j = g * kEach + m;
    if (j < ncols) scale[16 * j] = (uint8_t)v;
  }
}

// Quantise a patch along its rows (into `out`) and / or its columns (into `out_t`); an operand
// without codes, or that is switched off, is left out. f and ft may differ, but not be apart (see
// factors_apart).
template <int FMT, bool PACKED, bool ROWS, bool COLS, typename P>
__device__ __forceinline__ void quantize_patch(P& x, const Patch& p, int rows, int cols, int kp,
                                               const Mx4Out& out, const Mx4Out& out_t, Mx4Factor f,
                                               Mx4Factor ft, bool rows_on = true,
                                               bool cols_on = true) {
  constexpr int B = Mx4Fmt<FMT>::kBlock, PC = P::kCols;
  uint32_t rm[8], cm[PC];
  x.max_bits(rm, cm);
  if constexpr (ROWS) lanes_max<PACKED, 8, B / PC>(rm, 1);
  if constexpr (COLS) lanes_max<PACKED, PC, B / 8>(cm, 8);
  if constexpr (FMT == kNvfp4) {
    // Rare: a kept factor far too small (elements beyond 4096 f saturate wherever they lie, so
    // they may be cut off there before a quotient overflows), or a tiny one (see mx4_factor).
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, rm[i]);
    const float f0 = ROWS && COLS ? fmaxf(f.f, ft.f) : ROWS ? f.f : ft.f;
    const bool tiny = ROWS ? f.tiny : ft.tiny;  // (both or neither)
    if (tiny || m > __float_as_uint(4096.0f * f0)) {
      const float k = tiny ? kLift : 1.0f, lim = 4096.0f * (f0 * (1.0f / k));
      auto cut = [&](float v) { return fminf(fmaxf(v, -lim), lim) * k; };
      auto cut_bits = [&](uint32_t b) {
        return b >= 0x7f800000u ? b : __float_as_uint(fminf(__uint_as_float(b), lim) * k);
      };
      x.each(cut);
#pragma unroll
      for (int i = 0; i < 8; ++i) rm[i] = cut_bits(rm[i]);
#pragma unroll
      for (int j = 0; j < PC; ++j) cm[j] = cut_bits(cm[j]);
    }
  }
  // row scales: of the warp's first block; column scales: of this lane's
  const PatchOut o = PatchOut::of<FMT>(out, p.r, p.c, p.c - (threadIdx.x & 7) * PC);
  const PatchOut t = PatchOut::of<FMT>(out_t, p.c, p.r, p.r);
  const bool put_rows = ROWS && rows_on && out.codes && p.c < kp;
  const bool put_cols = COLS && cols_on && out_t.codes;
  uint64_t cinv[PC / 2], cfs[PC / 2];
  uint32_t cc[PC], cmask[PC];
  if constexpr (COLS) {
#pragma unroll
    for (int q = 0; q < PC / 2; ++q) {
      const Mx4Block a = mx4_block<FMT>(cm[2 * q], ft), b = mx4_block<FMT>(cm[2 * q + 1], ft);
      cinv[q] = f2_pack(a.inv, b.inv);
      cfs[q] = f2_pack(-a.fs, -b.fs);
      cmask[2 * q] = a.mask;
      cmask[2 * q + 1] = b.mask;
      cm[2 * q] = a.byte;
      cm[2 * q + 1] = b.byte;
    }
    put_col_scales<PC, B / 8>(cm, t.scale, put_cols ? cols - p.c : 0);
  }
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if constexpr (ROWS) {
        const Mx4Block s = mx4_block<FMT>(rm[i + h], f);
        const uint64_t inv = f2_pack(s.inv, s.inv), fs = f2_pack(-s.fs, -s.fs);
        float e[8];
#pragma unroll
        for (int q = 0; q < PC / 2; ++q)
          scaled2<FMT>(x.pair(i + h, q), inv, fs, e[2 * q], e[2 * q + 1]);
        if (put_rows && p.r + i + h < rows) {
          uint8_t* d = o.codes + (i + h) * o.step;
          if constexpr (PC == 8)
            *reinterpret_cast<uint32_t*>(d) = e2m1x8(e) & s.mask;
          else
            *reinterpret_cast<uint16_t*>(d) =
                (uint16_t)((e2m1x2(e[0], e[1]) | (e2m1x2(e[2], e[3]) << 8)) & s.mask);
        }
        rm[i + h] = s.byte;
      }
  }
  if constexpr (ROWS) {
    const long long left = rows - p.r;
    put_row_scales<8 * PC / B>(rm, o.scale, put_rows && left > 0 ? (int)(left < 8 ? left : 8) : 0);
  }
  if constexpr (COLS) {
#pragma unroll
    for (int q = 0; q < PC / 2; ++q) {
      float a[8], b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) scaled2<FMT>(x.pair(i, q), cinv[q], cfs[q], a[i], b[i]);
      cc[2 * q] = e2m1x8(a);
      cc[2 * q + 1] = e2m1x8(b);
    }
  }
  if constexpr (COLS) {
    if (put_cols) {
#pragma unroll
      for (int j = 0; j < PC; ++j)
        if (p.c + j < cols)
          *reinterpret_cast<uint32_t*>(t.codes + j * t.step) = cc[j] & cmask[j];
    }
  }
}

// (nvfp4 from fp32 both ways asks for four CTAs an SM, 128 registers: left alone it took 134 to 166.)
template <int FMT, typename T, bool ROWS, bool COLS>
__global__ void __launch_bounds__(kTileThreads, FMT == kNvfp4 && ROWS && COLS && sizeof(T) == 4 ? 4 : 0)
    mx4_quantize_kernel(int rows, int cols, const T* x, long long ldx, bool vec,
                        const float* factor, Mx4Out out, Mx4Out out_t) {
  launch_dependents();
  grid_dependency_wait();
  const Patch p = Patch::of<8>(cols);
  if (!COLS && p.r - (threadIdx.x & 24) >= rows) return;  // the whole warp is behind the last row
  const int kp = (cols + 127) & ~127;
  const Mx4Factor f = mx4_factor<FMT>(factor);
  constexpr bool kPacked = FMT == kMxfp4 || sizeof(T) == 2;
  if constexpr (sizeof(T) == 2) {
    PatchBf16 v;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      load8(v.w[i], x + (p.r + i) * ldx, p.c, cols, p.r + i < rows, vec);
    quantize_patch<FMT, kPacked, ROWS, COLS>(v, p, rows, cols, kp, out, out_t, f, f);
  } else {
    PatchF32<8> v;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      Vec8<T> w;
      load8(w, x + (p.r + i) * ldx, p.c, cols, p.r + i < rows, vec);
      w.get(v.v[i]);
    }
    quantize_patch<FMT, kPacked, ROWS, COLS>(v, p, rows, cols, kp, out, out_t, f, f);
  }
}

// ---------------------------------------------------------------------------- gated backward
// From da = dL/da and u = [gate | up]: dg = da * up * act'(gate), dup = da * act(gate), and
// a = act(gate) * up again. dg and dup leave quantised along the rows (for dX) and along the
// columns (for dW1), a along the columns (for dW2); none of them is written in 16 bits. Patches of
// 8 x 4: dg is quantised from registers while dup and a wait in shared memory, 16 bytes a lane,
// each lane its own. With all three in registers the same took 89 us instead of 81 (gelu 224
// instead of 124), and patches of 8 x 8 that read the inputs once per result 140.
//
// Bound by instructions (five quantisations an element: 55 % of the ALU's peak): 2048 x 11008 silu
// 76 / 93 us (mxfp4 / nvfp4; 195 MB, 2.6 TB/s), gelu 119 / 144, tanh gelu 99 / 118; 2048 x 11007 silu
// 136 / 153 (rows that do not start on eight bytes are read by words).
//
// du and dut have a factor each. Elements that saturate are cut off by the larger one (see
// quantize_patch), which is enough for the other as long as their quotient stays an fp32 number.
__device__ __forceinline__ bool factors_apart(const Mx4Factor& a, const Mx4Factor& b) {
  return a.tiny != b.tiny || fmaxf(a.f, b.f) > kLift * fminf(a.f, b.f);
}

struct Quad {  // four consecutive bf16
  uint2 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int c, int cols, bool row_ok,
                                       bool vec) {
    a = make_uint2(0, 0);
    if (!row_ok || c >= cols) return;
    if (vec && c + 4 <= cols) {
      a = ld8(row + c);
    } else if (c + 4 < cols) {  // the aligned words that hold them (see Vec8)
      const uintptr_t at = reinterpret_cast<uintptr_t>(row + c);
      const uint32_t* w = reinterpret_cast<const uint32_t*>(at & ~(uintptr_t)3);
      a = make_uint2(ld4(w), ld4(w + 1));
      if (at & 2) {
        a.x = prmt(a.x, a.y, 0x5432);
        a.y = prmt(a.y, ld4(w + 2), 0x5432);
      }
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

template <int FMT, int ACT>
__global__ void __launch_bounds__(kTileThreads, 4)
    mx4_gated_bwd_kernel(int rows, int F, const __nv_bfloat16* da,
                         long long ldda, bool vec_da, const __nv_bfloat16* u,
                         long long ldu, bool vec_g, bool vec_u, const float* f_du,
                         const float* f_dut, const float* f_at,
                         Mx4Out dg, Mx4Out dup, Mx4Out dgt, Mx4Out dupt, Mx4Out at) {
  __shared__ float4 kept[2][8][kTileThreads];
  grid_dependency_wait();
  const int kp = (F + 127) & ~127;
  if (!dg.codes) f_du = f_dut;
  if (!dgt.codes) f_dut = f_du;
  // Once, or where the factors are apart once for the rows and once for the columns.
#pragma unroll 1
  for (bool again = false;; again = true) {
    Patch p = Patch::of<4>(F);
    if (FMT == kNvfp4)  // (or all addresses are kept for the second turn)
      asm volatile("" : "+r"(p.c), "+l"(p.r));
    Quad wd[8], wg[8], wu[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const long long row = p.r + i;
      wd[i].load(da + row * ldda, p.c, F, row < rows, vec_da);
      wg[i].load(u + row * ldu, p.c, F, row < rows, vec_g);
      wu[i].load(u + row * ldu + F, p.c, F, row < rows, vec_u);
    }
    Mx4Factor fr = mx4_factor<FMT>(f_du), fc = mx4_factor<FMT>(f_dut);
    const bool apart = FMT == kNvfp4 && factors_apart(fr, fc);
    const bool rows_on = !again, cols_on = again || !apart;
    if (apart) (again ? fr : fc) = again ? fc : fr;
    PatchF32<4> v;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float b[4], a[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float h, dh;
        gate_and_grad<ACT>(wg[i].at(j), h, dh);
        const float d = wd[i].at(j), up = wu[i].at(j);
        v.v[i][j] = d * up * dh;
        b[j] = d * h;
        a[j] = h * up;
      }
      kept[0][i][threadIdx.x] = make_float4(b[0], b[1], b[2], b[3]);
      kept[1][i][threadIdx.x] = make_float4(a[0], a[1], a[2], a[3]);
    }
    asm volatile("" ::: "memory");  // (or the compiler keeps them in registers after all)
    auto take = [&](int k) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 w = kept[k][i][threadIdx.x];
        v.v[i][0] = w.x;
        v.v[i][1] = w.y;
        v.v[i][2] = w.z;
        v.v[i][3] = w.w;
      }
    };
    constexpr bool kPacked = FMT == kMxfp4;
    if (dg.codes || dgt.codes) {
      quantize_patch<FMT, kPacked, true, true>(v, p, rows, F, kp, dg, dgt, fr, fc, rows_on, cols_on);
      take(0);
      quantize_patch<FMT, kPacked, true, true>(v, p, rows, F, kp, dup, dupt, fr, fc, rows_on,
                                               cols_on);
    }
    if (!cols_on) continue;
    if (at.codes) {
      take(1);
      const Mx4Factor fa = mx4_factor<FMT>(f_at);
      quantize_patch<FMT, kPacked, false, true>(v, p, rows, F, kp, at, at, fa, fa);
    }
    return;
  }
}

// ---------------------------------------------------------------------------- and back
// A lane decodes eight columns of eight rows, four rows apart, so that a warp's stores cover 128
// consecutive bytes (bf16) of four rows. Rows of other alignment pass through shared memory, so that
// a warp's lanes write consecutive elements. Bound by HBM, mostly by its own stores: 4096 x 11008 to
// bf16 20 us (5.5 TB/s), to fp32 48; 4096 x 11007 27 and 48 us (150 and 185 with the lanes' own eight
// elements one by one).
template <int FMT, typename T>
__global__ void __launch_bounds__(kTileThreads)
    mx4_dequantize_kernel(int rows, int cols, const uint8_t* codes,
                          const uint8_t* scales, long long ld,
                          const float* factor, T* y, long long ldy,
                          bool vec) {
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tiles_c = (cols + 63) / 64;
  const unsigned tr = blockIdx.x / (unsigned)tiles_c, tc = blockIdx.x - tr * (unsigned)tiles_c;
  const long long r0 = (long long)tr * kTileRows + warp * 32;
  const int c = (int)tc * 64 + (lane & 7) * 8;
  if (r0 >= rows || (vec && c >= cols)) return;
  float f = 1.f;
  if constexpr (FMT == kNvfp4) f = factor[1];
  const int lr = lane >> 3;
  const uint8_t* cp = codes + ((r0 + lr) * ld + c) / 2;
  const uint8_t* sp = scales + mx4_scale_off<FMT>(r0 + lr, c / Mx4Fmt<FMT>::kBlock, ld);
  uint32_t w[8], sb[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool ok = r0 + lr + 4 * i < rows && c < cols;
    w[i] = ok ? ld4(cp + i * 2 * ld) : 0;
    sb[i] = ok ? sp[64 * i] : 0;
  }
  auto values = [&](int i, float (&v)[8]) {
    const float s = mx4_scale_value<FMT>(sb[i]);
    e2m1x8_values(w[i], v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = v[k] * s * f;  // (e2m1 times s is exact)
  };
  if (!vec) {
    __shared__ __align__(16) T stage[kTileThreads / 32][4][64];
    T(*st)[64] = stage[warp];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (r0 + 4 * i >= rows) break;
      float v[8];
      values(i, v);
      T* d = &st[lr][(lane & 7) * 8];
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(d) =
            make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7]));
      } else {
        reinterpret_cast<float4*>(d)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(d)[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
      __syncwarp();
      T e[8];  // all read before the first is written: shared loads stay behind global stores
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = st[j >> 1][(j & 1) * 32 + lane];
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const long long row = r0 + 4 * i + (j >> 1);
        const int col = (int)tc * 64 + (j & 1) * 32 + lane;
        if (row < rows && col < cols) y[row * ldy + col] = e[j];
      }
    }
    return;
  }
  T* o = y + (r0 + lr) * ldy + c;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (r0 + lr + 4 * i >= rows) break;
    float v[8];
    values(i, v);
    T* e = o + (long long)(4 * i) * ldy;
    if (c + 8 <= cols) {
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
  cudaError_t e = launch_kernel(true, mx4_zero2_kernel, dim3(1), dim3(1), 0, s, out);
  if (e != cudaSuccess) return e;
  const unsigned long long n = (unsigned long long)rows * groups8(cols);
  const dim3 grid(grid_for(n, 256 * 4, num_sms, 8));
  if (dtype)
    return launch_kernel(true, mx4_factor_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, rows, cols,
                         (const __nv_bfloat16*)x, ldx, row_vec(x, ldx, 2), out);
  return launch_kernel(true, mx4_factor_kernel<float>, grid, dim3(256), 0, s, rows, cols,
                       (const float*)x, ldx, row_vec(x, ldx, 4), out);
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
  auto k = fmt == kMxfp4 ? (act == 0   ? mx4_gated_bwd_kernel<kMxfp4, 0>
                            : act == 1 ? mx4_gated_bwd_kernel<kMxfp4, 1>
                                       : mx4_gated_bwd_kernel<kMxfp4, 2>)
                         : (act == 0   ? mx4_gated_bwd_kernel<kNvfp4, 0>
                            : act == 1 ? mx4_gated_bwd_kernel<kNvfp4, 1>
                                       : mx4_gated_bwd_kernel<kNvfp4, 2>);
  auto vec = [](const void* p, long long ld) {  // loads of four bf16
    return (reinterpret_cast<uintptr_t>(p) & 7) == 0 && ld % 4 == 0;
  };
  return launch_kernel(true, k, dim3(tile_grid(rows, F, 32)), dim3(kTileThreads), 0, s, rows, F,
                       db, ldda, vec(db, ldda), ub, ldu, vec(ub, ldu), vec(ub + F, ldu), f_du,
                       f_dut, f_at, dg, dup, dgt, dupt, at);
}

}  // namespace mgt
