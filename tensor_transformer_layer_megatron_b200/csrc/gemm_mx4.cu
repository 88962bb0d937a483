// Products of microscaled 4-bit operands on the tensor cores of sm_100a (tcgen05.mma with block
// scaling: kind::mxf4 for 32-element blocks with 2^e scales, kind::mxf4nvf4 for 16-element blocks
// with e4m3 scales; fp32 accumulators).
//
// C[m, n] = f_a f_b sum_b s_a(m, b) s_b(n, b) sum_{k in b} a(m, k) b(n, k): the tensor core takes
// the two 4-bit operands from shared memory and their scales from tensor memory and applies the
// scales inside the sum.
#include <cudaTypedefs.h>

#include <mutex>

#include "mx4_device.cuh"
#include "mx4_internal.h"

namespace mgt {
namespace {

// 2-D tiled bulk load into this CTA's shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load_2d(const CUtensorMap* m, uint64_t* bar, void* dst, int c0,
                                            int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}

// The same box into L2 only.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* m, int c0, int c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(c0), "r"(c1)
               : "memory");
}

// A 512-byte scale tile (128 rows by 4 blocks) to four tensor-memory columns: lane r % 32 of
// column r / 32 gets the four bytes of row r, in all four lane quarters. The source is 32 rows
// of 16 bytes, unswizzled: core matrices of 8 rows, 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
  uint64_t d = 0;
  d |= (uint64_t)((addr >> 4) & 0x3FFF);
  d |= (uint64_t)(128 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  return d;
}
__device__ __forceinline__ void tc_cp_scales(uint32_t taddr, uint32_t smem_addr) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr),
               "l"(scale_desc(smem_addr))
               : "memory");
}

// Instruction descriptor of the block-scaled kinds: both operands e2m1 (1), K-major. `id` selects
// the pair of scale bytes in a 32-bit scale word (mxfp4: 0 for the even 64-element step, 2 for
// the odd one; nvfp4 uses all four).
template <int FMT>
__device__ __forceinline__ uint32_t idesc_mx4(int M, int N, uint32_t id) {
  return (1u << 7) | (1u << 10) | (id << 4) | ((uint32_t)(N >> 3) << 17) |
         (FMT == kMxfp4 ? 1u << 23 : 0u) | ((uint32_t)(M >> 7) << 27) | (id << 29);
}
// a, b: low words of the operands' descriptors (start address >> 4, leading offset 1); the high
// word, the same for every K-major tile with 128-byte swizzle, joins them here.
template <int FMT, int GROUP>
__device__ __forceinline__ void tc_mma_mx4(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                           uint32_t sa, uint32_t sb, uint32_t accumulate) {
  constexpr uint32_t kHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
#define MX4_MMA(group, kind)                                                                  \
  asm volatile("{ .reg .pred p; .reg .b64 da, db; setp.ne.b32 p, %6, 0;\n\t"                  \
               "mov.b64 da, {%1, %7}; mov.b64 db, {%2, %7};\n\t"                              \
               "tcgen05.mma.cta_group::" group ".kind::" kind                                 \
               " [%0], da, db, %3, [%4], [%5], p; }" ::"r"(d),                                \
               "r"(a), "r"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate), "n"(kHigh)      \
               : "memory")
  if constexpr (FMT == kMxfp4 && GROUP == 1)
    MX4_MMA("1", "mxf4.block_scale.scale_vec::2X");
  else if constexpr (FMT == kMxfp4)
    MX4_MMA("2", "mxf4.block_scale.scale_vec::2X");
  else if constexpr (GROUP == 1)
    MX4_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X");
  else
    MX4_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X");
#undef MX4_MMA
}
__device__ __forceinline__ uint32_t desc_low(uint32_t addr) {
  return ((addr >> 4) & 0x3FFF) | (1u << 16);
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.b32 %0, 1, 0, p; }" : "=r"(p));
  return p != 0;
}

// The operands' tensor factors on a sum: their product x, and y = 1. A product outside fp32's normal
// numbers would make zero or infinity of sums that are neither (and NaN of zeros): there x and y
// are the two factors, whose smaller one then is above one or whose larger one is below 2^23.
template <int FMT>
__device__ __forceinline__ float2 sum_factors(const float* a, const float* b) {
  if constexpr (FMT == kMxfp4) return make_float2(1.f, 1.f);  // has none
  const float fa = a[1], fb = b[1], f = fa * fb;
  return f >= 1.17549435e-38f && f <= 3.40282347e38f ? make_float2(f, 1.f) : make_float2(fa, fb);
}
template <int FMT, int N>
__device__ __forceinline__ void scale_sums(float (&v)[N], float2 f) {
  if constexpr (FMT == kNvfp4) {
    if (f.y != 1.f) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] *= f.y;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= f.x;
  }
}

// v = act(v)
template <int N>
__device__ __forceinline__ void gate_all(float (&v)[N], int act) {
  float d;
  if (act == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) gate_and_grad<0>(v[i], v[i], d);
  } else if (act == 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) gate_and_grad<1>(v[i], v[i], d);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) gate_and_grad<2>(v[i], v[i], d);
  }
}

constexpr int kStageK = 256;          // elements of K per stage: 128 bytes of a row
constexpr int kPRows = kSkinnyRows;   // weight rows of a CTA's tile (per matrix)
constexpr int kPBytes = kPRows * 128;
constexpr int kPrefetchStages = 8;    // stages fetched into L2 ahead: 128 KB a CTA

// ---------------------------------------------------------------------------- weights as rows
// The weights' rows take the 128 lanes of the accumulator and up to 256 tokens its columns, so a
// few tokens cost no wasted operand traffic: each CTA streams its 128 weight rows once. The
// summed axis is split over a cluster of up to eight CTAs, whose fp32 partial tiles meet in
// distributed shared memory, added in rank order. Gated: two accumulators, gate and up rows of
// the same outputs.
//
// Bound by the weights' bytes and, at these sizes, by what comes before and after them (launch,
// first loads, sum over the cluster): one token, mxfp4, 12288 x 4096 7.8 us with its launch (26.7
// MB, 3.4 TB/s; nvfp4 8.5), 4096 x 11008 7.5; gated 2 x 11008 x 4096 11.1 us, any activation (nvfp4
// 12.9); 60 tokens with u kept 16.4 / 17.8; 90 tokens x 12288 x 4096 12.2 / 13.0. More tiles than
// places, 49152 x 4096: 384 CTAs on 296 places are 1.3 rounds, of which the second fills 30 % of
// the GPU: 28 us alone, 24 in a row of such calls, where the next call's weights are on their way.
struct SkinnyArgs {
  int M, N, kp;                 // tokens, weight rows (per matrix), K rounded up to 128
  int bnq, stages, tmem_cols;
  int vec;                      // C (u) takes stores of four elements
  const uint8_t* p_scales;
  const uint8_t* p2_scales;
  long long p_ld;
  const uint8_t* q_scales;
  long long q_ld;
  const float *p_factor, *q_factor;
  void* C;
  int c_f32;
  long long ldc;
  int act;
  Mx4Out a;
  const float* out_factor;
  __nv_bfloat16* u;
  long long ldu;
  int* err;
};

__device__ __forceinline__ float4 ld_dsmem4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

// Up to four consecutive outputs; vec: the address allows one store of all four.
__device__ __forceinline__ void store4(float* o, const float (&v)[4], int n, int vec) {
  if (vec && n >= 4) {
    *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) o[i] = v[i];
  }
}
__device__ __forceinline__ void store4(__nv_bfloat16* o, const float (&v)[4], int n, int vec) {
  if (vec && n >= 4) {
    *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) o[i] = __float2bfloat16_rn(v[i]);
  }
}

template <int FMT, bool GATED>
__global__ void __launch_bounds__(192)
    mx4_skinny_kernel(const __grid_constant__ CUtensorMap tmP,
                      const __grid_constant__ CUtensorMap tmP2,
                      const __grid_constant__ CUtensorMap tmQ, const SkinnyArgs g) {
  constexpr int NM = GATED ? 2 : 1;
  constexpr int kTps = kStageK / Mx4Fmt<FMT>::kTileCols;  // scale tiles per stage and 128 rows
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  // 128-row groups of the tokens' scales
  const int groups = !GATED && g.bnq > 128 ? 2 : 1;
  const int stage_bytes = NM * kPBytes + g.bnq * 128;
  const int sf_bytes = (NM + groups) * kTps * 512;
  uint8_t* sf = smem + g.stages * stage_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sf + g.stages * sf_bytes);
  uint64_t* empty = full + g.stages;
  uint64_t* tfull = empty + g.stages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t csize;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));
  const uint32_t rank = cluster_ctarank();
  const int p0 = (int)(blockIdx.x / csize) * kPRows;
  const int q0 = blockIdx.y * g.bnq;
  const int ki = (g.kp + kStageK - 1) / kStageK;
  const int k_begin = (int)((long long)ki * rank / csize);
  const int k_end = (int)((long long)ki * (rank + 1) / csize);
  const int k_tiles = g.kp / Mx4Fmt<FMT>::kTileCols;
  // groups of 128 tokens that have scales in the buffer
  const int q_groups = min(groups, (g.M - q0 + 127) / 128);

  if (warp == 2 && lane == 0) {
    // The weights' first stages into L2 while the previous kernel still runs. It may be the one
    // that writes them: L2 then takes its writes, and the copies to shared memory come after
    // grid_dependency_wait.
    const int end = min(k_end, k_begin + kPrefetchStages);
    for (int kt = k_begin; kt < end; ++kt) {
      tma_prefetch_2d(&tmP, kt * 128, p0);
      if (GATED) tma_prefetch_2d(&tmP2, kt * 128, p0);
    }
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < g.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmP);
    if (GATED) tma_prefetch_desc(&tmP2);
    tma_prefetch_desc(&tmQ);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, g.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t acc_cols = (uint32_t)(g.bnq + 31) & ~31u;
  launch_dependents();
  grid_dependency_wait();  // the operands are the previous kernel's results

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (int kt = k_begin; kt < k_end; ++kt) {
        if (!mbar_wait(&empty[stage], phase ^ 1, g.err, kErrTimeoutProducer, abort_flag)) break;
        const int n = min(kTps, k_tiles - kt * kTps);  // scale tiles of this stage
        mbar_arrive_expect_tx(&full[stage],
                              (uint32_t)(stage_bytes + (NM + q_groups) * n * 512));
        uint8_t* d = smem + stage * stage_bytes;
        uint8_t* s = sf + stage * sf_bytes;
        tma_load_2d(&tmP, &full[stage], d, kt * 128, p0);
        if (GATED) tma_load_2d(&tmP2, &full[stage], d + kPBytes, kt * 128, p0);
        tma_load_2d(&tmQ, &full[stage], d + NM * kPBytes, kt * 128, q0);
        const long long pt = (long long)(p0 / 128) * (g.p_ld / Mx4Fmt<FMT>::kTileCols) + kt * kTps;
        bulk_load_1d(s, g.p_scales + pt * 512, n * 512, &full[stage]);
        if (GATED) bulk_load_1d(s + kTps * 512, g.p2_scales + pt * 512, n * 512, &full[stage]);
        for (int q = 0; q < q_groups; ++q) {
          const long long qt =
              (long long)(q0 / 128 + q) * (g.q_ld / Mx4Fmt<FMT>::kTileCols) + kt * kTps;
          bulk_load_1d(s + (NM + q) * kTps * 512, g.q_scales + qt * 512, n * 512, &full[stage]);
        }
        if (++stage == g.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      for (int i = 1; i <= g.stages; ++i) {  // every copy has landed before the CTA may exit
        int s = stage - i;
        uint32_t ph = phase;
        if (s < 0) {
          s += g.stages;
          ph ^= 1;
        }
        mbar_wait(&full[s], ph, g.err, kErrTimeoutDrain, nullptr);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // The whole warp runs the loop and one elected lane issues: descriptors and addresses then
    // are warp-uniform values. Issued from a lone thread's registers, a stage's products and
    // scale copies took longer to issue than to run.
    const bool one = elect_one();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    int stage = 0;
    uint32_t phase = 0;
    const uint32_t sf_cols = (uint32_t)(NM + groups) * kTps * 4;
    for (int kt = k_begin; kt < k_end; ++kt) {
      if (!mbar_wait(&full[stage], phase, g.err, kErrTimeoutMma, abort_flag)) break;
      tc_fence_after();
      const int n = min(kTps, k_tiles - kt * kTps);
      const int steps = min(4, (g.kp - kt * kStageK) / 64);
      // Each stage has scale columns of its own: they are rewritten only after the producer
      // has seen the products of the stage's last use complete.
      const uint32_t sc = tm + NM * acc_cols + stage * sf_cols;
      const uint32_t ss = smem_u32(sf + stage * sf_bytes);
      const uint32_t pa = desc_low(smem_u32(smem + stage * stage_bytes));
      const uint32_t qa = pa + NM * (kPBytes >> 4);
      if (one) {
#pragma unroll
        for (int t = 0; t < kTps; ++t) {
          if (t < n) {
#pragma unroll
            for (int m = 0; m < NM; ++m)
              tc_cp_scales(sc + (m * kTps + t) * 4, ss + (m * kTps + t) * 512);
            tc_cp_scales(sc + (NM * kTps + t * groups) * 4, ss + (NM * kTps + t) * 512);
            if (groups == 2)
              tc_cp_scales(sc + (NM * kTps + t * 2 + 1) * 4, ss + ((NM + 1) * kTps + t) * 512);
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k < steps) {
            const int t = FMT == kMxfp4 ? k >> 1 : k;
            const uint32_t id = FMT == kMxfp4 ? (uint32_t)(k & 1) * 2 : 0u;
            const uint32_t idesc = idesc_mx4<FMT>(kPRows, g.bnq, id);
#pragma unroll
            for (int m = 0; m < NM; ++m)
              tc_mma_mx4<FMT, 1>(tm + m * acc_cols, pa + m * (kPBytes >> 4) + 2 * k, qa + 2 * k,
                                 idesc, sc + (m * kTps + t) * 4,
                                 sc + (NM * kTps + t * groups) * 4,
                                 k > 0 ? 1u : (uint32_t)(kt - k_begin));
          }
        }
        tc_commit(&empty[stage]);
      }
      __syncwarp();
      if (++stage == g.stages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (one) tc_commit(tfull);
    __syncwarp();
    mbar_wait(tfull, 0, g.err, kErrTimeoutDrain, nullptr);
  }

  // Partial tiles [matrix][token][128] in the operand stages' memory: all copies into it have
  // been consumed once the last product has completed.
  float* part = reinterpret_cast<float*>(smem);
  const bool epi = warp >= 2;
  const int ew = warp & 3;
  const int p = ew * 32 + lane;
  bool ok = true;
  if (epi) {
    ok = mbar_wait(tfull, 0, g.err, kErrTimeoutEpilogue, abort_flag) && !*abort_flag;
    tc_fence_after();
    if (ok) {
#pragma unroll 1
      for (int m = 0; m < NM; ++m)
#pragma unroll 1
        for (int c = 0; c < (int)acc_cols; c += 32) {
          float v[32];
          tmem_ld_32x32b_x32(tmem + m * acc_cols + c + ((uint32_t)(ew * 32) << 16), v);
          float* o = part + (m * g.bnq + c) * kPRows + p;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c + i < g.bnq) o[i * kPRows] = v[i];
        }
    }
    tc_fence_before();
  }
  __syncwarp();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, g.tmem_cols);
  }
  if (epi && ok) {
    // A warp takes a token of its CTA's share at a time, a lane four neighbouring weight rows.
    const float2 f = sum_factors<FMT>(g.p_factor, g.q_factor);
    const int tokens = min(g.bnq, g.M - q0);
    const uint32_t mine = smem_u32(part + lane * 4);
    const int col = p0 + lane * 4;
    const Mx4Factor of = mx4_factor<FMT>(GATED ? g.out_factor : nullptr);
#pragma unroll 2
    for (int t = (int)rank * 4 + (warp - 2); t < tokens; t += 4 * (int)csize) {
      float v[NM][4];
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        v[m][0] = v[m][1] = v[m][2] = v[m][3] = 0.f;
#pragma unroll
        for (uint32_t r = 0; r < 8; ++r) {
          if (r < csize) {
            const float4 w =
                ld_dsmem4(mapa_shared(mine + (uint32_t)((m * g.bnq + t) * kPRows * 4), r));
            v[m][0] += w.x;
            v[m][1] += w.y;
            v[m][2] += w.z;
            v[m][3] += w.w;
          }
        }
        scale_sums<FMT>(v[m], f);
      }
      const long long row = q0 + t;
      if constexpr (!GATED) {
        if (g.c_f32)
          store4(static_cast<float*>(g.C) + row * g.ldc + col, v[0], g.N - col, g.vec);
        else
          store4(static_cast<__nv_bfloat16*>(g.C) + row * g.ldc + col, v[0], g.N - col, g.vec);
      } else {
        if (g.u) {
          store4(g.u + row * g.ldu + col, v[0], g.N - col, g.vec);
          store4(g.u + row * g.ldu + g.N + col, v[NM - 1], g.N - col, g.vec);
        }
        float a[4];
        uint32_t mx = 0;
        gate_all(v[0], g.act);
#pragma unroll
        for (int i = 0; i < 4; ++i)  // columns behind the last are zeros
          a[i] = col + i < g.N ? v[0][i] * v[NM - 1][i] : 0.f;
        if (FMT == kNvfp4 && of.tiny) mx4_lift(a, of);
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = max(mx, abs_bits(a[i]));
        constexpr int B = Mx4Fmt<FMT>::kBlock;
#pragma unroll
        for (int o = B / 8; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const Mx4Block q = mx4_block<FMT>(mx, of);
        const float w[8] = {a[0], a[1], a[2], a[3], 0.f, 0.f, 0.f, 0.f};
        *reinterpret_cast<uint16_t*>(g.a.codes + (row * g.a.ld + col) / 2) =
            (uint16_t)mx4_codes8<FMT>(w, q, of);
        if (col % B == 0)
          g.a.scales[mx4_scale_off<FMT>(row, col / B, g.a.ld)] = (uint8_t)q.byte;
      }
    }
  }
  cluster_sync_all();  // no CTA leaves while a peer may still read its partial tile
}

// ---------------------------------------------------------------------------- CTA pairs
// Many rows: 256 x 256 tiles on pairs of CTAs (cta_group::2; each CTA holds 128 rows of A, 128 of
// B and the accumulators of its rows), persistent over the tiles. A stage holds 256 elements of K:
// 16 KB of A, 16 KB of B and the scales of the CTA's A rows and of all 256 B rows, which both
// tensor memories need. Operand bytes per multiply-add are those of bf16 at a quarter of the time,
// so wide tiles matter more than anything else here.
//
// Tensor memory: two 256-column accumulators and the scales do not fit 512 columns side by side.
// The accumulators overlap by 64 columns (0..255 and 192..447): the epilogue reads those first and
// frees them, and the next tile starts while it goes on with the other 192. Scales take columns
// 448..: two slots of 24 columns, a slot for 256 (mxfp4) or 128 (nvfp4) elements of K, rewritten
// once the products that read it have completed.
//
// Gated: B is 128 gate rows (CTA 0) and the 128 up rows of the same outputs (CTA 1).
//
// Bound by the tensor core and the shared memory that feeds it: a stage of 256 elements takes 650
// to 710 cycles where its products alone take 512, and the hand-over between tiles about 1,500. 8192
// x 24576 x 6144 mxfp4 451 us (5.5 PFLOP/s), nvfp4 477; 2048 x 12288 x 4096 47 / 49 us, 12288 x 4096
// x 2048 into fp32 61 / 66; gated 2048 x 2 * 11008 x 4096 silu 73 / 80 us, with u kept 82 / 89, gelu
// 92 / 99 (99 / 105), tanh gelu 86 / 105 (95 / 113). These are runs of a millisecond; after seconds of
// them the power cap holds the clock at 1.5 to 1.75 GHz and they take 8 to 17 % more (530 / 557, 55
// / 57, 69 / 76, gated silu 86 / 94).
struct PairArgs {
  int M, N, kp;
  int num_m, num_n, m_fast;
  int bn;                   // columns of a tile: 256 or 128
  const float *a_factor, *b_factor;
  void* C;
  int c_f32;
  long long ldc;
  bool tma;                 // C (u) takes bulk tensor stores
  int up_tiles;             // gated: scale tiles of rows before the first up row
  int act;
  Mx4Out a;
  const float* out_factor;
  __nv_bfloat16* u;
  long long ldu;
  int* err;
};

// Arrive on a barrier of the pair without ordering this thread's stores before it: the epilogue
// only reports tensor memory that it has read (tcgen05.wait::ld), and a releasing arrive waited
// 1500 cycles for the stores of the tile before.
__device__ __forceinline__ void arrive_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

constexpr int kPairThreads = 320;
constexpr int kScaleCol = 448;
constexpr int kSlotCols = 24;
constexpr int kStoreBytes = 5120;  // staging of one warp: 32 rows of at most 144 bytes, in whole KB

template <int FMT>
struct PairCfg {
  static constexpr int kTps = kStageK / Mx4Fmt<FMT>::kTileCols;
  static constexpr int kStages = FMT == kMxfp4 ? 5 : 4;
  static constexpr int kScaleBytes = 3 * kTps * 512;  // A's 128 rows and B's 256
  static constexpr int kOperandBytes = 2 * 128 * 128;
  static constexpr int kStageBytes = kOperandBytes + kScaleBytes;
  static constexpr int kSmem = 1024 + kStages * kStageBytes + 8 * kStoreBytes + 512;
};

__device__ __forceinline__ void tma_load_2d_pair(const CUtensorMap* m, uint32_t bar_cluster,
                                                 void* dst, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar_cluster), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void tc_cp_scales_pair(uint32_t taddr, uint32_t smem_addr) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr),
               "l"(scale_desc(smem_addr))
               : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, const void* src, int c0,
                                             int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1)
               : "memory");
}

// A warp's 32 rows by 32 columns (thread = row) to global memory through its staging buffer.
// Where the output's alignment allows it (map), by a bulk tensor store: bf16 blocks (2 KB) use two
// halves of the buffer in turn (`turn`), fp32 blocks (4 KB) all of it, 16-byte units of a row
// permuted as the map's swizzle has it.
template <typename T>
__device__ __forceinline__ void store_block_tma(uint8_t* stg, int& turn, const float (&v)[32],
                                                const CUtensorMap* map, int row0, int col0) {
  const int lane = threadIdx.x & 31;
  constexpr int kRow = 32 * (int)sizeof(T), kUnits = kRow / 16;
  uint8_t* buf = stg;
  if constexpr (sizeof(T) == 2) {
    buf += (turn & 1) * 2048;
    ++turn;
  }
  if (lane == 0) {  // the buffer's last store has read it
    if constexpr (sizeof(T) == 2)
      asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
    else
      bulk_wait_read0();
  }
  __syncwarp();
  const int swz = sizeof(T) == 2 ? (lane >> 1) & 3 : lane & 7;
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    uint4 w;
    if constexpr (sizeof(T) == 2)
      w = make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                     pack_bf16x2(v[8 * i + 4], v[8 * i + 5]),
                     pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
    else
      w = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                     __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
    *reinterpret_cast<uint4*>(buf + lane * kRow + ((i ^ swz) << 4)) = w;
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(map, buf, col0, row0);
    bulk_commit();
  }
}
// Elsewhere by stores in which consecutive lanes write consecutive elements of a row.
template <typename T>
__device__ __forceinline__ void store_block_any(uint8_t* stg, const float (&v)[32], T* base,
                                                long long ld, int row0, int rows, int col0,
                                                int cols) {
  const int lane = threadIdx.x & 31;
  constexpr int kRow = 32 * (int)sizeof(T) + 16;  // eight rows' 16-byte units meet no bank twice
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) * 2; ++i) {
    uint4 w;
    if constexpr (sizeof(T) == 2)
      w = make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                     pack_bf16x2(v[8 * i + 4], v[8 * i + 5]),
                     pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
    else
      w = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                     __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
    *reinterpret_cast<uint4*>(stg + lane * kRow + i * 16) = w;
  }
  __syncwarp();
  T* out = base + (long long)row0 * ld + col0;
  const int nr = min(32, rows - row0), nc = min(32, cols - col0);
  // Eight rows read before the first is written: the compiler does not move a shared load across a
  // global store, and one round trip per row made this the slowest part of ragged products (2048 x
  // 12287 x 4096 68 us row by row, 52 in eights; 47 for 12288, where bulk stores apply).
  T* o = out + lane;
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += 8) {
    T e[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) e[r] = reinterpret_cast<const T*>(stg + (r0 + r) * kRow)[lane];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      if (r0 + r < nr && lane < nc) *o = e[r];
      o += ld;
    }
  }
  __syncwarp();
}
template <typename T>
__device__ __forceinline__ void store_block(uint8_t* stg, int& turn, const float (&v)[32],
                                            const CUtensorMap* map, T* base, long long ld, int row0,
                                            int rows, int col0, int cols, bool tma) {
  if (tma)
    store_block_tma<T>(stg, turn, v, map, row0, col0);
  else
    store_block_any(stg, v, base, ld, row0, rows, col0, cols);
}

template <int FMT, bool GATED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    mx4_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmB2,
                    const __grid_constant__ CUtensorMap tmSA,
                    const __grid_constant__ CUtensorMap tmSB,
                    const __grid_constant__ CUtensorMap tmO,
                    const __grid_constant__ CUtensorMap tmO2, const PairArgs g) {
  using C = PairCfg<FMT>;
  constexpr int S = C::kStages, kTps = C::kTps;
  constexpr int kChunks = FMT == kMxfp4 ? 1 : 2;      // scale slots per stage
  constexpr int kTpc = kTps / kChunks;                // scale tiles per chunk (2)
  constexpr int kStepsPerChunk = 4 / kChunks;         // products of 64 elements per chunk
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* stg = smem + S * C::kOperandBytes;
  uint8_t* sf = stg + 8 * kStoreBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sf + S * C::kScaleBytes);
  uint64_t* empty = full + S;
  uint64_t* slot_free = empty + S;
  uint64_t* tfull = slot_free + 2;
  uint64_t* tempty = tfull + 2;
  uint64_t* overlap = tempty + 2;
  uint64_t* drain = overlap + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;
  const int num_tiles = g.num_m * g.num_n;
  const int ki = (g.kp + kStageK - 1) / kStageK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&slot_free[b], 1);
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 16);  // the epilogue warps of both CTAs
    }
    mbar_init(overlap, 16);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    if (GATED) tma_prefetch_desc(&tmB2);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist before any cross-CTA arrive or load
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();  // the operands are the previous kernel's results

  const int bn = GATED ? 256 : g.bn, sb = bn / 128;
  const bool shared_cols = bn == 256;            // the accumulators overlap
  const uint32_t acc1 = shared_cols ? 192 : bn;  // first column of the second
  auto tile_m = [&](int t) { return g.m_fast ? t % g.num_m : t / g.num_n; };
  auto tile_n = [&](int t) { return g.m_fast ? t / g.num_m : t % g.num_n; };

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int tile = pair; tile < num_tiles && ok; tile += num_pairs) {
      const int m0 = tile_m(tile) * 256 + (int)rank * 128;
      const int nt = tile_n(tile);
      const int sb0 = GATED ? nt : nt * bn / 128;
      const uint32_t stage_tx = 2 * (128 * 128 + bn / 2 * 128 + (1 + sb) * kTps * 512);
      for (int kt = 0; kt < ki; ++kt) {
        if (!mbar_wait(&empty[stage], phase ^ 1, g.err, kErrTimeoutProducer, abort_flag)) {
          ok = false;
          break;
        }
        if (leader) mbar_arrive_expect_tx(&full[stage], stage_tx);
        const uint32_t fb = mapa_shared(smem_u32(&full[stage]), 0);
        uint8_t* d = smem + stage * C::kOperandBytes;
        uint8_t* s = sf + stage * C::kScaleBytes;
        tma_load_2d_pair(&tmA, fb, d, kt * 128, m0);
        if (GATED)
          tma_load_2d_pair(rank ? &tmB2 : &tmB, fb, d + 128 * 128, kt * 128, nt * 128);
        else
          tma_load_2d_pair(&tmB, fb, d + 128 * 128, kt * 128, nt * bn + (int)rank * (bn / 2));
        tma_load_3d_pair(&tmSA, fb, s, 0, kt * kTps, m0 / 128);
        for (int q = 0; q < sb; ++q)
          tma_load_3d_pair(&tmSB, fb, s + (1 + q) * kTps * 512, 0, kt * kTps,
                           GATED && q ? g.up_tiles + nt : sb0 + q);
        if (++stage == S) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    // This CTA's loads complete on the leader's barriers: the leader sees all of them land, and
    // the peer waits for it at the last cluster barrier.
    if (leader) {
      for (int i = 1; i <= S; ++i) {
        int s = stage - i;
        uint32_t ph = phase;
        if (s < 0) {
          s += S;
          ph ^= 1;
        }
        mbar_wait(&full[s], ph, g.err, kErrTimeoutDrain, nullptr);
      }
    }
  } else if (leader && warp == 1) {
    // ------------------------------------------------------------ products (leader only)
    // The whole warp runs the loop and one elected lane issues, so that descriptors and
    // addresses are warp-uniform values: issued from a lone thread's registers, four products took
    // longer to issue than to run.
    const bool one = elect_one();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    int stage = 0, acc = 0, slot = 0;
    uint32_t phase = 0, acc_phase = 0, slot_phase = 0, ov_phase = 0;
    bool ok = true, first = true;
    for (int tile = pair; tile < num_tiles && ok; tile += num_pairs) {
      if (!mbar_wait(&tempty[acc], acc_phase ^ 1, g.err, kErrTimeoutMma, abort_flag)) break;
      if (!first && shared_cols) {  // the previous tile's share of the common columns has been read
        if (!mbar_wait(overlap, ov_phase, g.err, kErrTimeoutMma, abort_flag)) break;
        ov_phase ^= 1;
      }
      first = false;
      const uint32_t d = tm + (acc ? acc1 : 0);
      for (int kt = 0; kt < ki; ++kt) {
        if (!mbar_wait(&full[stage], phase, g.err, kErrTimeoutMma, abort_flag)) {
          ok = false;
          break;
        }
        const int steps = min(4, (g.kp - kt * kStageK) / 64);
        const uint32_t aa = desc_low(smem_u32(smem + stage * C::kOperandBytes));
        const uint32_t ba = aa + (128 * 128 >> 4);
        const uint32_t ss = smem_u32(sf + stage * C::kScaleBytes);
#pragma unroll
        for (int ch = 0; ch < kChunks; ++ch) {
          if (ch * kStepsPerChunk >= steps) break;
          if (!mbar_wait(&slot_free[slot], slot_phase ^ 1, g.err, kErrTimeoutMma, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sc = tm + kScaleCol + slot * kSlotCols;
          if (one) {
#pragma unroll
            for (int t = 0; t < kTpc; ++t) {
              tc_cp_scales_pair(sc + t * 4, ss + (ch * kTpc + t) * 512);
              tc_cp_scales_pair(sc + kTpc * 4 + t * sb * 4, ss + (kTps + ch * kTpc + t) * 512);
              if (sb == 2)
                tc_cp_scales_pair(sc + kTpc * 4 + t * 8 + 4, ss + (2 * kTps + ch * kTpc + t) * 512);
            }
#pragma unroll
            for (int j = 0; j < kStepsPerChunk; ++j) {
              const int k = ch * kStepsPerChunk + j;
              if (k < steps) {
                const int t = FMT == kMxfp4 ? j >> 1 : j;
                const uint32_t id = FMT == kMxfp4 ? (uint32_t)(j & 1) * 2 : 0u;
                tc_mma_mx4<FMT, 2>(d, aa + 2 * k, ba + 2 * k, idesc_mx4<FMT>(256, bn, id), sc + t * 4,
                                   sc + kTpc * 4 + t * 4 * sb, k > 0 ? 1u : (uint32_t)kt);
              }
            }
            tc_commit_pair(&slot_free[slot]);
          }
          __syncwarp();
          if (++slot == 2) {
            slot = 0;
            slot_phase ^= 1;
          }
        }
        if (!ok) break;
        if (one) tc_commit_pair_mc(&empty[stage], 0x3);
        __syncwarp();
        if (++stage == S) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
      if (one) tc_commit_pair_mc(&tfull[acc], 0x3);
      __syncwarp();
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1;
      }
    }
    if (one) tc_commit_pair(drain);
    __syncwarp();
    mbar_wait(drain, 0, g.err, kErrTimeoutDrain, nullptr);
  } else if (warp >= 2) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int ew = warp & 3, set = (warp - 2) >> 2;
    uint8_t* my = stg + (warp - 2) * kStoreBytes;
    const float2 f = sum_factors<FMT>(g.a_factor, g.b_factor);
    const Mx4Factor of = mx4_factor<FMT>(GATED ? g.out_factor : nullptr);
    const uint32_t tempty0 = mapa_shared(smem_u32(&tempty[0]), 0);
    const uint32_t overlap0 = mapa_shared(smem_u32(overlap), 0);
    int acc = 0, turn = 0;
    uint32_t acc_phase = 0;
    for (int tile = pair; tile < num_tiles; tile += num_pairs) {
      const int row0 = tile_m(tile) * 256 + (int)rank * 128 + ew * 32;
      const int row = row0 + lane;
      const int nt = tile_n(tile);
      if (!mbar_wait(&tfull[acc], acc_phase, g.err, kErrTimeoutEpilogue, abort_flag)) break;
      tc_fence_after();
      const uint32_t t0 = tmem + (acc ? acc1 : 0) + ((uint32_t)(ew * 32) << 16);
      if constexpr (!GATED) {
        // Up to four 32-column chunks per warp, all read into registers before any is stored. Where
        // the accumulators overlap, the first one lies in the common columns (6, 7 of the first
        // accumulator, 0, 1 of the second) and frees them.
        uint32_t r[4][32];
        const int half = (bn / 32 + 1) / 2, count = set ? bn / 32 - half : half;
        auto chunk = [&](int i) {
          if (!shared_cols) return set * half + i;
          return acc ? (i == 0 ? set : 1 + 3 * set + i) : (i == 0 ? 6 + set : 3 * set + i - 1);
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i < count) tmem_ld_32x32b_x32_nw(t0 + chunk(i) * 32, r[i]);
          if ((i == 0 && shared_cols) || i == 3) {
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_relaxed(i == 0 ? overlap0 : tempty0 + acc * 8);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) reg_fence(r[i]);
        if (FMT == kNvfp4 && f.y != 1.f) {  // (in place: further down it took registers)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < 32; ++k)
              r[i][k] = __float_as_uint(__uint_as_float(r[i][k]) * f.y);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int col0 = nt * bn + chunk(i) * 32;
          if (i < count && col0 < g.N && row0 < g.M) {
            float v[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(r[i][k]) * f.x;
            if (g.c_f32)
              store_block(my, turn, v, &tmO, static_cast<float*>(g.C), g.ldc, row0, g.M, col0, g.N,
                          g.tma);
            else
              store_block(my, turn, v, &tmO, static_cast<__nv_bfloat16*>(g.C), g.ldc, row0, g.M,
                          col0, g.N, g.tma);
          }
        }
      } else {
        // gate chunk c and up chunk c + 4 of the same outputs; c = 2, 3 first in the first
        // accumulator (their up chunks are common columns), 0, 1 first in the second
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          const int c = ((acc ? i : 1 - i) * 2) + set;
          float v[32], w[32];
          tmem_ld_32x32b_x32(t0 + c * 32, v);
          tmem_ld_32x32b_x32(t0 + 128 + c * 32, w);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_relaxed(i == 0 ? overlap0 : tempty0 + acc * 8);
          const int col0 = nt * 128 + c * 32;
          scale_sums<FMT>(v, f);
          scale_sums<FMT>(w, f);
          if (g.u && row0 < g.M) {
            if (col0 < g.N) {
              store_block(my, turn, v, &tmO, g.u, g.ldu, row0, g.M, col0, g.N, g.tma);
              store_block(my, turn, w, &tmO2, g.u + g.N, g.ldu, row0, g.M, col0, g.N, g.tma);
            }
          }
          gate_all(v, g.act);
          // Columns behind the last are zeros, and so are rows (whose scales may be anything: as
          // they come they would take the slow path of mx4_codes8).
          const int live = row < g.M ? g.N - col0 : 0;
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = k < live ? v[k] * w[k] : 0.f;
          if (FMT == kNvfp4 && of.tiny) mx4_lift(v, of);
          constexpr int B = Mx4Fmt<FMT>::kBlock;
          uint32_t codes[4], bytes = 0;
#pragma unroll
          for (int b = 0; b < 32 / B; ++b) {
            uint32_t mx = 0;
#pragma unroll
            for (int k = 0; k < B; ++k) mx = max(mx, abs_bits(v[b * B + k]));
            const Mx4Block q = mx4_block<FMT>(mx, of);
            bytes |= q.byte << (8 * b);
#pragma unroll
            for (int k = 0; k < B / 8; ++k) {
              float e[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) e[j] = v[b * B + k * 8 + j];
              codes[b * (B / 8) + k] = mx4_codes8<FMT>(e, q, of);
            }
          }
          if (row < g.M) {
            *reinterpret_cast<uint4*>(g.a.codes + ((long long)row * g.a.ld + col0) / 2) =
                make_uint4(codes[0], codes[1], codes[2], codes[3]);
            uint8_t* sp = g.a.scales + mx4_scale_off<FMT>(row, col0 / B, g.a.ld);
            if constexpr (FMT == kMxfp4)
              *sp = (uint8_t)bytes;
            else
              *reinterpret_cast<uint16_t*>(sp) = (uint16_t)bytes;
          }
        }
      }
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1;
      }
    }
  }
  if (warp >= 2 && lane == 0) bulk_wait0();  // the stores have left the staging buffers
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while its peer may still touch its barriers or TMEM
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ---------------------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

template <int RANK>
bool encode(CUtensorMap* m, CUtensorMapDataType type, const void* base,
            const cuuint64_t (&dims)[RANK], const cuuint64_t (&strides)[RANK - 1],
            const cuuint32_t (&box)[RANK], CUtensorMapSwizzle swizzle) {
  auto fn = encode_fn();
  cuuint32_t es[RANK];
  for (int i = 0; i < RANK; ++i) es[i] = 1;
  return fn && fn(m, type, RANK, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Codes of an operand as bytes, boxes of 128 bytes (256 elements) by box_rows rows with the
// swizzle that the tensor core reads; zeros out of bounds.
bool map_codes(CUtensorMap* m, const uint8_t* codes, int rows, int kp, long long ld, int box_rows) {
  return encode<2>(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes,
                   {(cuuint64_t)kp / 2, (cuuint64_t)rows}, {(cuuint64_t)ld / 2},
                   {128, (cuuint32_t)box_rows}, CU_TENSOR_MAP_SWIZZLE_128B);
}
// Scale tiles [rows of tiles][ld tiles], `tiles` of each row inside; boxes of box_tiles tiles.
bool map_tiles(CUtensorMap* m, const uint8_t* scales, long long tiles, long long rows,
               long long ld, int box_tiles) {
  return encode<3>(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, scales,
                   {128, (cuuint64_t)tiles, (cuuint64_t)rows}, {512, (cuuint64_t)ld * 512},
                   {128, (cuuint32_t)box_tiles, 1}, CU_TENSOR_MAP_SWIZZLE_NONE);
}
// Output, boxes of 32 by 32.
bool map_out(CUtensorMap* m, void* base, int cols, int rows, long long ld, bool f32) {
  return encode<2>(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                   base, {(cuuint64_t)cols, (cuuint64_t)rows}, {(cuuint64_t)ld * (f32 ? 4 : 2)},
                   {32, 32}, f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

bool store_vec4(const void* p, long long ld, int esz) {
  return (reinterpret_cast<uintptr_t>(p) & (4 * esz - 1)) == 0 && ld % 4 == 0;
}

template <int FMT, bool GATED>
cudaError_t launch_skinny(const Mx4Gemm& g, int num_sms, cudaStream_t s) {
  const SkinnyShape shape = skinny_shape(FMT == kNvfp4, GATED, g.M);
  if (!shape.stages) return cudaErrorInvalidConfiguration;
  const int bnq = shape.tokens;
  const int kp = (g.K + 127) & ~127, ki = (kp + kStageK - 1) / kStageK;

  const int up0 = (g.N + 127) & ~127;  // first up row of a gated weight operand
  CUtensorMap tp, tp2, tq;
  if (!map_codes(&tp, g.B.codes, g.N, kp, g.B.ld, kPRows) ||
      !map_codes(&tp2, g.B.codes + (GATED ? up0 * g.B.ld / 2 : 0), g.N, kp, g.B.ld, kPRows) ||
      !map_codes(&tq, g.A.codes, g.M, kp, g.A.ld, bnq))
    return cudaErrorInvalidValue;
  SkinnyArgs a = {};
  a.M = g.M; a.N = g.N; a.kp = kp;
  a.bnq = bnq; a.stages = shape.stages; a.tmem_cols = shape.tmem_cols;
  a.p_scales = g.B.scales;
  a.p2_scales = g.B.scales + (up0 / 128) * (g.B.ld / Mx4Fmt<FMT>::kTileCols) * 512;
  a.p_ld = g.B.ld;
  a.q_scales = g.A.scales; a.q_ld = g.A.ld;
  a.p_factor = g.b_factor; a.q_factor = g.a_factor;
  a.C = g.C; a.c_f32 = g.c_f32; a.ldc = g.ldc;
  a.act = g.act; a.a = g.a; a.out_factor = g.out_factor;
  a.u = static_cast<__nv_bfloat16*>(g.u); a.ldu = g.ldu;
  a.vec = GATED ? g.N % 4 == 0 && store_vec4(g.u, g.ldu, 2)
                : store_vec4(g.C, g.ldc, g.c_f32 ? 4 : 2);
  a.err = g.err;

  auto kern = mx4_skinny_kernel<FMT, GATED>;
  static SmemLimit limit;
  cudaError_t e = limit.allow(kern, 227 * 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(192);
  cfg.dynamicSmemBytes = (size_t)shape.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  // The sum is split as far as all clusters still run at once with a tenth of the places to spare:
  // the next kernel's first CTAs start there and fetch its weights. (12288 weight rows, K = 4096,
  // one token, with its quantisation: two CTAs a tile 9.2 us, three 14.1; 4096 rows, K = 11008: one
  // 20.3, four 10.1, eight 9.0.)
  const int tiles_p = (g.N + kPRows - 1) / kPRows, tiles_q = (g.M + bnq - 1) / bnq;
  const long long tiles = (long long)tiles_p * tiles_q;
  const int places = (shape.two ? 2 : 1) * num_sms;
  // With one CTA per SM, how many clusters of a size are resident at once depends on how they fill
  // the GPU's processor groups (16 clusters of eight do not: 4096 x 100 x 4096 took 18.7 us with
  // them, 11.0 without): the driver is asked, once per device, size and shape. With two per SM its answer
  // is lower than what runs best.
  static ResidentClusters resident;
  int split = ki < 8 ? ki : 8;
  for (; split > 1; --split) {
    if (tiles * split * 10 > 9 * places) continue;
    if (GATED || shape.two) break;
    int dev = 0, n = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = resident.get(dev, bnq / 16, split, &n, [&](int* clusters) {
      cfg.gridDim = dim3((unsigned)split);
      cfg.numAttrs = 1;
      attr[0].val.clusterDim.x = (unsigned)split;
      return cudaOccupancyMaxActiveClusters(clusters, kern, &cfg);
    });
    if (e != cudaSuccess) return e;
    if (tiles <= n) break;
  }
  attr[0].val.clusterDim.x = (unsigned)split;
  cfg.numAttrs = 2;
  cfg.gridDim = dim3((unsigned)(tiles_p * split), (unsigned)tiles_q);
  return cudaLaunchKernelEx(&cfg, kern, tp, tp2, tq, a);
}

// Columns of a pair's tile. A tile of 128 columns takes 0.8 of the time of one of 256 (6.1 us and
// 7.7 us at K = 4096), so it pays only where all of them run at once and 256 would leave pairs
// idle: 512 x 4096 x 4096 10.8 us against 12.4 us.
int pick_bn(const Mx4Gemm& g, int num_sms) {
  const long long tiles = (long long)((g.M + 255) / 256) * ((g.N + 127) / 128);
  return tiles <= num_sms / 2 ? 128 : 256;
}

template <int FMT, bool GATED>
cudaError_t launch_pair(const Mx4Gemm& g, int num_sms, cudaStream_t s) {
  using C = PairCfg<FMT>;
  const int kp = (g.K + 127) & ~127;
  const int up0 = (g.N + 127) & ~127;
  CUtensorMap ta, tb, tb2, tsa, tsb;
  const int b_rows = GATED ? 2 * up0 : g.N;
  const int bn = GATED ? 256 : pick_bn(g, num_sms);
  if (!map_codes(&ta, g.A.codes, g.M, kp, g.A.ld, 128) ||
      !map_codes(&tb, g.B.codes, g.N, kp, g.B.ld, bn / 2) ||
      !map_codes(&tb2, g.B.codes + (GATED ? up0 * g.B.ld / 2 : 0), g.N, kp, g.B.ld, 128) ||
      !map_tiles(&tsa, g.A.scales, kp / Mx4Fmt<FMT>::kTileCols, (g.M + 127) / 128,
                             g.A.ld / Mx4Fmt<FMT>::kTileCols, C::kTps) ||
      !map_tiles(&tsb, g.B.scales, kp / Mx4Fmt<FMT>::kTileCols, (b_rows + 127) / 128,
                             g.B.ld / Mx4Fmt<FMT>::kTileCols, C::kTps))
    return cudaErrorInvalidValue;
  PairArgs a = {};
  a.M = g.M; a.N = g.N; a.kp = kp;
  a.num_m = (g.M + 255) / 256;
  a.num_n = GATED ? up0 / 128 : (g.N + bn - 1) / bn;
  a.bn = bn;
  a.m_fast = g.M <= b_rows;  // the operand that every wave sweeps again is the smaller one
  a.a_factor = g.a_factor; a.b_factor = g.b_factor;
  a.C = g.C; a.c_f32 = g.c_f32; a.ldc = g.ldc;
  a.up_tiles = up0 / 128;
  a.act = g.act; a.a = g.a; a.out_factor = g.out_factor;
  a.u = static_cast<__nv_bfloat16*>(g.u); a.ldu = g.ldu;
  // Bulk tensor stores need 16-byte aligned bases and row strides, and rows that end on 16 bytes:
  // they write whole 16-byte units (seen with 129 fp32 columns in rows of 132). u's second half
  // starts at column N.
  CUtensorMap to = {}, to2 = {};
  auto out_map = [&](CUtensorMap* m, void* p, long long ld, int esz) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * esz) % 16 == 0 &&
           ((long long)g.N * esz) % 16 == 0 &&
           map_out(m, p, g.N, g.M, ld, esz == 4);
  };
  if (GATED)
    a.tma = a.u && out_map(&to, a.u, g.ldu, 2) && out_map(&to2, a.u + g.N, g.ldu, 2);
  else
    a.tma = out_map(&to, g.C, g.ldc, g.c_f32 ? 4 : 2);
  a.err = g.err;
  auto kern = mx4_pair_kernel<FMT, GATED>;
  static SmemLimit limit;
  cudaError_t e = limit.allow(kern, C::kSmem);
  if (e != cudaSuccess) return e;
  const int tiles = a.num_m * a.num_n;
  const int pairs = tiles < num_sms / 2 ? tiles : num_sms / 2;
  return launch_kernel(true, kern, dim3(2 * pairs), dim3(kPairThreads), (size_t)C::kSmem, s, ta, tb,
                       tb2, tsa, tsb, to, to2, a);
}

// Whether the weights-as-rows kernel is the faster one (times with the quantisation of the rows,
// mxfp4). It passes over the weights once per 64 or 256 rows and splits the sum; the pairs'
// tiles hold 256 rows. N x K = 12288 x 4096: 96 rows 15.0 us against 15.3, 128 rows 16.4 against
// 15.4; gated 11008 x 4096: 64 rows 18.9 against 22.3, 96 rows 25.8 against 22.5. Where the sum is
// long and the pairs' tiles leave most SMs idle the split wins further up: 4096 x 11008, 128 rows
// 16.9 against 22.2, 256 rows 21.2 against 22.7; and at any number of rows, by the CTAs that a tile
// of 256 x 128 can have and the 256-element stages of the sum (products alone; split against pairs):
// with six or more from 20 stages up (512 x 512 x 8192 10.3 against 15.2, 1000 x 128 x 16384 11.6
// against 25.6); with four 14.6 against 18.9 at 768 x 1024 x 11008 and 13.4 against 12.8 at 512 x 2048 x
// 6144; with three 18.0 against 19.1 at 512 x 2560 x 11008 and 16.4 against 15.6 at K = 8192; with two
// 32.8 against 36.1 at 1024 x 2048 x 24576 and 22.7 against 20.7 at K = 12288. All crossings were
// measured with mxfp4 and serve nvfp4 too, whose kernels take 4 to 15 % longer on both sides; the
// gated one at this one width and sum. A gated product of more than 64 rows is never split, so few
// tiles with a long sum (128 rows, 1024 outputs, K = 6144: 8 tiles) leave most pairs idle.
bool few_rows(const Mx4Gemm& g, int num_sms) {
  if (g.gated) return g.M <= kSkinnyGatedTokens;
  if (g.M <= 96) return true;
  const long long tiles = (long long)((g.M + 255) / 256) * ((g.N + 127) / 128);
  const int ki = (g.K + kStageK - 1) / kStageK;
  if (g.M <= 256 && tiles <= num_sms / 4 && ki > 32) return true;
  const long long ctas = 9 * num_sms / (10 * tiles);
  return ctas >= 6 ? ki >= 20 : ki >= 24 && ki * (ctas - 1) > 80;
}

template <int FMT, bool GATED>
cudaError_t launch_any(const Mx4Gemm& g, int num_sms, cudaStream_t s) {
  if (few_rows(g, num_sms)) return launch_skinny<FMT, GATED>(g, num_sms, s);
  return launch_pair<FMT, GATED>(g, num_sms, s);
}

}  // namespace

cudaError_t launch_gemm_mx4(const Mx4Gemm& g, int num_sms, cudaStream_t s) {
  if (g.fmt == kMxfp4)
    return g.gated ? launch_any<kMxfp4, true>(g, num_sms, s)
                   : launch_any<kMxfp4, false>(g, num_sms, s);
  return g.gated ? launch_any<kNvfp4, true>(g, num_sms, s)
                 : launch_any<kNvfp4, false>(g, num_sms, s);
}

}  // namespace mgt
