// Host check of the few-row 4-bit product's launch shapes, for every number of tokens, both formats, gated
// or not: what the kernel places in shared and tensor memory, counted again, fits what it is given.
// Exit status 0 on success.
#include <cstdio>

#include "../../tensor_transformer_layer_megatron_b200/csrc/mx4_internal.h"

int main() {
  int bad = 0, shapes = 0;
  for (int nv = 0; nv < 2; ++nv)
    for (int gated = 0; gated < 2; ++gated)
      for (int M = 1; M <= (gated ? mgt::kSkinnyGatedTokens : 1000); ++M) {
        const mgt::SkinnyShape s = mgt::skinny_shape(nv, gated, M);
        const int nm = gated ? 2 : 1, t = s.tokens;
        bool ok = t == (M <= 256 ? (M + 15) / 16 * 16 : 256);
        ok = ok && s.stages >= 2;
        // a stage: 128 bytes of each row of the operands, 512 bytes of scales per 128 rows and scale tile
        const int operands = nm * 128 * 128 + t * 128;
        const int tiles = (nm + (t > 128 ? 2 : 1)) * (nv ? 4 : 2);
        ok = ok && s.stage_bytes == operands + tiles * 512;
        // up to 1023 bytes to align, stages, two barriers a stage, one more, tensor-memory slot and flag
        const int used = 1023 + s.stages * (operands + tiles * 512) + (2 * s.stages + 1) * 8 + 8;
        ok = ok && used <= s.smem;
        // an SM has 228 KB, of which every CTA takes 1 KB beside its own
        ok = ok && (s.smem + 1024) * (s.two ? 2 : 1) <= 228 * 1024;
        // the partial tiles overwrite the operands only: scales of other copies are not under them
        ok = ok && nm * t * 128 * 4 <= s.stages * operands;
        // accumulators in whole 32-column reads, four columns a scale tile and stage
        const int cols = nm * ((t + 31) / 32 * 32) + s.stages * tiles * 4;
        ok = ok && cols <= s.tmem_cols && s.tmem_cols * (s.two ? 2 : 1) <= 512 && s.tmem_cols >= 32 &&
             (s.tmem_cols & (s.tmem_cols - 1)) == 0;
        if (!ok) std::printf("nv %d gated %d M %d: %d tokens, %d stages\n", nv, gated, M, t, s.stages);
        bad += !ok;
        ++shapes;
      }
  if (bad) std::printf("FAIL (%d of %d)\n", bad, shapes);
  else std::printf("ok (%d shapes)\n", shapes);
  return bad ? 1 : 0;
}
