// Host check of the cache of resident clusters behind the 4-bit products of few rows: each device, launch
// shape and cluster size has an answer of its own, asked for once; errors are not kept. Exit status 0
// on success.
#include <cstdio>

#include "../../tensor_transformer_layer_megatron_b200/csrc/mx4_internal.h"

int main() {
  static mgt::ResidentClusters cache;
  int bad = 0, asked = 0;
  auto answer = [](int dev, int shape, int size) { return 1000 * dev + 10 * shape + size; };
  for (int turn = 0; turn < 2; ++turn)
    for (int dev = 0; dev < 70; ++dev)
      for (int shape = 0; shape < 17; ++shape)
        for (int size = 2; size <= 8; ++size) {
          int n = -7;
          bad += cache.get(dev, shape, size, &n, [&](int* out) {
            ++asked;
            *out = answer(dev, shape, size);
            return cudaSuccess;
          }) != cudaSuccess;
          bad += n != answer(dev, shape, size);
        }
  // 64 devices once, six beyond them every time
  bad += asked != (64 + 2 * 6) * 17 * 7;
  static mgt::ResidentClusters fresh;
  int n = 0;
  for (int k = 0; k < 2; ++k)
    bad += fresh.get(1, 2, 3, &n, [](int*) { return cudaErrorInvalidValue; }) != cudaErrorInvalidValue;
  bad += fresh.get(1, 2, 3, &n, [](int* out) { return *out = 0, cudaSuccess; }) != cudaSuccess || n != 0;
  bad += fresh.get(1, 2, 3, &n, [](int*) { return cudaErrorInvalidValue; }) != cudaSuccess || n != 0;
  std::printf("%s (%d mismatches)\n", bad ? "FAIL" : "ok", bad);
  return bad ? 1 : 0;
}
