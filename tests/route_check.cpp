// Which kernel a chunk call takes (kvk_chunk_route.cuh); built and run by
// tests/test_chunk_route_host.py.
#include <cstdio>

#include "kvk_chunk_route.cuh"

int main() {
  struct Case {
    int path;
    bool tensor;
    int regs;
    bool fma;
    int want;
  };
  const int A = KVK_PATH_AUTO, T = KVK_PATH_TENSOR, C = KVK_PATH_CUDA_CORE, G = KVK_PATH_TENSOR_GENERAL;
  const Case cases[] = {
      {A, true, 128, true, T},   {A, true, -1, true, T},    // (a layout without a device)
      {A, true, 126, true, C},   {A, true, 0, true, C},     // built otherwise, or not known
      {A, true, 126, false, -1}, {A, false, 128, true, C},  {A, false, 128, false, -1},
      {T, true, 128, true, T},   {T, true, 126, true, -1},  {T, false, 128, true, -1},
      {G, true, 128, true, T},   {G, true, 120, true, -1},  {C, true, 128, true, C},
      {C, true, 128, false, -1},
  };
  int n = 0;
  for (const Case& c : cases) {
    const int got = kvk::chunk_route(c.path, c.tensor, c.regs, c.fma);
    if (got != c.want) return printf("case %d: %d, expected %d\n", n, got, c.want), 1;
    ++n;
  }
  printf("ok %d\n", n);
  return 0;
}
