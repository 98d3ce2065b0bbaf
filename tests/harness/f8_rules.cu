// Test harness (host only): rules of the 8-bit floating-point product that a host can run, on numbers read from stdin,
// one JSON line each on stdout.  Built and run by tests/test_ssm_forms.py; nothing here launches a kernel.
#include "../../depthwise_convolution_forward_gb300/csrc/mmf8.cu"

#include <cstdio>
#include <cstring>

namespace gconv {
CUresult encode_tiled(CUtensorMap*, CUtensorMapDataType, uint32_t, const void*, const uint64_t*, const uint64_t*,
                      const uint32_t*, const uint32_t*, CUtensorMapSwizzle) {
  return CUDA_SUCCESS;
}
}  // namespace gconv

using namespace gconv;

int main() {
  char what[16];
  int a, b, c, d;
  while (scanf("%15s %d %d %d %d", what, &a, &b, &c, &d) == 5) {
    if (!strcmp(what, "ring")) {  // steps, stages
      const OpenSteps o = open_steps(a, b);
      printf("{\"from\": %d, \"stage\": %d, \"phase\": %u}\n", o.from, o.stage, o.phase);
    } else if (!strcmp(what, "ymap")) {  // N, row stride, bytes of an element, offset of y
      MatmulF8Args m{};
      m.M = 256, m.N = a, m.ys = b, m.y = reinterpret_cast<void*>((uintptr_t)(4096 + d));
      CUtensorMap map;
      printf("{\"map\": %d}\n", (int)y_map(&map, m, c == 4 ? kF32 : kBF16));
    }
  }
  return 0;
}
