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
    }
  }
  return 0;
}
