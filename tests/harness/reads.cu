// Test harness (host only): which chunks and vectors the kernels that read rows by aligned words take by elements, on
// numbers read from stdin, one JSON line each on stdout.  Built and run by tests/test_ssm_forms.py.
#include "../../depthwise_convolution_forward_gb300/csrc/sscan.cuh"

#include <cstdio>
#include <cstring>

using namespace gconv;

int main() {
  char what[16];
  long long a, b, c, d, e;
  while (scanf("%15s %lld %lld %lld %lld %lld", what, &a, &b, &c, &d, &e) == 6) {
    const bool is = !strcmp(what, "chunk") ? end_chunk(a, b, c, d) : end_vector(a, (int)b, c, (int)d, (int)e);
    printf("{\"ends\": %d, \"tokens\": %d}\n", (int)is, kChunk);
  }
  return 0;
}
