// Test harness (host only): which vectors the kernel that reads rows by aligned words takes by elements, on
// numbers read from stdin, one JSON line each on stdout.  Built and run by tests/test_ssm_forms.py.
#include "../../depthwise_convolution_forward_gb300/csrc/seq_vec.cuh"

#include <cstdio>
#include <cstring>

using namespace gconv;

int main() {
  char what[16];
  long long a, b, c, d, e;
  while (scanf("%15s %lld %lld %lld %lld %lld", what, &a, &b, &c, &d, &e) == 6) {
    if (!strcmp(what, "vector")) printf("{\"ends\": %d}\n", (int)end_vector(a, (int)b, c, (int)d, (int)e));
  }
  return 0;
}
