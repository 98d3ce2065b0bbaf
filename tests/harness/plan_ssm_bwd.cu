// Test harness (host only): the selective scan's backward plan, its workspace and the sizes that both directions
// take, for problems read from stdin, one JSON line each on stdout.  Built and run by tests/test_ssm_forms.py.
#include "../../depthwise_convolution_forward_gb300/csrc/sscan_bwd.cu"

#include <cstdio>

using namespace gconv;

int main() {
  long long B, T, D, N, G;
  while (scanf("%lld %lld %lld %lld %lld", &B, &T, &D, &N, &G) == 5) {
    const bool fits = ssm_fits(B, T, (int)D, (int)N, (int)G);
    const SsmPlan p = fits ? bwd_plan(B, T, (int)D, (int)N, (int)G) : SsmPlan{};
    const Parts q = fits ? parts_of(p, B, T, (int)D, (int)N, (int)G) : Parts{};
    SsmArgs s{};
    s.B = B, s.T = T, s.D = (int)D, s.N = (int)N, s.G = (int)G;
    int64_t mix = 0;
    const int64_t blocks = fits ? sum_blocks(s, &mix) : 0;
    printf("{\"fits\": %s, \"CC\": %d, \"tpg\": %d, \"S\": %d, \"seg\": %lld, \"chunk\": %d, \"lanes\": %d, \"cols\": %lld, \"ends\": %lld, "
           "\"sums\": %lld, \"all\": %lld, \"sum_blocks\": %lld}\n",
           fits ? "true" : "false", p.CC, p.tpg, p.S, (long long)p.seg, kChunk, lanes_of((int)N), (long long)q.cols,
           (long long)q.ends, (long long)q.sums, (long long)q.all, (long long)blocks);
  }
  return 0;
}
