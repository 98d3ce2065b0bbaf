// Test harness (host only): the 8-bit product's planner and the scan's split and
// shared-memory sizes on problems read from stdin, one JSON line per problem on
// stdout.  Built and run by tests/test_seq_plans.py; nothing here launches a kernel.
#include "../../depthwise_convolution_forward_gb300/csrc/mmq.cu"
#include "../../depthwise_convolution_forward_gb300/csrc/scan.cu"

#include <cstdio>
#include <cstring>

namespace gconv {
CUresult encode_tiled(CUtensorMap*, CUtensorMapDataType, uint32_t, const void*, const uint64_t*, const uint64_t*,
                      const uint32_t*, const uint32_t*, CUtensorMapSwizzle) {
  return CUDA_ERROR_NOT_SUPPORTED;
}
}  // namespace gconv

using namespace gconv;

int main() {
  char what[16];
  long long a, b, c, sms;
  while (scanf("%15s %lld %lld %lld %lld", what, &a, &b, &c, &sms) == 5) {
    DeviceInfo dev{};
    dev.num_sms = (int)sms, dev.max_smem_optin = kDefaultSmemOptin;
    if (!strcmp(what, "matmul")) {
      MatmulQ8Args m{};
      m.M = a, m.N = (int)b, m.K = (int)c;
      TcPlan p{};
      if (!tc_plan(m, dev, &p)) {
        printf("{\"ok\": false}\n");
        continue;
      }
      printf("{\"ok\": true, \"BX\": %d, \"tiles\": %d, \"tiles_m\": %d, \"tiles_n\": %d, \"ksteps\": %d, \"raw_stages\": %d, "
             "\"raw_bytes\": %u, \"wide_bytes\": %u, \"teams\": %d, \"threads\": %d, \"wide_col\": %d, \"max_bx\": %d}\n",
             p.BX, p.tiles, p.tiles_m, p.tiles_n, p.ksteps, p.raw_stages, p.raw_bytes, p.wide_bytes, kTeams, kTcThreads,
             kWideCol, kMaxBX);
    } else if (!strcmp(what, "share")) {  // a product's M, N, K
      MatmulQ8Args m{};
      m.M = a, m.N = (int)b, m.K = (int)c;
      TcPlan p{};
      tc_plan(m, dev, &p);
      printf("{\"split\": %d, \"per\": %d, \"BX\": %d, \"tiles\": %d, \"ksteps\": %d, \"ring\": %u, \"most\": %d, \"room\": %d}\n",
             p.split, p.per, p.BX, p.tiles, p.ksteps, p.raw_stages * p.raw_bytes, kMaxShare, share_sms(p.split, dev.num_sms));
    } else {  // units, tokens in a sequence, tokens of a block's tile
      printf("{\"fwd\": %d, \"bwd\": %d, \"most\": %d, \"smem\": [%d, %d, %d, %d]}\n", split_of(a, b, (int)c, (int)sms, 3),
             split_of(a, b, (int)c, (int)sms, 1), kMaxSplit, ScanRing<2, 16, 4, 2, 3>::kBytes, ScanRing<1, 16, 4, 2, 3>::kBytes,
             ScanRing<2, 8, 8, 3, 4>::kBytes, ScanRing<1, 8, 8, 3, 4>::kBytes);
    }
  }
  return 0;
}
