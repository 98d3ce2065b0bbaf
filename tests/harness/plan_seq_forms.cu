// Test harness (host only): the plans of the 8-bit product's form without TMA, the
// scan's splits as its launchers take them, and the rings of shared memory that they
// ask for, on problems read from stdin, one JSON line per problem on stdout.  Built and
// run by tests/test_seq_forms.py; nothing here launches a kernel.
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
    if (!strcmp(what, "any")) {  // M, N, K
      MatmulQ8Args m{};
      m.M = a, m.N = (int)b, m.K = (int)c;
      TcPlan p{};
      const bool ok = tc_plan(m, dev, &p, true);
      printf("{\"ok\": %s, \"BX\": %d, \"tiles_m\": %d, \"tiles_n\": %d, \"tiles\": %d, \"ksteps\": %d, \"split\": %d, \"per\": %d, "
             "\"ring\": %u, \"wide\": %u, \"places\": %d, \"most\": %d}\n",
             ok ? "true" : "false", p.BX, p.tiles_m, p.tiles_n, p.tiles, p.ksteps, p.split, p.per, p.raw_stages * p.raw_bytes,
             kTeams * p.wide_bytes, kTeams * kWideW * kStageBytes, share_sms(p.split, dev.num_sms));
    } else {  // slabs of all sequences, tokens of a sequence, bytes of an element
      const bool wide = c == 4;
      printf("{\"fwd\": %d, \"bwd\": %d, \"most\": %d, \"six\": [%d, %d], \"eight\": [%d, %d], \"forward\": [%d, %d]}\n",
             wide ? fwd_split<float>(a, b, 64, (int)sms) : fwd_split<__half>(a, b, 64, (int)sms),
             split_of(a, b, 64, (int)sms, wide ? 2 : 1), kMaxSplit, ScanRing<2, 8, 6, 2, 4>::kBytes, ScanRing<1, 8, 6, 2, 4>::kBytes,
             ScanRing<2, 8, 8, 3, 4>::kBytes, ScanRing<1, 8, 8, 3, 4>::kBytes, ScanRing<2, 16, 4, 2, 3>::kBytes,
             ScanRing<1, 16, 4, 2, 3>::kBytes);
    }
  }
  return 0;
}
