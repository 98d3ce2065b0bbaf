// Test harness (host only): the argument checks of the sequence operators' C ABI
// with launches that do nothing, so that a call which passes them can be told from
// one that is refused, with made-up addresses and without a GPU.  Built and loaded by
// tests/test_seq_overlap.py.
#include "../../depthwise_convolution_forward_gb300/csrc/seq_api.cu"

namespace gconv {
gconv_status set_last_error(gconv_status s, const char*, ...) { return s; }
cudaError_t current_device(DeviceInfo* info, int** status) {
  *info = DeviceInfo{0, kDefaultSms, kDefaultSmemOptin};
  *status = nullptr;
  return cudaSuccess;
}
cudaError_t conv1d_fwd_launch(const ConvSeqArgs&, const LaunchArgs&, const DeviceInfo&) { return cudaSuccess; }
cudaError_t conv1d_bwd_launch(const ConvSeqArgs&, const LaunchArgs&, const DeviceInfo&) { return cudaSuccess; }
cudaError_t scan_fwd_launch(const ScanArgs&, const LaunchArgs&, const DeviceInfo&) { return cudaSuccess; }
cudaError_t scan_bwd_launch(const ScanArgs&, const LaunchArgs&, const DeviceInfo&) { return cudaSuccess; }
cudaError_t norm_q8_launch(const NormArgs&, const LaunchArgs&, const DeviceInfo&) { return cudaSuccess; }
cudaError_t matmul_q8_launch(const MatmulQ8Args&, const LaunchArgs&, const DeviceInfo&) { return cudaSuccess; }
int64_t conv1d_bwd_workspace_bytes(int64_t, int64_t, int, int) { return 16; }
int64_t scan_saved_bytes(int64_t, int64_t, int) { return 16; }
int64_t scan_bwd_workspace_bytes(int64_t, int64_t, int) { return 16; }
}  // namespace gconv
