// Internal interface between the C-ABI layer of the sequence operators
// (seq_api.cu) and their kernels.  Not installed, not part of the ABI.
#pragma once

#include "../../include/gconv_seq.h"
#include "kernels.h"

namespace gconv {

// A [B, T, D] tensor: element strides of batch and token.
struct SeqStride {
  int64_t b, t;
};

struct ConvSeqArgs {
  const void* x;
  const void* w;
  const void* bias;       // may be null
  const void* state_in;   // may be null
  const int32_t* lens;    // may be null
  void* y;
  void* state_out;        // may be null
  // backward only
  const void* dy;
  const void* dstate_out;  // may be null
  void* dx;
  void* dw;
  void* dbias;      // may be null
  void* dstate_in;  // may be null
  float* ws;
  int64_t B, T;
  int D, K, act;
  SeqStride sx, sy;
};
cudaError_t conv1d_fwd_launch(const ConvSeqArgs& c, const LaunchArgs& a, const DeviceInfo& dev);
cudaError_t conv1d_bwd_launch(const ConvSeqArgs& c, const LaunchArgs& a, const DeviceInfo& dev);
int64_t conv1d_bwd_workspace_bytes(int64_t B, int64_t T, int D, int K);

struct ScanArgs {
  const void* x;
  const void* r;
  const void* i;
  const float* lam;
  const float* h0;      // may be null
  const int32_t* lens;  // may be null
  void* y;
  float* hT;     // may be null
  float* saved;  // forward: may be null
  // backward only
  const void* dy;
  const float* dhT;  // may be null
  void* dx;
  void* dr;
  void* di;
  float* dlam;
  float* dh0;  // may be null
  float* ws;
  int64_t B, T;
  int D;
  float decay;
  SeqStride sx, sr, si, sy;
};
cudaError_t scan_fwd_launch(const ScanArgs& s, const LaunchArgs& a, const DeviceInfo& dev);
cudaError_t scan_bwd_launch(const ScanArgs& s, const LaunchArgs& a, const DeviceInfo& dev);
int64_t scan_saved_bytes(int64_t B, int64_t T, int D);
int64_t scan_bwd_workspace_bytes(int64_t B, int64_t T, int D);

struct NormArgs {
  const void* x;
  const void* res;  // may be null
  const void* w;    // may be null
  void* res_out;    // may be null
  void* y;          // may be null
  int8_t* q;        // may be null
  float* scale;     // null with q
  int64_t rows;
  int D;
  float eps;
  int64_t sx, sr, sy;
  bool norm;  // false: quantise the rows as they are
};
cudaError_t norm_q8_launch(const NormArgs& n, const LaunchArgs& a, const DeviceInfo& dev);

struct MatmulQ8Args {
  const int8_t* xq;
  const float* sx;
  const int8_t* wq;
  const float* sw;
  const void* bias;  // may be null
  void* y;
  int64_t M;
  int N, K;
  int64_t ys;
};
cudaError_t matmul_q8_launch(const MatmulQ8Args& m, const LaunchArgs& a, const DeviceInfo& dev);

// The current device's properties and status word (api.cu).
cudaError_t current_device(DeviceInfo* info, int** status);

}  // namespace gconv
