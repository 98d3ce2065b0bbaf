// Test harness (host only): two threads raise one kernel's shared-memory limit, the
// smaller setting slower than the larger one.  Prints the limit that is left, which has
// to be the larger.  The driver call is a stand-in.  Built and run by
// tests/test_smem_attr.py.
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>

enum cudaError_t { cudaSuccess = 0, cudaErrorInvalidDevice = 101 };
enum cudaFuncAttribute { cudaFuncAttributeMaxDynamicSharedMemorySize = 8 };
std::atomic<int> limit{0}, calls{0}, in_small{0};
template <typename F>
cudaError_t cudaFuncSetAttribute(F*, cudaFuncAttribute, int bytes) {
  ++calls;
  if (bytes == 100) {
    in_small = 1;
    for (int k = 0; k < 200 && limit != 200; ++k) std::this_thread::sleep_for(std::chrono::milliseconds(1));
  }
  limit = bytes;
  return cudaSuccess;
}

#include "../../depthwise_convolution_forward_gb300/csrc/plan_cache.h"

void kernel() {}

int main() {
  gconv::SmemAttr attr;
  std::thread small([&] { attr.ensure(kernel, 0, 100); });
  while (!in_small) std::this_thread::yield();
  std::thread large([&] { attr.ensure(kernel, 0, 200); });
  small.join();
  large.join();
  const int both = calls;
  attr.ensure(kernel, 0, 50), attr.ensure(kernel, 0, 200);
  printf("%d %d %d\n", (int)limit, both, calls - both);
  return 0;
}
