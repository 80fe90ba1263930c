// A launch that the runtime refuses is reported once: the launch helpers leave no
// error behind that the thread's next launch would report although its kernel runs.
// Linked with --wrap for the two runtime calls below: they stand in for the runtime's,
// refuse a launch when told to and keep the last error as it does.  Needs no GPU.
// Exit code 0 = as expected.
#include <cstdio>

#include "common.cuh"

static cudaError_t next_result = cudaSuccess, last_error = cudaSuccess;
static int launches = 0;

extern "C" {
cudaError_t __wrap_cudaLaunchKernelExC(const cudaLaunchConfig_t *, const void *, void **) {
  ++launches;
  if (next_result != cudaSuccess) last_error = next_result;
  return next_result;
}
cudaError_t __wrap_cudaGetLastError() {
  const cudaError_t e = last_error;
  last_error = cudaSuccess;
  return e;
}
}

static void kernel(int) {}

template <typename F>
static bool check(const char *what, F launch) {
  next_result = cudaErrorInvalidConfiguration;
  const moe_status refused = launch();
  const cudaError_t left = last_error;
  next_result = cudaSuccess;
  const moe_status after = launch();
  std::printf("%s: refused %d, left behind %d, the next %d\n", what, (int)refused, (int)left, (int)after);
  return refused == MOE_ERR_CUDA && left == cudaSuccess && after == MOE_OK;
}

int main() {
  bool ok = check("programmatic", [] { return moe_host::launch_pdl(kernel, dim3(1), dim3(32), 0, nullptr, 1); });
  ok &= check("cooperative", [] { return moe_host::launch_coop_pdl(kernel, dim3(1), dim3(32), 0, nullptr, 1); });
  ok &= launches == 4;
  if (ok) std::printf("launch status ok\n");
  return !ok;
}
