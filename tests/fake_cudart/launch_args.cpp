// launch_args.cpp -- the runtime without a GPU (fake_cudart.cpp), which also
// notes what the first launch of the attention over the 8-bit cache is given.
#define cudaLaunchKernelExC counted_launch
#include "fake_cudart.cpp"
#undef cudaLaunchKernelExC

// (launch_fields.cu)
extern "C" void attention_workspace(const void* args, const void** ws, unsigned long long* bytes);

namespace {
const void* g_ws;
unsigned long long g_ws_bytes;
}  // namespace

extern "C" {
// (cache_attention_kernel takes a tensor map and its arguments)
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* cfg, const void* kernel, void** args) {
  if (g_launches == 0) attention_workspace(args[1], &g_ws, &g_ws_bytes);
  return counted_launch(cfg, kernel, args);
}
const void* fake_workspace() { return g_ws; }
unsigned long long fake_workspace_bytes() { return g_ws_bytes; }
}
