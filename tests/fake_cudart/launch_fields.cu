// launch_fields.cu -- the workspace among the arguments of the attention over the 8-bit cache.
#include "../../gemm_pt_block_gb300/csrc/internal.h"

extern "C" void attention_workspace(const void* args, const void** ws, unsigned long long* bytes) {
  const auto* a = static_cast<const mx::AttentionArgs*>(args);
  *ws = a->ws;
  *bytes = a->ws_bytes;
}
