// Attention of drafted trees on tensor cores: not there yet, every plan takes the
// CUDA-core kernel (tree_simt.cu).
#include "rpa_internal.h"

namespace rpa {

bool tree_tc_supported(int32_t, int32_t, int32_t) { return false; }
int launch_tree_attn(const Plan& plan, const Args& a, void* stream) { return launch_tree_simt(plan, a, stream); }

}  // namespace rpa
