// Instances of the windowed attention forward kernel, dense tensors, bf16 operands.
#include "attn_window.cuh"

namespace fa {
template cudaError_t launch_attn_window<kBF16, 64, false>(const WinLaunch&);
template cudaError_t launch_attn_window<kBF16, 128, false>(const WinLaunch&);
template cudaError_t launch_attn_window<kBF16, 256, false>(const WinLaunch&);
}  // namespace fa
