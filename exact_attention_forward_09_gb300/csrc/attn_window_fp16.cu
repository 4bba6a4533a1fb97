// Instances of the windowed attention forward kernel, dense tensors, fp16 operands.
#include "attn_window.cuh"

namespace fa {
template cudaError_t launch_attn_window<kFP16, 64, false>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 128, false>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 256, false>(const WinLaunch&);
}  // namespace fa
