// Instances of the windowed attention forward kernel, dense tensors, fp16 operands.
#include "attn_window.cuh"

namespace fa {
template cudaError_t launch_attn_window<kFP16, 64, false, WIN_PAIR>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 128, false, WIN_PAIR>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 256, false, WIN_ONE>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 64, false, WIN_TWO>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 64, false, WIN_SPLIT>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 128, false, WIN_SPLIT>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 256, false, WIN_SPLIT>(const WinLaunch&);
}  // namespace fa
