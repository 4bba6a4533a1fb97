// Instances of the windowed attention forward kernel, paged key/value cache, fp16 operands.
#include "attn_window.cuh"

namespace fa {
template cudaError_t launch_attn_window<kFP16, 64, true, WIN_FEW2>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 64, true, WIN_ONE>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 64, true, WIN_PAIR>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 128, true, WIN_FEW>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 128, true, WIN_FEW2>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 128, true, WIN_ONE>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 128, true, WIN_PAIR>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 256, true, WIN_FEW>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 256, true, WIN_ONE>(const WinLaunch&);
}  // namespace fa
