// Instances of the windowed attention forward kernel, trees over a paged key/value cache, fp16 operands.
#include "attn_window.cuh"

namespace fa {
template cudaError_t launch_attn_window<kFP16, 64, true, WIN_FEW2, true>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 64, true, WIN_ONE, true>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 64, true, WIN_PAIR, true>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 128, true, WIN_FEW, true>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 128, true, WIN_FEW2, true>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 128, true, WIN_ONE, true>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 128, true, WIN_PAIR, true>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 256, true, WIN_FEW, true>(const WinLaunch&);
template cudaError_t launch_attn_window<kFP16, 256, true, WIN_ONE, true>(const WinLaunch&);
}  // namespace fa
