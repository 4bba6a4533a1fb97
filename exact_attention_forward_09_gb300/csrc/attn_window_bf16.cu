// Instances of the windowed attention forward kernel, dense tensors, bf16 operands.
#include "attn_window.cuh"

namespace fa {
template cudaError_t launch_attn_window<kBF16, 64, false, WIN_PAIR>(const WinLaunch&);
template cudaError_t launch_attn_window<kBF16, 128, false, WIN_PAIR>(const WinLaunch&);
template cudaError_t launch_attn_window<kBF16, 256, false, WIN_ONE>(const WinLaunch&);
template cudaError_t launch_attn_window<kBF16, 64, false, WIN_TWO>(const WinLaunch&);
template cudaError_t launch_attn_window<kBF16, 64, false, WIN_SPLIT>(const WinLaunch&);
template cudaError_t launch_attn_window<kBF16, 128, false, WIN_SPLIT>(const WinLaunch&);
template cudaError_t launch_attn_window<kBF16, 256, false, WIN_SPLIT>(const WinLaunch&);

int window_clusters(int dev, int n) {
  // (what a d = 128 CTA needs leaves room for no second one, as every WIN_SPLIT CTA does)
  using C = WinCfg<kBF16, 128, false, WIN_SPLIT>;
  static int known[64][4] = {};
  const int k = n == 8 ? 3 : n == 4 ? 2 : 1;
  if (dev < 0 || dev >= 64) return 0;
  if (known[dev][k] == 0) {
    auto kern = attn_window_kernel<kBF16, 128, false, WIN_SPLIT, false>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)n, 1, 1);
    cfg.blockDim = dim3(C::THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)n;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int count = 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&count, kern, &cfg) != cudaSuccess || count < 1) {
      cudaGetLastError();
      count = -1;  // clusters of this size do not run here
    }
    known[dev][k] = count;
  }
  return known[dev][k];
}
}  // namespace fa
