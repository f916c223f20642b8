// Instantiations and launches of the block-scaled FP8 GEMM.
#include <atomic>

#include "block.h"

namespace fp8mlp {

namespace {

// large problems: 256 x 256 tiles of a CTA pair
using CfgLin2 = BlockCfg<2, 256, 5, false>;
using CfgUp2 = BlockCfg<2, 256, 4, true>;
// few tiles: 128 x 128 tiles of one CTA, so that more SMs take part
using CfgLin1 = BlockCfg<1, 128, 5, false>;
using CfgUp1 = BlockCfg<1, 128, 5, true>;

constexpr int kMaxDevices = 64;

template <class C>
cudaError_t launch_cfg(BlockGemmParams& p, int num_sms, cudaStream_t s) {
  // set once per device; two threads racing here set the same value
  static std::atomic<bool> attr_done[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices || !attr_done[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(gemm_block_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    if (C::SPLIT_REGS) {
      // the epilogue's larger share has to be there to be taken, or it would wait for good
      cudaFuncAttributes fa;
      e = cudaFuncGetAttributes(&fa, gemm_block_kernel<C>);
      if (e != cudaSuccess) return e;
      if (fa.numRegs * C::THREADS < C::REGS_SUM) return cudaErrorLaunchOutOfResources;
    }
    if (dev >= 0 && dev < kMaxDevices) attr_done[dev].store(true, std::memory_order_release);
  }
  p.tiles_m = (p.M + C::TILE_M - 1) / C::TILE_M;
  p.tiles_n = (p.N + C::BN - 1) / C::BN;
  const long long tiles = static_cast<long long>(p.tiles_m) * p.tiles_n;
  const int units = num_sms / C::CG;
  const int grid = static_cast<int>(tiles < units ? tiles : units) * C::CG;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(C::THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C::CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, gemm_block_kernel<C>, p);
  count_launches(1);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

bool block_gemm_pairs(int M, int N, int num_sms) {
  const long long big = static_cast<long long>((M + 255) / 256) * ((N + 255) / 256);
  return 2 * big > num_sms / 2;
}

cudaError_t launch_block_gemm(bool relu2, bool pairs, BlockGemmParams& p, int num_sms, cudaStream_t s) {
  if (pairs) return relu2 ? launch_cfg<CfgUp2>(p, num_sms, s) : launch_cfg<CfgLin2>(p, num_sms, s);
  return relu2 ? launch_cfg<CfgUp1>(p, num_sms, s) : launch_cfg<CfgLin1>(p, num_sms, s);
}

}  // namespace fp8mlp
