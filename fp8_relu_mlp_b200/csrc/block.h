// Host-side declarations of the block-scaled FP8 product, the gated norms and
// the optimizer step.
#pragma once

#include <atomic>

#include "gemm_block_sm100.cuh"
#include "internal.h"

namespace fp8mlp {

constexpr int kBlock = 128;  // elements that share one scale

namespace dev {

// magnitude bits of the largest of eight BF16 values (NaN above infinity
// above every finite value, so an integer max is exact)
__device__ __forceinline__ unsigned int amax8(const uint4& v) {
  const unsigned int w[4] = {v.x, v.y, v.z, v.w};
  unsigned int m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) m = max(m, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
  return m;
}

__device__ __forceinline__ uint2 quant8(const uint4& v, float s) {
  const unsigned int w[4] = {v.x, v.y, v.z, v.w};
  uint32_t q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) q[j] = pack_e4m3x2(__fmul_rn(bf16lo_to_f32(w[j]), s), __fmul_rn(bf16hi_to_f32(w[j]), s));
  return make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
}

}  // namespace dev

// Sets a kernel's shared memory limit once per device; two threads racing here
// set the same value.
template <class F>
cudaError_t allow_smem(F* kernel, std::atomic<bool> (&done)[64], int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < 64;
  if (known && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess && known) done[dev].store(true, std::memory_order_release);
  return e;
}

// whether a product of these sizes runs on 256 x 256 tiles of CTA pairs (else
// on 128 x 128 tiles of single CTAs)
bool block_gemm_pairs(int M, int N, int num_sms);
cudaError_t launch_block_gemm(bool relu2, bool pairs, BlockGemmParams& p, int num_sms, cudaStream_t s);

// the product for few rows; x: bf16, quantised on the way (xq and xs are
// written), or NULL: xq and xs are read
constexpr int kGemvMaxM = 8, kGemvMaxUp = 4;
// whether it is the faster form
bool block_gemv_fits(bool relu2, int M, int K, int N);
cudaError_t launch_block_gemv(int M, int K, int N, const uint16_t* x, uint8_t* xq, float* xs, const uint8_t* Wq,
                              const float* ws, uint16_t* y, int num_sms, cudaStream_t s);
cudaError_t launch_block_gemv_up(int M, int K, int N, const uint16_t* x, uint8_t* xq, float* xs, const uint8_t* Wq,
                                 const float* ws, uint16_t* post, uint8_t* post_q, float* post_s, cudaStream_t s);

cudaError_t launch_quantize_block(int M, int K, const uint16_t* x, uint8_t* xq, float* xs, cudaStream_t s);
cudaError_t launch_weight_block(int N, int K, const uint16_t* W, uint8_t* Wq, float* ws, uint8_t* Wq_t, float* ws_t,
                                cudaStream_t s);

// norms after a block and before the next one with gate and residual scale
constexpr int kNormMaxD = 8192;
struct NormGateFwd {
  int M, d, rows;
  float eps;
  const uint16_t *r, *y, *w_post, *gate, *w_pre;
  const float* alpha;
  uint16_t *r_next, *x;
  float *rstd_post, *rstd_pre;
  uint8_t* xq;
  float* xs;
};
cudaError_t launch_norm_gate_fwd(const NormGateFwd& p, cudaStream_t s);

struct NormGateBwd {
  int M, d, rows;
  const uint16_t *r, *y, *w_post, *gate, *w_pre;
  const float* alpha;
  const float *rstd_post, *rstd_pre;
  const uint16_t *r_next, *dx, *dr_next;
  uint16_t *dr, *dy;
  float *dw_post, *dgate, *dalpha, *dw_pre;
  float* workspace;
};
size_t norm_gate_bwd_workspace(int M, int d, int rows);
cudaError_t launch_norm_gate_bwd(const NormGateBwd& p, cudaStream_t s);

// optimizer
cudaError_t launch_adamw_state_init(fp8mlp_adamw_state* st, float lr, unsigned int seed, int step, cudaStream_t s);
size_t grad_norm_workspace(int n, const fp8mlp_adamw_tensor* t);
cudaError_t launch_grad_norm(int n, const fp8mlp_adamw_tensor* t, float max_norm, float* out, double* workspace,
                             cudaStream_t s);
cudaError_t launch_adamw(int n, const fp8mlp_adamw_tensor* t, fp8mlp_adamw_state* st, int state_bits, float beta1,
                         float beta2, float eps, const float* grad_coef, unsigned int* status, cudaStream_t s);

}  // namespace fp8mlp
