// Host-side declarations of the block-scaled FP8 product, the gated norms and
// the optimizer step.
#pragma once

#include "gemm_block_sm100.cuh"
#include "internal.h"

namespace fp8mlp {

constexpr int kBlock = 128;  // elements that share one scale

// whether a product of these sizes runs on 256 x 256 tiles of CTA pairs (else
// on 128 x 128 tiles of single CTAs)
bool block_gemm_pairs(int M, int N, int num_sms);
cudaError_t launch_block_gemm(bool relu2, bool pairs, BlockGemmParams& p, int num_sms, cudaStream_t s);

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
