// Quantisers of the block-scaled FP8 product.
#include "block.h"

namespace fp8mlp {

namespace {

using namespace dev;

// x [M,K] bf16 -> codes and inverse scales of groups of 128 along K.  HBM-bound:
// 16384 x 768 in 6.5 us (5.8 TB/s), 8192 x 4096 in 15.2 (6.6).  Sixteen
// lanes hold one group (16 bytes each), so its maximum takes four shuffles.
// A half-warp walks kGroups groups of one row, all loads first: 64 bytes in
// flight per thread keep HBM busy at 2048 threads per SM.
constexpr int kGroups = 4;
__global__ void __launch_bounds__(256) quantize_block_kernel(int M, int K, const uint16_t* __restrict__ x,
                                                             uint8_t* __restrict__ xq, float* __restrict__ xs) {
  pdl_wait();
  pdl_launch_dependents();
  const int sub = threadIdx.x & 15;
  const int m = blockIdx.x * 16 + (threadIdx.x >> 4);
  const int kb0 = blockIdx.y * kGroups;
  const bool row_ok = m < M;
  const size_t base = static_cast<size_t>(m) * K;
  uint4 v[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const int k = (kb0 + g) * kBlock + sub * 8;
    v[g] = make_uint4(0, 0, 0, 0);
    if (row_ok && k < K) v[g] = *reinterpret_cast<const uint4*>(x + base + k);
  }
  unsigned int top[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    top[g] = amax8(v[g]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top[g] = max(top[g], __shfl_xor_sync(0xffffffffu, top[g], o));
  }
  // lane g works out the scale of group g: two divisions for all of them
  unsigned int mine = top[0];
#pragma unroll
  for (int g = 1; g < kGroups; ++g) mine = sub == g ? top[g] : mine;
  float inv;
  const float s = block_scale(__uint_as_float(mine << 16), &inv);
  if (row_ok && sub < kGroups && (kb0 + sub) * kBlock < K) xs[static_cast<size_t>(kb0 + sub) * M + m] = inv;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const int k = (kb0 + g) * kBlock + sub * 8;
    const float sg = __shfl_sync(0xffffffffu, s, g, 16);
    if (row_ok && k < K) *reinterpret_cast<uint2*>(xq + base + k) = quant8(v[g], sg);
  }
}

// One 128 x 128 block of W [N,K] per CTA, read once into registers (eight
// 16-byte rows per thread): maximum, scale, codes, and the transposed codes
// through shared memory.  4096 x 1024 from HBM: 4.4 us the plain layout, 6.6 the
// transposed one, 6.8 both (floors 1.9, 1.9, 2.6: one round of 256 CTAs, bound by
// latency), 50304 x 768 20, 33 and 35 (17.7, 17.7, 23.6: the transposed codes go
// to shared memory byte by byte).
__global__ void __launch_bounds__(256) weight_block_kernel(int N, int K, const uint16_t* __restrict__ W,
                                                           uint8_t* __restrict__ Wq, float* __restrict__ ws,
                                                           uint8_t* __restrict__ Wq_t, float* __restrict__ ws_t) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ unsigned int wmax[8];
  __shared__ __align__(16) uint8_t tile[kBlock][kBlock + 4];  // [k][n]
  const int sub = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  const int kb = blockIdx.x, nb = blockIdx.y;
  const int k = kb * kBlock + sub * 8;
  uint4 v[8];
  unsigned int a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = nb * kBlock + r0 + 16 * i;
    v[i] = make_uint4(0, 0, 0, 0);
    if (n < N && k < K) v[i] = *reinterpret_cast<const uint4*>(W + static_cast<size_t>(n) * K + k);
    a = max(a, amax8(v[i]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = a;
  __syncthreads();
  a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, wmax[i]);
  float inv;
  const float s = block_scale(__uint_as_float(a << 16), &inv);
  if (threadIdx.x == 0) {
    if (ws != nullptr) ws[static_cast<size_t>(kb) * gridDim.y + nb] = inv;
    if (ws_t != nullptr) ws_t[static_cast<size_t>(nb) * gridDim.x + kb] = inv;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = nb * kBlock + r0 + 16 * i;
    const uint2 c = quant8(v[i], s);
    if (Wq != nullptr && n < N && k < K) *reinterpret_cast<uint2*>(Wq + static_cast<size_t>(n) * K + k) = c;
    if (Wq_t != nullptr) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        tile[sub * 8 + j][r0 + 16 * i] = static_cast<uint8_t>(c.x >> (8 * j));
        tile[sub * 8 + 4 + j][r0 + 16 * i] = static_cast<uint8_t>(c.y >> (8 * j));
      }
    }
  }
  if (Wq_t == nullptr) return;
  __syncthreads();
  // rows of Wq_t: 128 bytes each, eight bytes per lane (N is a multiple of 16)
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int kr = r0 + 16 * i;
    const int n = nb * kBlock + sub * 8;
    if (kb * kBlock + kr < K && n < N) {
      const uint32_t* src = reinterpret_cast<const uint32_t*>(&tile[kr][sub * 8]);
      *reinterpret_cast<uint2*>(Wq_t + static_cast<size_t>(kb * kBlock + kr) * N + n) = make_uint2(src[0], src[1]);
    }
  }
}

}  // namespace

cudaError_t launch_quantize_block(int M, int K, const uint16_t* x, uint8_t* xq, float* xs, cudaStream_t s) {
  const int kb = (K + kBlock - 1) / kBlock;
  const dim3 grid((M + 15) / 16, (kb + kGroups - 1) / kGroups);
  const cudaError_t e = launch_pdl(quantize_block_kernel, grid, dim3(256), 0, s, M, K, x, xq, xs);
  count_launches(1);
  return e;
}

cudaError_t launch_weight_block(int N, int K, const uint16_t* W, uint8_t* Wq, float* ws, uint8_t* Wq_t, float* ws_t,
                                cudaStream_t s) {
  const dim3 grid((K + kBlock - 1) / kBlock, (N + kBlock - 1) / kBlock);
  const cudaError_t e = launch_pdl(weight_block_kernel, grid, dim3(256), 0, s, N, K, W, Wq, ws, Wq_t, ws_t);
  count_launches(1);
  return e;
}

}  // namespace fp8mlp
