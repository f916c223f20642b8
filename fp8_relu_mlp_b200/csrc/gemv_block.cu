// The block-scaled FP8 product for few tokens:
//
//   y[m, n] = sum_kb xs[kb, m] ws[kb, n / 128] sum_{k in kb} xq[m, k] Wq[n, k]
//
// With up to eight rows the product is a pass over the weights, and what
// counts is latency: one launch instead of two, no tensor maps, and every SM
// takes part.  Each CTA quantises all of x (or unpacks its codes) to fp32 in
// shared memory while its first weights are under way; a warp then takes two
// rows of Wq at a time, 16 codes per lane and load.  e4m3 products are exact
// in fp32; a lane's sixteen belong to one scale block, so the factor
// xs * ws is applied once per sixteen.
#include <atomic>
#include <cmath>

#include "block.h"

namespace fp8mlp {

namespace {

using namespace dev;

constexpr int kThreads = 256;
constexpr int kRows = 2;    // of Wq per warp: neighbours, so of one weight block
constexpr int kAhead = 4;   // loads of 512 codes per row that are under way together
constexpr int kSmemMost = 96 * 1024;

// two e4m3 codes in the low half of v
__device__ __forceinline__ float2 e4m3x2_values(uint32_t v) {
  uint32_t h;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(v));
  float2 f;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
__device__ __forceinline__ float4 e4m3x4_values(uint32_t v) {
  const float2 a = e4m3x2_values(v), b = e4m3x2_values(v >> 16);
  return make_float4(a.x, a.y, b.x, b.y);
}

// x in shared memory: 16 values of a lane's step side by side, their four
// vectors swapped so that eight neighbouring lanes hit all banks
__device__ __forceinline__ int x_vec(int chunk, int q) { return chunk * 4 + (q ^ ((chunk >> 1) & 3)); }

// All of x to shared memory: [M][K / 4] vectors, then the scales [M][kblocks].
// x: bf16 (its codes and scales are written, by the first CTA), or NULL: the
// codes are read.
template <int M>
__device__ __forceinline__ void stage_x(int K, const uint16_t* __restrict__ x, uint8_t* xq, float* xs, float4* sx,
                                        float* sscale) {
  const int kblocks = (K + kBlock - 1) / kBlock;
  if (x != nullptr) {
    // sixteen lanes per group of 128
    const int sub = threadIdx.x & 15;
    for (int g0 = 0; g0 < M * kblocks; g0 += kThreads / 16) {  // uniform: the shuffles need whole warps
      const int g = g0 + (threadIdx.x >> 4);
      const int m = g / kblocks, kb = g - m * kblocks, k = kb * kBlock + sub * 8;
      const bool in = g < M * kblocks && k < K;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (in) v = __ldg(reinterpret_cast<const uint4*>(x + static_cast<size_t>(m) * K + k));
      unsigned int am = amax8(v);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
      float inv;
      const float s = block_scale(__uint_as_float(am << 16), &inv);
      if (in) {
        const uint2 q = quant8(v, s);
        float4* row = sx + static_cast<size_t>(m) * (K / 4);
        row[x_vec(k >> 4, (k >> 2) & 3)] = e4m3x4_values(q.x);
        row[x_vec(k >> 4, ((k >> 2) & 3) + 1)] = e4m3x4_values(q.y);
        if (blockIdx.x == 0) *reinterpret_cast<uint2*>(xq + static_cast<size_t>(m) * K + k) = q;
        if (sub == 0) {
          sscale[g] = inv;
          if (blockIdx.x == 0) xs[static_cast<size_t>(kb) * M + m] = inv;
        }
      }
    }
  } else {
    for (int i = threadIdx.x; i < M * (K / 16); i += kThreads) {
      const int m = i / (K / 16), c = i - m * (K / 16);
      const uint4 v = *reinterpret_cast<const uint4*>(xq + static_cast<size_t>(m) * K + c * 16);
      float4* row = sx + static_cast<size_t>(m) * (K / 4);
      row[x_vec(c, 0)] = e4m3x4_values(v.x);
      row[x_vec(c, 1)] = e4m3x4_values(v.y);
      row[x_vec(c, 2)] = e4m3x4_values(v.z);
      row[x_vec(c, 3)] = e4m3x4_values(v.w);
    }
    for (int i = threadIdx.x; i < M * kblocks; i += kThreads) {
      const int m = i / kblocks, kb = i - m * kblocks;
      sscale[i] = xs[static_cast<size_t>(kb) * M + m];
    }
  }
}

// Two rows of Wq against x: 512 codes of each per load, kAhead loads at once.
struct WRows {
  uint4 w[kAhead][kRows];
  __device__ __forceinline__ void load(const uint8_t* __restrict__ Wq, int K, int N, int n, int k0, int lane) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int k = k0 + a * 512 + lane * 16;
        w[a][r] = k < K && n + r < N ? __ldg(reinterpret_cast<const uint4*>(Wq + static_cast<size_t>(n + r) * K + k))
                                     : make_uint4(0, 0, 0, 0);
      }
  }
};

// acc[r][m], whole in every lane; `w` holds the first loads
template <int M>
__device__ __forceinline__ void rows_product(WRows& w, int K, int N, int n, const uint8_t* __restrict__ Wq,
                                             const float* __restrict__ ws, const float4* sx, const float* sscale, int lane,
                                             float (&acc)[kRows][M]) {
  const int kblocks = (K + kBlock - 1) / kBlock, n_blocks = (N + kBlock - 1) / kBlock;
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int m = 0; m < M; ++m) acc[r][m] = 0.f;
  const float* wsc = ws + (n >> 7);
  for (int k0 = 0; k0 < K; k0 += kAhead * 512) {
    if (k0 > 0) w.load(Wq, K, N, n, k0, lane);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int k = k0 + a * 512 + lane * 16;
      if (k < K) {
        const int kb = k >> 7, c = k >> 4;
        const float wf = __ldg(wsc + static_cast<size_t>(kb) * n_blocks);
        float f[kRows][16];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const uint32_t v[4] = {w.w[a][r].x, w.w[a][r].y, w.w[a][r].z, w.w[a][r].w};
#pragma unroll
          for (int q = 0; q < 4; ++q) *reinterpret_cast<float4*>(&f[r][4 * q]) = e4m3x4_values(v[q]);
        }
#pragma unroll
        for (int m = 0; m < M; ++m) {
          const float scale = __fmul_rn(sscale[m * kblocks + kb], wf);
          float p[kRows];
#pragma unroll
          for (int r = 0; r < kRows; ++r) p[r] = 0.f;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float4 xv = sx[static_cast<size_t>(m) * (K / 4) + x_vec(c, q)];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
              p[r] = fmaf(xv.x, f[r][4 * q], p[r]);
              p[r] = fmaf(xv.y, f[r][4 * q + 1], p[r]);
              p[r] = fmaf(xv.z, f[r][4 * q + 2], p[r]);
              p[r] = fmaf(xv.w, f[r][4 * q + 3], p[r]);
            }
          }
#pragma unroll
          for (int r = 0; r < kRows; ++r) acc[r][m] = fmaf(p[r], scale, acc[r][m]);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[r][m] += __shfl_xor_sync(0xffffffffu, acc[r][m], o);
}

template <int M>
__global__ void __launch_bounds__(kThreads) gemv_block_kernel(int K, int N, const uint16_t* __restrict__ x, uint8_t* xq,
                                                              float* xs, const uint8_t* __restrict__ Wq,
                                                              const float* __restrict__ ws, uint16_t* __restrict__ y) {
  pdl_wait();
  pdl_launch_dependents();
  extern __shared__ __align__(16) float4 sx[];
  float* sscale = reinterpret_cast<float*>(sx + static_cast<size_t>(M) * (K / 4));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int step = gridDim.x * (kThreads / 32) * kRows;
  int n = (blockIdx.x * (kThreads / 32) + warp) * kRows;
  WRows w;
  w.load(Wq, K, N, n, 0, lane);
  stage_x<M>(K, x, xq, xs, sx, sscale);
  __syncthreads();
  for (; n < N; n += step) {
    float acc[kRows][M];
    rows_product<M>(w, K, N, n, Wq, ws, sx, sscale, lane, acc);
    // N is even: a pair of columns per row of y
#pragma unroll
    for (int m = 0; m < M; ++m)
      if (lane == m) *reinterpret_cast<uint32_t*>(y + static_cast<size_t>(m) * N + n) = pack_bf16x2(acc[0][m], acc[1][m]);
    if (n + step < N) w.load(Wq, K, N, n + step, 0, lane);
  }
}

// The up-projection: a cluster of four CTAs per 128 columns, so that more SMs
// read weights; their row maxima meet through distributed shared memory.
constexpr int kCluster = 4;
template <int M>
__global__ void __launch_bounds__(kThreads)
    gemv_up_kernel(int K, int N, const uint16_t* __restrict__ x, uint8_t* xq, float* xs, const uint8_t* __restrict__ Wq,
                   const float* __restrict__ ws, uint16_t* __restrict__ post, uint8_t* __restrict__ post_q,
                   float* __restrict__ post_s) {
  pdl_wait();
  pdl_launch_dependents();
  extern __shared__ __align__(16) float4 sx[];
  __shared__ float val[M][kBlock / kCluster];  // relu(acc)^2 of this CTA's columns
  __shared__ float top[kCluster][M];
  float* sscale = reinterpret_cast<float*>(sx + static_cast<size_t>(M) * (K / 4));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int blk = blockIdx.x / kCluster, col0 = blk * kBlock + static_cast<int>(rank) * (kBlock / kCluster);
  int c = warp * 4;  // four columns per warp, two at a time
  WRows w;
  w.load(Wq, K, N, col0 + c, 0, lane);
  stage_x<M>(K, x, xq, xs, sx, sscale);
  cluster_sync();  // for x, and so that the others' shared memory is there to be written
#pragma unroll 1
  for (int i = 0; i < 2; ++i, c += kRows) {
    float acc[kRows][M];
    rows_product<M>(w, K, N, min(col0 + c, N - kRows), Wq, ws, sx, sscale, lane, acc);
    if (i == 0) w.load(Wq, K, N, col0 + c + kRows, 0, lane);
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const float a = col0 + c + r < N ? max_nan(acc[r][m], 0.f) : 0.f;
        if (lane == r * M + m) val[m][c + r] = __fmul_rn(a, a);
      }
  }
  __syncthreads();
  if (warp < M) {
    float a = val[warp][lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
    if (lane < kCluster) {
      const uint32_t dst = mapa_shared(smem_u32(&top[rank][warp]), lane);
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst), "f"(a) : "memory");
    }
  }
  cluster_sync();
  if (warp < M) {
    float a = top[0][warp];
#pragma unroll
    for (int k = 1; k < kCluster; ++k) a = max_nan(a, top[k][warp]);
    float inv;
    const float s = block_scale(a, &inv);
    const int n = col0 + lane;
    const float v = val[warp][lane];
    if (n < N) {
      post[static_cast<size_t>(warp) * N + n] = static_cast<uint16_t>(pack_bf16x2(v, 0.f));
      post_q[static_cast<size_t>(warp) * N + n] = static_cast<uint8_t>(pack_e4m3x2(__fmul_rn(v, s), 0.f));
    }
    if (rank == 0 && lane == 0) post_s[static_cast<size_t>(blk) * M + warp] = inv;
  }
}

size_t gemv_smem(int M, int K) { return static_cast<size_t>(M) * K * 4 + static_cast<size_t>(M) * ((K + 127) / 128) * 4; }

template <int M>
cudaError_t launch_up_m(int K, int N, const uint16_t* x, uint8_t* xq, float* xs, const uint8_t* Wq, const float* ws,
                        uint16_t* post, uint8_t* post_q, float* post_s, cudaStream_t s) {
  static std::atomic<bool> done[64] = {};
  cudaError_t e = allow_smem(gemv_up_kernel<M>, done, kSmemMost);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((N + kBlock - 1) / kBlock * kCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = gemv_smem(M, K);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, gemv_up_kernel<M>, K, N, x, xq, xs, Wq, ws, post, post_q, post_s);
  count_launches(1);
  return e;
}

template <int M>
cudaError_t launch_m(int K, int N, const uint16_t* x, uint8_t* xq, float* xs, const uint8_t* Wq, const float* ws,
                     uint16_t* y, int num_sms, cudaStream_t s) {
  static std::atomic<bool> done[64] = {};
  cudaError_t e = allow_smem(gemv_block_kernel<M>, done, kSmemMost);
  if (e != cudaSuccess) return e;
  const int need = (N + kThreads / 32 * kRows - 1) / (kThreads / 32 * kRows), most = (M == 1 ? 4 : 2) * num_sms;  // what the registers allow
  e = launch_pdl(gemv_block_kernel<M>, dim3(need < most ? need : most), dim3(kThreads), gemv_smem(M, K), s, K, N, x, xq,
                 xs, Wq, ws, y);
  count_launches(1);
  return e;
}

}  // namespace

// Estimated times of both forms in ns, fitted to 310 measured shapes (M 1 to 8,
// K 16 to 4096, N 16 to 50304, weights from HBM) and checked on 400 others.  The
// pass over the weights: a start, groups of 128 quantised or unpacked 16 at a
// time by every CTA, and per column the sums over lanes (by M) and loads of 512
// codes (by K); the up-projection's start has its clusters'.  The tensor cores: a
// start, a k-block after the other, and the weights' way.  Calls from BF16 rows,
// whose quantiser the pass takes along, and from codes take the same form, so
// that they give the same bits: the starts are the mean of both.  The choice
// takes 1 to 3 % more than the faster form on average and half as much again
// at most.  Us from BF16 rows: 1 x 768 -> 2304 2.6 by the pass and 5.8 by the
// tensor cores, 8 x 768 -> 4096 7.5 and 6.1, 8 x 512 -> 16384 15.3 and 8.5, 1 x 4096
// -> 50304 53 and 69; up-projection from codes 1 x 1024 -> 4096 5.8 and 6.1,
// 4 x 1024 -> 4096 6.4 and 6.1.
bool block_gemv_fits(bool relu2, int M, int K, int N) {
  if (M > (relu2 ? kGemvMaxUp : kGemvMaxM) || gemv_smem(M, K) > static_cast<size_t>(kSmemMost)) return false;
  const float kb = static_cast<float>((K + kBlock - 1) / kBlock), loads = static_cast<float>((K + 511) / 512);
  const float rounds = ceilf(M * kb / 16), m = static_cast<float>(M), n = static_cast<float>(N) * 1e-3f;
  float pass, tensor;
  if (relu2) {
    pass = 2325.f + 1250.f * rounds + n * (35.f + 65.f * m + loads * (150.f + 5.f * m));
    tensor = 3500.f + 260.f * kb + n * (120.f + 32.f * kb);
  } else {
    pass = 1125.f + 740.f * rounds + 85.f * m + n * (45.f * m + loads * (105.f + 20.f * m));
    tensor = 2900.f + 260.f * kb + n * (100.f + 26.f * kb);
  }
  return pass < tensor;
}

cudaError_t launch_block_gemv(int M, int K, int N, const uint16_t* x, uint8_t* xq, float* xs, const uint8_t* Wq,
                              const float* ws, uint16_t* y, int num_sms, cudaStream_t s) {
  switch (M) {
    case 1: return launch_m<1>(K, N, x, xq, xs, Wq, ws, y, num_sms, s);
    case 2: return launch_m<2>(K, N, x, xq, xs, Wq, ws, y, num_sms, s);
    case 3: return launch_m<3>(K, N, x, xq, xs, Wq, ws, y, num_sms, s);
    case 4: return launch_m<4>(K, N, x, xq, xs, Wq, ws, y, num_sms, s);
    case 5: return launch_m<5>(K, N, x, xq, xs, Wq, ws, y, num_sms, s);
    case 6: return launch_m<6>(K, N, x, xq, xs, Wq, ws, y, num_sms, s);
    case 7: return launch_m<7>(K, N, x, xq, xs, Wq, ws, y, num_sms, s);
    case 8: return launch_m<8>(K, N, x, xq, xs, Wq, ws, y, num_sms, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_block_gemv_up(int M, int K, int N, const uint16_t* x, uint8_t* xq, float* xs, const uint8_t* Wq,
                                 const float* ws, uint16_t* post, uint8_t* post_q, float* post_s, cudaStream_t s) {
  switch (M) {
    case 1: return launch_up_m<1>(K, N, x, xq, xs, Wq, ws, post, post_q, post_s, s);
    case 2: return launch_up_m<2>(K, N, x, xq, xs, Wq, ws, post, post_q, post_s, s);
    case 3: return launch_up_m<3>(K, N, x, xq, xs, Wq, ws, post, post_q, post_s, s);
    case 4: return launch_up_m<4>(K, N, x, xq, xs, Wq, ws, post, post_q, post_s, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fp8mlp
