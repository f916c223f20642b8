// AdamW over many tensors, moments in fp32 or in 8 bits, and the gradient
// norm that clips it.
//
//   g' = coef g          m' = b1 m + (1 - b1) g'       v' = b2 v + (1 - b2) g'^2
//   p' = p - lr wd p - (lr / (1 - b1^t)) m' / (sqrt(v') / sqrt(1 - b2^t) + eps)
//
// Memory-bound: every array is read and written once.  The tensors'
// descriptors travel as kernel arguments (no device table to fill, nothing
// read from the host when a captured graph is replayed); a CTA finds its
// tensor by a binary search over the running count of chunks.  The products
// and sums are rounded one by one (no contraction), so the result does not
// depend on how the loop is compiled.
//
// 8-bit moments: blocks of 128 share a scale.  A warp holds a block, four
// elements per lane, so the block's maximum takes five shuffles.  v is held as
// sqrt(v), which halves the exponent range: e4m3 spans a factor 2^17.8 below
// the block's largest sqrt(v), 2^35 in v.  A positive sqrt(v) never becomes
// zero, or a small gradient's next step would divide by eps alone.  The codes
// are rounded stochastically: with round-to-nearest a moment whose change per
// step (1 - b2 of it) is under half a code step would never move again.
#include <climits>

#include "block.h"

namespace fp8mlp {

namespace {

using namespace dev;

constexpr int kMaxTensors = 48;       // descriptors per launch (kernel arguments hold 4 KB on every driver)
constexpr int kChunk = 4096;          // elements per CTA: 256 threads x 4 x 4
constexpr int kThreads = 256;

struct TensorArg {
  long long n;
  float* p;
  uint16_t* p_bf16;
  const float* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  float lr_mult, weight_decay;
};

struct AdamArgs {
  TensorArg t[kMaxTensors];
  int first_chunk[kMaxTensors + 1];
  int n_tensors;
  int tensor0;  // index of t[0] in the call (part of the random numbers)
  float beta1, beta2, om_beta1, om_beta2, eps;
  int last;  // this launch ends the call: the step count advances
  fp8mlp_adamw_state* st;
  const float* coef;
  unsigned int* status;
};

template <class Args>
__device__ __forceinline__ int find_tensor(const Args& a, int chunk) {
  int lo = 0, hi = a.n_tensors - 1;  // first_chunk[lo] <= chunk
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.first_chunk[mid] <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// the 32-bit finaliser of MurmurHash3 (A. Appleby, public domain)
__device__ __forceinline__ uint32_t mix32(uint32_t h) {
  h ^= h >> 16;
  h *= 0x85EBCA6Bu;
  h ^= h >> 13;
  h *= 0xC2B2AE35u;
  return h ^ (h >> 16);
}

// scaled value (|a| <= 448) -> the e4m3 value below or above it, the one above
// with the probability of its share of the step; u in [0, 1).  a / q and the
// multiplication back are by powers of two; q is the step of a's binade.
__device__ __forceinline__ float e4m3_stochastic(float a, float u) {
  const uint32_t mag = __float_as_uint(a) & 0x7FFFFFFFu;
  const uint32_t e = max(mag >> 23, 121u);  // exponents below -6 share the subnormal step 2^-9
  const float invq = __uint_as_float((257u - e) << 23), q = __uint_as_float((e - 3u) << 23);
  const float k = floorf(__fadd_rn(__fmul_rn(__uint_as_float(mag), invq), u));
  return copysignf(fminf(__fmul_rn(k, q), FP8MLP_E4M3_MAX), a);
}

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  // two codes -> two halves (exact); the upper one is unused
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(code & 0xFFu)));
  float f;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(h));
  return f;
}

struct StepScalars {
  float coef, size, inv_bc2;
};

struct Moments {
  float m, v;
};

__device__ __forceinline__ Moments moments(float m, float v, float g, const AdamArgs& a, float coef) {
  const float ge = __fmul_rn(g, coef);
  Moments r;
  r.m = __fadd_rn(__fmul_rn(m, a.beta1), __fmul_rn(ge, a.om_beta1));
  r.v = __fadd_rn(__fmul_rn(v, a.beta2), __fmul_rn(__fmul_rn(ge, ge), a.om_beta2));
  return r;
}

__device__ __forceinline__ float new_weight(float p, const Moments& x, float sqrt_v, float eps, float size, float inv_bc2,
                                            float decay) {
  const float den = __fadd_rn(__fmul_rn(sqrt_v, inv_bc2), eps);
  return __fsub_rn(__fsub_rn(p, __fmul_rn(p, decay)), __fmul_rn(__fdiv_rn(x.m, den), size));
}

__device__ __forceinline__ uint16_t bf16_stochastic(float x, uint32_t bits16) {
  const uint32_t u = __float_as_uint(x);
  if ((u & 0x7F800000u) == 0x7F800000u) return static_cast<uint16_t>(pack_bf16x2(x, 0.f));  // inf, NaN
  return static_cast<uint16_t>((u + bits16) >> 16);
}

// BITS: of the moments.  A warp takes blocks of 128 elements, four per lane.
template <int BITS>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ AdamArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ double corr[2];
  const int step = a.st->step + 1;
  const float lr = a.st->lr;
  const float coef = a.coef != nullptr ? *a.coef : 1.f;
  const uint32_t seed = a.st->seed;
  if (threadIdx.x < 2) {
    // beta^step by squaring, in double
    double b = threadIdx.x == 0 ? a.beta1 : a.beta2, r = 1.0;
    for (int k = step; k > 0; k >>= 1) {
      if (k & 1) r *= b;
      b *= b;
    }
    corr[threadIdx.x] = 1.0 - r;
  }
  __syncthreads();
  const bool skip = !(fabsf(coef) <= 3.4028234664e38f);  // a NaN or infinite coefficient: the step is not taken
  if (!skip) {
    const int ti = find_tensor(a, blockIdx.x);
    const TensorArg& t = a.t[ti];
    const float lr_t = __fmul_rn(lr, t.lr_mult);
    const float size = static_cast<float>(static_cast<double>(lr_t) / corr[0]);
    const float inv_bc2 = static_cast<float>(1.0 / sqrt(corr[1]));
    const float decay = __fmul_rn(lr_t, t.weight_decay);
    const uint32_t key = mix32(static_cast<uint32_t>(a.tensor0 + ti) * 0x9E3779B9u +
                               static_cast<uint32_t>(step) * 0x7F4A7C15u + seed);
    const long long base = static_cast<long long>(blockIdx.x - a.first_chunk[ti]) * kChunk;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 2
    for (int it = 0; it < kChunk / 1024; ++it) {
      const long long i0 = base + it * 1024 + warp * 128 + lane * 4;
      if (i0 - lane * 4 >= t.n) break;  // the whole warp is past the end
      const int valid = t.n - i0 >= 4 ? 4 : (t.n > i0 ? static_cast<int>(t.n - i0) : 0);
      const bool full = valid == 4;
      float g[4] = {0.f, 0.f, 0.f, 0.f}, p[4] = {0.f, 0.f, 0.f, 0.f};
      Moments x[4];
      float m[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
      const long long blk = i0 >> 7;
      if (full) {
        const float4 q = *reinterpret_cast<const float4*>(t.g + i0);
        g[0] = q.x, g[1] = q.y, g[2] = q.z, g[3] = q.w;
        if (t.p != nullptr) {
          const float4 w = *reinterpret_cast<const float4*>(t.p + i0);
          p[0] = w.x, p[1] = w.y, p[2] = w.z, p[3] = w.w;
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(t.p_bf16 + i0);
          p[0] = bf16lo_to_f32(w.x), p[1] = bf16hi_to_f32(w.x), p[2] = bf16lo_to_f32(w.y), p[3] = bf16hi_to_f32(w.y);
        }
        if constexpr (BITS == 32) {
          const float4 a4 = *reinterpret_cast<const float4*>(static_cast<const float*>(t.m) + i0);
          const float4 b4 = *reinterpret_cast<const float4*>(static_cast<const float*>(t.v) + i0);
          m[0] = a4.x, m[1] = a4.y, m[2] = a4.z, m[3] = a4.w;
          v[0] = b4.x, v[1] = b4.y, v[2] = b4.z, v[3] = b4.w;
        } else {
          const uint32_t cm = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.m) + i0);
          const uint32_t cv = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.v) + i0);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            m[k] = e4m3_value(cm >> (8 * k));
            v[k] = e4m3_value(cv >> (8 * k));
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k < valid) {
            g[k] = t.g[i0 + k];
            p[k] = t.p != nullptr ? t.p[i0 + k] : bf16lo_to_f32(t.p_bf16[i0 + k]);
            if constexpr (BITS == 32) {
              m[k] = static_cast<const float*>(t.m)[i0 + k];
              v[k] = static_cast<const float*>(t.v)[i0 + k];
            } else {
              m[k] = e4m3_value(static_cast<const uint8_t*>(t.m)[i0 + k]);
              v[k] = e4m3_value(static_cast<const uint8_t*>(t.v)[i0 + k]);
            }
          }
        }
      }
      if constexpr (BITS == 8) {
        const float sm = t.m_scale[blk], sv = t.v_scale[blk];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          m[k] = __fmul_rn(m[k], sm);
          v[k] = __fmul_rn(v[k], sv);
          v[k] = __fmul_rn(v[k], v[k]);
        }
      }
      float root[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[k] = moments(m[k], v[k], g[k], a, coef);
        root[k] = __fsqrt_rn(x[k].v);
        p[k] = new_weight(p[k], x[k], root[k], a.eps, size, inv_bc2, decay);
      }
      uint32_t bits[4];
      if (BITS == 8 || t.p == nullptr) {
#pragma unroll
        for (int k = 0; k < 4; ++k) bits[k] = mix32(mix32(static_cast<uint32_t>(i0 + k) ^ key) + key);
      }
      uint16_t w16[4];
      if (t.p != nullptr) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w16[k] = static_cast<uint16_t>(pack_bf16x2(p[k], 0.f));
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) w16[k] = bf16_stochastic(p[k], mix32(bits[k] ^ 0x5BD1E995u) & 0xFFFFu);
      }
      uint32_t cm = 0, cv = 0;
      if constexpr (BITS == 8) {
        float am = 0.f, av = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k < valid) {
            am = max_nan(am, fabsf(x[k].m));
            av = max_nan(av, root[k]);
          }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, o));
          av = max_nan(av, __shfl_xor_sync(0xffffffffu, av, o));
        }
        float im, iv;
        const float sm = block_scale(am, &im), sv = block_scale(av, &iv);
        if (lane == 0) {
          t.m_scale[blk] = im;
          t.v_scale[blk] = iv;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float um = static_cast<float>(bits[k] & 0xFFFFu) * 0x1p-16f, uv = static_cast<float>(bits[k] >> 16) * 0x1p-16f;
          const float em = fminf(fmaxf(__fmul_rn(x[k].m, sm), -FP8MLP_E4M3_MAX), FP8MLP_E4M3_MAX);
          const float ev = fminf(__fmul_rn(root[k], sv), FP8MLP_E4M3_MAX);
          float qm = e4m3_stochastic(em, um), qv = e4m3_stochastic(ev, uv);
          if (root[k] > 0.f && qv == 0.f) qv = 0x1p-9f;
          cm |= (pack_e4m3x2(qm, 0.f) & 0xFFu) << (8 * k);
          cv |= (pack_e4m3x2(qv, 0.f) & 0xFFu) << (8 * k);
        }
      }
      if (full) {
        if (t.p != nullptr) *reinterpret_cast<float4*>(t.p + i0) = make_float4(p[0], p[1], p[2], p[3]);
        if (t.p_bf16 != nullptr)
          *reinterpret_cast<uint2*>(t.p_bf16 + i0) =
              make_uint2(w16[0] | (static_cast<uint32_t>(w16[1]) << 16), w16[2] | (static_cast<uint32_t>(w16[3]) << 16));
        if constexpr (BITS == 32) {
          *reinterpret_cast<float4*>(static_cast<float*>(t.m) + i0) = make_float4(x[0].m, x[1].m, x[2].m, x[3].m);
          *reinterpret_cast<float4*>(static_cast<float*>(t.v) + i0) = make_float4(x[0].v, x[1].v, x[2].v, x[3].v);
        } else {
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.m) + i0) = cm;
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.v) + i0) = cv;
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k < valid) {
            if (t.p != nullptr) t.p[i0 + k] = p[k];
            if (t.p_bf16 != nullptr) t.p_bf16[i0 + k] = w16[k];
            if constexpr (BITS == 32) {
              static_cast<float*>(t.m)[i0 + k] = x[k].m;
              static_cast<float*>(t.v)[i0 + k] = x[k].v;
            } else {
              static_cast<uint8_t*>(t.m)[i0 + k] = static_cast<uint8_t>(cm >> (8 * k));
              static_cast<uint8_t*>(t.v)[i0 + k] = static_cast<uint8_t>(cv >> (8 * k));
            }
          }
        }
      }
    }
  }
  if (!a.last) return;
  // the last CTA to get here advances the step count: every CTA has read it
  // (a CTA arrives after its reads; launches of one call run one after another)
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    const unsigned int n = atomicAdd(&a.st->arrived, 1u);
    if (n == gridDim.x - 1) {
      a.st->arrived = 0;
      if (skip) {
        a.st->skipped += 1;
        atomicOr(a.status, static_cast<unsigned int>(FP8MLP_STATUS_STEP_SKIPPED));
      } else {
        a.st->step = step;
      }
      __threadfence();
    }
  }
}

__global__ void adamw_state_init_kernel(fp8mlp_adamw_state* st, float lr, unsigned int seed, int step) {
  pdl_wait();
  pdl_launch_dependents();
  st->lr = lr;
  st->step = step;
  st->seed = seed;
  st->arrived = 0;
  st->skipped = 0;
  for (int i = 0; i < 3; ++i) st->pad[i] = 0;
}

// ---- gradient norm ------------------------------------------------------------
// Squares and sums in double: fp32 squares overflow from 1.8e19 on and
// underflow below 1e-23, and 82 million terms lose digits.  A CTA's part goes
// to the workspace and one CTA adds the parts in a fixed order.
constexpr int kNormTensors = 128;
constexpr int kNormChunk = 16384;

struct NormArgs {
  const float* g[kNormTensors];
  long long n[kNormTensors];
  int first_chunk[kNormTensors + 1];
  int n_tensors;
  double* part;
};

__global__ void __launch_bounds__(kThreads) grad_sq_kernel(const __grid_constant__ NormArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ double sh[kThreads / 32];
  const int ti = find_tensor(a, blockIdx.x);
  const float* g = a.g[ti];
  const long long n = a.n[ti];
  const long long base = static_cast<long long>(blockIdx.x - a.first_chunk[ti]) * kNormChunk;
  double s0 = 0.0, s1 = 0.0;
#pragma unroll 4
  for (int it = 0; it < kNormChunk / (4 * kThreads); ++it) {
    const long long i = base + (it * kThreads + threadIdx.x) * 4;
    if (i + 4 <= n) {
      const float4 v = *reinterpret_cast<const float4*>(g + i);
      s0 = fma(static_cast<double>(v.x), static_cast<double>(v.x), s0);
      s1 = fma(static_cast<double>(v.y), static_cast<double>(v.y), s1);
      s0 = fma(static_cast<double>(v.z), static_cast<double>(v.z), s0);
      s1 = fma(static_cast<double>(v.w), static_cast<double>(v.w), s1);
    } else {
      for (long long k = i; k < n; ++k) s0 = fma(static_cast<double>(g[k]), static_cast<double>(g[k]), s0);
    }
  }
  double s = s0 + s1;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < kThreads / 32; ++k) s += sh[k];
    a.part[blockIdx.x] = s;
  }
}

__global__ void __launch_bounds__(1024) grad_norm_kernel(const double* part, long long n, float max_norm, float* out) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ double sh[32];
  double s = 0.0;
  for (long long i = threadIdx.x; i < n; i += 1024) s += part[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    for (int k = 0; k < 32; ++k) s += sh[k];
    const float norm = static_cast<float>(sqrt(s));
    out[0] = norm;
    // NaN where the norm is not finite, which makes the step skip itself
    out[1] = norm <= 3.4028234664e38f ? fminf(1.f, __fdiv_rn(max_norm, __fadd_rn(norm, 1e-6f))) : __int_as_float(0x7fc00000);
  }
}

long long chunks_of(long long n, int chunk) { return (n + chunk - 1) / chunk; }

}  // namespace

cudaError_t launch_adamw_state_init(fp8mlp_adamw_state* st, float lr, unsigned int seed, int step, cudaStream_t s) {
  const cudaError_t e = launch_pdl(adamw_state_init_kernel, dim3(1), dim3(1), 0, s, st, lr, seed, step);
  count_launches(1);
  return e;
}

size_t grad_norm_workspace(int n, const fp8mlp_adamw_tensor* t) {
  size_t parts = 0;
  for (int i = 0; i < n; ++i) parts += static_cast<size_t>(chunks_of(t[i].n, kNormChunk));
  return parts * sizeof(double);
}

cudaError_t launch_grad_norm(int n, const fp8mlp_adamw_tensor* t, float max_norm, float* out, double* workspace,
                             cudaStream_t s) {
  long long parts = 0;
  NormArgs a;
  a.n_tensors = 0;
  a.first_chunk[0] = 0;
  a.part = workspace;
  for (int i = 0; i <= n; ++i) {
    const bool flush = i == n || a.n_tensors == kNormTensors;
    if (flush && a.n_tensors > 0) {
      const int grid = a.first_chunk[a.n_tensors];
      const cudaError_t e = launch_pdl(grad_sq_kernel, dim3(grid), dim3(kThreads), 0, s, a);
      count_launches(1);
      if (e != cudaSuccess) return e;
      parts += grid;
      a.part = workspace + parts;
      a.n_tensors = 0;
    }
    if (i == n) break;
    if (t[i].n == 0) continue;
    a.g[a.n_tensors] = t[i].g;
    a.n[a.n_tensors] = t[i].n;
    a.first_chunk[a.n_tensors + 1] = a.first_chunk[a.n_tensors] + static_cast<int>(chunks_of(t[i].n, kNormChunk));
    ++a.n_tensors;
  }
  const cudaError_t e = launch_pdl(grad_norm_kernel, dim3(1), dim3(1024), 0, s, static_cast<const double*>(workspace),
                                   parts, max_norm, out);
  count_launches(1);
  return e;
}

cudaError_t launch_adamw(int n, const fp8mlp_adamw_tensor* t, fp8mlp_adamw_state* st, int state_bits, float beta1,
                         float beta2, float eps, const float* grad_coef, unsigned int* status, cudaStream_t s) {
  AdamArgs a;
  a.beta1 = beta1;
  a.beta2 = beta2;
  a.om_beta1 = static_cast<float>(1.0 - static_cast<double>(beta1));
  a.om_beta2 = static_cast<float>(1.0 - static_cast<double>(beta2));
  a.eps = eps;
  a.st = st;
  a.coef = grad_coef;
  a.status = status;
  int last = -1;  // the last tensor with elements
  for (int i = 0; i < n; ++i)
    if (t[i].n > 0) last = i;
  for (int i = 0; i <= last;) {
    a.n_tensors = 0;
    a.first_chunk[0] = 0;
    a.tensor0 = i;
    // consecutive tensors: the random numbers go by a tensor's place in the call
    for (; i <= last && a.n_tensors < kMaxTensors; ++i) {
      TensorArg& d = a.t[a.n_tensors];
      d.n = t[i].n;
      d.p = t[i].p;
      d.p_bf16 = t[i].p_bf16;
      d.g = t[i].g;
      d.m = t[i].m;
      d.v = t[i].v;
      d.m_scale = t[i].m_scale;
      d.v_scale = t[i].v_scale;
      d.lr_mult = t[i].lr_mult;
      d.weight_decay = t[i].weight_decay;
      a.first_chunk[a.n_tensors + 1] = a.first_chunk[a.n_tensors] + static_cast<int>(chunks_of(t[i].n, kChunk));
      ++a.n_tensors;
    }
    a.last = i > last;
    const int grid = a.first_chunk[a.n_tensors];
    if (grid == 0) continue;  // only empty tensors, and more to come
    const cudaError_t e = state_bits == 32 ? launch_pdl(adamw_kernel<32>, dim3(grid), dim3(kThreads), 0, s, a)
                                           : launch_pdl(adamw_kernel<8>, dim3(grid), dim3(kThreads), 0, s, a);
    count_launches(1);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace fp8mlp
