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
// Measured over 42.5 M elements: fp32 states 211 to 220 us (30 bytes an element,
// 6.0 to 5.8 TB/s; on BF16 weights alone 169, 24 bytes), 8-bit states 173 us (18
// bytes: here the 113 instructions an element bound it, 15 of them random bits,
// 19 the rounded division and square root; the SMs issue in 4 of 5 cycles), on
// BF16 weights alone 179 (126 instructions); the norm 31 us (5.5 TB/s).
//
// 8-bit moments: blocks of 128 share a scale.  v is held as
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

constexpr int kFew = 64, kMany = 256;  // descriptors per launch: as kernel arguments (at most 32764 bytes)
constexpr int kThreads = 256;
constexpr int kStep = 8 * kThreads;  // elements a CTA takes at a time: two blocks of 128 per warp
constexpr int kSms = 148;

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

template <int CAP>
struct AdamArgs {
  TensorArg t[CAP];
  int first_chunk[CAP + 1];
  int n_tensors;
  int steps;    // per chunk, the CTAs' unit of work
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

// Scaled value (|a| <= 448) -> the e4m3 value below or above it, the one above
// with the probability of its share of the step: floor(|a| / q + u) q, with q
// the step of a's binade and u in [0, 1) a multiple of 2^-16.
//
// From 2^-6 on, q is 2^-3 of the binade, so |a| / q + u is the mantissa with u
// added 20 bits below the ones that stay, and a carry moves on to the next
// binade by itself: one integer addition and a mask.
__device__ __forceinline__ float stochastic_normal(float a, uint32_t u16) {
  return __uint_as_float((__float_as_uint(a) + (u16 << 4)) & 0xFFF00000u);
}
// Below 2^-6 the step is 2^-9.
__device__ __forceinline__ float stochastic_subnormal(float a, uint32_t u16) {
  const float u = __uint_as_float(0x3F800000u + (u16 << 7)) - 1.f;  // u16 2^-16
  const float k = __fadd_rd(__fmaf_rn(fabsf(a), 512.f, u), 0x1p23f) - 0x1p23f;  // floor
  return copysignf(k * 0x1p-9f, a);
}

// four e4m3 codes -> values (exact)
__device__ __forceinline__ void e4m3x4_values(uint32_t codes, float (&f)[4]) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(f[0]), "=f"(f[1])
      : "r"(lo));
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(f[2]), "=f"(f[3])
      : "r"(hi));
}

// A product that goes into a sum: as two single ones, since a packed product
// followed by a packed sum is contracted to one rounding whatever its modifier.
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  float x, y, u, v;
  f2_unpack(a, x, y);
  f2_unpack(b, u, v);
  return f2_pack(__fmul_rn(x, u), __fmul_rn(y, v));
}

// Two elements' step: m, v in and out, sqrt(v) and the weight out.  A
// difference is a sum with the factor's sign turned.
struct StepScalars {
  uint64_t beta1, beta2, om_beta1, om_beta2, coef, inv_bc2, eps, nsize, ndecay;
};
__device__ __forceinline__ uint64_t both(float x) { return f2_pack(x, x); }

__device__ __forceinline__ void step2(float (&p)[2], float (&m)[2], float (&v)[2], float (&root)[2], const float (&g)[2],
                                      const StepScalars& c) {
  const uint64_t ge = f2_mul(f2_pack(g[0], g[1]), c.coef);
  f2_unpack(f2_add(mul2(f2_pack(m[0], m[1]), c.beta1), mul2(ge, c.om_beta1)), m[0], m[1]);
  f2_unpack(f2_add(mul2(f2_pack(v[0], v[1]), c.beta2), mul2(f2_mul(ge, ge), c.om_beta2)), v[0], v[1]);
  root[0] = __fsqrt_rn(v[0]);
  root[1] = __fsqrt_rn(v[1]);
  float den[2];
  f2_unpack(f2_add(mul2(f2_pack(root[0], root[1]), c.inv_bc2), c.eps), den[0], den[1]);
  const uint64_t q = f2_pack(__fdiv_rn(m[0], den[0]), __fdiv_rn(m[1], den[1])), w = f2_pack(p[0], p[1]);
  f2_unpack(f2_add(f2_add(w, mul2(w, c.ndecay)), mul2(q, c.nsize)), p[0], p[1]);
}

__device__ __forceinline__ uint32_t bf16_stochastic(float x, uint32_t bits16) {
  return x == x ? (__float_as_uint(x) + bits16) >> 16 : 0x7FFFu;  // an infinity keeps its exponent
}

// Four elements from a, or the first `valid` of them and zeros (FULL: all).
template <bool FULL>
__device__ __forceinline__ void load4(const float* a, int valid, float (&f)[4]) {
  if constexpr (FULL) {
    const float4 q = *reinterpret_cast<const float4*>(a);
    f[0] = q.x, f[1] = q.y, f[2] = q.z, f[3] = q.w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = k < valid ? a[k] : 0.f;
  }
}
template <bool FULL>
__device__ __forceinline__ void load4(const uint16_t* a, int valid, float (&f)[4]) {
  if constexpr (FULL) {
    const uint2 w = *reinterpret_cast<const uint2*>(a);
    f[0] = bf16lo_to_f32(w.x), f[1] = bf16hi_to_f32(w.x), f[2] = bf16lo_to_f32(w.y), f[3] = bf16hi_to_f32(w.y);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = k < valid ? bf16lo_to_f32(a[k]) : 0.f;
  }
}
template <bool FULL>
__device__ __forceinline__ uint32_t load4(const uint8_t* a, int valid) {
  if constexpr (FULL) return *reinterpret_cast<const uint32_t*>(a);
  uint32_t w = 0;
  for (int k = 0; k < valid; ++k) w |= static_cast<uint32_t>(a[k]) << (8 * k);
  return w;
}
template <bool FULL>
__device__ __forceinline__ void store4(float* a, int valid, const float (&f)[4]) {
  if constexpr (FULL) {
    *reinterpret_cast<float4*>(a) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < valid) a[k] = f[k];
  }
}
template <bool FULL>
__device__ __forceinline__ void store4(uint16_t* a, int valid, uint2 w) {
  if constexpr (FULL) {
    *reinterpret_cast<uint2*>(a) = w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < valid) a[k] = static_cast<uint16_t>((k < 2 ? w.x : w.y) >> (16 * (k & 1)));
  }
}
template <bool FULL>
__device__ __forceinline__ void store4(uint8_t* a, int valid, uint32_t w) {
  if constexpr (FULL) {
    *reinterpret_cast<uint32_t*>(a) = w;
  } else {
    for (int k = 0; k < valid; ++k) a[k] = static_cast<uint8_t>(w >> (8 * k));
  }
}

// One warp, 256 elements from `base` on (fewer without FULL).
template <int BITS, bool FULL>
__device__ __forceinline__ void warp_step(const TensorArg& t, const StepScalars& sc, long long base, int lane, uint32_t key) {
  const long long i = base + lane * 4;  // and + 128
  int valid[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const long long left = t.n - i - b * 128;
    valid[b] = FULL || left >= 4 ? 4 : left > 0 ? static_cast<int>(left) : 0;
  }
  float g[2][4], p[2][4], m[2][4], v[2][4], root[2][4];
  uint32_t cm[2], cv[2];
  const float* gp = t.g + i;
  float* pp = t.p + i;
  uint16_t* p16 = t.p_bf16 + i;
  float *m32 = static_cast<float*>(t.m) + i, *v32 = static_cast<float*>(t.v) + i;
  uint8_t *m8 = static_cast<uint8_t*>(t.m) + i, *v8 = static_cast<uint8_t*>(t.v) + i;
  const long long blk = base >> 7;
  float sm[2], sv[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    load4<FULL>(gp + b * 128, valid[b], g[b]);
    if (t.p != nullptr)
      load4<FULL>(pp + b * 128, valid[b], p[b]);
    else
      load4<FULL>(p16 + b * 128, valid[b], p[b]);
    if constexpr (BITS == 32) {
      load4<FULL>(m32 + b * 128, valid[b], m[b]);
      load4<FULL>(v32 + b * 128, valid[b], v[b]);
    } else {
      cm[b] = load4<FULL>(m8 + b * 128, valid[b]);
      cv[b] = load4<FULL>(v8 + b * 128, valid[b]);
      const bool in = FULL || (blk + b) * 128 < t.n;
      sm[b] = in ? t.m_scale[blk + b] : 0.f;
      sv[b] = in ? t.v_scale[blk + b] : 0.f;
    }
  }
  uint32_t bits[2][4];
  if (BITS == 8 || t.p == nullptr) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        bits[b][k] = mix32(mix32(static_cast<uint32_t>(i + b * 128 + k) ^ key) + key);
        asm volatile("" : "+r"(bits[b][k]));  // once: the compiler would compute them again for each use
      }
  }
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    if constexpr (BITS == 8) {
      e4m3x4_values(cm[b], m[b]);
      e4m3x4_values(cv[b], v[b]);
      const uint64_t s1 = both(sm[b]), s2 = both(sv[b]);
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        f2_unpack(f2_mul(f2_pack(m[b][k], m[b][k + 1]), s1), m[b][k], m[b][k + 1]);
        const uint64_t u = f2_mul(f2_pack(v[b][k], v[b][k + 1]), s2);
        f2_unpack(f2_mul(u, u), v[b][k], v[b][k + 1]);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      float tp[2] = {p[b][k], p[b][k + 1]}, tm[2] = {m[b][k], m[b][k + 1]}, tv[2] = {v[b][k], v[b][k + 1]}, tr[2];
      const float tg[2] = {g[b][k], g[b][k + 1]};
      step2(tp, tm, tv, tr, tg, sc);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        p[b][k + j] = tp[j];
        m[b][k + j] = tm[j];
        v[b][k + j] = tv[j];
        root[b][k + j] = tr[j];
      }
    }
    if (t.p != nullptr) {
      store4<FULL>(pp + b * 128, valid[b], p[b]);
      if (t.p_bf16 != nullptr)
        store4<FULL>(p16 + b * 128, valid[b], make_uint2(pack_bf16x2(p[b][0], p[b][1]), pack_bf16x2(p[b][2], p[b][3])));
    } else {
      // bits of their own: the moments use up all 32, and shared ones would tie
      // a weight's rounding to its moments'
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = bf16_stochastic(p[b][k], mix32(bits[b][k] ^ 0x5BD1E995u) & 0xFFFFu);
      store4<FULL>(p16 + b * 128, valid[b], make_uint2((w[0] & 0xFFFFu) | (w[1] << 16), (w[2] & 0xFFFFu) | (w[3] << 16)));
    }
    if constexpr (BITS == 32) {
      store4<FULL>(m32 + b * 128, valid[b], m[b]);
      store4<FULL>(v32 + b * 128, valid[b], v[b]);
    }
  }
  if constexpr (BITS == 8) {
    // block maxima, as integers: magnitudes order like their bits, NaN above
    // infinity; elements past the end are zero
    uint32_t top[4];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const float am = max3_nan(max_nan(fabsf(m[b][0]), fabsf(m[b][1])), fabsf(m[b][2]), fabsf(m[b][3]));
      const float av = max3_nan(max_nan(root[b][0], root[b][1]), root[b][2], root[b][3]);
      top[b] = __reduce_max_sync(0xffffffffu, __float_as_uint(am) & 0x7FFFFFFFu);
      top[2 + b] = __reduce_max_sync(0xffffffffu, __float_as_uint(av) & 0x7FFFFFFFu);
    }
    const int q = lane >> 3;  // m of block 0 and 1, v of block 0 and 1
    float inv;
    const float s = block_scale(__uint_as_float(q == 0 ? top[0] : q == 1 ? top[1] : q == 2 ? top[2] : top[3]), &inv);
    if ((lane & 7) == 0 && (FULL || (blk + (q & 1)) * 128 < t.n)) (q < 2 ? t.m_scale : t.v_scale)[blk + (q & 1)] = inv;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const float s1 = __shfl_sync(0xffffffffu, s, b * 8), s2 = __shfl_sync(0xffffffffu, s, 16 + b * 8);
      const uint64_t s1x2 = both(s1), s2x2 = both(s2);
      float em[4], ev[4], qm[4], qv[4];
      uint32_t low = 0xFFFFFFFFu;  // bits of the smallest magnitude above zero, twice, less one
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        f2_unpack(f2_mul(f2_pack(m[b][k], m[b][k + 1]), s1x2), em[k], em[k + 1]);
        f2_unpack(f2_mul(f2_pack(root[b][k], root[b][k + 1]), s2x2), ev[k], ev[k + 1]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t w = bits[b][k];
        qm[k] = stochastic_normal(em[k], w & 0xFFFFu);
        qv[k] = stochastic_normal(ev[k], w >> 16);
        low = min(low, min(2u * __float_as_uint(em[k]) - 1u, 2u * __float_as_uint(ev[k]) - 1u));
      }
      // magnitudes below 2^-6 are rare; a positive sqrt(v) so far below its
      // block's largest that the product is zero needs a scale under 2^-54
      if (low < 2u * 0x3C800000u - 1u || s2 < 0x1p-50f) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t w = bits[b][k];
          const float sub_m = stochastic_subnormal(em[k], w & 0xFFFFu), sub_v = stochastic_subnormal(ev[k], w >> 16);
          qm[k] = fabsf(em[k]) < 0x1p-6f ? sub_m : qm[k];
          qv[k] = ev[k] < 0x1p-6f ? (root[b][k] > 0.f ? fmaxf(sub_v, 0x1p-9f) : 0.f) : qv[k];
        }
      }
      store4<FULL>(m8 + b * 128, valid[b], pack_e4m3x2(qm[0], qm[1]) | (pack_e4m3x2(qm[2], qm[3]) << 16));
      store4<FULL>(v8 + b * 128, valid[b], pack_e4m3x2(qv[0], qv[1]) | (pack_e4m3x2(qv[2], qv[3]) << 16));
    }
  }
}

// BITS: of the moments.  CTAs are persistent (the powers of beta take as long
// as a chunk).  A warp takes two blocks of 128 elements at a time, four
// elements of each per lane; its four block maxima take one integer reduction
// each, and a quarter of the warp works out each block's scale.
template <int BITS, int CAP>
__global__ void __launch_bounds__(kThreads, BITS == 8 ? 4 : 3) adamw_kernel(const __grid_constant__ AdamArgs<CAP> a) {
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
  const int chunks = skip ? 0 : a.first_chunk[a.n_tensors];
  StepScalars sc;
  sc.beta1 = both(a.beta1);
  sc.beta2 = both(a.beta2);
  sc.om_beta1 = both(a.om_beta1);
  sc.om_beta2 = both(a.om_beta2);
  sc.coef = both(coef);
  sc.inv_bc2 = both(static_cast<float>(1.0 / sqrt(corr[1])));
  sc.eps = both(a.eps);
  sc.nsize = sc.ndecay = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int known = -1;  // tensor that sc's last two and the key belong to
  uint32_t key = 0;
  for (int chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x) {
    const int ti = find_tensor(a, chunk);
    const TensorArg& t = a.t[ti];
    if (ti != known) {
      const float lr_t = __fmul_rn(lr, t.lr_mult);
      sc.nsize = both(-static_cast<float>(static_cast<double>(lr_t) / corr[0]));
      sc.ndecay = both(-__fmul_rn(lr_t, t.weight_decay));
      key = mix32(static_cast<uint32_t>(a.tensor0 + ti) * 0x9E3779B9u + static_cast<uint32_t>(step) * 0x7F4A7C15u + seed);
      known = ti;
    }
    long long base = (static_cast<long long>(chunk - a.first_chunk[ti]) * a.steps * 8 + warp) * 256;
#pragma unroll 1
    for (int k = 0; k < a.steps; ++k, base += kStep) {
      if (base >= t.n) break;
      if (base + 256 <= t.n)
        warp_step<BITS, true>(t, sc, base, lane, key);
      else
        warp_step<BITS, false>(t, sc, base, lane, key);
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
#pragma unroll 1
  for (int it = 0; it < kNormChunk / (4 * kThreads); it += 8) {
    const long long i0 = base + (it * kThreads + threadIdx.x) * 4;
    if (i0 + 28 * kThreads + 4 <= n) {
      float4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = *reinterpret_cast<const float4*>(g + i0 + 4 * kThreads * k);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        s0 = fma(static_cast<double>(v[k].x), static_cast<double>(v[k].x), s0);
        s1 = fma(static_cast<double>(v[k].y), static_cast<double>(v[k].y), s1);
        s0 = fma(static_cast<double>(v[k].z), static_cast<double>(v[k].z), s0);
        s1 = fma(static_cast<double>(v[k].w), static_cast<double>(v[k].w), s1);
      }
    } else {
      for (int k = 0; k < 8; ++k)
        for (long long i = i0 + 4 * kThreads * k, e = i + 4; i < e && i < n; ++i)
          s0 = fma(static_cast<double>(g[i]), static_cast<double>(g[i]), s0);
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

template <int CAP>
cudaError_t launch_adamw_cap(int n, const fp8mlp_adamw_tensor* t, fp8mlp_adamw_state* st, int state_bits, float beta1,
                             float beta2, float eps, const float* grad_coef, unsigned int* status, cudaStream_t s) {
  AdamArgs<CAP> a;
  a.beta1 = beta1;
  a.beta2 = beta2;
  a.om_beta1 = static_cast<float>(1.0 - static_cast<double>(beta1));
  a.om_beta2 = static_cast<float>(1.0 - static_cast<double>(beta2));
  a.eps = eps;
  a.st = st;
  a.coef = grad_coef;
  a.status = status;
  int last = -1;  // the last tensor with elements
  long long all = 0;
  for (int i = 0; i < n; ++i) {
    if (t[i].n > 0) last = i;
    all += t[i].n;
  }
  // chunks of up to eight steps, as long as every CTA gets four of them
  const int most = kSms * (state_bits == 8 ? 4 : 3);
  const long long fit = all / (static_cast<long long>(kStep) * most * 4);
  a.steps = fit < 1 ? 1 : fit > 8 ? 8 : static_cast<int>(fit);
  for (int i = 0; i <= last;) {
    a.n_tensors = 0;
    a.first_chunk[0] = 0;
    a.tensor0 = i;
    // consecutive tensors: the random numbers go by a tensor's place in the call
    for (; i <= last && a.n_tensors < CAP; ++i) {
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
      a.first_chunk[a.n_tensors + 1] = a.first_chunk[a.n_tensors] + static_cast<int>(chunks_of(t[i].n, a.steps * kStep));
      ++a.n_tensors;
    }
    a.last = i > last;
    const int chunks = a.first_chunk[a.n_tensors];
    if (chunks == 0) continue;  // only empty tensors, and more to come
    const dim3 grid(chunks < most ? chunks : most);
    const cudaError_t e = state_bits == 32 ? launch_pdl(adamw_kernel<32, CAP>, grid, dim3(kThreads), 0, s, a)
                                           : launch_pdl(adamw_kernel<8, CAP>, grid, dim3(kThreads), 0, s, a);
    count_launches(1);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

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
  return n <= kFew ? launch_adamw_cap<kFew>(n, t, st, state_bits, beta1, beta2, eps, grad_coef, status, s)
                   : launch_adamw_cap<kMany>(n, t, st, state_bits, beta1, beta2, eps, grad_coef, status, s);
}

}  // namespace fp8mlp
