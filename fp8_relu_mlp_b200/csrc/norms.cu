// Norms after one block and before the next, fused with the gate and the
// residual scale, and their gradient.
//
//   n  = y * rstd(y)               r' = alpha r + gate (n w_post)
//   x  = r' * rstd(r') * w_pre     (and the e4m3 copy of x, one scale per 1 x 128)
//
// Memory-bound: the row is read once into registers, both norms and the
// quantiser work on it there, and every output is rounded once from fp32.  A
// worker owns a row: a warp where a lane can hold its share (d <= 1024), else
// a CTA.
#include "block.h"

namespace fp8mlp {

namespace {

using namespace dev;

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const unsigned int w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = bf16lo_to_f32(w[j]);
    f[2 * j + 1] = bf16hi_to_f32(w[j]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ uint4 ones8() {
  return make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
}

__device__ __forceinline__ uint4 load8(const uint16_t* p, int c) { return *reinterpret_cast<const uint4*>(p + c); }

// sums of N values over the worker's threads; `red` is two buffers used in
// turn, so that one barrier per call is enough
template <bool CTA, int N>
__device__ __forceinline__ void worker_sum(float (&v)[N], float (*red)[32][N], int& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if constexpr (CTA) {
    const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[turn][warp][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
    for (int k = 0; k < nw; ++k) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += red[turn][k][i];
    }
    turn ^= 1;
  }
}

// VPT 16-byte vectors per thread; CTA: one row per CTA, else one per warp
template <int VPT, bool CTA>
__global__ void __launch_bounds__(256) norm_gate_fwd_kernel(const NormGateFwd p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float red[2][32][1];
  int turn = 0;
  const int tpr = CTA ? blockDim.x : 32;
  const int t = CTA ? threadIdx.x : threadIdx.x & 31;
  const int workers = CTA ? gridDim.x : gridDim.x * (blockDim.x >> 5);
  const int first = CTA ? blockIdx.x : blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const bool post = p.y != nullptr, pre = p.x != nullptr;
  const float alpha = p.alpha != nullptr ? *p.alpha : 1.f;
  const float inv_d = 1.f / static_cast<float>(p.d);
  for (int m = first; m < p.M; m += workers) {
    const size_t base = static_cast<size_t>(m) * p.d;
    uint4 vr[VPT], vy[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = (t + j * tpr) * 8;
      vr[j] = vy[j] = make_uint4(0, 0, 0, 0);
      if (c < p.d) {
        vr[j] = load8(p.r + base, c);
        if (post) vy[j] = load8(p.y + base, c);
      }
    }
    float rn[VPT][8];
    float sum[1];
    if (post) {
      sum[0] = 0.f;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        float y[8];
        unpack8(vy[j], y);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[0] = fmaf(y[i], y[i], sum[0]);
      }
      worker_sum<CTA>(sum, red, turn);
      const float b = __fdiv_rn(1.f, __fsqrt_rn(fmaf(sum[0], inv_d, p.eps)));
      if (t == 0) p.rstd_post[m] = b;
      const uint16_t* gate = p.gate != nullptr ? p.gate + static_cast<size_t>(m / p.rows) * p.d : nullptr;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int c = (t + j * tpr) * 8;
        float r[8], y[8], g[8], wp[8];
        unpack8(vr[j], r);
        unpack8(vy[j], y);
        unpack8(gate != nullptr && c < p.d ? load8(gate, c) : ones8(), g);
        unpack8(p.w_post != nullptr && c < p.d ? load8(p.w_post, c) : ones8(), wp);
#pragma unroll
        for (int i = 0; i < 8; ++i) rn[j][i] = fmaf(g[i], y[i] * b * wp[i], alpha * r[i]);
        if (c < p.d) *reinterpret_cast<uint4*>(p.r_next + base + c) = pack8(rn[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < VPT; ++j) unpack8(vr[j], rn[j]);
    }
    if (!pre) continue;
    sum[0] = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[0] = fmaf(rn[j][i], rn[j][i], sum[0]);
    worker_sum<CTA>(sum, red, turn);
    const float a = __fdiv_rn(1.f, __fsqrt_rn(fmaf(sum[0], inv_d, p.eps)));
    if (t == 0) p.rstd_pre[m] = a;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = (t + j * tpr) * 8;
      float x[8], wp[8];
      unpack8(p.w_pre != nullptr && c < p.d ? load8(p.w_pre, c) : ones8(), wp);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = rn[j][i] * a * wp[i];
      if (c < p.d) *reinterpret_cast<uint4*>(p.x + base + c) = pack8(x);
      if (p.xq != nullptr) {
        // sixteen lanes hold one group of 128 columns
        float am = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) am = max_nan(am, fabsf(x[i]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, o));
        float inv;
        const float s = block_scale(am, &inv);
        if (c < p.d) {
          uint32_t q[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) q[i] = pack_e4m3x2(__fmul_rn(x[2 * i], s), __fmul_rn(x[2 * i + 1], s));
          *reinterpret_cast<uint2*>(p.xq + base + c) = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
          if ((t & 15) == 0) p.xs[static_cast<size_t>(c >> 7) * p.M + m] = inv;
        }
      }
    }
  }
}

// ---- gradient ---------------------------------------------------------------
// With xh = r' rstd_pre, n = y rstd_post, gw = gate w_post and
// E = dr_next + rstd_pre w_pre dx:
//   D  = dL/dr' = E - rstd_pre xh c1,        c1 = mean(w_pre dx xh)
//   dr = alpha D
//   dy = rstd_post (D gw - n c2),            c2 = mean(D gw n)
// c2 needs D, but mean(D gw n) = mean(E gw n) - rstd_pre c1 mean(xh gw n), so
// the three sums are taken in one pass and one reduction.  The sums over the
// rows (gains, gate, alpha) stay in each worker's registers; a worker walks
// units, a unit being a run of rows of one gate row, and a second kernel adds
// the workers' parts in a fixed order.
struct NormBwdSplit {
  int workers;  // each owns one partial row of the gains' gradients
  int slices;   // units per gate row
  int len;      // rows per unit
  int groups;   // gate rows
};

constexpr int kBwdWarpCtas = 296;  // CTAs in warp mode: two per SM
constexpr int kBwdWarps = 4;
constexpr int kBwdCtas = 592;      // CTAs in CTA mode: four per SM

__host__ __device__ inline bool bwd_by_cta(int d) { return d > 768; }

NormBwdSplit norm_bwd_split(int M, int d, int rows) {
  NormBwdSplit s;
  const int rpg = rows < M ? rows : M;
  s.groups = (M + rpg - 1) / rpg;
  const int most = bwd_by_cta(d) ? kBwdCtas : kBwdWarpCtas * kBwdWarps;
  int n = (most + s.groups - 1) / s.groups;
  if (n > rpg) n = rpg;
  s.len = (rpg + n - 1) / n;
  s.slices = (rpg + s.len - 1) / s.len;
  const long long units = static_cast<long long>(s.groups) * s.slices;
  s.workers = units < most ? static_cast<int>(units) : most;
  return s;
}

template <int VPT, bool CTA>
__global__ void __launch_bounds__(CTA ? 512 : 32 * kBwdWarps) norm_gate_bwd_kernel(const NormGateBwd p, const NormBwdSplit sp) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float red[2][32][3];
  int turn = 0;
  const int tpr = CTA ? blockDim.x : 32;
  const int t = CTA ? threadIdx.x : threadIdx.x & 31;
  const int me = CTA ? blockIdx.x : blockIdx.x * kBwdWarps + (threadIdx.x >> 5);
  if (me >= sp.workers) return;  // whole warps (or CTAs) leave
  const bool post = p.y != nullptr, pre = p.dx != nullptr;
  const float alpha = p.alpha != nullptr ? *p.alpha : 1.f;
  const float inv_d = 1.f / static_cast<float>(p.d);
  const int rpg = p.rows < p.M ? p.rows : p.M;
  float* part_gain = p.workspace;  // [2][workers][d]
  float* part_gate = part_gain + 2 * static_cast<size_t>(sp.workers) * p.d;  // [units][d] when slices > 1
  float swpre[VPT][8], swpost[VPT][8];
  double salpha = 0.0;
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) swpre[j][i] = swpost[j][i] = 0.f;

  const long long units = static_cast<long long>(sp.groups) * sp.slices;
  for (long long u = me; u < units; u += sp.workers) {
    const int g = static_cast<int>(u / sp.slices);
    const int sl = static_cast<int>(u - static_cast<long long>(g) * sp.slices);
    const int g0 = g * rpg;  // < M
    const int gend = p.M - g0 < rpg ? p.M : g0 + rpg;
    const int m0 = gend - g0 < sl * sp.len ? gend : g0 + sl * sp.len;
    const int m1 = gend - m0 < sp.len ? gend : m0 + sp.len;
    float sgate[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) sgate[j][i] = 0.f;
    const uint16_t* gate = p.gate != nullptr ? p.gate + static_cast<size_t>(g) * p.d : nullptr;
    for (int m = m0; m < m1; ++m) {
      const size_t base = static_cast<size_t>(m) * p.d;
      const float a = pre ? p.rstd_pre[m] : 0.f, b = post ? p.rstd_post[m] : 0.f;
      uint4 vrn[VPT], vdx[VPT], vdr[VPT], vy[VPT], vr[VPT];
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int c = (t + j * tpr) * 8;
        const uint4 z = make_uint4(0, 0, 0, 0);
        vrn[j] = vdx[j] = vdr[j] = vy[j] = vr[j] = z;
        if (c < p.d) {
          if (pre) {
            vrn[j] = load8(p.r_next + base, c);
            vdx[j] = load8(p.dx + base, c);
          }
          if (p.dr_next != nullptr) vdr[j] = load8(p.dr_next + base, c);
          if (post) vy[j] = load8(p.y + base, c);
          if (p.dalpha != nullptr) vr[j] = load8(p.r + base, c);
        }
      }
      float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int c = (t + j * tpr) * 8;
        float rn[8], dx[8], dr[8], y[8], wpre[8], wpost[8], gt[8];
        unpack8(vrn[j], rn);
        unpack8(vdx[j], dx);
        unpack8(vdr[j], dr);
        unpack8(vy[j], y);
        unpack8(p.w_pre != nullptr && c < p.d ? load8(p.w_pre, c) : ones8(), wpre);
        unpack8(p.w_post != nullptr && c < p.d ? load8(p.w_post, c) : ones8(), wpost);
        unpack8(gate != nullptr && c < p.d ? load8(gate, c) : ones8(), gt);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xh = rn[i] * a, dxw = dx[i] * wpre[i], gn = gt[i] * wpost[i] * (y[i] * b);
          s[0] = fmaf(dxw, xh, s[0]);
          s[1] = fmaf(fmaf(a, dxw, dr[i]), gn, s[1]);
          s[2] = fmaf(xh, gn, s[2]);
        }
      }
      worker_sum<CTA>(s, red, turn);
      const float ac1 = a * (s[0] * inv_d);
      const float c2 = (s[1] - ac1 * s[2]) * inv_d;
      float row_alpha = 0.f;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int c = (t + j * tpr) * 8;
        float rn[8], dx[8], dr[8], y[8], r[8], wpre[8], wpost[8], gt[8], odr[8], ody[8];
        unpack8(vrn[j], rn);
        unpack8(vdx[j], dx);
        unpack8(vdr[j], dr);
        unpack8(vy[j], y);
        unpack8(vr[j], r);
        unpack8(p.w_pre != nullptr && c < p.d ? load8(p.w_pre, c) : ones8(), wpre);
        unpack8(p.w_post != nullptr && c < p.d ? load8(p.w_post, c) : ones8(), wpost);
        unpack8(gate != nullptr && c < p.d ? load8(gate, c) : ones8(), gt);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xh = rn[i] * a, n = y[i] * b;
          const float D = fmaf(-xh, ac1, fmaf(a, dx[i] * wpre[i], dr[i]));
          odr[i] = alpha * D;
          ody[i] = b * fmaf(-n, c2, D * gt[i] * wpost[i]);
          swpre[j][i] = fmaf(dx[i], xh, swpre[j][i]);
          swpost[j][i] = fmaf(D * gt[i], n, swpost[j][i]);
          sgate[j][i] = fmaf(D * wpost[i], n, sgate[j][i]);
          row_alpha = fmaf(D, r[i], row_alpha);
        }
        if (c < p.d) {
          *reinterpret_cast<uint4*>(p.dr + base + c) = pack8(odr);
          if (post) *reinterpret_cast<uint4*>(p.dy + base + c) = pack8(ody);
        }
      }
      salpha += static_cast<double>(row_alpha);
    }
    if (p.dgate != nullptr) {
      float* out = sp.slices > 1 ? part_gate + static_cast<size_t>(u) * p.d : p.dgate + static_cast<size_t>(g) * p.d;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int c = (t + j * tpr) * 8;
        if (c < p.d) {
          *reinterpret_cast<float4*>(out + c) = make_float4(sgate[j][0], sgate[j][1], sgate[j][2], sgate[j][3]);
          *reinterpret_cast<float4*>(out + c + 4) = make_float4(sgate[j][4], sgate[j][5], sgate[j][6], sgate[j][7]);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = (t + j * tpr) * 8;
    if (c < p.d) {
      float* o = part_gain + static_cast<size_t>(me) * p.d + c;
      float* o2 = o + static_cast<size_t>(sp.workers) * p.d;
      if (p.dw_pre != nullptr) {
        *reinterpret_cast<float4*>(o) = make_float4(swpre[j][0], swpre[j][1], swpre[j][2], swpre[j][3]);
        *reinterpret_cast<float4*>(o + 4) = make_float4(swpre[j][4], swpre[j][5], swpre[j][6], swpre[j][7]);
      }
      if (p.dw_post != nullptr) {
        *reinterpret_cast<float4*>(o2) = make_float4(swpost[j][0], swpost[j][1], swpost[j][2], swpost[j][3]);
        *reinterpret_cast<float4*>(o2 + 4) = make_float4(swpost[j][4], swpost[j][5], swpost[j][6], swpost[j][7]);
      }
    }
  }
  if (p.dalpha != nullptr) {
    double* part_alpha = reinterpret_cast<double*>(part_gate + (sp.slices > 1 ? static_cast<size_t>(units) * p.d : 0));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) salpha += __shfl_xor_sync(0xffffffffu, salpha, o);
    if constexpr (CTA) {
      __shared__ double reda[32];
      if ((threadIdx.x & 31) == 0) reda[threadIdx.x >> 5] = salpha;
      __syncthreads();
      if (threadIdx.x == 0) {
        salpha = 0.0;
        for (int k = 0; k < static_cast<int>(blockDim.x >> 5); ++k) salpha += reda[k];
      }
    }
    if (t == 0) part_alpha[me] = salpha;
  }
}

// Adds the workers' parts: blockIdx.y = 0, 1 the gains, 2.. the gate rows
// (when they were split).  32 columns x 32 interleaved partial sums per CTA.
__global__ void __launch_bounds__(1024) norm_gate_bwd_sum_kernel(const NormGateBwd p, const NormBwdSplit sp) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float sh[32][33];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const float* part_gate = p.workspace + 2 * static_cast<size_t>(sp.workers) * p.d;
  const int job = blockIdx.y;
  if (p.dalpha != nullptr && blockIdx.x == 0 && job == 0 && row == 31) {
    const size_t units = static_cast<size_t>(sp.groups) * sp.slices;
    const double* pa = reinterpret_cast<const double*>(part_gate + (sp.slices > 1 ? units * p.d : 0));
    double s = 0.0;
    for (int k = lane; k < sp.workers; k += 32) s += pa[k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) *p.dalpha = static_cast<float>(s);
  }
  float* out = job == 0 ? p.dw_pre : job == 1 ? p.dw_post : p.dgate + static_cast<size_t>(job - 2) * p.d;
  if (out == nullptr) return;
  const float* src;
  int n;
  if (job < 2) {
    src = p.workspace + static_cast<size_t>(job) * sp.workers * p.d;
    n = sp.workers;
  } else {
    src = part_gate + static_cast<size_t>(job - 2) * sp.slices * p.d;
    n = sp.slices;
  }
  float s = 0.f;
  if (c < p.d)
    for (int k = row; k < n; k += 32) s += src[static_cast<size_t>(k) * p.d + c];
  sh[row][lane] = s;
  __syncthreads();
  // transposed: warp `row` adds column `row`
  s = sh[lane][row];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int col = blockIdx.x * 32 + row;
  if (lane == 0 && col < p.d) out[col] = s;
}

template <int VPT, bool CTA>
cudaError_t fwd_one(const NormGateFwd& p, int grid, int threads, cudaStream_t s) {
  const cudaError_t e = launch_pdl(norm_gate_fwd_kernel<VPT, CTA>, dim3(grid), dim3(threads), 0, s, p);
  count_launches(1);
  return e;
}

template <int VPT, bool CTA>
cudaError_t bwd_one(const NormGateBwd& p, const NormBwdSplit& sp, int threads, cudaStream_t s) {
  const int grid = CTA ? sp.workers : (sp.workers + kBwdWarps - 1) / kBwdWarps;
  const cudaError_t e = launch_pdl(norm_gate_bwd_kernel<VPT, CTA>, dim3(grid), dim3(threads), 0, s, p, sp);
  count_launches(1);
  return e;
}

int threads_for(int nvec, int vpt) { return (nvec + 32 * vpt - 1) / (32 * vpt) * 32; }

}  // namespace

cudaError_t launch_norm_gate_fwd(const NormGateFwd& p, int num_sms, cudaStream_t s) {
  const int nvec = p.d / 8;
  if (nvec <= 128) {
    // a warp per row, eight rows per CTA
    const int need = (p.M + 7) / 8, most = num_sms * 8;
    const int grid = need < most ? need : most;
    if (nvec <= 32) return fwd_one<1, false>(p, grid, 256, s);
    if (nvec <= 64) return fwd_one<2, false>(p, grid, 256, s);
    if (nvec <= 96) return fwd_one<3, false>(p, grid, 256, s);
    return fwd_one<4, false>(p, grid, 256, s);
  }
  const int most = num_sms * 16;
  const int grid = p.M < most ? p.M : most;
  if (nvec <= 256) return fwd_one<1, true>(p, grid, threads_for(nvec, 1), s);
  if (nvec <= 512) return fwd_one<2, true>(p, grid, threads_for(nvec, 2), s);
  return fwd_one<4, true>(p, grid, threads_for(nvec, 4), s);
}

size_t norm_gate_bwd_workspace(int M, int d, int rows) {
  const NormBwdSplit sp = norm_bwd_split(M, d, rows);
  const size_t units = static_cast<size_t>(sp.groups) * sp.slices;
  const size_t floats = (2 * static_cast<size_t>(sp.workers) + (sp.slices > 1 ? units : 0)) * d;
  return floats * 4 + static_cast<size_t>(sp.workers) * 8;
}

cudaError_t launch_norm_gate_bwd(const NormGateBwd& p, int num_sms, cudaStream_t s) {
  (void)num_sms;
  const NormBwdSplit sp = norm_bwd_split(p.M, p.d, p.rows);
  const int nvec = p.d / 8;
  cudaError_t e;
  if (!bwd_by_cta(p.d)) {
    const int threads = 32 * kBwdWarps;
    if (nvec <= 32)
      e = bwd_one<1, false>(p, sp, threads, s);
    else if (nvec <= 64)
      e = bwd_one<2, false>(p, sp, threads, s);
    else
      e = bwd_one<3, false>(p, sp, threads, s);
  } else if (nvec <= 256) {
    e = bwd_one<1, true>(p, sp, threads_for(nvec, 1), s);
  } else {
    e = bwd_one<2, true>(p, sp, threads_for(nvec, 2), s);
  }
  if (e != cudaSuccess) return e;
  const bool gate_parts = p.dgate != nullptr && sp.slices > 1;
  if (p.dw_pre == nullptr && p.dw_post == nullptr && !gate_parts && p.dalpha == nullptr) return cudaSuccess;
  const dim3 grid((p.d + 31) / 32, 2 + (gate_parts ? sp.groups : 0));
  e = launch_pdl(norm_gate_bwd_sum_kernel, grid, dim3(1024), 0, s, p, sp);
  count_launches(1);
  return e;
}

}  // namespace fp8mlp
