// Norms after one block and before the next, fused with the gate and the
// residual scale, and their gradient.
//
//   n  = y * rstd(y)               r' = alpha r + gate (n w_post)
//   x  = r' * rstd(r') * w_pre     (and the e4m3 copy of x, one scale per 1 x 128)
//
// Memory-bound: every row is read once, both norms and the quantiser work on
// it in registers, and every output is rounded once from fp32.  A worker owns
// a row: 4, 8 or 16 lanes where they can hold it, a warp up to d = 1024, else
// a CTA.  Workers are persistent and copy their next rows to shared memory
// while they compute the current one (cp.async, each thread its own 16-byte
// vectors, so no barrier is needed): the two dependent reductions of a row
// would otherwise leave HBM idle.  Measured back to back at 16384 x 768: forward
// with the FP8 copy 19.5 us (5.8 TB/s, 0.89 of the copy rate; 24.1 without the
// ring), gradient 38 us (4.6 TB/s: 735 instructions per row and warp with eight
// warps per SM, which its registers allow, come next to HBM); 7777 x 2064 with a
// gate per 1000 rows, a CTA per row, 66 us.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "block.h"

namespace fp8mlp {

namespace {

using namespace dev;

constexpr int kSmemCta = 224 * 1024;
constexpr int kRingGateRows = 16;  // gradient: gate rows shorter than this are streamed, longer ones stay in registers
constexpr int kSms = 148;  // CTAs per residency slot; the workspace's size must not depend on the device

__device__ __forceinline__ void unpack8(const uint4& v, uint64_t (&f)[4]) {
  const unsigned int w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = f2_pack(bf16lo_to_f32(w[j]), bf16hi_to_f32(w[j]));
}

__device__ __forceinline__ uint4 pack8(const uint64_t (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a, b;
    f2_unpack(f[j], a, b);
    w[j] = pack_bf16x2(a, b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void product8(const uint4& a, const uint4& b, uint64_t (&f)[4]) {
  uint64_t x[4], y[4];
  unpack8(a, x);
  unpack8(b, y);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2_mul(x[i], y[i]);
}

__device__ __forceinline__ uint4 ones8() {
  return make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
}

__device__ __forceinline__ uint4 load8(const uint16_t* p, int c) { return *reinterpret_cast<const uint4*>(p + c); }

// columns c.. of a vector that may be absent (ones); zero past the row's end
__device__ __forceinline__ uint4 gain8(const uint16_t* p, int c, int d) {
  if (c >= d) return make_uint4(0, 0, 0, 0);
  return p != nullptr ? load8(p, c) : ones8();
}

// 16 bytes to this thread's slot, zeros where `valid` is false
__device__ __forceinline__ void copy16(uint32_t slot, const uint16_t* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(slot), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// until at most depth - 1 copy groups are under way
__device__ __forceinline__ void copy_wait(int depth) {
  if (depth == 2)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 2;" ::: "memory");
}

__device__ __forceinline__ float hsum(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return a + b;
}

// m / d for m < 2^31 by a product: with 2^(s-1) < d <= 2^s and
// k = ceil(2^(31+s) / d), m k 2^-(31+s) exceeds m / d by less than 1 / d
struct FastDiv {
  uint32_t mul;
  int shift;  // -1: d = 1
  __device__ __forceinline__ int operator()(int m) const {
    return shift < 0 ? m : static_cast<int>(__umulhi(static_cast<uint32_t>(m), mul) >> shift);
  }
};

FastDiv fast_div(int d) {
  int s = 0;
  while ((1ll << s) < d) ++s;
  if (s == 0) return {0, -1};
  return {static_cast<uint32_t>(((1ull << (31 + s)) + d - 1) / d), s - 1};
}

// The ring: each warp has its own, stage by stage the vectors of its 32 lanes
// next to each other, so that a copy is 512 contiguous bytes and every offset
// but the stage's is a constant.
constexpr int kVec = 512;

// Sums of N values over a worker's threads: LPR lanes, or the CTA's warps
// through `red`, two buffers used in turn, so that one barrier per call is
// enough.
template <int LPR, bool CTA, int N>
__device__ __forceinline__ void worker_sum(float (&v)[N], float (*red)[11][N], int& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
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

// How rows are dealt out: VPT 16-byte vectors per thread, LPR lanes per row
// (CTA: all threads of the CTA), `per_sm` CTAs per SM, a ring of `depth` rows.
// A row's fixed costs (reductions, divisions, addresses) are paid per warp, so
// a thread takes three or four vectors where the row has them.
struct NormShape {
  int vpt, lpr;
  bool cta;
  int threads, per_sm, depth;
  size_t smem;
};

constexpr int kSmemSm = 227 * 1024, kSmemStatic = 1024 + 1536;  // per CTA: reserved by the system, and declared below

// threads1..4: of a CTA whose workers are warps or less with 1..4 vectors per
// lane; warps: resident per SM for rows that take a CTA, 3 and 4 vectors per
// thread; tensors: in the ring; extra: further 16-byte vectors per thread and
// vector
NormShape norm_shape(int d, const int (&threads)[4], const int (&vpts)[2], const int (&warps)[2], int largest, int tensors, int extra) {
  const int nvec = d / 8;
  NormShape s = {};
  s.lpr = nvec <= 4 ? 4 : nvec <= 8 ? 8 : nvec <= 16 ? 16 : 32;
  s.cta = nvec > 128;
  s.per_sm = 1;
  if (!s.cta) {
    s.vpt = (nvec + 31) / 32;
    s.threads = threads[s.vpt - 1];
  } else {
    // the smaller VPT unless it takes a larger CTA than there is, or wastes more lanes
    const int ta = (nvec + 32 * vpts[0] - 1) / (32 * vpts[0]) * 32, tb = (nvec + 32 * vpts[1] - 1) / (32 * vpts[1]) * 32;
    const int k = ta > largest || vpts[0] * ta > vpts[1] * tb ? 1 : 0;
    s.vpt = vpts[k];
    s.threads = k == 0 ? ta : tb;
    s.per_sm = std::max(1, warps[k] * 32 / s.threads);
  }
  const size_t stage = static_cast<size_t>(tensors * s.vpt) * 16 * s.threads;
  const size_t other = static_cast<size_t>(extra) * s.vpt * s.threads * 16 + kSmemStatic;
  while (s.per_sm > 1 && s.per_sm * (2 * stage + other) > kSmemSm) --s.per_sm;
  s.depth = s.per_sm * (3 * stage + other) <= kSmemSm ? 3 : 2;
  s.smem = s.depth * stage + other - kSmemStatic;
  return s;
}

// ---- forward ------------------------------------------------------------------
// `ring_gate`: several gate rows; a row's own is copied ahead like r and y
template <int VPT, int LPR, bool CTA>
__global__ void __launch_bounds__(CTA ? 384 : 512) norm_gate_fwd_kernel(const NormGateFwd p, const FastDiv by_rows,
                                                                        const int depth, const bool ring_gate) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kGroupLanes = LPR < 16 ? LPR : 16;  // that hold one scale block (tpr is a multiple of them)
  constexpr int R = 0, Y = VPT, G = 2 * VPT;        // first vectors of the tensors in the ring
  extern __shared__ __align__(16) char ring[];
  __shared__ float red[2][11][1];
  int turn = 0;
  constexpr int tpr = LPR;  // vectors between two of a thread's; a CTA's warps own runs of 32 VPT vectors
  const int t = CTA ? (threadIdx.x >> 5) * (32 * VPT) + (threadIdx.x & 31) : threadIdx.x % LPR;
  constexpr int kPerCta = CTA ? 1 : 512 / LPR;
  const int workers = gridDim.x * kPerCta;
  // few rows spread over the CTAs; many are dealt in runs of neighbours, whose
  // scales share sectors
  const int first = CTA ? blockIdx.x
                        : p.M < workers ? blockIdx.x + gridDim.x * (threadIdx.x / LPR)
                                        : blockIdx.x * kPerCta + threadIdx.x / LPR;
  const bool post = p.y != nullptr, pre = p.x != nullptr;
  const float alpha = p.alpha != nullptr ? *p.alpha : 1.f;
  const uint64_t alpha2 = f2_pack(alpha, alpha);
  const float inv_d = 1.f / static_cast<float>(p.d);
  const uint32_t stage_bytes = (ring_gate ? 3 : 2) * VPT * kVec, ring_end = depth * stage_bytes;
  const char* mine = ring + (threadIdx.x >> 5) * ring_end + (threadIdx.x & 31) * 16;
  const uint32_t mine32 = smem_u32(mine);
  auto vec = [&](uint32_t off, int v) { return *reinterpret_cast<const uint4*>(mine + off + v * kVec); };
  // columns of vector j: col + j * tpr * 8, in the row for j < nv
  const int col = t * 8;
  int nv = 0;
#pragma unroll
  for (int j = 0; j < VPT; ++j) nv += col + j * tpr * 8 < p.d ? 1 : 0;
  auto fetch = [&](uint32_t off, int m) {
    if (m < p.M) {
      const size_t base = static_cast<size_t>(m) * p.d + col;
      const size_t gbase = ring_gate ? static_cast<size_t>(by_rows(m)) * p.d + col : 0;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const bool in = j < nv;
        const int o = in ? j * tpr * 8 : 0;  // a vector past the row's end: zeros, from a valid address
        const size_t a = (nv > 0 ? base : 0) + o;
        copy16(mine32 + off + (R + j) * kVec, p.r + a, in);
        if (post) copy16(mine32 + off + (Y + j) * kVec, p.y + a, in);
        if (ring_gate) copy16(mine32 + off + (G + j) * kVec, p.gate + (nv > 0 ? gbase : 0) + o, in);
      }
    }
    copy_commit();
  };
  uint4 wpost[VPT], wpre[VPT], gate[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    wpost[j] = gain8(p.w_post, col + j * tpr * 8, p.d);
    wpre[j] = gain8(p.w_pre, col + j * tpr * 8, p.d);
    gate[j] = gain8(p.gate, col + j * tpr * 8, p.d);  // the only row, unless the ring brings others
  }
  auto next = [&](int m) { return p.M - m > workers ? m + workers : p.M; };
  int m = first < p.M ? first : p.M, ahead = m;
  uint32_t off = 0, foff = (depth - 1) * stage_bytes;
  for (int s = 0; s < depth - 1; ++s) {
    fetch(s * stage_bytes, ahead);
    ahead = next(ahead);
  }
  // uniform over the warp (a CTA's threads share m)
  while (__any_sync(0xffffffffu, m < p.M)) {
    fetch(foff, ahead);
    ahead = next(ahead);
    copy_wait(depth);
    const bool on = m < p.M;
    const size_t base = static_cast<size_t>(on ? m : 0) * p.d + col;
    uint64_t rn[VPT][4];
    if (post) {
      if (ring_gate) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) gate[j] = vec(off, G + j);
      }
      uint64_t yy = 0;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        uint64_t y[4];
        unpack8(vec(off, Y + j), y);
#pragma unroll
        for (int i = 0; i < 4; ++i) yy = f2_fma(y[i], y[i], yy);
      }
      float sum[1] = {hsum(yy)};
      worker_sum<LPR, CTA>(sum, red, turn);
      const float b = __frsqrt_rn(fmaf(sum[0], inv_d, p.eps));
      if (on && t == 0) p.rstd_post[m] = b;
      const uint64_t b2 = f2_pack(b, b);
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        uint64_t r[4], y[4], g[4], w[4];
        unpack8(vec(off, R + j), r);
        unpack8(vec(off, Y + j), y);
        unpack8(gate[j], g);
        unpack8(wpost[j], w);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          rn[j][i] = f2_fma(g[i], f2_mul(f2_mul(y[i], b2), w[i]), f2_mul(alpha2, r[i]));
        if (on && j < nv) *reinterpret_cast<uint4*>(p.r_next + base + j * tpr * 8) = pack8(rn[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < VPT; ++j) unpack8(vec(off, R + j), rn[j]);
    }
    if (pre) {
      uint64_t rr = 0;
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) rr = f2_fma(rn[j][i], rn[j][i], rr);
      float sum[1] = {hsum(rr)};
      worker_sum<LPR, CTA>(sum, red, turn);
      const float a = __frsqrt_rn(fmaf(sum[0], inv_d, p.eps));
      if (on && t == 0) p.rstd_pre[m] = a;
      const uint64_t a2 = f2_pack(a, a);
      float am[VPT];
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        uint64_t w[4];
        unpack8(wpre[j], w);
#pragma unroll
        for (int i = 0; i < 4; ++i) rn[j][i] = f2_mul(f2_mul(rn[j][i], a2), w[i]);
        if (on && j < nv) *reinterpret_cast<uint4*>(p.x + base + j * tpr * 8) = pack8(rn[j]);
        if (p.xq != nullptr) {
          // sixteen lanes (or the row's few) hold one group of 128 columns
          am[j] = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float u, v;
            f2_unpack(rn[j][i], u, v);
            am[j] = max3_nan(am[j], fabsf(u), fabsf(v));
          }
#pragma unroll
          for (int o = kGroupLanes / 2; o > 0; o >>= 1) am[j] = max_nan(am[j], __shfl_xor_sync(0xffffffffu, am[j], o));
        }
      }
      if (p.xq != nullptr) {
        // lane j of a group works out the scale of its j-th block: two
        // divisions per row instead of two per vector
        const int l = t & (kGroupLanes - 1);
        float top = am[0];
#pragma unroll
        for (int j = 1; j < VPT; ++j) top = l == j ? am[j] : top;
        float inv;
        const float s = block_scale(top, &inv);
        if (on && l < VPT) {
          const int c = (t - l + l * tpr) * 8;
          if (c < p.d) p.xs[static_cast<size_t>(c >> 7) * p.M + m] = inv;
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
          const float sj = __shfl_sync(0xffffffffu, s, j, kGroupLanes);
          const uint64_t s2 = f2_pack(sj, sj);
          uint32_t q[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float u, v;
            f2_unpack(f2_mul(rn[j][i], s2), u, v);
            q[i] = pack_e4m3x2(u, v);
          }
          if (on && j < nv)
            *reinterpret_cast<uint2*>(p.xq + base + j * tpr * 8) = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
        }
      }
    }
    m = next(m);
    off = off + stage_bytes == ring_end ? 0 : off + stage_bytes;
    foff = foff + stage_bytes == ring_end ? 0 : foff + stage_bytes;
  }
}

// ---- gradient ---------------------------------------------------------------
// With xh = r' rstd_pre, n = y rstd_post, gw = gate w_post and
// E = dr_next + rstd_pre w_pre dx:
//   D  = dL/dr' = E - rstd_pre xh c1,        c1 = mean(w_pre dx xh)
//   dr = alpha D
//   dy = rstd_post (D gw - n c2),            c2 = mean(D gw n)
// c2 needs D, but mean(D gw n) = mean(E gw n) - rstd_pre c1 mean(xh gw n), so
// the three sums are taken in one pass and one reduction.
//
// Sums over rows: a worker keeps T = sum(D n) of the gate row it is in, in
// registers.  At the gate row's end w_post T goes to dgate, or to the
// workspace where several workers share the gate row, and gate T is added to
// its part of dw_post.  With one gate row for all, T itself is the worker's
// part: dgate = w_post sum(T), dw_post = gate sum(T).  The CTA adds its
// workers' parts, a second kernel those of the CTAs, all in a fixed order.
//
// The rows are cut into one run per team of workers, and a team deals out its
// run's rows in turn, so that what is in flight lies close together: a run
// per worker instead, 14 rows of 768, took 51 us where this takes 37
// (16384 x 768), as HBM then opens a page for each worker.  Larger teams share
// more gate rows: a worker leaves one part per gate row of its team's run, or
// per row where gate rows are no longer than the team.  Short gate rows are
// dealt whole and leave no parts.
struct NormBwdSplit {
  int ctas, groups;  // gate rows
  int rpg;           // rows per gate row, at most M
  int team, run;     // workers per team, rows per team
  int unit;          // neighbouring rows dealt at once: 1, or a whole gate row
  int slots;         // parts of gate rows per worker: of the most that it can touch
  bool by_row;       // 1: each of a worker's rows is of another gate row, a part is a row
  int spread;        // 1: fewer rows than workers, workers counted across the CTAs
};

constexpr int kBwdOneCta = 16;    // up to so many rows one CTA does everything, in one launch
constexpr int kBwdFewGroups = 64;  // a CTA column sums each gate row; beyond, a warp
// Gate rows that may be dealt whole: up to 32 rows, or 16 KB of each tensor.
// 1M x 32 with 33 rows each takes 106 us dealt whole and 172 in shared parts,
// 1M x 64 with 100 rows 221 and 318, 300k x 128 with 48 rows 126 and 183;
// 300k x 256 with 100 rows (51 KB) 252 and 222.  Half as many gate rows as
// workers are enough, as shared parts cost more than idle workers: at 0.55 of
// them 0.58 to 0.91 of the time from 2 x 16 to 32 x 1024, at 0.4 of them 0.59
// to 1.22.  With a CTA per row parts are few, and all of them are asked for.
constexpr int kBwdUnit = 32, kBwdUnitElements = 8192;
constexpr int kBwdThreads[4] = {512, 384, 256, 256};
constexpr int kBwdCtaVpt[2] = {2, 4}, kBwdCtaWarps[2] = {16, 8};  // what the registers allow

// with the gate in the ring (6 tensors) or not (5); the split is made without,
// as the workspace's size must not depend on which
NormShape norm_bwd_shape(int d, int groups, int tensors) {
  return norm_shape(d, kBwdThreads, kBwdCtaVpt, kBwdCtaWarps, 160, tensors, groups > 1 ? 2 : 0);
}

NormBwdSplit norm_bwd_split(int M, int d, int rows) {
  NormBwdSplit s = {};
  s.rpg = rows < M ? rows : M;
  s.groups = (M - 1) / s.rpg + 1;
  const NormShape sh = norm_bwd_shape(d, s.groups, 5);
  const int per_cta = sh.cta ? 1 : sh.threads / sh.lpr;
  int total = kSms * sh.per_sm * per_cta;
  if (!sh.cta && M <= kBwdOneCta) total = per_cta;
  s.ctas = std::min(total / per_cta, M);
  s.spread = M <= total ? 1 : 0;
  s.unit = 1;
  const bool short_rows = s.rpg <= kBwdUnit || static_cast<long long>(s.rpg) * d <= kBwdUnitElements;
  const bool whole = s.rpg == 1 || (short_rows && (sh.cta ? 1LL : 2LL) * s.groups >= total);
  if (s.groups == 1) {
    s.team = total;
    s.run = M;
  } else if (whole) {
    // whole gate rows, no shared ones
    s.unit = s.rpg;
    s.team = s.spread ? 1 : per_cta * (sh.cta ? 16 : 8);
    while (total % s.team != 0) s.team /= 2;
    const int teams = total / s.team;
    s.run = ((s.groups + teams - 1) / teams) * s.rpg;
  } else if (s.spread) {
    s.team = s.run = 1;
  } else {
    // the largest team whose run touches at most two gate rows
    for (s.team = per_cta * (sh.cta ? 16 : 8);; s.team /= 2) {
      if (total % s.team != 0) continue;
      const int teams = total / s.team;
      s.run = (M - 1) / teams + 1;
      if (s.run - 1 <= s.rpg || s.team == per_cta) break;
    }
  }
  // A worker's rows are a team apart: where that is a gate row or more, no two
  // of them share one, and a part per row takes less than one per gate row of
  // the run (138 MB at 65536 x 32 with 8 rows each, 9.7 so; 84 us, 18).  With a
  // warp per row teams are small, and the place's arithmetic would spill.
  s.by_row = s.groups > 1 && !whole && s.team >= s.rpg && sh.lpr < 32;
  s.slots = s.groups == 1 || whole ? 0
            : s.by_row             ? (s.run + s.team - 1) / s.team
            : s.run < 2            ? 1
                                   : (s.run - 2) / s.rpg + 2;
  return s;
}

struct NormBwdWorkspace {
  double* alpha;  // [ctas]
  float* gain;    // [2][ctas][d]
  float* gate;    // [workers][slots][d], with several gate rows: parts of the gate rows in the team's run
};

__host__ __device__ inline size_t bwd_alpha_floats(int ctas) { return 4 * static_cast<size_t>((ctas + 1) / 2); }

__device__ __forceinline__ NormBwdWorkspace bwd_workspace(float* base, int ctas, int d) {
  NormBwdWorkspace w;
  w.alpha = reinterpret_cast<double*>(base);
  w.gain = base + bwd_alpha_floats(ctas);
  w.gate = w.gain + 2 * static_cast<size_t>(ctas) * d;
  return w;
}

__device__ __forceinline__ float4 f32x4(uint64_t lo, uint64_t hi) {
  float4 f;
  f2_unpack(lo, f.x, f.y);
  f2_unpack(hi, f.z, f.w);
  return f;
}
__device__ __forceinline__ void store_f32x8(float* o, const uint64_t (&v)[4]) {
  *reinterpret_cast<float4*>(o) = f32x4(v[0], v[1]);
  *reinterpret_cast<float4*>(o + 4) = f32x4(v[2], v[3]);
}

// The sum over rows for column c, where it goes: a part (`last` false) or the
// gradients it stands for.
__device__ __forceinline__ void gain_out(const NormGateBwd& p, const NormBwdWorkspace& ws, int job, bool one, bool last,
                                         int ctas, int c, float s) {
  if (!last) {
    ws.gain[(static_cast<size_t>(job) * ctas + blockIdx.x) * p.d + c] = s;
  } else if (job == 0) {
    p.dw_pre[c] = s;
  } else if (!one) {
    p.dw_post[c] = s;
  } else {
    if (p.dw_post != nullptr) p.dw_post[c] = p.gate != nullptr ? bf16lo_to_f32(p.gate[c]) * s : s;
    if (p.dgate != nullptr) p.dgate[c] = p.w_post != nullptr ? bf16lo_to_f32(p.w_post[c]) * s : s;
  }
}

template <int VPT, int LPR, bool CTA>
__global__ void __launch_bounds__(CTA ? 256 : kBwdThreads[VPT - 1], CTA && VPT == 2 ? 2 : 1)
    norm_gate_bwd_kernel(const NormGateBwd p, const NormBwdSplit sp, const FastDiv by_rpg, const int depth,
                         const bool ring_gate, const bool direct) {
  pdl_wait();
  pdl_launch_dependents();
  // first vectors of the tensors in the ring: r', dx, dr_next, y, r, gate
  constexpr int RN = 0, DX = VPT, DR = 2 * VPT, Y = 3 * VPT, R = 4 * VPT, G = 5 * VPT;
  extern __shared__ __align__(16) uint4 smem[];
  __shared__ float red[2][11][3];
  __shared__ double reda[16];
  int turn = 0;
  const int tid = threadIdx.x, nthr = CTA ? blockDim.x : kBwdThreads[VPT - 1];
  constexpr int tpr = LPR;  // vectors between two of a thread's; a CTA's warps own runs of 32 VPT vectors
  const int t = CTA ? (tid >> 5) * (32 * VPT) + (tid & 31) : tid % LPR;
  const bool one = sp.groups == 1;
  const bool post = p.y != nullptr, pre = p.dx != nullptr;
  const int per_cta = CTA ? 1 : nthr / LPR;
  const int sub = CTA ? 0 : tid / LPR;
  const int me = sp.spread ? blockIdx.x + gridDim.x * sub : blockIdx.x * per_cta + sub;
  const float alpha = p.alpha != nullptr ? *p.alpha : 1.f;
  const uint64_t alpha2 = f2_pack(alpha, alpha);
  const float inv_d = 1.f / static_cast<float>(p.d);
  const NormBwdWorkspace ws = bwd_workspace(p.workspace, gridDim.x, p.d);
  // shared memory: this thread's part of dw_post (several gate rows), then the ring
  uint4* spost = smem + tid;
  char* ring = reinterpret_cast<char*>(smem + (one ? 0 : 2 * VPT * nthr));
  const uint32_t stage_bytes = (ring_gate ? 6 : 5) * VPT * kVec, ring_end = depth * stage_bytes;
  char* mine = ring + (tid >> 5) * ring_end + (tid & 31) * 16;
  const uint32_t mine32 = smem_u32(mine);
  auto vec = [&](uint32_t off, int v) { return *reinterpret_cast<const uint4*>(mine + off + v * kVec); };
  const uint4 zero = make_uint4(0, 0, 0, 0);
  if (!pre || !post || p.dr_next == nullptr || p.dalpha == nullptr) {
    // tensors that are left out read as zero: nothing is copied over this
    for (uint32_t o = 0; o < ring_end; o += stage_bytes)
      for (int v = 0; v < 5 * VPT; ++v) *reinterpret_cast<uint4*>(mine + o + v * kVec) = zero;
  }
  // rows m0, m0 + 1, .. of a unit, then the worker's next unit, below m1
  const int team = me / sp.team;
  const long long r0 = static_cast<long long>(team) * sp.run;
  const int m1 = static_cast<int>(min(r0 + sp.run, static_cast<long long>(p.M)));
  const int m0 = static_cast<int>(min(r0 + static_cast<long long>(me - team * sp.team) * sp.unit, static_cast<long long>(m1)));
  const int skip = min((sp.team - 1) * static_cast<long long>(sp.unit), static_cast<long long>(p.M));
  struct Row {
    int m, left;  // rows of the unit from m on
  };
  auto next = [&](Row k) {
    if (k.left > 1) return Row{k.m + 1 < m1 ? k.m + 1 : m1, k.left - 1};
    return Row{m1 - k.m > skip + 1 ? k.m + 1 + skip : m1, sp.unit};
  };
  // columns of vector j: col + j * tpr * 8, in the row for j < nv
  const int col = t * 8;
  int nv = 0;
#pragma unroll
  for (int j = 0; j < VPT; ++j) nv += col + j * tpr * 8 < p.d ? 1 : 0;
  // the row's statistics are read with it, up to two rows ahead
  float qa[2] = {0.f, 0.f}, qb[2] = {0.f, 0.f};
  auto fetch = [&](uint32_t off, int m, float& a, float& b) {
    a = b = 0.f;
    if (m < m1) {
      const size_t base = nv > 0 ? static_cast<size_t>(m) * p.d + col : 0;
      const size_t gbase = ring_gate && nv > 0 ? static_cast<size_t>(by_rpg(m)) * p.d + col : 0;
      if (pre) a = p.rstd_pre[m];
      if (post) b = p.rstd_post[m];
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const bool in = j < nv;
        const int o = in ? j * tpr * 8 : 0;  // a vector past the row's end: zeros, from a valid address
        const uint32_t dst = mine32 + off + j * kVec;
        if (pre) {
          copy16(dst + RN * kVec, p.r_next + base + o, in);
          copy16(dst + DX * kVec, p.dx + base + o, in);
        }
        if (p.dr_next != nullptr) copy16(dst + DR * kVec, p.dr_next + base + o, in);
        if (post) copy16(dst + Y * kVec, p.y + base + o, in);
        if (p.dalpha != nullptr) copy16(dst + R * kVec, p.r + base + o, in);
        if (ring_gate) copy16(dst + G * kVec, p.gate + gbase + o, in);
      }
    }
    copy_commit();
  };

  uint4 wpre[VPT], wpost[VPT], gate[VPT];
  uint64_t gw[VPT][4], swpre[VPT][4], T[VPT][4];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = col + j * tpr * 8;
    wpre[j] = gain8(p.w_pre, c, p.d);
    wpost[j] = gain8(p.w_post, c, p.d);
    gate[j] = zero;
#pragma unroll
    for (int i = 0; i < 4; ++i) gw[j][i] = swpre[j][i] = T[j][i] = 0;
    if (!one) spost[(2 * j) * nthr] = spost[(2 * j + 1) * nthr] = zero;
  }
  double salpha = 0.0;
  // what a gate row's place among the worker's parts is counted from
  const int first = LPR < 32 && sp.by_row ? m0 : by_rpg(r0 < p.M ? static_cast<int>(r0) : 0);
  int g = -1;      // gate row of T
  int g_end = m0;  // where it ends
  // T of gate row g to its place, and its share of dw_post
  auto flush = [&]() {
    float* dst = nullptr;
    int part = g - first;
    if constexpr (LPR < 32) {
      // by row, the worker's only row of gate row g is its first one from g * rpg on
      if (sp.by_row) part = (g * sp.rpg - first + sp.team - 1) / sp.team;
    }
    if (p.dgate != nullptr)
      dst = sp.slots == 0 ? p.dgate + static_cast<size_t>(g) * p.d
                          : ws.gate + (static_cast<size_t>(me) * sp.slots + part) * p.d;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      uint64_t w[4], o[4], f[4];
      unpack8(wpost[j], w);
      unpack8(gate[j], f);
      const uint4 a = spost[(2 * j) * nthr], b = spost[(2 * j + 1) * nthr];
      uint64_t s[4] = {f2_pack(__uint_as_float(a.x), __uint_as_float(a.y)), f2_pack(__uint_as_float(a.z), __uint_as_float(a.w)),
                       f2_pack(__uint_as_float(b.x), __uint_as_float(b.y)), f2_pack(__uint_as_float(b.z), __uint_as_float(b.w))};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[i] = f2_mul(T[j][i], w[i]);
        s[i] = f2_fma(T[j][i], f[i], s[i]);
        T[j][i] = 0;
      }
      if (dst != nullptr && j < nv) store_f32x8(dst + col + j * tpr * 8, o);
      *reinterpret_cast<float4*>(&spost[(2 * j) * nthr]) = f32x4(s[0], s[1]);
      *reinterpret_cast<float4*>(&spost[(2 * j + 1) * nthr]) = f32x4(s[2], s[3]);
    }
  };

  Row cur{m0, sp.unit}, ahead = cur;
  uint32_t off = 0, foff = (depth - 1) * stage_bytes;
  fetch(0, ahead.m, qa[0], qb[0]);
  ahead = next(ahead);
  if (depth == 3) {
    fetch(stage_bytes, ahead.m, qa[1], qb[1]);
    ahead = next(ahead);
  }
  // uniform over the warp (a CTA's threads share m)
  while (__any_sync(0xffffffffu, cur.m < m1)) {
    const int m = cur.m;
    float fa, fb;
    fetch(foff, ahead.m, fa, fb);
    ahead = next(ahead);
    const bool on = m < m1;
    if (on && m >= g_end && post) {
      // the next gate row
      if (!one && g >= 0) flush();
      g = by_rpg(m);
      g_end = p.M - g * sp.rpg < sp.rpg ? p.M : (g + 1) * sp.rpg;
      if (!ring_gate) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
          gate[j] = gain8(p.gate != nullptr ? p.gate + static_cast<size_t>(g) * p.d : nullptr, col + j * tpr * 8, p.d);
          product8(gate[j], wpost[j], gw[j]);
        }
      }
    }
    copy_wait(depth);
    if (ring_gate && on) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        gate[j] = vec(off, G + j);
        product8(gate[j], wpost[j], gw[j]);
      }
    }
    const size_t base = static_cast<size_t>(on ? m : 0) * p.d + col;
    const float a = qa[0], b = qb[0];
    const uint64_t a2 = f2_pack(a, a), b2 = f2_pack(b, b);
    uint64_t s0 = 0, s1 = 0, s2 = 0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      uint64_t rn[4], dx[4], dr[4], y[4], w[4];
      unpack8(vec(off, RN + j), rn);
      unpack8(vec(off, DX + j), dx);
      unpack8(vec(off, DR + j), dr);
      unpack8(vec(off, Y + j), y);
      unpack8(wpre[j], w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t xh = f2_mul(rn[i], a2), dxw = f2_mul(dx[i], w[i]), gn = f2_mul(gw[j][i], f2_mul(y[i], b2));
        s0 = f2_fma(dxw, xh, s0);
        s1 = f2_fma(f2_fma(a2, dxw, dr[i]), gn, s1);
        s2 = f2_fma(xh, gn, s2);
      }
    }
    float s[3] = {hsum(s0), hsum(s1), hsum(s2)};
    worker_sum<LPR, CTA>(s, red, turn);
    const float ac1 = a * (s[0] * inv_d);
    const float c2 = (s[1] - ac1 * s[2]) * inv_d;
    const uint64_t nac1 = f2_pack(-ac1, -ac1), nc2 = f2_pack(-c2, -c2);
    asm volatile("" ::: "memory");  // the vectors are read again: kept, they would spill
    uint64_t ra = 0;
    if (on) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        uint64_t rn[4], dx[4], dr[4], y[4], r[4], w[4], odr[4], ody[4];
        unpack8(vec(off, RN + j), rn);
        unpack8(vec(off, DX + j), dx);
        unpack8(vec(off, DR + j), dr);
        unpack8(vec(off, Y + j), y);
        unpack8(vec(off, R + j), r);
        unpack8(wpre[j], w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t xh = f2_mul(rn[i], a2), n = f2_mul(y[i], b2);
          const uint64_t D = f2_fma(xh, nac1, f2_fma(a2, f2_mul(dx[i], w[i]), dr[i]));
          odr[i] = f2_mul(alpha2, D);
          ody[i] = f2_mul(b2, f2_fma(n, nc2, f2_mul(D, gw[j][i])));
          swpre[j][i] = f2_fma(dx[i], xh, swpre[j][i]);
          T[j][i] = f2_fma(D, n, T[j][i]);
          ra = f2_fma(D, r[i], ra);
        }
        if (j < nv) {
          *reinterpret_cast<uint4*>(p.dr + base + j * tpr * 8) = pack8(odr);
          if (post) *reinterpret_cast<uint4*>(p.dy + base + j * tpr * 8) = pack8(ody);
        }
      }
      salpha += static_cast<double>(hsum(ra));
    }
    qa[0] = depth == 2 ? fa : qa[1];
    qb[0] = depth == 2 ? fb : qb[1];
    qa[1] = fa;
    qb[1] = fb;
    cur = next(cur);
    off = off + stage_bytes == ring_end ? 0 : off + stage_bytes;
    foff = foff + stage_bytes == ring_end ? 0 : foff + stage_bytes;
  }
  if (!one && g >= 0) flush();

  // ---- the CTA's parts of dw_pre (job 0) and of T or dw_post (job 1)
  asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
  for (int job = 0; job < 2; ++job) {
    if (job == 0 ? p.dw_pre == nullptr : (p.dw_post == nullptr && !(one && p.dgate != nullptr))) continue;
    uint64_t v[VPT][4];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (job == 1 && !one) {
        const uint4 a = spost[(2 * j) * nthr], b = spost[(2 * j + 1) * nthr];
        v[j][0] = f2_pack(__uint_as_float(a.x), __uint_as_float(a.y));
        v[j][1] = f2_pack(__uint_as_float(a.z), __uint_as_float(a.w));
        v[j][2] = f2_pack(__uint_as_float(b.x), __uint_as_float(b.y));
        v[j][3] = f2_pack(__uint_as_float(b.z), __uint_as_float(b.w));
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = job == 0 ? swpre[j][i] : T[j][i];
      }
    }
    if constexpr (!CTA) {
      // over a warp's workers by shuffles, over the warps through the ring
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int o = LPR; o < 32; o <<= 1) v[j][i] = f2_add(v[j][i], __shfl_xor_sync(0xffffffffu, v[j][i], o));
      const int warp = tid >> 5, nw = nthr >> 5;
      float* buf = reinterpret_cast<float*>(ring);
      const int width = LPR * VPT * 8;
      __syncthreads();  // the ring (and the other job's sums) are done with
      if ((tid & 31) < LPR) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) store_f32x8(buf + warp * width + (t + j * LPR) * 8, v[j]);
      }
      __syncthreads();
      for (int c = tid; c < p.d; c += nthr) {
        float s = 0.f;
        for (int k = 0; k < nw; ++k) s += buf[k * width + c];
        gain_out(p, ws, job, one, direct, gridDim.x, c, s);
      }
    } else {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int c = (t + j * tpr) * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x, y;
          f2_unpack(v[j][i], x, y);
          if (c < p.d) {
            gain_out(p, ws, job, one, direct, gridDim.x, c + 2 * i, x);
            gain_out(p, ws, job, one, direct, gridDim.x, c + 2 * i + 1, y);
          }
        }
      }
    }
  }
  if (p.dalpha != nullptr) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) salpha += __shfl_xor_sync(0xffffffffu, salpha, o);
    if ((tid & 31) == 0) reda[tid >> 5] = salpha;
    __syncthreads();
    if (tid == 0) {
      salpha = 0.0;
      for (int k = 0; k < nthr >> 5; ++k) salpha += reda[k];
      if (direct)
        *p.dalpha = static_cast<float>(salpha);
      else
        ws.alpha[blockIdx.x] = salpha;
    }
  }
}

__device__ __forceinline__ void add2(float2& s, const float* p) {
  const float2 v = *reinterpret_cast<const float2*>(p);
  s.x += v.x;
  s.y += v.y;
}

// Parts of gate row g for columns c.. that are `k0` modulo `kn` in their order.
__device__ __forceinline__ float2 gate_parts(const NormGateBwd& p, const NormBwdSplit& sp, const float* gate, int g, int c,
                                             int k0, int kn) {
  const uint32_t run = sp.run, team = sp.team, rpg = sp.rpg;
  const uint32_t r0 = g * rpg, r1 = min(r0 + rpg, static_cast<uint32_t>(p.M));
  if (sp.by_row) {
    float2 s = make_float2(0.f, 0.f);
#pragma unroll 4
    for (uint32_t row = r0 + k0; row < r1; row += kn) {
      const uint32_t t = row / run, i = row - t * run, slot = i / team;
      add2(s, gate + (static_cast<size_t>(t * team + i - slot * team) * sp.slots + slot) * p.d + c);
    }
    return s;
  }
  const uint32_t t0 = r0 / run, parts = ((r1 - 1) / run - t0 + 1) * team;
  float2 s = make_float2(0.f, 0.f);
#pragma unroll 4
  for (uint32_t i = k0; i < parts; i += kn) {
    const uint32_t t = t0 + i / team, k = i % team;
    const uint32_t c0 = t * run, a = max(r0, c0), b = min(r1, c0 + run);
    // the team's worker k has rows a.. of it if the first one dealt to it is below b
    const uint32_t behind = (a - c0) % team, row = a + (k >= behind ? k - behind : k + team - behind);
    if (row < b) add2(s, gate + (static_cast<size_t>(t * team + k) * sp.slots + (g - c0 / rpg)) * p.d + c);
  }
  return s;
}

// Adds the CTAs' parts: blockIdx.y = 0, 1 the gains, 2.. gate rows that several
// workers share.  64 columns x 32 interleaved partial sums per CTA; beyond
// kBwdFewGroups gate rows a warp adds each.
__global__ void __launch_bounds__(1024) norm_gate_bwd_sum_kernel(const NormGateBwd p, const NormBwdSplit sp) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ __align__(8) float sh[32][66];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int c = blockIdx.x * 64 + lane * 2;
  const NormBwdWorkspace ws = bwd_workspace(p.workspace, sp.ctas, p.d);
  const int job = blockIdx.y;
  const bool one = sp.groups == 1;
  if (p.dalpha != nullptr && blockIdx.x == 0 && job == 0 && row == 31) {
    double s = 0.0;
    for (int k = lane; k < sp.ctas; k += 32) s += ws.alpha[k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) *p.dalpha = static_cast<float>(s);
  }
  if (job >= 2 && sp.groups > kBwdFewGroups) {
    for (int g = (job - 2) * 32 + row; g < sp.groups && c < p.d; g += 32 * (gridDim.y - 2))
      *reinterpret_cast<float2*>(p.dgate + static_cast<size_t>(g) * p.d + c) = gate_parts(p, sp, ws.gate, g, c, 0, 1);
    return;
  }
  float2 v = make_float2(0.f, 0.f);
  if (job < 2) {
    if (job == 0 ? p.dw_pre == nullptr : (p.dw_post == nullptr && !(one && p.dgate != nullptr))) return;
    const float* src = ws.gain + static_cast<size_t>(job) * sp.ctas * p.d + c;
    if (c < p.d) {
#pragma unroll 4
      for (int k = row; k < sp.ctas; k += 32) add2(v, src + static_cast<size_t>(k) * p.d);
    }
  } else if (c < p.d) {
    v = gate_parts(p, sp, ws.gate, job - 2, c, row, 32);
  }
  *reinterpret_cast<float2*>(&sh[row][lane * 2]) = v;
  __syncthreads();
  // sixteen lanes add a column
  const int col = threadIdx.x >> 4, part = threadIdx.x & 15;
  float s = sh[part][col] + sh[part + 16][col];
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int out = blockIdx.x * 64 + col;
  if (part == 0 && out < p.d) {
    if (job < 2)
      gain_out(p, ws, job, one, true, sp.ctas, out, s);
    else
      p.dgate[static_cast<size_t>(job - 2) * p.d + out] = s;
  }
}

template <int VPT, int LPR, bool CTA>
cudaError_t fwd_one(const NormGateFwd& p, const NormShape& sh, bool ring_gate, cudaStream_t s) {
  static std::atomic<bool> done[64] = {};
  cudaError_t e = allow_smem(norm_gate_fwd_kernel<VPT, LPR, CTA>, done, kSmemCta);
  if (e != cudaSuccess) return e;
  const int most = kSms * sh.per_sm;
  e = launch_pdl(norm_gate_fwd_kernel<VPT, LPR, CTA>, dim3(p.M < most ? p.M : most), dim3(sh.threads), sh.smem, s, p,
                 fast_div(p.rows), sh.depth, ring_gate);
  count_launches(1);
  return e;
}

template <int VPT, int LPR, bool CTA>
cudaError_t bwd_one(const NormGateBwd& p, const NormBwdSplit& sp, const NormShape& sh, bool ring_gate, bool direct,
                    cudaStream_t s) {
  static std::atomic<bool> done[64] = {};
  cudaError_t e = allow_smem(norm_gate_bwd_kernel<VPT, LPR, CTA>, done, kSmemCta);
  if (e != cudaSuccess) return e;
  e = launch_pdl(norm_gate_bwd_kernel<VPT, LPR, CTA>, dim3(sp.ctas), dim3(sh.threads), sh.smem, s, p, sp,
                 fast_div(sp.rpg), sh.depth, ring_gate, direct);
  count_launches(1);
  return e;
}

template <class F>
cudaError_t by_shape(const NormShape& s, F&& f) {
  using std::integral_constant;
  if (s.cta) {
    if (s.vpt == 2) return f(integral_constant<int, 2>(), integral_constant<int, 32>(), std::true_type());
    if (s.vpt == 3) return f(integral_constant<int, 3>(), integral_constant<int, 32>(), std::true_type());
    return f(integral_constant<int, 4>(), integral_constant<int, 32>(), std::true_type());
  }
  if (s.lpr == 4) return f(integral_constant<int, 1>(), integral_constant<int, 4>(), std::false_type());
  if (s.lpr == 8) return f(integral_constant<int, 1>(), integral_constant<int, 8>(), std::false_type());
  if (s.lpr == 16) return f(integral_constant<int, 1>(), integral_constant<int, 16>(), std::false_type());
  if (s.vpt == 1) return f(integral_constant<int, 1>(), integral_constant<int, 32>(), std::false_type());
  if (s.vpt == 2) return f(integral_constant<int, 2>(), integral_constant<int, 32>(), std::false_type());
  if (s.vpt == 3) return f(integral_constant<int, 3>(), integral_constant<int, 32>(), std::false_type());
  return f(integral_constant<int, 4>(), integral_constant<int, 32>(), std::false_type());
}

}  // namespace

cudaError_t launch_norm_gate_fwd(const NormGateFwd& p, cudaStream_t s) {
  const bool ring_gate = p.gate != nullptr && p.rows < p.M;
  const int threads[4] = {512, 512, 512, 512}, cta_vpt[2] = {3, 4}, cta_warps[2] = {12, 12};
  const NormShape sh = norm_shape(p.d, threads, cta_vpt, cta_warps, 256, ring_gate ? 3 : 2, 0);
  return by_shape(sh, [&](auto vpt, auto lpr, auto cta) {
    return fwd_one<decltype(vpt)::value, decltype(lpr)::value, decltype(cta)::value>(p, sh, ring_gate, s);
  });
}

size_t norm_gate_bwd_workspace(int M, int d, int rows) {
  const NormBwdSplit sp = norm_bwd_split(M, d, rows);
  const size_t teams = (static_cast<size_t>(M) + sp.run - 1) / sp.run;
  const size_t rows_of_parts = 2 * static_cast<size_t>(sp.ctas) + teams * sp.team * sp.slots;
  return (bwd_alpha_floats(sp.ctas) + rows_of_parts * d) * sizeof(float);
}

cudaError_t launch_norm_gate_bwd(const NormGateBwd& p, cudaStream_t s) {
  const NormBwdSplit sp = norm_bwd_split(p.M, p.d, p.rows);
  // gate rows that several workers share
  const bool shared_gates = p.dgate != nullptr && sp.slots > 0;
  const bool direct = sp.ctas == 1 && !shared_gates;
  // the gate in the ring too, where its rows are short and the ring still holds two rows of everything
  NormShape sh = norm_bwd_shape(p.d, sp.groups, 6);
  const bool ring_gate =
      p.gate != nullptr && sp.rpg < kRingGateRows && sp.groups > 1 && sh.smem <= static_cast<size_t>(kSmemCta);
  if (!ring_gate) sh = norm_bwd_shape(p.d, sp.groups, 5);
  cudaError_t e = by_shape(sh, [&](auto vpt, auto lpr, auto cta) {
    return bwd_one<decltype(vpt)::value, decltype(lpr)::value, decltype(cta)::value>(p, sp, sh, ring_gate, direct, s);
  });
  if (e != cudaSuccess || direct) return e;
  const bool one_gate = p.dgate != nullptr && sp.groups == 1;
  if (p.dw_pre == nullptr && p.dw_post == nullptr && !one_gate && !shared_gates && p.dalpha == nullptr) return e;
  const int jobs = 2 + (!shared_gates ? 0 : sp.groups > kBwdFewGroups ? std::min((sp.groups + 31) / 32, 4096) : sp.groups);
  e = launch_pdl(norm_gate_bwd_sum_kernel, dim3((p.d + 63) / 64, jobs), dim3(1024), 0, s, p, sp);
  count_launches(1);
  return e;
}

}  // namespace fp8mlp
