// Warp-specialised, persistent tcgen05 GEMM on e4m3 operands with a scale for
// each block of 128:
//
//   y[m, n] = sum_kb xs[kb, m] * ws[kb, n / 128] * sum_{k in kb} xq[m, k] Wq[n, k]
//
// The scales vary along K, so a sum over all of K cannot stay in TMEM.  One
// pipeline stage is one 128-byte swizzle row of e4m3, which is one scale
// block: its four UMMAs start a fresh TMEM accumulator, and the epilogue
// warps add that partial sum, times xs * ws, to fp32 sums in registers while
// the tensor cores fill the next accumulator (512 TMEM columns hold 512 / BN
// of them).  A thread owns one row and 128 columns, i.e. one weight block: the
// factor is one number per thread and k-block, and for the relu^2 output the
// thread holds a whole 1 x 128 scale block, so its maximum needs no exchange.
//   warp 0      TMA producer: A/B k-blocks into a STAGES-deep ring
//   warp 1      allocates TMEM, issues the UMMAs from one thread
//   warp 2      pairs: stores finished tiles (TMA)
//   next        scales of each k-block to shared memory
//   then        4 * BN / 128 epilogue warps
// What bounds it: a k-block of a 256 x 256 tile is 512 cycles of tensor work;
// issuing it takes 500 to 560, and its promotion (128 columns of TMEM and 128
// multiply-adds per epilogue thread) some 600 (clock reads in a copy of the
// kernel), with the hand-over of two accumulators between them.  Back to back,
// 8192 x 4096 -> 1024 takes 30 to 31 us (2.2 PFLOP/s; an unscaled e4m3 library
// product of that size 24.4), 16384 x 768 -> 2304, where writing y weighs as much
// as the six k-blocks, 29.4 to 30 (2.0; 29.0).  Steps that gained, in us of the
// latter as each was built: no release fence in the hand-over and pipelined TMEM
// reads 80 to 41, 128-byte output rows 38, one commit per k-block 37, a store
// thread 35, elected issue 34.5, scales by a warp of their own 30.5.  Measured and
// not taken: 256 x 128 tiles (L2 and hand-over bound, 50), 16 epilogue warps (47),
// output straight from registers (44), A kept in shared memory along N (38).
// CG = 2: the CTAs of a cluster pair share a 2-CTA UMMA over 256 rows, as in
// gemm_sm100.cuh.  TMA zero-fills rows and columns past the edges and clips
// the stores.
#pragma once

#include "gemm_sm100.cuh"

namespace fp8mlp {

struct alignas(64) BlockGemmParams {
  CUtensorMap tmA, tmB;
  CUtensorMap tmOut;   // bf16 output, STORE_ROWS rows x 64 columns
  CUtensorMap tmOut2;  // relu^2: e4m3 copy, STORE_ROWS rows x 128 columns
  int M, N, K;
  int tiles_m, tiles_n;
  int n_blocks;          // ceil(N / 128): row length of ws
  const float* xs;       // [ceil(K / 128)][M]
  const float* ws;       // [ceil(K / 128)][n_blocks]
  float* post_s;         // relu^2: [n_blocks][M] inverse scales of the e4m3 copy
  unsigned int* status;
  unsigned long long timeout_ns;
  int debug_flags;
};

// CG CTAs per tile, BN tile columns
template <int CG_, int BN_, int STAGES_, bool RELU2_>
struct BlockCfg {
  static constexpr int CG = CG_;
  static constexpr int BM = 128;
  static constexpr int TILE_M = BM * CG;
  static constexpr int BN = BN_;
  static constexpr int B_ROWS = BN / CG;           // rows of B per CTA
  static constexpr int STAGES = STAGES_;
  static constexpr bool RELU2 = RELU2_;
  static constexpr int BK = 128;
  static constexpr int A_BYTES = BM * BK;
  static constexpr int B_BYTES = B_ROWS * BK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGE_TX = CG * STAGE_BYTES;
  static constexpr uint32_t IDESC = dev::instr_desc(dev::FMT_E4M3, dev::FMT_E4M3, false, false, TILE_M, BN);
  static constexpr int NBUF = 512 / BN;            // TMEM accumulators
  static constexpr int NEPI = 4 * BN / 128;
  // A pair's CTAs have tile after tile: a thread of its own stores them, since
  // a TMA store waits for its place in the queue, up to 1000 cycles behind the
  // others of its tile and the loads, which the epilogue would lose.  A single
  // CTA has one tile, mostly: each epilogue warp stores its part when it has
  // it, which ends 0.4 us sooner than gathering the warps' parts.
  static constexpr bool STORE_WARP = CG == 2;
  static constexpr int STORE_ROWS = STORE_WARP ? 128 : 32;
  static constexpr int SCALE_WARP = STORE_WARP ? 3 : 2;
  static constexpr int EPI0 = SCALE_WARP + 1;      // first epilogue warp
  static constexpr int THREADS = 32 * (EPI0 + NEPI);
  // With eight epilogue warps a thread needs more than its even share of the
  // registers: the first warpgroup hands some over.
  static constexpr bool SPLIT_REGS = NEPI == 8;
  static constexpr int REGS_CONTROL = 72, REGS_EPI = 216;
  static constexpr int REGS_SUM = 128 * REGS_CONTROL + 32 * NEPI * REGS_EPI;  // of the launch, at least
  // output: chunks of 128 rows x 128 bytes, 64 columns of bf16 or 128 codes
  static constexpr int CHUNK = BM * 128;
  static constexpr int OUT_CHUNKS = BN / 64 + (RELU2 ? BN / 128 : 0);
  // ring of scales: a k-block's are 128 rows' and BN / 128 weight blocks'.
  // A single CTA announces them with its loads: the UMMAs wait for both, and
  // their completion tells the epilogue.  A slot is free once the UMMAs NBUF
  // k-blocks behind its last use are done (they waited for that use's
  // accumulator); the wait for those must not see the barrier's next phase,
  // which holds for SRING <= NBUF + STAGES.
  // A pair's UMMAs are issued by one CTA: that way would pass signals between
  // CTAs, which order the other's own shared memory only with a release at
  // cluster scope (1000 cycles behind the loads under way).  So each CTA of a
  // pair has barriers of its own for the slots (the up-projection takes 1 to 2 %
  // longer for it, the plain product no longer); a single CTA with few tiles
  // would lose 5 to 20 %.
  static constexpr int SCALES = 132 * 4;
  static constexpr int SRING = NBUF == 2 ? 4 : 8;
  static constexpr bool SLOT_BARS = CG == 2;
  static_assert(SLOT_BARS || (SRING > NBUF && SRING <= NBUF + STAGES && SRING - NBUF <= STAGES), "scale ring");
  static constexpr int NUM_BARS = 2 * STAGES + NBUF + (SLOT_BARS ? 2 * SRING : 0) + 3;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + SRING * SCALES + OUT_CHUNKS * CHUNK + NUM_BARS * 8 + 16;
  static_assert(CG == 1 || CG == 2, "CTA group");
  static_assert(BN == 128 || BN == 256, "accumulators");
  static_assert(SMEM_BYTES <= 232448, "shared memory");
};

namespace dev {

template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// A load that stays where it is written: the compiler would sink a plain one
// to its use, four k-blocks later, and put its latency back into the loop.
__device__ __forceinline__ float ld_scale(const float* p, bool valid) {
  float v;
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\tmov.f32 %0, 0f00000000;\n\t"
      "@q ld.global.nc.f32 %0, [%1];\n\t}"
      : "=f"(v)
      : "l"(p), "r"(static_cast<int>(valid)));
  return v;
}

// one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// max that keeps NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// conversions of the positive part, NaN kept
__device__ __forceinline__ uint32_t pack_bf16x2_relu(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.relu.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t pack_e4m3x2_relu(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.relu.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return static_cast<uint32_t>(d);
}

// Scale of a block of 128 whose largest magnitude is `amax`: s maps amax onto
// 448 and is at most 2^120, so that 1/s stays a normal number; an all-zero
// block takes s = 1.  A block that holds an infinity or NaN takes s = 1 and
// stores 1/s = NaN, so that what is computed from it is NaN instead of a
// saturated code that looks finite.
__device__ __forceinline__ float block_scale(float amax, float* inv) {
  if (!(amax <= 3.4028234664e38f)) {
    *inv = __int_as_float(0x7fc00000);
    return 1.f;
  }
  const float s = amax > 0.f ? fminf(__fdiv_rn(FP8MLP_E4M3_MAX, amax), 1.329227995784916e36f) : 1.f;
  *inv = __fdiv_rn(1.f, s);
  return s;
}

}  // namespace dev

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) gemm_block_kernel(const __grid_constant__ BlockGemmParams p) {
  using namespace dev;
  constexpr int CG = C::CG;
  // no room to align by hand; without static shared memory the base is aligned
  extern __shared__ __align__(1024) uint8_t smem_aligned[];
  if ((smem_u32(smem_aligned) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(p.status, STATUS_TIMEOUT);
    return;
  }
  uint8_t* sStage = smem_aligned;
  uint8_t* sOut = sStage + C::STAGES * C::STAGE_BYTES;
  float* sScale = reinterpret_cast<float*>(sOut + C::OUT_CHUNKS * C::CHUNK);
  uint64_t* full = reinterpret_cast<uint64_t*>(sScale + C::SRING * (C::SCALES / 4));
  uint64_t* done = full + C::STAGES;
  uint64_t* tempty = done + C::STAGES;
  uint64_t* sfull = tempty + C::NBUF;    // SLOT_BARS: a slot's scales are there,
  uint64_t* sempty = sfull + C::SRING;   // and have been read
  uint64_t* oready = sfull + (C::SLOT_BARS ? 2 * C::SRING : 0);  // a tile's output is in shared memory
  uint64_t* ofree = oready + 1;          // it has been read from there
  uint64_t* fin = ofree + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(fin + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int unit = static_cast<int>(blockIdx.x) / CG;
  const int nunits = static_cast<int>(gridDim.x) / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], C::SLOT_BARS ? 1 : 2);  // the loads, and the scales
      mbar_init(&done[s], 1);
    }
    for (int a = 0; a < C::NBUF; ++a) {
      mbar_init(&tempty[a], C::NEPI * CG);  // one arrival per epilogue warp of the pair
    }
    for (int i = 0; C::SLOT_BARS && i < C::SRING; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&sempty[i], C::NEPI);
    }
    mbar_init(oready, C::NEPI);
    mbar_init(ofree, 1);
    mbar_init(fin, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc<CG>(tmem_holder, 512);
    tmem_relinquish<CG>();
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  const WaitCtx w{p.status, abort_flag, p.timeout_ns};
  const int num_tiles = p.tiles_m * p.tiles_n;
  const int num_kb = (p.K + C::BK - 1) / C::BK;

  if (warp < C::EPI0) {
    if constexpr (C::SPLIT_REGS) reg_dec<C::REGS_CONTROL>();
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      if (lane == 0 && !(p.debug_flags & FP8MLP_DEBUG_STALL_PRODUCER)) {
        tma_prefetch_desc(&p.tmA);
        tma_prefetch_desc(&p.tmB);
        uint32_t stage = 0, phase = 0;
        long long issued = 0;
        bool ok = true;
        for (int t = unit; t < num_tiles && ok; t += nunits) {
          const int mb = t / p.tiles_n, nb = t - mb * p.tiles_n;
          const int m0 = mb * C::TILE_M + static_cast<int>(rank) * C::BM;
          const int n0 = nb * C::BN + static_cast<int>(rank) * C::B_ROWS;
          for (int kb = 0; kb < num_kb; ++kb) {
            if (!mbar_wait(&done[stage], phase ^ 1u, w)) {
              ok = false;
              break;
            }
            uint8_t* a = sStage + stage * C::STAGE_BYTES;
            uint8_t* b = a + C::A_BYTES;
            if constexpr (CG == 1) {
              mbar_arrive_expect_tx(&full[stage], C::STAGE_TX);
              tma_load_2d(a, &p.tmA, &full[stage], kb * C::BK, m0);
              tma_load_2d(b, &p.tmB, &full[stage], kb * C::BK, n0);
            } else {
              if (leader) mbar_arrive_expect_tx(&full[stage], C::STAGE_TX);
              const uint32_t fb = mapa_shared(smem_u32(&full[stage]), 0);
              tma_load_2d_cg2(a, &p.tmA, fb, kb * C::BK, m0);
              tma_load_2d_cg2(b, &p.tmB, fb, kb * C::BK, n0);
            }
            ++issued;
            if (++stage == C::STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        // the last copy into each stage must have landed before exit
        if (leader) {
          const long long n_drain = issued < C::STAGES ? issued : C::STAGES;
          for (long long i = 0; i < n_drain; ++i) {
            const long long n = issued - 1 - i;
            mbar_wait_drain(&full[n % C::STAGES], static_cast<uint32_t>((n / C::STAGES) & 1), p.timeout_ns);
          }
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      // The whole warp runs the loop and one elected lane issues: what it
      // issues is then known to be uniform and needs no moves to uniform
      // registers, which took longer than the UMMAs.
      if (leader) {
        const bool elected = elect_one();
        uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 0;
        bool ok = true;
        for (int t = unit; t < num_tiles && ok; t += nunits) {
          for (int kb = 0; kb < num_kb; ++kb) {
            if (!mbar_wait_inline(&full[stage], phase, w) || !mbar_wait_inline(&tempty[buf], buf_phase ^ 1u, w)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a0 = smem_u32(sStage + stage * C::STAGE_BYTES);
            const uint32_t b0 = a0 + C::A_BYTES;
            if (elected) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma<CG, true>(tmem_base + buf * C::BN, smem_desc(a0 + k * 32, 16, 1024),
                               smem_desc(b0 + k * 32, 16, 1024), C::IDESC, k != 0 ? 1u : 0u);
              if constexpr (CG == 1)
                tc_commit(&done[stage]);
              else
                tc_commit_cg2_mc(&done[stage], 0x3);
            }
            __syncwarp();
            if (++buf == C::NBUF) {
              buf = 0;
              buf_phase ^= 1u;
            }
            if (++stage == C::STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        // every UMMA issued must be complete before TMEM is freed
        if (elected) {
          if constexpr (CG == 1)
            tc_commit(fin);
          else
            tc_commit_cg2(fin);
          mbar_wait_drain(fin, 0, p.timeout_ns);
        }
        __syncwarp();
      }
    } else if (C::STORE_WARP && warp == 2) {
      // ---------------------------------------------------------- store
      if (lane == 0) {
        uint32_t phase = 0;
        for (int t = unit; t < num_tiles; t += nunits) {
          const int mb = t / p.tiles_n, nb = t - mb * p.tiles_n;
          const int row0 = mb * C::TILE_M + static_cast<int>(rank) * C::BM;
          if (!mbar_wait(oready, phase, w)) break;
#pragma unroll
          for (int c = 0; c < C::BN / 64; ++c) tma_store_2d(&p.tmOut, sOut + c * C::CHUNK, nb * C::BN + c * 64, row0);
          if constexpr (C::RELU2) {
#pragma unroll
            for (int c = 0; c < C::BN / 128; ++c)
              tma_store_2d(&p.tmOut2, sOut + (C::BN / 64 + c) * C::CHUNK, nb * C::BN + c * 128, row0);
          }
          bulk_commit();
          bulk_wait_read<0>();
          mbar_arrive(ofree);
          phase ^= 1u;
        }
        bulk_wait<0>();
      }
    } else if (warp == C::SCALE_WARP) {
      // ---------------------------------------------------------- scales
      // The epilogue would have to wait for loads of its own (each k-block
      // takes less time than one from L2), so this warp keeps four k-blocks'
      // scales under way and puts them beside their stage.
      int st = unit, skb = 0;
      const float *px = nullptr, *pw = nullptr;  // of k-block 0
      int rows = 0;
      bool wlane = false;
      auto seek = [&]() {
        rows = 0;
        wlane = false;
        if (st >= num_tiles) return;
        const int mb = st / p.tiles_n, nb = st - mb * p.tiles_n;
        const int m = mb * C::TILE_M + static_cast<int>(rank) * C::BM + lane;
        const int nblk = nb * (C::BN / 128) + lane;
        rows = p.M - m;
        wlane = lane < C::BN / 128 && nblk < p.n_blocks;
        px = p.xs + m;
        pw = p.ws + nblk;
      };
      auto load = [&](float (&v)[5]) {
        const float* x = px + static_cast<size_t>(skb) * p.M;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = ld_scale(x + i * 32, rows > i * 32);
        v[4] = ld_scale(pw + static_cast<size_t>(skb) * p.n_blocks, wlane);
        if (++skb == num_kb) {
          skb = 0;
          st += nunits;
          seek();
        }
      };
      seek();
      float v[4][5];
#pragma unroll
      for (int j = 0; j < 4; ++j) load(v[j]);
      const long long my_tiles = unit < num_tiles ? (num_tiles - unit + nunits - 1) / nunits : 0;
      const long long steps = my_tiles * num_kb;
      // from here on a slot, or its stage's barrier, is not in its first round
      constexpr int kFirst = C::SRING < C::STAGES ? C::SRING : C::STAGES;
      uint32_t stage = 0, slot = 0, sphase = 1, wstage = kFirst - C::SRING + C::NBUF, wphase = 0;
      bool ok = true;
      for (long long g0 = 0; g0 < steps && ok; g0 += 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (g0 + j >= steps) break;
          if constexpr (C::SLOT_BARS) {
            ok = mbar_wait_inline(&sempty[slot], sphase, w);
          } else if (g0 + j >= kFirst) {
            ok = mbar_wait_inline(&done[wstage], wphase, w);
            if (++wstage == C::STAGES) {
              wstage = 0;
              wphase ^= 1u;
            }
          }
          if (!ok) break;
          float* s = sScale + slot * (C::SCALES / 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[lane + i * 32] = v[j][i];
          if (lane < C::BN / 128) s[128 + lane] = v[j][4];
          __syncwarp();
          if (lane == 0) mbar_arrive(C::SLOT_BARS ? &sfull[slot] : &full[stage]);
          load(v[j]);
          if (++slot == C::SRING) {
            slot = 0;
            sphase ^= 1u;
          }
          if (++stage == C::STAGES) stage = 0;
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    if constexpr (C::SPLIT_REGS) reg_inc<C::REGS_EPI>();
    const int q = warp & 3;  // TMEM lane quarter
    const int e = warp - C::EPI0;
    const int c0 = (e >> 2) * 128;  // first column of the tile that is this warp's
    const uint32_t tmem_mine = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + c0;
    const uint32_t tempty0 = CG == 2 ? mapa_shared(smem_u32(&tempty[0]), 0) : 0u;
    const uint32_t orow = smem_u32(sOut) + (e >> 2) * (2 * C::CHUNK) + (q * 32 + lane) * 128;  // this thread's row, bf16
    const uint32_t qrow = smem_u32(sOut) + (C::BN / 64 + (e >> 2)) * C::CHUNK + (q * 32 + lane) * 128;  // codes
    const uint32_t xor16 = (lane & 7) << 4;  // of the 128-byte swizzle
    uint32_t buf = 0, stage = 0, phase = 0, slot = 0, sphase = 0, ofree_phase = 1;

    // this warp's rows of a chunk, out
    auto store_part = [&](const CUtensorMap* map, int chunk, int col, int row) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(map, sOut + chunk * C::CHUNK + q * 4096, col, row);
        bulk_commit();
      }
    };
    bool ok = true;
    for (int t = unit; t < num_tiles; t += nunits) {
      const int mb = t / p.tiles_n, nb = t - mb * p.tiles_n;
      const int row0 = mb * C::TILE_M + static_cast<int>(rank) * C::BM + q * 32;
      const int n0 = nb * C::BN + c0;
      uint64_t acc[64];  // 128 fp32 sums as pairs
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0;
      for (int kb = 0; kb < num_kb; ++kb) {
        float f = 0.f;
        auto factor = [&]() {
          const float* sc = sScale + slot * (C::SCALES / 4);
          f = __fmul_rn(sc[q * 32 + lane], sc[128 + (c0 >> 7)]);
        };
        if constexpr (C::SLOT_BARS) {
          if (!mbar_wait_inline(&sfull[slot], sphase, w)) {
            ok = false;
            break;
          }
          factor();
        }
        if (!mbar_wait_inline(&done[stage], phase, w)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // sixteen columns are multiplied while the next sixteen are read
        uint32_t v[2][16];
        const uint32_t src = tmem_mine + buf * C::BN;
        tmem_ld16_issue(src, v[0]);
        if constexpr (!C::SLOT_BARS) factor();
        const uint64_t f2 = f2_pack(f, f);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          tmem_wait16(v[c & 1]);
          if (c < 7) {
            tmem_ld16_issue(src + (c + 1) * 16, v[(c + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if constexpr (CG == 1)
                mbar_arrive(&tempty[buf]);
              else
                mbar_arrive_cluster_relaxed(tempty0 + buf * 8u);
              if constexpr (C::SLOT_BARS) mbar_arrive(&sempty[slot]);
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            acc[c * 8 + i] = f2_fma(
                f2_pack(__uint_as_float(v[c & 1][2 * i]), __uint_as_float(v[c & 1][2 * i + 1])), f2, acc[c * 8 + i]);
        }
        if (++buf == C::NBUF) buf = 0;
        if (++slot == C::SRING) {
          slot = 0;
          sphase ^= 1u;
        }
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      float s = 1.f;
      if constexpr (C::RELU2) {
        // acc |acc| in place, whose positive part is post (the conversions drop
        // the rest), the maximum over this 1 x 128 block (columns past N are
        // zero), and the block's scale.  The codes are rounded once, from the
        // fp32 value.
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          float u, v;
          f2_unpack(acc[i], u, v);
          amax = max3_nan(amax, u, v);
          acc[i] = f2_pack(__fmul_rn(u, fabsf(u)), __fmul_rn(v, fabsf(v)));
        }
        amax = __fmul_rn(amax, amax);  // squaring is monotone, its rounding too
        float inv;
        s = block_scale(amax, &inv);
        if (row0 + lane < p.M && n0 < p.N)
          p.post_s[static_cast<size_t>(n0 >> 7) * p.M + row0 + lane] = inv;
      }
      // the previous tile has left shared memory
      if constexpr (C::STORE_WARP) {
        if (!mbar_wait_inline(ofree, ofree_phase, w)) break;
        ofree_phase ^= 1u;
      } else {
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        uint32_t pk[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float u, v;
          f2_unpack(acc[j * 4 + i], u, v);
          pk[i] = C::RELU2 ? pack_bf16x2_relu(u, v) : pack_bf16x2(u, v);
        }
        st_shared_v4(orow + (j >> 3) * C::CHUNK + (((j & 7) * 16) ^ xor16), pk[0], pk[1], pk[2], pk[3]);
        if (!C::STORE_WARP && (j & 7) == 7) store_part(&p.tmOut, j >> 3, n0 + (j >> 3) * 64, row0);
      }
      if constexpr (C::RELU2) {
        const uint64_t s2 = f2_pack(s, s);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t qk[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float u0, u1, u2, u3;
            f2_unpack(f2_mul(acc[j * 8 + 2 * i], s2), u0, u1);
            f2_unpack(f2_mul(acc[j * 8 + 2 * i + 1], s2), u2, u3);
            qk[i] = pack_e4m3x2_relu(u0, u1) | (pack_e4m3x2_relu(u2, u3) << 16);
          }
          st_shared_v4(qrow + ((j * 16) ^ xor16), qk[0], qk[1], qk[2], qk[3]);
        }
        if (!C::STORE_WARP) store_part(&p.tmOut2, C::BN / 64, n0, row0);
      }
      if constexpr (C::STORE_WARP) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(oready);
      }
    }
    if (!C::STORE_WARP && lane == 0) bulk_wait<0>();
    __syncwarp();
  }

  __syncwarp();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc<CG>(tmem_base, 512);
  }
}

}  // namespace fp8mlp
