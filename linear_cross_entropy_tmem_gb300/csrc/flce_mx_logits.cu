// flce_mx_logits.cu — a head's logits from a weight in 4 bits: the block-scaled
// tcgen05 product, and its C entry point.
//
//   z[n, v] = logit_scale (sum over blocks of 2^(kh + kw) sum of ch cw  + bias[v]),  out = rn(cap(z))
//
// Few tokens: bound by the weight's bytes, 17/32 of V D.  The weight is the MMA's
// A operand (128 vocabulary entries, TMEM lanes), the tokens its B operand (16 to
// 208 TMEM columns), so that a single token costs a tile of 16 columns and not of
// 128 rows.  4096 x 151936: 55 us for one token (the bytes alone 49), 59 for 64, 73 for
// 208.
//
// Many tokens: 2047 take 490 us, 5.2 PFLOP/s.  What a tile takes from L2 (43 KB for 128 x
// 192 x 256) takes 335 us by itself; the products, which run under it, add 20, the copies of
// the scales, in line with them, 60, the epilogue's work on TMEM and its stores 70.  (CTA
// pairs with tiles of 256 x 192 take a third less from L2, but the loads alone took them
// longer, also with seven stages under way: 550 and 633 us.)
//
//   warp 8     TMA producer: per stage 256 columns (128 bytes of a row, one
//              swizzle atom) of both operands, and their scales as they lie in
//              memory.  As many stages as fit.
//   warp 9     issuer: copies a stage's scales from shared memory to TMEM
//              (tcgen05.cp; each stage has TMEM columns of its own, so that they are
//              free when the stage is), then four MMAs of K = 64.
//   warps 0-7  two epilogue groups, one for each of two accumulators: bias,
//              scale, soft cap, rounding, store.
//
// The weight's copies of the first stages are issued before the hidden states'
// quantisation (the launch before this one) is waited for.  Waits are bounded as
// in the other products.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cuda.h>

#include "flce_mxfp4.cuh"

namespace flce {
namespace {

constexpr int kMxM = 128;              // vocabulary entries of a tile
constexpr int kMxMaxN = 208;           // tokens of a tile, at most: two accumulators and four stages' scales fill TMEM
constexpr int kMxManyN = 192;          // the same where there are more tiles than one: five stages fit
constexpr int kMxK = 256;              // columns of a stage
constexpr int kMxRow = kMxK / 2;       // bytes
constexpr int kMxMaxStages = 10;
constexpr int kMxSmem = 216 << 10;     // for the stages
constexpr uint32_t kTmemAll = 512;
constexpr int kMxTurn = 4096;          // bytes in which an epilogue group turns its output round
constexpr int kMxTurnTokens = 17;      // from so many tokens on (8 tokens: 58.4 us either way)

struct MxLogitsParams {
  const uint8_t *a_scales, *b_scales;
  const void* bias;
  void* out;
  int64_t os;
  int32_t tokens, vocab, cols;
  int32_t tile_n, halves, groups, kbs;     // kbs: stages of a tile
  int32_t m_tiles, n_tiles, stages;
  int32_t stage_bytes, b_off, as_off, bs_off;
  int32_t sf_col, sf_cols;                 // TMEM columns of the scales: the first, and a stage's
  int32_t bias_dtype;
  float scale, cap, inv_cap;
};

// E2M1 operands, power-of-two scales, fp32 sums, K-major, M = 128, N = n; the scales of K step
// `half` of two are bytes 2 half and 2 half + 1 of a TMEM word.
__device__ __forceinline__ uint32_t instr_desc_mxf4(uint32_t n, uint32_t half) {
  return (half * 2u) << 4        // B's scale byte
         | (1u << 7)             // A: e2m1
         | (1u << 10)            // B: e2m1
         | ((n >> 3) << 17)      // N / 8
         | (1u << 23)            // scales: e8m0
         | ((kMxM >> 4) << 24)   // M / 16
         | (half * 2u) << 29;    // A's scale byte
}
// These are issued by the lane with `lead`, from code that the whole warp runs: where
// control flow is uniform the descriptors stay in uniform registers.  (Issued from one
// thread's own branch, a stage's four copies and four MMAs took 600 cycles, more than
// the stage's bytes: one token of 4096 x 151936 took 63 us in place of 55, 2047 tokens 676 in
// place of 522 at the time.)
__device__ __forceinline__ void umma_mxf4(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                          uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "setp.ne.b32 q, %7, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit_to(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(smem_u32(bar)), "r"(lead)
      : "memory");
}
// 512 bytes of scales (32 rows of 16 bytes) to 4 TMEM columns, the same in each
// quarter of the lanes: lane l, column c holds the scales of row 32 c + l.
__device__ __forceinline__ uint64_t scale_desc(uint32_t smem) {  // no swizzle; groups of 8 rows are 128 bytes apart
  return static_cast<uint64_t>((smem & 0x3FFFFu) >> 4) | static_cast<uint64_t>(128 >> 4) << 32 | uint64_t(1) << 46;
}
__device__ __forceinline__ void copy_scales(uint32_t lead, uint32_t taddr, uint64_t desc) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}\n" ::"r"(taddr), "l"(desc), "r"(lead)
      : "memory");
}
// Untiled copy of a multiple of 16 bytes, completion counted on an mbarrier.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// tanh, relative error about 3 units of fp32's last place, without a branch: below 1 Lambert's
// continued fraction to u^2 / 9, else (e - 1) / (e + 1) with e = e^(2 u); one reciprocal.
__device__ __forceinline__ float tanh_both(float u) {
  const float t = fminf(fmaxf(u * (2.f * kLog2e), -60.f), 60.f), e = ex2_approx(t), s = u * u;
  const bool low = s < 1.f;
  const float num = low ? u * fmaf(s, s + 105.f, 945.f) : e - 1.f;
  const float den = low ? fmaf(s, fmaf(s, 15.f, 420.f), 945.f) : e + 1.f;
  const float y = num * rcp_approx(den);
  return u != u ? u : y;  // (the bounds of t would hide a NaN)
}

constexpr int kMxBarrierBytes = 1024;
struct MxSmem {
  uint8_t* stage;
  uint64_t *full, *empty, *tfull, *tempty, *drain;
  uint32_t* tmem_slot;
  CtaControl* ctl;
  uint8_t* turn;
};
__device__ __forceinline__ MxSmem carve(uint8_t* raw, int stages, int stage_bytes) {
  MxSmem s;
  s.stage = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  s.full = reinterpret_cast<uint64_t*>(s.stage + stages * stage_bytes);
  s.empty = s.full + kMxMaxStages;
  s.tfull = s.empty + kMxMaxStages;
  s.tempty = s.tfull + kAccBufs;
  s.drain = s.tempty + kAccBufs;
  s.tmem_slot = reinterpret_cast<uint32_t*>(s.drain + 1);
  s.ctl = reinterpret_cast<CtaControl*>(s.tmem_slot + 2);
  s.turn = s.stage + stages * stage_bytes + kMxBarrierBytes;
  return s;
}

// As mbar_wait, but the clock and the abort flag are looked at once in 64 tries: these waits end within a
// microsecond, and their wake-up is on the way of every stage.
__device__ __forceinline__ bool stage_wait(uint64_t* bar, uint32_t parity, CtaControl* ctl, int* status) {
  const uint32_t addr = smem_u32(bar);
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(addr, parity)) return true;
    if (i & 63u) continue;
    if (ctl->abort) return false;
    const uint64_t t = global_timer_ns();
    if (t0 == 0) t0 = t;
    if (t - t0 > kWaitTimeoutNs) {
      ctl->abort = 1u;
      if (status) atomicCAS(status, 0, kStatusTimeout);
      return false;
    }
  }
}

// For a whole warp, which gives up as one (a vote is uniform).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, CtaControl* ctl, int* status) {
  const uint32_t addr = smem_u32(bar);
  if (__all_sync(0xffffffffu, mbar_try_wait(addr, parity))) return true;
  return __all_sync(0xffffffffu, stage_wait(bar, parity, ctl, status));
}

// The four warps of an epilogue group.
__device__ __forceinline__ void group_sync(int grp) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + grp) : "memory");
}
__device__ __forceinline__ bool group_all(int grp, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, %2, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}\n"
      : "=r"(all)
      : "r"(uint32_t(ok)), "r"(1 + grp)
      : "memory");
  return all != 0;
}

// Until a copy or an MMA that this thread started has ended (bounded all the same).
__device__ __forceinline__ void wait_teardown(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(smem_u32(bar), parity))
    if (global_timer_ns() - t0 > kWaitTimeoutNs) return;
}

// The tile's tokens are the faster index: blocks that run together share weight tiles.
__device__ __forceinline__ void tile_of(const MxLogitsParams& p, int u, int& m, int& n) {
  m = u / p.n_tiles;
  n = u - m * p.n_tiles;
}

// A CTA's steps, a stage each: `kbs` per tile, tiles `stride` apart; counted up, without divisions.
struct Step {
  int m, n, kb = 0, dm, dn;
  __device__ __forceinline__ Step(const MxLogitsParams& p, int first, int stride) {
    tile_of(p, first, m, n);
    tile_of(p, stride, dm, dn);
  }
  __device__ __forceinline__ void next(const MxLogitsParams& p) {
    if (++kb < p.kbs) return;
    kb = 0;
    m += dm;
    n += dn;
    if (n >= p.n_tiles) {
      n -= p.n_tiles;
      ++m;
    }
  }
};

// kTurned: rows of the output start on 16-byte boundaries.  TMEM's lanes are vocabulary entries, so
// that a warp has 32 of a token's logits; the group's four warps turn 128 of several tokens' round in
// shared memory, and store lines of 256 or 512 bytes (2047 tokens 490 us in place of 522 with
// 64 bytes from a warp; 64 tokens to fp32, 128256 x 2048, 34 in place of 37).
template <class O, bool kTurned>
__global__ void __launch_bounds__(kThreads, 1)
    mx_logits_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                     const __grid_constant__ MxLogitsParams p, int* status) {
  extern __shared__ uint8_t smem_raw[];
  const MxSmem sm = carve(smem_raw, p.stages, p.stage_bytes);
  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0);  // (uniform)
  const int units = p.m_tiles * p.n_tiles, first = int(blockIdx.x), stride = int(gridDim.x);
  if (threadIdx.x == kTmaWarp * 32) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int b = 0; b < kAccBufs; ++b) {
      mbar_init(&sm.tfull[b], 1);
      mbar_init(&sm.tempty[b], kEpilogueWarps);
    }
    mbar_init(sm.drain, 1);
    sm.ctl->abort = 0u;
    fence_mbar_init();
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_b);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(sm.tmem_slot, kTmemAll);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *sm.tmem_slot, 0);

  if (warp == kTmaWarp) {
    // ---------------------------------------------------------------- producer
    if (elect_one()) {
      const int mine = units > first ? (units - 1 - first) / stride + 1 : 0;
      const int64_t steps = int64_t(mine) * p.kbs;
      // Half of a stage: the weight's (with the count of all bytes that the stage waits for), or the tokens'.
      auto load = [&](const Step& s, int stage, bool weight) {
        const int m = s.m, n = s.n, kb = s.kb;
        uint8_t* at = sm.stage + stage * p.stage_bytes;
        uint64_t* bar = &sm.full[stage];
        const int groups = min(2, p.groups - 2 * kb);
        if (weight) {
          mbar_arrive_expect_tx(bar, uint32_t((kMxM + p.tile_n) * kMxRow + groups * (1 + p.halves) * kScaleTile));
          tma_load_2d(at, &map_a, bar, kb * kMxRow, m * kMxM);
          bulk_load(at + p.as_off, p.a_scales + (int64_t(m) * p.groups + 2 * kb) * kScaleTile, groups * kScaleTile, bar);
        } else {
          tma_load_2d(at + p.b_off, &map_b, bar, kb * kMxRow, n * p.tile_n);
          bulk_load(at + p.bs_off, p.b_scales + (int64_t(n) * p.groups + 2 * kb) * p.halves * kScaleTile,
                    groups * p.halves * kScaleTile, bar);
        }
      };
      const int ahead = int(min(int64_t(p.stages), steps));
      Step w(p, first, stride), t = w;
      for (int i = 0; i < ahead; ++i, w.next(p)) load(w, i, true);
      griddep_wait();  // the hidden states are quantised, the status word is cleared
      for (int i = 0; i < ahead; ++i, t.next(p)) load(t, i, false);
      int stage = 0;
      uint32_t phase = 0;
      int64_t i = ahead;
      if (ahead == p.stages) {
        for (; i < steps; ++i) {
          if (!stage_wait(&sm.empty[stage], phase, sm.ctl, status)) break;
          load(w, stage, true);
          load(w, stage, false);
          w.next(p);
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // Every copy this thread issued has to land before the CTA may exit.
      for (int64_t j = max(int64_t(0), i - p.stages); j < i; ++j)
        wait_teardown(&sm.full[j % p.stages], uint32_t((j / p.stages) & 1));
    }
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- issuer
    {
      const uint32_t lead = elect_one() ? 1u : 0u;
      const uint32_t idesc0 = instr_desc_mxf4(uint32_t(p.tile_n), 0), idesc1 = instr_desc_mxf4(uint32_t(p.tile_n), 1);
      const uint32_t smem0 = smem_u32(sm.stage);
      const uint64_t a0 = smem_desc_sw128(smem0, 16, 1024), b0 = smem_desc_sw128(smem0 + uint32_t(p.b_off), 16, 1024);
      const uint64_t as0 = scale_desc(smem0 + uint32_t(p.as_off)), bs0 = scale_desc(smem0 + uint32_t(p.bs_off));
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int u = first; ok && u < units; u += stride) {
        if (!warp_wait(&sm.tempty[acc], acc_phase ^ 1u, sm.ctl, status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + uint32_t(acc * p.tile_n);
        for (int kb = 0; kb < p.kbs; ++kb) {
          if (!warp_wait(&sm.full[stage], phase, sm.ctl, status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          // (descriptors hold addresses in units of 16 bytes, below 2^14 of them: sums do not carry over)
          const uint64_t off = uint64_t(uint32_t(stage * p.stage_bytes) >> 4);
          const uint32_t sf = tmem + uint32_t(p.sf_col + stage * p.sf_cols);
          const int groups = p.groups - 2 * kb;
          copy_scales(lead, sf, as0 + off);
          copy_scales(lead, sf + 8, bs0 + off);
          if (p.halves == 2) copy_scales(lead, sf + 12, bs0 + off + kScaleTile / 16);
          if (groups > 1) {
            copy_scales(lead, sf + 4, as0 + off + kScaleTile / 16);
            copy_scales(lead, sf + 8 + p.halves * 4, bs0 + off + p.halves * (kScaleTile / 16));
            if (p.halves == 2) copy_scales(lead, sf + 20, bs0 + off + 3 * (kScaleTile / 16));
          }
          const int left = p.cols - kb * kMxK;
          const uint32_t sfb = sf + 8, sfb1 = sfb + p.halves * 4;
          umma_mxf4(lead, d, a0 + off, b0 + off, idesc0, sf, sfb, uint32_t(kb));
          if (left > 64) umma_mxf4(lead, d, a0 + off + 2, b0 + off + 2, idesc1, sf, sfb, 1u);
          if (left > 128) umma_mxf4(lead, d, a0 + off + 4, b0 + off + 4, idesc0, sf + 4, sfb1, 1u);
          if (left > 192) umma_mxf4(lead, d, a0 + off + 6, b0 + off + 6, idesc1, sf + 4, sfb1, 1u);
          commit_to(lead, &sm.empty[stage]);
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        commit_to(lead, &sm.tfull[acc]);
        if (++acc == kAccBufs) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      commit_to(lead, sm.drain);
      wait_teardown(sm.drain, 0);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- epilogue
    const int grp = warp / kEpilogueWarps, quarter = warp % kEpilogueWarps;
    const uint32_t taddr = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(grp * p.tile_n);
    uint32_t phase = 0;
    int seq = 0;
    for (int u = first; u < units; u += stride, ++seq) {
      if ((seq & 1) != grp) continue;
      // (the warp gives up as one, and where the group's warps share a buffer, they do)
      bool ok;
      if constexpr (kTurned) {
        ok = group_all(grp, stage_wait(&sm.tfull[grp], phase, sm.ctl, status));
      } else {
        ok = warp_wait(&sm.tfull[grp], phase, sm.ctl, status);
      }
      if (!ok) break;
      tc_fence_after();
      int m, n;
      tile_of(p, u, m, n);
      const int v0 = m * kMxM, v = v0 + quarter * 32 + int(lane_id());
      const float bias = p.bias && v < p.vocab ? load_as(p.bias, p.bias_dtype, v) : 0.f;
      const int n0 = n * p.tile_n, count = min(p.tile_n, p.tokens - n0);
      O* out0 = static_cast<O*>(p.out) + int64_t(n0) * p.os + v0;
      for (int c = 0; c < count; c += 32) {
        uint32_t r[32];
        tmem_ld32(taddr + uint32_t(c), r);
        tmem_ld_wait(r);
        auto logit = [&](int j) {
          float z = (__uint_as_float(r[j]) + bias) * p.scale;
          if (p.cap > 0.f) z = p.cap * tanh_both(z * p.inv_cap);
          return from_f32<O>(z);
        };
        if constexpr (kTurned) {
          constexpr int kRows = kMxTurn / (kMxM * int(sizeof(O))), kE = 16 / int(sizeof(O)), kPerRow = kMxM / kE;
          O* turn = reinterpret_cast<O*>(sm.turn + grp * kMxTurn);
          const int t = quarter * 32 + int(lane_id());
#pragma unroll
          for (int k = 0; k < 32; k += kRows) {
            if (c + k >= count) break;
            group_sync(grp);  // the rows before are read
#pragma unroll
            for (int j = 0; j < kRows; ++j) turn[j * kMxM + t] = logit(k + j);
            group_sync(grp);
#pragma unroll
            for (int i = t; i < kRows * kPerRow; i += 128) {
              const int row = c + k + i / kPerRow, at = i % kPerRow * kE;
              if (row >= count) break;
              const Vec<O, kE> x = load_vec<O, kE>(turn + i * kE);
              O* to = out0 + int64_t(row) * p.os + at;
              if (v0 + at + kE <= p.vocab) {
                store_vec<O, kE>(to, x);
              } else {
#pragma unroll
                for (int e = 0; e < kE; ++e)
                  if (v0 + at + e < p.vocab) to[e] = x.v[e];
              }
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c + j < count && v < p.vocab) out0[int64_t(c + j) * p.os + (v - v0)] = logit(j);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane_id() == 0) mbar_arrive(&sm.tempty[grp]);
      phase ^= 1u;
    }
  }
  griddep_release();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemAll);
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
struct MxPlan {
  int tile_n, n_tiles, halves, stages, stage_bytes;
  size_t codes, scales, bytes;  // places in the workspace
};
MxPlan plan(const flce_mxfp4_logits_problem* p) {
  MxPlan l;
  const int most = p->tokens <= kMxMaxN ? kMxMaxN : kMxManyN;
  l.n_tiles = int(std::max<int64_t>(1, mx_cdiv(p->tokens, most)));
  l.tile_n = int(std::max<int64_t>(16, mx_cdiv(mx_cdiv(p->tokens, l.n_tiles), 16) * 16));
  l.halves = l.tile_n > 128 ? 2 : 1;
  l.stage_bytes = int(mx_cdiv((kMxM + l.tile_n) * kMxRow + 2 * (1 + l.halves) * kScaleTile, 1024) * 1024);
  // TMEM: two accumulators, and 8 + 8 halves columns of scales for each stage
  const int by_tmem = (int(kTmemAll) - 2 * l.tile_n) / (8 + 8 * l.halves);
  l.stages = std::min({kMxMaxStages, kMxSmem / l.stage_bytes, by_tmem});
  l.codes = 256;
  l.scales = l.codes + size_t(p->tokens) * size_t(mx_row_bytes(p->cols));
  l.scales = (l.scales + 255) / 256 * 256;
  l.bytes = l.scales + size_t(l.n_tiles) * size_t(l.halves) * size_t(mx_groups(p->cols)) * kScaleTile;
  return l;
}

int validate(const flce_mxfp4_logits_problem* p) {
  if (!p) return FLCE_ERR_INVALID_ARG;
  if (p->tokens < 0 || p->tokens > (1 << 24) || p->vocab < 1 || p->vocab >= INT32_MAX - 256 || p->cols < 1 ||
      p->cols > (1 << 20) || p->hidden_stride < 0 || p->out_stride < 0)
    return FLCE_ERR_INVALID_ARG;
  if (mx_cdiv(p->vocab, kMxM) * mx_cdiv(std::max<int64_t>(1, p->tokens), 16) > INT32_MAX / 2) return FLCE_ERR_INVALID_ARG;
  if (!known_dtype(p->hidden_dtype) || !known_dtype(p->out_dtype) || !known_dtype(p->bias_dtype))
    return FLCE_ERR_UNSUPPORTED_DTYPE;
  if (!std::isfinite(p->logit_scale) || !std::isfinite(p->softcap) || p->softcap < 0.f) return FLCE_ERR_INVALID_ARG;
  return FLCE_OK;
}

template <class O, bool kTurned>
cudaError_t launch_logits(const CUtensorMap& a, const CUtensorMap& b, const MxLogitsParams& q, int* status, int num_sms,
                          cudaStream_t st) {
  auto kern = mx_logits_kernel<O, kTurned>;
  const int smem = 1024 + q.stages * q.stage_bytes + kMxBarrierBytes + 2 * kMxTurn;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             1024 + kMxSmem + kMxBarrierBytes + 2 * kMxTurn);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(std::min(q.m_tiles * q.n_tiles, num_sms)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, b, q, status);
}
template <class O>
cudaError_t launch_logits(const CUtensorMap& a, const CUtensorMap& b, const MxLogitsParams& q, int* status, int num_sms,
                          cudaStream_t st) {
  const bool lines = q.tokens >= kMxTurnTokens && aligned_to(q.out, 16) && q.os * int64_t(sizeof(O)) % 16 == 0;
  return lines ? launch_logits<O, true>(a, b, q, status, num_sms, st)
               : launch_logits<O, false>(a, b, q, status, num_sms, st);
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

int flce_mxfp4_logits_workspace_size(const flce_mxfp4_logits_problem* problem, size_t* bytes) {
  if (!bytes) return FLCE_ERR_INVALID_ARG;
  FLCE_TRY(validate(problem));
  *bytes = plan(problem).bytes + 256;
  return FLCE_OK;
}

int flce_mxfp4_logits(const flce_mxfp4_logits_problem* problem, const void* hidden, const void* codes,
                      const void* scales, const void* bias, void* out, void* workspace, size_t workspace_bytes,
                      flce_stream_t stream) {
  const flce_mxfp4_logits_problem* p = problem;
  size_t need = 0;
  FLCE_TRY(flce_mxfp4_logits_workspace_size(p, &need));
  if (p->tokens == 0) return FLCE_OK;
  if (!hidden || !codes || !scales || !out || !workspace || (p->tokens > 1 && p->out_stride < p->vocab))
    return FLCE_ERR_INVALID_ARG;
  if (!aligned_to(hidden, elem_size(p->hidden_dtype)) || !aligned_to(codes, 16) || !aligned_to(scales, 16) ||
      !aligned_to(out, elem_size(p->out_dtype)) || !aligned_to(workspace, 16) ||
      (bias && !aligned_to(bias, elem_size(p->bias_dtype))))
    return FLCE_ERR_MISALIGNED;
  if (workspace_bytes < need) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  DeviceInfo dev;
  FLCE_TRY(get_device(&dev));
  FLCE_TRY(check_local(dev, hidden, codes, scales, bias, out, workspace));
  const MxPlan l = plan(p);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  CUtensorMap a, b;
  const uint64_t row = uint64_t(mx_row_bytes(p->cols));
  FLCE_TRY(make_byte_map(&a, codes, row, uint64_t(p->vocab), kMxRow, kMxM));
  FLCE_TRY(make_byte_map(&b, ws + l.codes, row, uint64_t(p->tokens), kMxRow, uint32_t(l.tile_n)));
  MxQuantParams h{};
  h.x = hidden;
  h.codes = ws + l.codes;
  h.scales = ws + l.scales;
  h.status = reinterpret_cast<int*>(ws);
  h.rows = p->tokens;
  h.stride = p->hidden_stride;
  h.cols = int32_t(p->cols);
  h.tile_rows = l.tile_n;
  FLCE_TRY(logged(FLCE_LAUNCH_OTHER, st,
                  [&] { return launch_mx_quantize(h, p->hidden_dtype, int64_t(l.n_tiles) * l.tile_n, dev.num_sms, st); }));
  MxLogitsParams q{};
  q.a_scales = static_cast<const uint8_t*>(scales);
  q.b_scales = ws + l.scales;
  q.bias = bias;
  q.out = out;
  q.os = p->out_stride;
  q.tokens = int32_t(p->tokens);
  q.vocab = int32_t(p->vocab);
  q.cols = int32_t(p->cols);
  q.tile_n = l.tile_n;
  q.halves = l.halves;
  q.groups = int32_t(mx_groups(p->cols));
  q.kbs = int32_t(mx_cdiv(p->cols, kMxK));
  q.m_tiles = int32_t(mx_cdiv(p->vocab, kMxM));
  q.n_tiles = l.n_tiles;
  q.stages = l.stages;
  q.stage_bytes = l.stage_bytes;
  q.b_off = kMxM * kMxRow;
  q.as_off = q.b_off + l.tile_n * kMxRow;
  q.bs_off = q.as_off + 2 * kScaleTile;
  q.sf_col = 2 * l.tile_n;
  q.sf_cols = 8 + 8 * l.halves;
  q.bias_dtype = p->bias_dtype;
  q.scale = p->logit_scale;
  q.cap = p->softcap;
  // (1 / cap of the smallest numbers is beyond fp32: an infinity would make a logit of 0 not a number)
  q.inv_cap = p->softcap > 0.f ? std::min(1.f / p->softcap, FLT_MAX) : 0.f;
  int* status = reinterpret_cast<int*>(ws);
  return logged(FLCE_LAUNCH_OTHER, st, [&] {
    if (p->out_dtype == FLCE_F32) return launch_logits<float>(a, b, q, status, dev.num_sms, st);
    if (p->out_dtype == FLCE_BF16) return launch_logits<__nv_bfloat16>(a, b, q, status, dev.num_sms, st);
    return launch_logits<__half>(a, b, q, status, dev.num_sms, st);
  });
}

}  // extern "C"
