// Grouped block-scaled FP8 products for few rows per expert (decoding, small ragged
// batches), sm_100a: the forward and DGrad of a layer with one weight per expert,
//
//   out[i, j] = sum_r  sA(i, r) * sB(e, j / 128, r) * sum_{l in slice r} qA[i, l] * qB_e[j, l]
//
// for the rows i of expert e, with the arithmetic of the large-tile kernel (each 128-wide
// slice an FP8 tensor-core product in fp32, acc = fma(P_r, sA * sB, acc) in increasing r
// from +0), so that a row has the same bits whichever kernel the sizes select.
//
// With a few rows per expert the product is bound by reading every active expert's FP8
// weights once (2 flops per weight byte and row, far below the tensor cores' rate), so:
//
//  * The weights are the MMA's M side: a tile is 128 weight rows x at most kNT token rows,
//    so an expert with few tokens costs an MMA of N = kNT (32 .. 128) and the token rows
//    ride along, instead of 128 or 256 mostly empty token rows per MMA.
//  * Persistent CTAs, one per SM, walk the tiles of all experts that have rows (expert by
//    expert, the token tiles of a strip next to each other so that they share its weights
//    in L2); the copies of the next tile start while this one is multiplied, promoted and
//    stored, so the weight stream does not stop between tiles or experts.
//  * A ring of stages of kG consecutive slices, up to 200 KB in all (a strip lower than 128
//    rows fills a part of each stage: 16 of 40 KB at 32 weight and 32 token rows): one 3D
//    tensor copy brings kG * 128 bytes of each of the weight rows, another the token rows of
//    the same slices (single-slice stages measured 1-4 % slower: twice the copies and
//    barriers).
//  * Warp 0 is the producer; warps 1 and 2 issue the MMAs of alternate stages into up to 8
//    TMEM buffers of kG slices; warp 3 multiplies each slice's token scales by its block
//    scale, in shared memory; the other warps promote a buffer at a time (figures at
//    launch_grouped_strips), in the 16x256b shape: a lane holds 4 weight rows x a quarter of
//    its warpgroup's tokens (all of them, or half in each of two warpgroups from 64 tokens
//    on), so that it reads a quarter of the scale products. With a weight row per lane every
//    lane read all of them, 16-byte broadcasts that filled the shared-memory pipe: 16 experts
//    of 3584 x 1024, 64 rows each, took 18.7 us, 14.4 this way (four warpgroups: 18.0; captured
//    calls whose operands stay in L2).
//  * Epilogue: 16 tokens at a time through shared memory by a transposing stmatrix, so that
//    a warp stores 64 bytes of each of 8 tokens at once.
//
// The first token row of an expert's tiles is rounded down to a multiple of 4 (the row
// scales come by tensor copy, whose innermost coordinate is a multiple of 16 bytes); rows
// of other experts in a tile are multiplied and not stored.
// Every mbarrier wait is bounded; a wait that gives up records FP8Q_ERR_TIMEOUT in the
// device error word and the CTA winds down.
#include <algorithm>
#include <atomic>

#include "fp8q_device.cuh"
#include "fp8q_grouped.cuh"
#include "fp8q_host.h"

namespace fp8q {
namespace {

constexpr int kGmIssuers = 2;    // warps 1 and 2
constexpr int kGmScaleWarp = 3;  // forms the scale products
constexpr int kGmPromote = 4;    // first promotion warp
constexpr int kGmRows = 128;     // weight rows of a tile
constexpr int kGmBK = 128;
constexpr int kGmMaxStages = 8;
constexpr int kGmScRing = 8;     // row-scale slots (one per stage's slices)
constexpr uint32_t kGmMaxSmem = 232448;
constexpr uint32_t kGmStaging = 1024;  // a promotion warp's outputs: 16 tokens x 32 weight rows

template <int kNT>
struct GmShape {
  static constexpr int kG = 2;  // slices per stage, accumulator buffer and row-scale slot
  static constexpr int kBufs = kNT * kG <= 64 ? 8 : 512 / (kNT * kG);  // accumulator buffers
  static constexpr uint32_t kTmemCols = kBufs * kG * kNT;
  static constexpr int kHalves = kNT >= 64 ? 2 : 1;        // promotion warpgroups
  static constexpr int kCols = kNT / kHalves;              // token columns of each
  static constexpr int kThreads = 32 * (kGmPromote + 4 * kHalves);
  static constexpr uint32_t kWBytes = kG * kGmRows * kGmBK;
  static constexpr uint32_t kXBytes = kG * kNT * kGmBK;
  static constexpr uint32_t kStage = kWBytes + kXBytes;
  static constexpr uint32_t kSlot = kG * kNT * 4;  // a multiple of 128
  static constexpr uint32_t kBars = 2 * kGmMaxStages + 2 * kBufs + 3 * kGmScRing + 1;
  static constexpr uint32_t kStaging = 4 * kHalves * kGmStaging;
  static constexpr uint32_t kFixed = kGmScRing * kSlot + kStaging + kBars * 8 + 16;
  static_assert(kBufs % kGmIssuers == 0, "an accumulator buffer is always the same issuer's");
  static_assert(kNT % 32 == 0 && kNT <= 256 && kSlot % 128 == 0, "MMA N and copy alignment");
  static_assert((kTmemCols & (kTmemCols - 1)) == 0 && kTmemCols >= 32 && kTmemCols <= 512,
                "TMEM allocations are powers of two");
};

struct GmParams {
  const int32_t* offsets;
  int32_t experts, rows;
  int32_t strips;    // strips of one expert's weight
  int32_t kblocks;   // slices of the reduction
  int32_t stages;
  int32_t height;    // weight rows of a strip: 128, 64 or 32
  int32_t wy_step;   // an expert's step in the weight map: rows
  int32_t wz_step;   // and slices
  const float* sb;   // block scale of (e, strip, slice): sb[e*sb_se + strip*sb_sj + slice*sb_sr]
  int64_t sb_se, sb_sj, sb_sr;
  uint16_t* y;
  int64_t ldy;
  unsigned* err;
  uint64_t wait_limit_ns;
};

struct GmTile {
  int e, strip, row0, lo, hi;
};

template <int kNT>
__device__ __forceinline__ int gm_token_tiles(int lo, int hi) {
  return hi > lo ? (hi - (lo & ~3) + kNT - 1) / kNT : 0;
}

template <int kNT>
__device__ __forceinline__ GmTile gm_tile(int t, const GmParams& p, const int* off,
                                          const int* first) {
  GmTile g;
  g.e = group_find(first, p.experts, t / p.strips);
  const int tt = first[g.e + 1] - first[g.e];
  const int w = t - first[g.e] * p.strips;
  g.strip = w / tt;
  g.lo = off[g.e];
  g.hi = off[g.e + 1];
  g.row0 = (g.lo & ~3) + (w - g.strip * tt) * kNT;
  return g;
}

__device__ __forceinline__ void gm_wait_drain(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  const uint32_t a = smem_u32(bar);
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(a, parity)) {
    if (global_timer_ns() - t0 > limit_ns) return;
  }
}

// 16 lanes x 32 or 64 accumulator columns in the 16x256b shape.
template <int kR>
__device__ __forceinline__ void gm_tmem_load(uint32_t taddr, uint32_t (&r)[kR]) {
  static_assert(kR == 16 || kR == 32, "tcgen05.ld widths");
  if constexpr (kR == 16) tmem_ld_16x256b_x4(taddr, r);
  else tmem_ld_16x256b_x8(taddr, r);
}

template <int kNT>
__global__ void __launch_bounds__(GmShape<kNT>::kThreads, 1) grouped_strip_kernel(
    const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
    const __grid_constant__ CUtensorMap tmSA, const GmParams p) {
  using S = GmShape<kNT>;
  constexpr int kBufs = S::kBufs, kG = S::kG;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int stages = p.stages;
  uint8_t* slots = smem + static_cast<uint32_t>(stages) * S::kStage;
  uint8_t* staging = slots + kGmScRing * S::kSlot;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + S::kStaging);
  uint64_t* empty = full + kGmMaxStages;
  uint64_t* tfull = empty + kGmMaxStages;
  uint64_t* tempty = tfull + kBufs;
  uint64_t* sfull = tempty + kBufs;
  uint64_t* sempty = sfull + kGmScRing;
  uint64_t* pfull = sempty + kGmScRing;  // scale products of a slot
  uint64_t* done = pfull + kGmScRing;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* off = reinterpret_cast<int*>(tmem_slot + 4);
  int* first = off + p.experts + 1;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, kGmIssuers);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(tfull + b, 1);
      mbar_init(tempty + b, (p.height >> 5) * S::kHalves);
    }
    for (int i = 0; i < kGmScRing; ++i) {
      mbar_init(sfull + i, 1);
      mbar_init(pfull + i, 1);
      mbar_init(sempty + i, (p.height >> 5) * S::kHalves);
    }
    mbar_init(done, kGmIssuers);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&tmW);
    prefetch_tensormap(&tmX);
    prefetch_tensormap(&tmSA);
  }
  wait_for_previous_kernel();
  group_table_fill(off, first, p.offsets, p.experts, p.rows, p.err, gm_token_tiles<kNT>);
  if (warp == 1) tmem_alloc<S::kTmemCols>(tmem_slot);  // while warp 0 scans the table
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  let_next_kernel_start();
  const uint32_t tmem_base = *tmem_slot;
  const WaitCtl ctl{abort_flag, p.err, p.wait_limit_ns};
  const int num_tiles = first[p.experts] * p.strips;
  const int KB = p.kblocks;
  const int nst = (KB + kG - 1) / kG;  // accumulator buffers of a tile
  const int quarters = p.height >> 5;  // TMEM lane quarters that hold weight rows

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int s = 0, si = 0;
      uint32_t ph = 0, sph = 0;
      uint32_t issued = 0, par = 0, sc_issued = 0, sc_par = 0;  // as in the large-tile kernel
      bool ok = true;
      for (int t = blockIdx.x; ok && t < num_tiles; t += gridDim.x) {
        const GmTile g = gm_tile<kNT>(t, p, off, first);
        const int wy = g.e * p.wy_step + g.strip * p.height, wz = g.e * p.wz_step;
        for (int kb = 0; kb < KB; kb += kG) {
          if (!mbar_wait(empty + s, ph ^ 1u, ctl)) { ok = false; break; }
          mbar_arrive_expect_tx(full + s, kG * kGmBK * p.height + S::kXBytes);
          tma_load_3d(smem + s * S::kStage, &tmW, 0, wy, wz + kb, full + s);
          tma_load_3d(smem + s * S::kStage + S::kWBytes, &tmX, 0, g.row0, kb, full + s);
          issued |= 1u << s;
          par = (par & ~(1u << s)) | (ph << s);
          if (++s == stages) { s = 0; ph ^= 1u; }
          if (!mbar_wait(sempty + si, sph ^ 1u, ctl)) { ok = false; break; }
          mbar_arrive_expect_tx(sfull + si, S::kSlot);
          tma_load_2d(slots + si * S::kSlot, &tmSA, g.row0, kb, sfull + si);
          sc_issued |= 1u << si;
          sc_par = (sc_par & ~(1u << si)) | (sph << si);
          if (++si == kGmScRing) { si = 0; sph ^= 1u; }
        }
      }
      if (!ok) {  // let the copies still in flight land before the CTA exits
        for (int i = 0; i < stages; ++i)
          if ((issued >> i) & 1u) gm_wait_drain(full + i, (par >> i) & 1u, p.wait_limit_ns);
        for (int i = 0; i < kGmScRing; ++i)
          if ((sc_issued >> i) & 1u) gm_wait_drain(sfull + i, (sc_par >> i) & 1u, p.wait_limit_ns);
      }
    }
    __syncwarp();
  } else if (warp <= kGmIssuers) {
    // ------------------------------------------------------------ MMA issuers
    if (lane == 0) {
      // Issuer i takes the accumulator buffers i, i + 2, ... of this CTA: kG slices of kNT
      // columns each, then one commit for the buffer. Both issuers follow every stage (the
      // other one's they hand back at once): an issuer that met a stage only every second
      // time it is filled could not tell those two phases apart by their parity.
      const uint32_t issuer = static_cast<uint32_t>(warp - 1);
      const uint32_t idesc = idesc_e4m3_f32(kGmRows, kNT);
      int s = 0;
      uint32_t ph = 0, it = 0;  // it: accumulator buffers filled by this CTA so far
      bool ok = true;
      for (int t = blockIdx.x; ok && t < num_tiles; t += gridDim.x) {
        for (int kb = 0; ok && kb < KB; kb += kG, ++it) {
          const bool mine = it % kGmIssuers == issuer;
          const uint32_t buf = it % kBufs, tph = (it / kBufs) & 1u;
          if (mine && !mbar_wait(tempty + buf, tph ^ 1u, ctl)) { ok = false; break; }
          if (!mbar_wait(full + s, ph, ctl)) { ok = false; break; }
          if (mine) {
            tc_fence_after();
            const uint32_t w0 = smem_u32(smem + s * S::kStage);
            const uint32_t x0 = w0 + S::kWBytes;
#pragma unroll
            for (int j = 0; j < kG; ++j)
              if (kb + j < KB)
                mma_f8f6f4_slice(tmem_base + (buf * kG + j) * kNT,
                                 smem_desc_k_sw128(w0 + j * p.height * kGmBK),
                                 smem_desc_k_sw128(x0 + j * kNT * kGmBK), idesc);
            mma_commit(tfull + buf);
            mma_commit(empty + s);
          } else {
            mbar_arrive(empty + s);
          }
          if (++s == stages) { s = 0; ph ^= 1u; }
        }
      }
      mma_commit(done);
      gm_wait_drain(done, 0, p.wait_limit_ns);
    }
    __syncwarp();
  } else if (warp == kGmScaleWarp) {
    // ------------------------------------------------------------ scale products
    // Each slot's row scales times the slice's block scale, in place: one product per token
    // and slice instead of one per token, slice and promoting thread (as many packed
    // multiplications there as the promotion has FMAs).
    uint32_t si = 0, sph = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < num_tiles; t += gridDim.x) {
      const GmTile g = gm_tile<kNT>(t, p, off, first);
      const float* sbp = p.sb + g.e * p.sb_se + ((g.strip * p.height) >> 7) * p.sb_sj;
      // 32 slices at a time: lane l holds slice 32 * (kb / 32) + l; the next ones 16 ahead
      auto sb_fetch = [&](int kk) -> float { return kk < KB ? ld_after_wait(sbp + kk * p.sb_sr) : 0.0f; };
      float sbv = sb_fetch(lane), sbx = 0.0f;
      for (int kb = 0; kb < KB; kb += kG) {
        if ((kb & 31) == 16) sbx = sb_fetch(kb + 16 + lane);
        if ((kb & 31) == 0 && kb > 0) sbv = sbx;
        if (!mbar_wait_warp(sfull + si, sph, ctl)) { ok = false; break; }
        float* sc = reinterpret_cast<float*>(slots + si * S::kSlot);
#pragma unroll
        for (int j = 0; j < kG; ++j) {
          const float sb = __shfl_sync(0xFFFFFFFFu, sbv, (kb + j) & 31);
#pragma unroll
          for (int i = 0; i < kNT; i += 32)
            sc[j * kNT + i + lane] = __fmul_rn(sc[j * kNT + i + lane], sb);
        }
        fence_proxy_async_smem();  // before a later copy into this slot
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull + si);
        if (++si == kGmScRing) { si = 0; sph ^= 1u; }
      }
    }
  } else {
    // ------------------------------------------------------------ promotion + epilogue
    const int q = warp & 3;  // TMEM lane quarter this warp may access
    const int my_tiles = q < quarters ? num_tiles : 0;  // a low strip leaves quarters idle
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    // acc[(2 * b + h) * kCols / 4 + 2 * k + {0, 1}] is weight row 16b + 8h + lane / 4 of the
    // warp's quarter, tokens 8k + 2 * (lane % 4) + {0, 1} of its warpgroup
    constexpr int kCols = S::kCols, kOct = kCols / 8;
    constexpr int kFly = kCols == 32 ? kG : 1;  // slices whose loads are in flight together
    const int col0 = ((warp - kGmPromote) >> 2) * kCols;  // this warpgroup's tokens
    uint8_t* stg = staging + (warp - kGmPromote) * kGmStaging;
    // this lane's address in a transposing store of 8 tokens (64-byte lines, the 16-byte
    // pieces swizzled so that 8 tokens meet all banks), its token and piece in the read back
    const uint32_t st_put = smem_u32(stg) + (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
    const int tok = lane >> 2, piece = lane & 3;
    const uint8_t* st_get = stg + tok * 64 + ((piece ^ ((tok >> 1) & 3)) << 4);
    uint32_t it = 0, si = 0, sph = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < my_tiles; t += gridDim.x) {
      float acc[kCols];
#pragma unroll
      for (int i = 0; i < kCols; ++i) acc[i] = 0.0f;
      for (int k = 0; k < nst; ++k) {
        const int kb = k * kG;
        if (!mbar_wait_warp(pfull + si, sph, ctl)) { ok = false; break; }
        const float2* sa = reinterpret_cast<const float2*>(slots + si * S::kSlot) + col0 / 2 + (lane & 3);
        const uint32_t buf = it % kBufs, tph = (it / kBufs) & 1u;
        if (!mbar_wait_warp(tfull + buf, tph, ctl)) { ok = false; break; }
        tc_fence_after();
        const bool whole = kb + kG <= KB;  // a last stage may hold fewer slices
#pragma unroll
        for (int j0 = 0; j0 < kG; j0 += kFly) {
          uint32_t r[kFly][2][kCols / 2];
#pragma unroll
          for (int j = 0; j < kFly; ++j)
#pragma unroll
            for (int b = 0; b < 2; ++b)
              gm_tmem_load(lane_base + (static_cast<uint32_t>(16 * b) << 16) + (buf * kG + j0 + j) * kNT + col0,
                           r[j][b]);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < kFly; ++j) {
            if (j0 + j == 0 || whole) {
#pragma unroll
              for (int k = 0; k < kOct; ++k) {
                const float2 sc = sa[(j0 + j) * (kNT / 2) + 4 * k];
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    float* a = acc + (2 * b + h) * (kCols / 4) + 2 * k;
                    const uint32_t* p2 = r[j][b] + 4 * k + 2 * h;
                    fma2(a[0], a[1], __uint_as_float(p2[0]), __uint_as_float(p2[1]), sc.x, sc.y);
                  }
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(tempty + buf);
          mbar_arrive(sempty + si);
        }
        ++it;
        if (++si == kGmScRing) { si = 0; sph ^= 1u; }
      }
      if (!ok) break;
      const GmTile o = gm_tile<kNT>(t, p, off, first);
      uint16_t* dst = p.y + static_cast<int64_t>(o.row0 + col0 + tok) * p.ldy + o.strip * p.height +
                      q * 32 + 8 * piece;
      const int lo = o.lo - o.row0 - col0 - tok, hi = o.hi - o.row0 - col0 - tok;
#pragma unroll
      for (int k = 0; k < kOct; k += 2) {
#pragma unroll
        for (int kk = k; kk < k + 2; ++kk) {
          uint32_t v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[i] = pack_bf16x2(acc[i * (kCols / 4) + 2 * kk], acc[i * (kCols / 4) + 2 * kk + 1]);
          stmatrix_trans_x4(st_put + (kk - k) * 512, v[0], v[1], v[2], v[3]);
        }
        __syncwarp();
#pragma unroll
        for (int kk = k; kk < k + 2; ++kk)
          if (8 * kk >= lo && 8 * kk < hi)
            *reinterpret_cast<uint4*>(dst + 8 * kk * p.ldy) =
                *reinterpret_cast<const uint4*>(st_get + (kk - k) * 512);
        __syncwarp();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<S::kTmemCols>(tmem_base);
  }
}

template <int kNT>
fp8q_status launch_strips(const GroupedGemm& g, int64_t token_tiles, int sms,
                          cudaStream_t stream) {
  using S = GmShape<kNT>;
  const int64_t KB = g.Kg / kGmBK;
  const uint32_t fixed = 1024 + S::kFixed + group_table_bytes(static_cast<int>(g.E));
  GmParams p = {};
  p.stages = static_cast<int32_t>(
      std::min<uint32_t>(kGmMaxStages, (kGmMaxSmem - fixed) / S::kStage));
  const size_t smem = fixed + static_cast<size_t>(p.stages) * S::kStage;
  // Strip height: 128 rows fill the MMA; where its tiles would leave half of the SMs without
  // one, lower strips (the rest of the MMA's rows is whatever the stage holds, its lanes are
  // never read) put more SMs on the weights (8 experts of 512 x 2048, 2 rows each, captured
  // calls: 8.5 to 9.3 us with 128 rows, 8.35 with 32). The stages keep their size, so a lower
  // strip has less in flight.
  p.height = kGmRows;
  while (p.height > 32 && token_tiles * (g.Ng / p.height) * 2 <= sms) p.height /= 2;
  CUtensorMap tmW, tmX, tmSA;
  const uint64_t wdims[3] = {kGmBK, static_cast<uint64_t>(g.b_outer),
                             static_cast<uint64_t>(g.b_inner / kGmBK)};
  const uint64_t wstr[2] = {static_cast<uint64_t>(g.b_inner), kGmBK};
  const uint32_t wbox[3] = {kGmBK, static_cast<uint32_t>(p.height), S::kG};
  const uint64_t xdims[3] = {kGmBK, static_cast<uint64_t>(g.rows), static_cast<uint64_t>(KB)};
  const uint64_t xstr[2] = {static_cast<uint64_t>(g.Kg), kGmBK};
  const uint32_t xbox[3] = {kGmBK, kNT, S::kG};
  if (!encode_tmap_3d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.B, wdims, wstr, wbox,
                      CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tmap_3d(&tmX, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.A, xdims, xstr, xbox,
                      CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tmap_2d(&tmSA, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, g.sa, g.rows, KB, g.ldsa * 4, kNT,
                      S::kG, CU_TENSOR_MAP_SWIZZLE_NONE))
    return FP8Q_ERR_UNSUPPORTED;
  p.offsets = g.offsets;
  p.experts = static_cast<int32_t>(g.E);
  p.rows = static_cast<int32_t>(g.rows);
  p.strips = static_cast<int32_t>(g.Ng / p.height);
  p.kblocks = static_cast<int32_t>(KB);
  p.wy_step = static_cast<int32_t>(g.by_step);
  p.wz_step = static_cast<int32_t>(g.bx_step / kGmBK);
  p.sb = g.sb;
  p.sb_se = g.sb_se;
  p.sb_sj = g.sb_sj;
  p.sb_sr = g.sb_sr;
  p.y = static_cast<uint16_t*>(g.y);
  p.ldy = g.ldy;
  p.err = device_error_word();
  p.wait_limit_ns = kWaitLimitNs;
  if (!p.err) return FP8Q_ERR_CUDA;
  // token tiles at most: each expert with rows adds a partial tile and up to 3 rows
  const int64_t tiles = (g.rows + (kNT + 2) * std::min(g.E, g.rows)) / kNT * p.strips;
  if (tiles > 0x7FFFFFFF) return FP8Q_ERR_SHAPE;
  static std::atomic<int> smem_ok[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FP8Q_ERR_CUDA;
  if (!smem_ok[dev].load(std::memory_order_acquire)) {
    const cudaError_t e =
        cudaFuncSetAttribute(grouped_strip_kernel<kNT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kGmMaxSmem));
    if (e != cudaSuccess) {
      set_last_error("cudaFuncSetAttribute(grouped strips)", e);
      cudaGetLastError();
      return FP8Q_ERR_CUDA;
    }
    smem_ok[dev].store(1, std::memory_order_release);
  }
  return launch_overlapped("grouped_strip_kernel launch", grouped_strip_kernel<kNT>,
                           static_cast<int>(std::min<int64_t>(tiles, sms)), S::kThreads, smem, stream,
                           tmW, tmX, tmSA, p);
}

}  // namespace

// The choice goes by the sizes alone (the routing itself is known on the device only: rows
// is what the buffers hold); every kernel takes every routing and gives the same bits.
// Measured on one B200, us a call in a captured graph whose calls take other weights each
// (300 MB or more in all), experts of 0.75 to 1.25 times the average, two runs within 4 %
// but where a range is given. 64 experts at 16384 rows in buffers of which 128 are routed: 340
// with the large tiles that rows selects, 159 with buffers of 128 rows.
//
// 1. Where one tile per SM holds the whole product, its time is the serial walk over the
//    slices: the narrowest tile that fits. One expert of 4096 x 4096, 1 row: 10.5 / 14.4 /
//    19.3 with tiles of 32 / 64 / 128 token rows, 20.8 with large tiles; 512 x 5120, 300
//    rows: 12.5 / 12.7 / 15.5, large 25.4; DGrad, 16 experts of 3584 x 1024, at 16 rows each
//    14.9 / 15.5 / 16.3, large 21.8; at 32, 18.8 / 14.9 / 16.1, large 21.7; at 64, 23.4 /
//    20.0 / 16.2, large 22.4. An expert's rows are taken as one and a half times the average
//    (an expert over the tile's width needs a second tile).
// 2. Otherwise few rows per expert are bound by the weights (strips), many by the tensor
//    cores (large tiles). Forward, 64 experts of 4096 x 4096, at 16 / 32 / 56 / 80 / 128 /
//    160 / 192 rows each: 32-row tiles 165 / 198 / 266 / 340 / 482 / 581 / 675, 64-row 168 /
//    170 / 192-204 / 289 / 375 / 444 / 508, 128-row 225 / 231 / 227 / 259 / 348 / 432 / 444,
//    large 354 / 358 / 361 / 368 / 361 / 365 / 367; 8 experts at 80 / 128 / 160 / 192: 64-row
//    38 / 45 / 49 / 60, 128-row 31 / 41-44 / 56 / 55, large 47 / 50 / 51 / 51. Behind a fill
//    of L2 and a pause of 1 ms, 64 experts at 128 / 160: 128-row 287 / 362, large 310 / 312;
//    8 experts: 48 / 58, large 52 / 53.
fp8q_status launch_grouped_strips(const GroupedGemm& g, bool& taken, cudaStream_t stream) {
  taken = true;
  const int sms = sm100_sm_count();
  if (!sms) return FP8Q_ERR_UNSUPPORTED;
  const int64_t used = std::min(g.E, g.rows);  // experts that can have rows
  const int64_t avg = (g.rows + used - 1) / used;
  const int64_t likely = used == 1 ? avg : avg + avg / 2;
  auto token_tiles = [&](int64_t nt) { return used * ((likely + 3 + nt - 1) / nt); };
  const int64_t strips = g.Ng / kGmRows;
  if (token_tiles(32) * strips <= sms) return launch_strips<32>(g, token_tiles(32), sms, stream);
  if (token_tiles(64) * strips <= sms) return launch_strips<64>(g, token_tiles(64), sms, stream);
  if (token_tiles(128) * strips <= sms) return launch_strips<128>(g, token_tiles(128), sms, stream);
  if (g.rows <= 16 * g.E) return launch_strips<32>(g, token_tiles(32), sms, stream);
  if (g.rows <= 56 * g.E) return launch_strips<64>(g, token_tiles(64), sms, stream);
  if (g.rows <= 128 * g.E) return launch_strips<128>(g, token_tiles(128), sms, stream);
  taken = false;
  return FP8Q_OK;
}

}  // namespace fp8q
