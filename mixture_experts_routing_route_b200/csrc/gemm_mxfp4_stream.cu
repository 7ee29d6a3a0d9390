// Grouped MXFP4 GEMM for a few rows: at most 32 in all, as in a decode step.
//
// Nothing is reused there, the weights of the chosen experts are read once and
// that is the time; the kernel is a weight stream with tensor cores in it.
// Against the CTA-pair kernel (gemm_mxfp4.cu):
//  - the operands change places: 128 weight rows (output columns) are the M
//    side, up to 32 tokens the N side, so an MMA costs a tenth and a tile of
//    one token wastes no operand loads (a pair's tile costs 512 cycles of MMA
//    per stage whatever its rows, 69 GB/s of weights an SM);
//  - every SM gets the same number of stages (128 weight rows x 256 values of
//    K): the stages of all tiles in one line, cut into equal pieces. A tile cut
//    between SMs is finished by the SM that arrives last, which adds the pieces
//    in the order of K (the same order whoever is last: the same bits);
//  - a block takes less than half of the shared and tensor memory, so that the
//    down projection's blocks move in next to the up projection's: they set up
//    and load their first weights while those still run.
//
// CTA = 6 warps: producer, MMA issuer, four epilogue warps (a thread per weight
// row, a warp per block of 32 of h; a block's largest magnitude is one
// reduction across the warp).
// Every wait is bounded; a time-out sets MOE_DEVERR_TIMEOUT and unwinds.
#include "mxfp4_gemm.cuh"
#include <algorithm>

namespace moe {

namespace {

constexpr int kTok = kMxStreamRows;  // token columns of an MMA
constexpr int kThreads = 192;
constexpr int kEpiThreads = 128;

template <int EPI>
struct SCfg {
  static constexpr int MATS = EPI == EPI_SWIGLU ? 2 : 1;
  static constexpr int OPERANDS = MATS * kBoxBytes + kTok * 128;
  static constexpr int STAGE_BYTES = OPERANDS + (MATS + 1) * 2 * kScaleTile;  // a multiple of 1024
  static constexpr int STAGES = EPI == EPI_SWIGLU ? 3 : EPI == EPI_GELU ? 5 : 4;
  static constexpr int SF_COL = 128;    // after two accumulators of MATS x 32 columns
  static constexpr int TMEM_COLS = 256;
  static constexpr size_t SMEM = static_cast<size_t>(STAGES) * STAGE_BYTES + 1024;
};

// The first stage of block c of W <= stages.
__device__ __forceinline__ int stage_begin(int c, long long stages, int W) {
  return static_cast<int>(c * stages / W);
}
// The block that has stage s.
__device__ __forceinline__ int stage_owner(long long s, long long stages, int W) {
  return static_cast<int>(((s + 1) * W - 1) / stages);
}

// Eight token columns from c on of each matrix's accumulator.
template <int MATS>
__device__ __forceinline__ void load_columns(uint32_t tbase, int c, float (&v)[MATS][8]) {
  uint32_t r[MATS][8];
#pragma unroll
  for (int m = 0; m < MATS; ++m)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[m][0]), "=r"(r[m][1]), "=r"(r[m][2]), "=r"(r[m][3]), "=r"(r[m][4]), "=r"(r[m][5]),
                   "=r"(r[m][6]), "=r"(r[m][7])
                 : "r"(tbase + m * kTok + c));
  tmem_ld_wait();
#pragma unroll
  for (int m = 0; m < MATS; ++m)
#pragma unroll
    for (int k = 0; k < 8; ++k) v[m][k] = __uint_as_float(r[m][k]);
}

__device__ __forceinline__ void epi_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(kEpiThreads) : "memory"); }

template <int EPI>
__global__ void __launch_bounds__(kThreads, 2)
stream_mxf4(const __grid_constant__ CUtensorMap tmW0, const __grid_constant__ CUtensorMap tmW1,
            const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmSW0,
            const __grid_constant__ CUtensorMap tmSW1, const __grid_constant__ CUtensorMap tmSX, MxArgs args,
            float* partials) {
  using C = SCfg<EPI>;
  constexpr int MATS = C::MATS, STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[STAGES], empty_bar[STAGES];
  __shared__ __align__(8) uint64_t tfull_bar[2], tfree_bar[2], drain_bar;
  __shared__ uint32_t tmem_base_s;
  __shared__ int late_s, flag_s[2];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) { mbar_init(&full_bar[s], 1); mbar_init(&empty_bar[s], 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(&tfull_bar[b], 1); mbar_init(&tfree_bar[b], 4); }
    mbar_init(&drain_bar, 1);
    fence_mbar_init();
    prefetch_tmap(&tmW0);
    prefetch_tmap(&tmW1);
    prefetch_tmap(&tmX);
    prefetch_tmap(&tmSW0);
    prefetch_tmap(&tmSW1);
    prefetch_tmap(&tmSX);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_s, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // see MxArgs::early
  const bool early = args.early != 0;
  if (!early) pdl_begin();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, tmem_base_s, 0);
  const int me = blockIdx.x;
  const int katoms = args.K / 128;  // scale tiles along K
  const int nkb = (katoms + 1) / 2;

  // Every role walks the same tiles.
  TileList<kTok> list;
  list.build(args, args.N / 128, lane);
  const long long stages = static_cast<long long>(list.total) * nkb;
  // blocks that take part: each has a stage at least
  const int W = static_cast<int>(min(static_cast<long long>(gridDim.x), stages));
  const int beg = me < W ? stage_begin(me, stages, W) : 0, end = me < W ? stage_begin(me + 1, stages, W) : 0;

  if (warp == 0) {
    int u = -1;
    MxTile t{};
    auto at_stage = [&](int s) -> int {  // the tile of stage s into t; returns its block of K
      const int su = s / nkb;
      if (su != u) {
        u = su;
        t = list.tile(u, 128, lane);
      }
      return s - su * nkb;
    };
    auto load_weights = [&](int stage, int kb) {
      uint8_t* sw = smem + stage * C::STAGE_BYTES;
      uint8_t* ss = sw + C::OPERANDS;
      const int row = t.e * args.N + t.n0;
      const int g = (row / 128) * katoms + 2 * kb;
      mbar_arrive_expect_tx(&full_bar[stage], C::STAGE_BYTES);
      tma_load_2d(sw, &tmW0, &full_bar[stage], kb * 128, row);
      tma_load_2d(ss, &tmSW0, &full_bar[stage], 0, g);
      if (MATS == 2) {
        tma_load_2d(sw + kBoxBytes, &tmW1, &full_bar[stage], kb * 128, row);
        tma_load_2d(ss + 2 * kScaleTile, &tmSW1, &full_bar[stage], 0, g);
      }
    };
    // early: the first weights go out before the wait for the previous kernel
    const int ahead = early ? min(STAGES, end - beg) : 0;
    for (int i = 0; i < ahead; ++i) {
      const int kb = at_stage(beg + i);
      if (elect_one()) load_weights(i, kb);
      __syncwarp();
    }
    if (early) pdl_begin();
    int stage = 0;
    uint32_t phase = 0;
    uint32_t issued_mask = (1u << ahead) - 1u, last_parity = 0;
    for (int s = beg; s < end; ++s) {
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&empty_bar[stage], phase ^ 1u))) {
        set_error(args.ctl, MOE_DEVERR_TIMEOUT);
        break;
      }
      const int kb = at_stage(s);
      if (elect_one()) {
        if (s - beg >= ahead) load_weights(stage, kb);
        uint8_t* sx = smem + stage * C::STAGE_BYTES + MATS * kBoxBytes;
        tma_load_2d(sx, &tmX, &full_bar[stage], kb * 128, t.row0);
        tma_load_2d(sx + kTok * 128 + MATS * 2 * kScaleTile, &tmSX, &full_bar[stage], 0, t.group * katoms + 2 * kb);
      }
      __syncwarp();
      issued_mask |= 1u << stage;
      last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
      if (++stage == STAGES) { stage = 0; phase ^= 1u; }
    }
    // Every load issued must have landed before the CTA may exit.
    for (int s = 0; s < STAGES; ++s)
      if (issued_mask & (1u << s))
        if (!mbar_wait_bounded(&full_bar[s], (last_parity >> s) & 1u)) set_error(args.ctl, MOE_DEVERR_TIMEOUT);
  } else if (warp == 1) {
    if (early) pdl_begin();
    constexpr uint32_t kIdesc0 = make_idesc_mxf4(128, kTok, 0);
    constexpr uint32_t kIdesc2 = make_idesc_mxf4(128, kTok, 2);
    const uint32_t base = smem_u32(smem);
    const uint64_t wdesc0 = make_sw128_desc(base, 16, 1024);
    const uint64_t xdesc0 = make_sw128_desc(base + MATS * kBoxBytes, 16, 1024);
    const uint64_t sdesc0 = make_scale_desc(base + C::OPERANDS);
    int stage = 0;
    uint32_t phase = 0;
    uint32_t set = 0;
    bool dead = false, issued_any = false;  // in the issuing thread
    int u = beg / nkb, kb = beg - u * nkb, i = 0;  // i: tiles begun here
    bool fresh = true;
    for (int s = beg; s < end; ++s) {
      const uint32_t d_tmem = tmem_base + (i & 1) * (MATS * kTok);
      const uint32_t so = stage * (C::STAGE_BYTES >> 4);
      const int atoms = min(2, katoms - 2 * kb);
      const bool done = kb == nkb - 1 || s == end - 1;  // the last stage of this tile here
      if (elect_one()) {
        if (!dead) dead = !mbar_wait_bounded(&full_bar[stage], phase);
        // two accumulators: the epilogue has read this one
        if (fresh && i >= 2 && !dead) dead = !mbar_wait_bounded(&tfree_bar[i & 1], ((i >> 1) - 1) & 1);
        if (!dead) {
          tc_fence_after();
#pragma unroll
          for (int at = 0; at < 2; ++at) {
            if (at < atoms) {
              const uint32_t sf = tmem_base + C::SF_COL + (set ^ at) * 16;
#pragma unroll
              for (int j = 0; j <= MATS; ++j)  // weights, then tokens
                copy_scales<1>(sf + 4 * j, sdesc0 + so + (j * 2 + at) * (kScaleTile >> 4));
#pragma unroll
              for (int kk = 0; kk < 2; ++kk) {
                const uint32_t off = so + (at * 2 + kk) * 2;
#pragma unroll
                for (int m = 0; m < MATS; ++m)
                  umma_mxf4<1>(d_tmem + m * kTok, wdesc0 + off + m * (kBoxBytes >> 4), xdesc0 + off,
                               kk == 0 ? kIdesc0 : kIdesc2, sf + 4 * m, sf + 4 * MATS,
                               !fresh || at != 0 || kk != 0 ? 1u : 0u);
              }
            }
          }
          umma_commit(&empty_bar[stage]);
          if (done) umma_commit(&tfull_bar[i & 1]);
          issued_any = true;
        }
      }
      __syncwarp();
      set ^= atoms & 1;
      fresh = false;
      if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      if (++kb == nkb) {
        kb = 0;
        ++u;
        ++i;
        fresh = true;
      }
    }
    if (__any_sync(0xffffffffu, dead)) set_error(args.ctl, MOE_DEVERR_TIMEOUT);
    if (__any_sync(0xffffffffu, issued_any)) {
      // Tensor memory is freed below: wait until every MMA issued is done.
      if (elect_one()) umma_commit(&drain_bar);
      __syncwarp();
      (void)mbar_wait_bounded(&drain_bar, 0);
    }
  } else {
    if (early) pdl_begin();
    const int q = warp & 3;  // tensor-memory lane quarter
    const int col = q * 32 + lane;  // output column in the tile
    const bool lead = threadIdx.x == kThreads - kEpiThreads;
    int i = 0;
    for (int s = beg; s < end; ++i) {
      const int u = s / nkb;
      const int s_end = min(end, (u + 1) * nkb);
      const MxTile t = list.tile(u, 128, lane);
      // A tile cut between blocks c0..c1: whoever comes last adds the pieces, in
      // the order of K, the others leave theirs in the workspace. Usually that
      // is the block where the tile begins, at the end of its stages: the next
      // one had its piece first. So look before the wait for the MMAs whether
      // the other pieces are there; then this one need not go through memory.
      const long long s0 = static_cast<long long>(u) * nkb;
      const int c0 = stage_owner(s0, stages, W), c1 = stage_owner(s0 + nkb - 1, stages, W);
      const uint32_t others = static_cast<uint32_t>(c1 - c0);
      auto piece = [&](int c) -> float* {  // block c's: 0 for a tile begun before its stages, else 1
        return partials + (static_cast<size_t>(c) * 2 + (stage_begin(c, stages, W) > s0 ? 0 : 1)) * (MATS * kTok * 128) + col;
      };
      // tickets: a byte per block in which a cut tile begins
      uint32_t* word = &args.ctl->stream_ticket[c0 >> 2];
      const int sh = 8 * (c0 & 3);
      // one thread decides for the four warps, which share barriers and so have
      // to leave together
      if (lead) {
        bool last = true;
        if (others > 0) {
          last = ((*reinterpret_cast<volatile uint32_t*>(word) >> sh) & 255u) == others;
          if (last) atomicSub(word, others << sh);
          __threadfence();
        }
        const bool ok = mbar_wait_bounded(&tfull_bar[i & 1], (i >> 1) & 1);
        flag_s[i & 1] = (ok ? 1 : 0) | (last ? 2 : 0);
      }
      epi_barrier();
      const int flag = flag_s[i & 1];
      if ((flag & 1) == 0) {
        set_error(args.ctl, MOE_DEVERR_TIMEOUT);
        break;
      }
      (void)mbar_try_wait(&tfull_bar[i & 1], (i >> 1) & 1);  // complete: each thread observes it
      tc_fence_after();
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + (i & 1) * (MATS * kTok);
      bool finish = (flag & 2) != 0;
      if (!finish) {
        float* mine = piece(me);
#pragma unroll 1
        for (int c = 0; c < t.rows; c += 8) {
          float v[MATS][8];
          load_columns(tb, c, v);
#pragma unroll
          for (int m = 0; m < MATS; ++m)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (c + k < t.rows) __stcg(mine + (m * kTok + c + k) * 128, v[m][k]);
        }
        __threadfence();
        epi_barrier();
        if (lead) {
          const uint32_t before = (atomicAdd(word, 1u << sh) >> sh) & 255u;
          if (before == others) atomicSub(word, (others + 1u) << sh);
          late_s = before == others;
          __threadfence();
        }
        epi_barrier();
        finish = late_s != 0;
      }
      if (finish) {
#pragma unroll 1
        for (int c = 0; c < t.rows; c += 8) {
          float v[MATS][8];
          load_columns(tb, c, v);
          if (others > 0) {
            float own[MATS][8];
#pragma unroll
            for (int m = 0; m < MATS; ++m)
#pragma unroll
              for (int k = 0; k < 8; ++k) { own[m][k] = v[m][k]; v[m][k] = 0.f; }
#pragma unroll 1
            for (int b = c0; b <= c1; ++b) {
              const float* p = piece(b);
#pragma unroll
              for (int m = 0; m < MATS; ++m)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  v[m][k] += b == me ? own[m][k] : c + k < t.rows ? __ldcg(p + (m * kTok + c + k) * 128) : 0.f;
            }
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (c + k >= t.rows) break;
            const size_t row = static_cast<size_t>(t.row0) + c + k;
            if constexpr (EPI == EPI_STORE) {
              args.out[row * args.N + t.n0 + col] = __float2bfloat16_rn(v[0][k]);
            } else {
              const float h = EPI == EPI_SWIGLU ? silu_fast(v[0][k]) * v[MATS - 1][k] : gelu_fast(v[0][k]);
              const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7fffffffu);
              const uint32_t sb = mx_scale_byte(top);
              // eight lanes' codes to one word
              uint32_t w = sb == 255u ? 0u : e2m1(h * mx_inv_scale(sb)) << (4 * (lane & 7));
              w |= __shfl_xor_sync(0xffffffffu, w, 1);
              w |= __shfl_xor_sync(0xffffffffu, w, 2);
              w |= __shfl_xor_sync(0xffffffffu, w, 4);
              if ((lane & 7) == 0)
                *reinterpret_cast<uint32_t*>(args.out_codes + row * (args.N / 2) + (t.n0 + col) / 2) = w;
              if (lane == 0)
                args.out_scales[mx_scale_at(t.group, args.N / 128, c + k, t.n0 / 32 + q)] = static_cast<uint8_t>(sb);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tfree_bar[i & 1]);
      s = s_end;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

template <int EPI>
cudaError_t run_stream(const MxRows& x, const MxWeights& w0, const MxWeights& w1, const MxArgs& args,
                       float* partials, cudaStream_t s) {
  using C = SCfg<EPI>;
  CUtensorMap tw0, tw1, tx, sw0, sw1, sx;
  const uint64_t wrows = static_cast<uint64_t>(args.E) * args.N, katoms = args.K / 128;
  const uint64_t xtiles = (static_cast<uint64_t>(args.rows_max) / 128 + args.E) * katoms;
  if (!make_tma_codes(&tw0, w0.codes, wrows, args.K / 2, 128) ||
      !make_tma_codes(&tw1, w1.codes, wrows, args.K / 2, 128) ||
      !make_tma_codes(&tx, x.codes, static_cast<uint64_t>(args.rows_max), args.K / 2, kTok) ||
      !make_tma_scales(&sw0, w0.scales, wrows / 128 * katoms) ||
      !make_tma_scales(&sw1, w1.scales, wrows / 128 * katoms) || !make_tma_scales(&sx, x.scales, xtiles))
    return cudaErrorInvalidValue;
  auto kern = stream_mxf4<EPI>;
  cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::SMEM));
  return launch_pdl(kern, dim3(stream_blocks()), dim3(kThreads), C::SMEM, s, false, tw0, tw1, tx, sw0, sw1, sx, args,
                    partials);
}

}  // namespace

int stream_blocks() { return std::min(num_sms(), kMxStreamBlocks); }

cudaError_t launch_stream_mxfp4_up(const MxRows& x, const MxWeights& w1, const MxWeights& w3, moe_act_t act,
                                   const MxArgs& args, float* partials, cudaStream_t s) {
  if (act == MOE_ACT_SWIGLU) return run_stream<EPI_SWIGLU>(x, w1, w3, args, partials, s);
  return run_stream<EPI_GELU>(x, w1, w1, args, partials, s);
}

cudaError_t launch_stream_mxfp4_down(const MxRows& h, const MxWeights& w2, const MxArgs& args, float* partials,
                                     cudaStream_t s) {
  return run_stream<EPI_STORE>(h, w2, w2, args, partials, s);
}

}  // namespace moe
