// The experts' FFN on MXFP4 rows and weights for a few rows: at most 32 in all,
// as in a decode step.
//
// Nothing is reused there: the weights of the chosen experts are read once and
// that is the time. One kernel streams them, up projection, then down
// projection, with tensor cores in the stream. Against the tiles of
// gemm_mxfp4.cu:
//  - the operands change places: 128 weight rows (output columns) are the M
//    side, up to 32 tokens the N side, so an MMA costs a tenth and a tile of
//    one token wastes no operand loads (a tile there costs 512 cycles of MMA per
//    stage whatever its rows, 69 GB/s of weights an SM);
//  - every SM gets the same number of stages (128 weight rows x 256 or 512
//    values of K) of each projection: the stages of all tiles in one line, cut
//    into as many equal ranges as there are blocks. A tile cut between ranges is
//    finished by the block that comes to it last, which adds the pieces in the
//    order of K (the same order whoever is last: the same bits);
//  - both projections are one launch. The down projection's first weights are
//    loaded before h is complete, into the ring that the up projection drains.
//    As two launches, h crossed a kernel boundary of 3 to 4 us. (Prefetching the
//    rest of them to L2 as well held up the blocks still at the up projection:
//    126 -> 136 us with all eight experts of a Mixtral-shaped layer.)
//
// Blocks take ranges from a counter, the up projection's first, and wait for h
// only with a range of the down projection in hand. So whatever blocks are
// resident, those of the up projection's ranges that are not done are being
// worked on, and no wait needs a block that has not started (no cooperative
// launch, which cost 5 us between kernels).
//
// CTA = 6 warps: producer, MMA issuer, four epilogue warps (a thread per weight
// row, a warp per block of 32 of h; a block's largest magnitude is one
// reduction across the warp).
// Every wait is bounded; a time-out sets MOE_DEVERR_TIMEOUT and unwinds.
#include "mxfp4_gemm.cuh"
#include <algorithm>
#include <type_traits>

namespace moe {

namespace {

constexpr int kTok = kMxStreamRows;  // token columns of an MMA
constexpr int kThreads = 192;
constexpr int kEpiThreads = 128;

// A stage: BOXES boxes of 128 weight rows x 256 values of K (up projection: of
// its matrices; down projection: of neighbouring blocks of K), the token rows,
// their scales.
template <int UP>
struct SCfg {
  static constexpr int BOXES = UP == EPI_SWIGLU ? 2 : 1;
  static constexpr int TOK_OFF = BOXES * kBoxBytes;
  static constexpr int SF_OFF = TOK_OFF + BOXES * kTok * 128;  // scales: tokens, then weights, a box each
  static constexpr int STAGE_BYTES = SF_OFF + 2 * BOXES * 2 * kScaleTile;  // a multiple of 1024
  static constexpr int STAGES = UP == EPI_SWIGLU ? 5 : 8;
  static constexpr int SF_COL = 128;    // after two accumulators of two x 32 columns
  static constexpr int TMEM_COLS = 256;
  static constexpr size_t SMEM = static_cast<size_t>(STAGES) * STAGE_BYTES + 1024;
};

struct StreamMaps {
  CUtensorMap w[3], sw[3];  // W_gate or W1, W_up, W_down: codes and scales
  CUtensorMap x[2], sx[2];  // rows of the up and of the down projection
};

// One projection: tiles of 128 columns, scale tiles along K, stages of a tile,
// and all stages cut into W ranges of q or (the first `more`) q + 1 stages.
struct Share {
  int ntn, katoms, nkb, W, q, more;
  __device__ __forceinline__ Share(int active, int N, int K, int atoms) {  // atoms: scale tiles along K in a stage
    ntn = N / 128;
    katoms = K / 128;
    nkb = (katoms + atoms - 1) / atoms;
    const int stages = active * ntn * nkb;
    W = min(static_cast<int>(gridDim.x), stages);
    q = W > 0 ? stages / W : 0;
    more = stages - q * W;
  }
  __device__ __forceinline__ int begin(int r) const { return r * q + min(r, more); }
  // The range that has stage s.
  __device__ __forceinline__ int owner(int s) const {
    const int cut = more * (q + 1);
    return s < cut ? s / (q + 1) : more + (s - cut) / q;
  }
};

constexpr int kItemSlots = 2;

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

__device__ __forceinline__ uint32_t load_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ void epi_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(kEpiThreads) : "memory"); }

template <int UP>
__global__ void __launch_bounds__(kThreads, 1)
stream_ffn_mxf4(const __grid_constant__ StreamMaps maps, MxArgs args) {
  using C = SCfg<UP>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[STAGES], empty_bar[STAGES];
  __shared__ __align__(8) uint64_t tfull_bar[2], tfree_bar[2], drain_bar;
  __shared__ __align__(8) uint64_t item_full[kItemSlots], item_empty[kItemSlots];
  __shared__ volatile int item_ring[kItemSlots];  // a range: the up projection's, then the down projection's; -1: the end
  __shared__ Segments segments;
  __shared__ uint32_t tmem_base_s;
  __shared__ int late_s, flag_s[2];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) { mbar_init(&full_bar[s], 1); mbar_init(&empty_bar[s], 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(&tfull_bar[b], 1); mbar_init(&tfree_bar[b], 4); }
    mbar_init(&drain_bar, 1);
    for (int i = 0; i < kItemSlots; ++i) { mbar_init(&item_full[i], 1); mbar_init(&item_empty[i], 5); }
    fence_mbar_init();
    for (int m = 0; m < 3; ++m) { prefetch_tmap(&maps.w[m]); prefetch_tmap(&maps.sw[m]); }
    for (int m = 0; m < 2; ++m) { prefetch_tmap(&maps.x[m]); prefetch_tmap(&maps.sx[m]); }
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
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, tmem_base_s, 0);
  if (!early) pdl_begin();
  // Every role walks the same tiles: active expert u / ntn, columns u % ntn.
  TileList<kTok> list;
  // The first range is taken while the segments load (early: the counters were
  // reset before the previous kernel began, too).
  unsigned taken = 0;
  if (threadIdx.x == 0) taken = atomicAdd(&args.ctl->stream_next, 1u);
  load_segments(segments, args, threadIdx.x, kThreads);
  __syncthreads();
  list.build(args, segments, 1, lane);
  const Share up(list.total, args.F, args.d, 2), down(list.total, args.d, args.F, 2 * C::BOXES);

  // The next range, by a whole warp; -1 at the end or after a time-out.
  auto read_item = [&](int slot) -> int {
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(&item_full[slot & 1], (slot >> 1) & 1))) {
      set_error(args.ctl, MOE_DEVERR_TIMEOUT);
      return -1;
    }
    const int v = item_ring[slot & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_empty[slot & 1]);
    return v;
  };

  // Wait until every range of the up projection is done: h is complete, and
  // tickets and pieces are free for the down projection.
  auto up_done = [&]() -> bool {
    const uint64_t limit = wait_limit_ns(args.ctl), t0 = globaltimer_ns();
    for (;;) {
      if (load_acquire(&args.ctl->stream_up_done) >= static_cast<unsigned>(up.W)) return true;
      if (globaltimer_ns() - t0 > limit) return false;
    }
  };

  if (warp == 0) {
    int u = -1, stage = 0, slot = 0;
    uint32_t phase = 0;
    uint32_t issued_mask = 0, last_parity = 0;
    MxTile t{};
    auto at_stage = [&](const Share& sh, int s) -> int {  // the tile of stage s into t; returns its block of K
      const int su = s / sh.nkb;
      if (su != u) {
        u = su;
        t = list.tile(su / sh.ntn, 0, lane);
        t.n0 = su % sh.ntn * 128;
      }
      return s - su * sh.nkb;
    };
    // p: 0 up projection (a box per matrix), 1 down projection (a box per block
    // of K; the last stage of K may have fewer)
    auto boxes = [&](const Share& sh, auto p, int kb) -> int {
      return decltype(p)::value == 0 ? 1 : min(C::BOXES, (sh.katoms - 2 * C::BOXES * kb + 1) / 2);
    };
    auto load_weights = [&](const Share& sh, auto p, int st, int kb) {
      uint8_t* sw = smem + st * C::STAGE_BYTES;
      uint8_t* ss = sw + C::SF_OFF + C::BOXES * 2 * kScaleTile;
      const int row = t.e * (sh.ntn * 128) + t.n0;
      const int g = (row / 128) * sh.katoms;
      const int tok = boxes(sh, p, kb);
      const int wgt = decltype(p)::value == 0 ? C::BOXES : tok;
      mbar_arrive_expect_tx(&full_bar[st], wgt * (kBoxBytes + 2 * kScaleTile) + tok * (kTok * 128 + 2 * kScaleTile));
#pragma unroll
      for (int j = 0; j < C::BOXES; ++j) {
        if (j >= wgt) break;
        const int m = decltype(p)::value == 0 ? j : 2, k = decltype(p)::value == 0 ? kb : kb * C::BOXES + j;
        tma_load_2d(sw + j * kBoxBytes, &maps.w[m], &full_bar[st], k * 128, row);
        tma_load_2d(ss + j * 2 * kScaleTile, &maps.sw[m], &full_bar[st], 0, g + 2 * k);
      }
    };
    auto load_tokens = [&](const Share& sh, auto p, int st, int kb) {
      uint8_t* sx = smem + st * C::STAGE_BYTES;
      constexpr int P = decltype(p)::value;
      const int tok = boxes(sh, p, kb);
#pragma unroll
      for (int j = 0; j < (P == 0 ? 1 : C::BOXES); ++j) {
        if (j >= tok) break;
        const int k = P == 0 ? kb : kb * C::BOXES + j;
        tma_load_2d(sx + C::TOK_OFF + j * kTok * 128, &maps.x[P], &full_bar[st], k * 128, t.row0);
        tma_load_2d(sx + C::SF_OFF + j * 2 * kScaleTile, &maps.sx[P], &full_bar[st], 0, t.group * sh.katoms + 2 * k);
      }
    };
    auto slot_free = [&]() -> bool {
      if (__all_sync(0xffffffffu, mbar_wait_bounded(&empty_bar[stage], phase ^ 1u))) return true;
      set_error(args.ctl, MOE_DEVERR_TIMEOUT);
      return false;
    };
    auto next_slot = [&] {
      issued_mask |= 1u << stage;
      last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
      if (++stage == STAGES) { stage = 0; phase ^= 1u; }
    };
    // The next range, taken and published to this block's other roles.
    auto next_item = [&]() -> int {
      int v = -1;
      if (lane == 0) {
        const unsigned n = slot == 0 ? taken : atomicAdd(&args.ctl->stream_next, 1u);
        if (n < static_cast<unsigned>(up.W + down.W)) v = static_cast<int>(n);
        if (!mbar_wait_bounded(&item_empty[slot & 1], ((slot >> 1) & 1) ^ 1u)) {
          set_error(args.ctl, MOE_DEVERR_TIMEOUT);
          v = -1;
        }
        item_ring[slot & 1] = v;
        mbar_arrive(&item_full[slot & 1]);
      }
      ++slot;
      return __shfl_sync(0xffffffffu, v, 0);
    };
    // One range: its first weights, as far as the ring has room, `ready` (what
    // the rows wait for), the rows of those stages, then the rest.
    auto stream = [&](const Share& sh, int range, auto p, bool weights_first, auto&& ready) -> bool {
      u = -1;
      const int beg = sh.begin(range), end = sh.begin(range + 1);
      const int ahead = weights_first ? min(STAGES, end - beg) : 0;
      const int stage0 = stage;
      for (int i = 0; i < ahead; ++i) {
        if (!slot_free()) return false;
        const int kb = at_stage(sh, beg + i);
        if (elect_one()) load_weights(sh, p, stage, kb);
        __syncwarp();
        next_slot();
      }
      const bool go = ready();
      // rows of the stages that have their weights (also after a time-out: a
      // stage armed has to complete)
      u = -1;
      for (int i = 0; i < ahead; ++i) {
        const int st = stage0 + i < STAGES ? stage0 + i : stage0 + i - STAGES;
        const int kb = at_stage(sh, beg + i);
        if (elect_one()) load_tokens(sh, p, st, kb);
        __syncwarp();
      }
      if (!go) return false;
      for (int s = beg + ahead; s < end; ++s) {
        if (!slot_free()) return false;
        const int kb = at_stage(sh, s);
        if (elect_one()) {
          load_weights(sh, p, stage, kb);
          load_tokens(sh, p, stage, kb);
        }
        __syncwarp();
        next_slot();
      }
      return true;
    };
    bool waited = !early, ok = true;
    int item = -1;
    while (ok && (item = next_item()) >= 0) {
      if (item < up.W) {
        ok = stream(up, item, std::integral_constant<int, 0>{}, !waited, [&] {
          if (!waited) pdl_begin();
          waited = true;
          return true;
        });
      } else {
        ok = stream(down, item - up.W, std::integral_constant<int, 1>{}, true, [&]() -> bool {
          if (!waited) pdl_begin();
          waited = true;
          const bool there = up_done();
          // h was written by ordinary stores and is read by TMA
          asm volatile("fence.proxy.async;" ::: "memory");
          if (__all_sync(0xffffffffu, there)) return true;
          set_error(args.ctl, MOE_DEVERR_TIMEOUT);
          return false;
        });
      }
    }
    if (!waited) pdl_begin();
    if (item >= 0) {  // gave up: the other roles' end
      if (lane == 0 && mbar_wait_bounded(&item_empty[slot & 1], ((slot >> 1) & 1) ^ 1u)) {
        item_ring[slot & 1] = -1;
        mbar_arrive(&item_full[slot & 1]);
      }
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
    const uint64_t xdesc0 = make_sw128_desc(base + C::TOK_OFF, 16, 1024);
    const uint64_t sdesc0 = make_scale_desc(base + C::SF_OFF);
    int stage = 0, i = 0;  // i: tiles begun here
    uint32_t phase = 0;
    uint32_t set = 0;
    bool dead = false, issued_any = false;  // in the issuing thread
    auto multiply = [&](const Share& sh, int range, auto p) {
      constexpr int P = decltype(p)::value;
      constexpr int MATS = P == 0 ? C::BOXES : 1;  // accumulators
      constexpr int KBOX = P == 0 ? 1 : C::BOXES;  // boxes along K
      const int beg = sh.begin(range), end = sh.begin(range + 1);
      int kb = beg % sh.nkb;
      bool fresh = true;
      for (int s = beg; s < end; ++s) {
        const uint32_t d_tmem = tmem_base + (i & 1) * (2 * kTok);
        const uint32_t so = stage * (C::STAGE_BYTES >> 4);
        const int atoms = min(2 * KBOX, sh.katoms - 2 * KBOX * kb);
        const bool done = kb == sh.nkb - 1 || s == end - 1;  // the last stage of this tile here
        if (elect_one()) {
          if (!dead) dead = !mbar_wait_bounded(&full_bar[stage], phase);
          // two accumulators: the epilogue has read this one
          if (fresh && i >= 2 && !dead) dead = !mbar_wait_bounded(&tfree_bar[i & 1], ((i >> 1) - 1) & 1);
          if (!dead) {
            tc_fence_after();
#pragma unroll
            for (int at = 0; at < 2 * KBOX; ++at) {
              if (at < atoms) {
                const int box = at >> 1;
                const uint32_t sf = tmem_base + C::SF_COL + (set ^ (at & 1)) * 16;
                copy_scales<1>(sf, sdesc0 + so + at * (kScaleTile >> 4));  // tokens
#pragma unroll
                for (int m = 0; m < MATS; ++m)
                  copy_scales<1>(sf + 4 + 4 * m, sdesc0 + so + (2 * (C::BOXES + m) + at) * (kScaleTile >> 4));
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                  const uint32_t off = so + ((at & 1) * 2 + kk) * 2;
#pragma unroll
                  for (int m = 0; m < MATS; ++m)
                    umma_mxf4<1>(d_tmem + m * kTok, wdesc0 + off + (m + box) * (kBoxBytes >> 4),
                                 xdesc0 + off + box * ((kTok * 128) >> 4), kk == 0 ? kIdesc0 : kIdesc2, sf + 4 + 4 * m,
                                 sf, !fresh || at != 0 || kk != 0 ? 1u : 0u);
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
        fresh = done;
        if (done) ++i;
        if (++kb == sh.nkb) kb = 0;
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
    };
    for (int slot = 0, item; (item = read_item(slot)) >= 0; ++slot) {
      if (item < up.W) multiply(up, item, std::integral_constant<int, 0>{});
      else multiply(down, item - up.W, std::integral_constant<int, 1>{});
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
    auto finish_tiles = [&](const Share& sh, int range, auto epi) -> bool {
      constexpr int EPI = decltype(epi)::value;
      constexpr int MATS = EPI == EPI_SWIGLU ? 2 : 1;
      const int beg = sh.begin(range), end = sh.begin(range + 1);
      for (int s = beg; s < end; ++i) {
        const int u = s / sh.nkb;
        const int s_end = min(end, (u + 1) * sh.nkb);
        MxTile t = list.tile(u / sh.ntn, 0, lane);
        t.n0 = u % sh.ntn * 128;
        // A tile cut between ranges c0..c1: whoever comes last adds the pieces,
        // in the order of K, the others leave theirs in the workspace. Usually
        // that is the range where the tile begins, at the end of its stages: the
        // next one had its piece first. So look before the wait for the MMAs
        // whether the other pieces are there; then this one need not go through
        // memory.
        const int s0 = u * sh.nkb;
        const int c0 = s0 >= beg ? range : sh.owner(s0);
        const int c1 = s0 + sh.nkb <= end ? range : sh.owner(s0 + sh.nkb - 1);
        const uint32_t others = static_cast<uint32_t>(c1 - c0);
        auto piece = [&](int c) -> float* {  // range c's: 0 for a tile begun before its stages, else 1
          return args.partials + (static_cast<size_t>(c) * 2 + (sh.begin(c) > s0 ? 0 : 1)) * (2 * kTok * 128) + col;
        };
        // tickets: a byte per range in which a cut tile begins
        uint32_t* word = &args.ctl->stream_ticket[c0 >> 2];
        const int shift = 8 * (c0 & 3);
        // one thread decides for the four warps, which share barriers and so
        // have to leave together
        if (lead) {
          bool last = true, ok = true;
          if (others > 0) {
            // the up projection's tiles count in the same bytes
            if (EPI == EPI_STORE) ok = up_done();
            // acquire: the pieces counted are visible
            last = ok && ((load_acquire(word) >> shift) & 255u) == others;
            if (last) (void)atomicSub(word, others << shift);
          }
          if (ok) ok = mbar_wait_bounded(&tfull_bar[i & 1], (i >> 1) & 1);
          flag_s[i & 1] = (ok ? 1 : 0) | (last ? 2 : 0);
        }
        epi_barrier();
        const int flag = flag_s[i & 1];
        if ((flag & 1) == 0) {
          set_error(args.ctl, MOE_DEVERR_TIMEOUT);
          return false;
        }
        (void)mbar_try_wait(&tfull_bar[i & 1], (i >> 1) & 1);  // complete: each thread observes it
        tc_fence_after();
        const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + (i & 1) * (2 * kTok);
        bool finish = (flag & 2) != 0;
        if (!finish) {
          float* mine = piece(range);
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
            const uint32_t before = (atomicAdd(word, 1u << shift) >> shift) & 255u;
            if (before == others) {
              (void)atomicSub(word, (others + 1u) << shift);
              __threadfence();
            }
            late_s = before == others;
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
                    v[m][k] += b == range ? own[m][k] : c + k < t.rows ? __ldcg(p + (m * kTok + c + k) * 128) : 0.f;
              }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              if (c + k >= t.rows) break;
              const size_t row = static_cast<size_t>(t.row0) + c + k;
              if constexpr (EPI == EPI_STORE) {
                args.out[row * args.d + t.n0 + col] = __float2bfloat16_rn(v[0][k]);
              } else {
                const float h = EPI == EPI_SWIGLU ? silu_fast(v[0][k]) * v[MATS - 1][k] : gelu2<PhiTail>(v[0][k], 0.0f).x;
                const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7fffffffu);
                const uint32_t sb = mx_scale_byte(top);
                // eight lanes' codes to one word
                uint32_t w = sb == 255u ? 0u : e2m1(h * mx_inv_scale(sb)) << (4 * (lane & 7));
                w |= __shfl_xor_sync(0xffffffffu, w, 1);
                w |= __shfl_xor_sync(0xffffffffu, w, 2);
                w |= __shfl_xor_sync(0xffffffffu, w, 4);
                if ((lane & 7) == 0)
                  *reinterpret_cast<uint32_t*>(args.out_codes + row * (args.F / 2) + (t.n0 + col) / 2) = w;
                if (lane == 0)
                  args.out_scales[mx_scale_at(t.group, args.F / 128, c + k, t.n0 / 32 + q)] = static_cast<uint8_t>(sb);
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tfree_bar[i & 1]);
        s = s_end;
      }
      return true;
    };
    for (int slot = 0, item; (item = read_item(slot)) >= 0; ++slot) {
      if (item < up.W) {
        if (!finish_tiles(up, item, std::integral_constant<int, UP>{})) break;
        // this range's part of h is written
        __threadfence();
        epi_barrier();
        if (lead) atomicAdd(&args.ctl->stream_up_done, 1u);
      } else if (!finish_tiles(down, item - up.W, std::integral_constant<int, EPI_STORE>{})) {
        break;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // The last block to finish resets the counters for the next launch.
  if (threadIdx.x == 0 && atomicAdd(&args.ctl->stream_done, 1u) == gridDim.x - 1u) {
    atomicExch(&args.ctl->stream_next, 0u);
    atomicExch(&args.ctl->stream_up_done, 0u);
    atomicExch(&args.ctl->stream_done, 0u);
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

template <int UP>
cudaError_t run_stream(const MxRows& x, const MxWeights& w1, const MxWeights& w3, const MxWeights& w2,
                       const MxRows& h, const MxArgs& args, cudaStream_t s) {
  using C = SCfg<UP>;
  StreamMaps m;
  const uint64_t E = args.E, d = args.d, F = args.F, rows = static_cast<uint64_t>(args.rows_max);
  const uint64_t groups = rows / 128 + E;
  if (!make_tma_codes(&m.w[0], w1.codes, E * F, d / 2, 128) || !make_tma_codes(&m.w[1], w3.codes, E * F, d / 2, 128) ||
      !make_tma_codes(&m.w[2], w2.codes, E * d, F / 2, 128) || !make_tma_codes(&m.x[0], x.codes, rows, d / 2, kTok) ||
      !make_tma_codes(&m.x[1], h.codes, rows, F / 2, kTok) ||
      !make_tma_scales(&m.sw[0], w1.scales, E * (F / 128) * (d / 128)) ||
      !make_tma_scales(&m.sw[1], w3.scales, E * (F / 128) * (d / 128)) ||
      !make_tma_scales(&m.sw[2], w2.scales, E * (F / 128) * (d / 128)) ||
      !make_tma_scales(&m.sx[0], x.scales, groups * (d / 128)) ||
      !make_tma_scales(&m.sx[1], h.scales, groups * (F / 128)))
    return cudaErrorInvalidValue;
  auto kern = stream_ffn_mxf4<UP>;
  cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::SMEM));
  return launch_pdl(kern, dim3(std::min(num_sms(), kMxStreamBlocks)), dim3(kThreads), C::SMEM, s, false, m, args);
}

}  // namespace

cudaError_t launch_stream_ffn_mxfp4(const MxRows& x, const MxWeights& w1, const MxWeights& w3, const MxWeights& w2,
                                    moe_act_t act, const MxRows& h, const MxArgs& args, cudaStream_t s) {
  if (act == MOE_ACT_SWIGLU) return run_stream<EPI_SWIGLU>(x, w1, w3, w2, h, args, s);
  return run_stream<EPI_GELU>(x, w1, w1, w2, h, args, s);
}

}  // namespace moe
