// Grouped expert GEMM on MXFP4 operands (tcgen05 kind::mxf4, block scales in
// tensor memory), for the experts' FFN with 4-bit weights and rows.
//
//   C[rows of e, n-tile] = epilogue( A[rows of e, :] . B[e][n-tile, :]^T )
//   A: codes [rows_max, K/2], B: codes [E, N, K/2], both K-major; scales as
//      mxfp4.cuh lays them out (the order tcgen05.cp takes them in)
//   epilogue: SwiGLU (W_gate and W_up side by side in one N = 256 MMA) or GELU,
//      then the row's 32-column blocks quantised to MXFP4 again (codes and
//      scales of h); or the plain bf16 store of the down projection. Sums and
//      activations are fp32; h is rounded once (to E2M1), y once (to bf16).
//
// Two forms of one kernel, both persistent. GROUP 2, for experts with many rows
// and long K: the two CTAs of a cluster compute one 256-row x N tile together
// (cta_group::2); CTA r holds A rows [row0 + 128 r, +128) and its half of the B
// columns (SwiGLU: CTA 0 W_gate's, CTA 1 W_up's of the same output columns), its
// rows' scales and the scales of all B columns. GROUP 1: a CTA computes a
// 128-row x N tile and holds all B columns. A CTA's warps:
//   warp 0   producer: per stage (256 values of K) the A and B boxes by TMA (128
//            bytes = 256 codes a row, 128-byte swizzle) and the scale tiles (two
//            of 512 bytes per 128 rows)
//   warp 1   MMA issuer (of a pair: the even CTA's): per 128 values of K one
//            thread copies the scale tiles to tensor memory (of both CTAs;
//            tcgen05.cp, replicated to the four lane quarters) and issues two
//            MMAs of K = 64
//   8 or 16  epilogue: a thread per row and a half or a quarter of the columns,
//            32 columns (one block) at a time
//   the last scheduler: hands out tiles
// Why pairs: a stage of a 128 x 256 tile is 51 KB that come from L2 and go
// through one CTA's shared memory twice (written, read by the MMAs), some 790
// clocks at 128 bytes a clock for 512 clocks of MMA (measured: 800). A pair's CTA
// has 35 KB a stage for the same MMA time: 525 to 540 clocks (K = 4096 and 14336).
//
// Tensor memory: two accumulators of 256 columns and the scales do not fit in
// 512 columns, so the accumulators overlap by 32 columns (columns 0-255 and
// 224-479) and the scales use 480-511 (two sets of 12, taken in turn). The
// epilogue reads the overlapping columns first and frees them at once; the
// next tile's MMAs start then, while the rest of the tile is still read.
//
// Work is handed out dynamically, as in the bf16 CTA-pair kernel, so that CTAs
// sharing a weight block read it at nearly the same time: the even CTA's
// scheduler (GROUP 1: each CTA's) takes the next tile from a counter in the
// control block, decodes it, publishes it to its CTA's roles and hands it to the
// odd CTA's scheduler, if there is one, which does the same there. The
// three-slot ring keeps this chain (some 3000 cycles a tile of a pair: the
// counter, a search with a division, waits and releases at cluster scope) off
// every other role's path, and takes no tile so early that a slow pair would
// hold work an idle one could do.
// Every wait is bounded; a time-out sets MOE_DEVERR_TIMEOUT and unwinds.
// Times in the comments below are those of short runs, before the power cap.
#include "mxfp4_gemm.cuh"

namespace moe {

namespace {

constexpr int kUnitSlots = 3;              // ring of tiles published to a CTA's roles

// Arrive on another CTA's mbarrier without a release: for arrivals that order
// tensor-memory loads only (complete, and fenced by tcgen05.fence).
__device__ __forceinline__ void arrive_relaxed_cluster(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

// The instructions of one CTA (GROUP 1) or of a pair (GROUP 2).
template <int GROUP>
__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  if constexpr (GROUP == 2) {
    tma_load_2d_pair(dst, map, bar, c0, c1);
  } else {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1) : "memory");
  }
}
// Arrive on `bar` in each CTA of the group once the MMAs issued so far are done.
template <int GROUP>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (GROUP == 2) umma_commit_pair_mc(bar, 0x3);
  else umma_commit(bar);
}
template <int GROUP>
__device__ __forceinline__ void group_sync() {
  if constexpr (GROUP == 2) cluster_sync();
  else __syncthreads();
}

template <int EPI, int NMMA, int GROUP>
struct Cfg {
  static constexpr int TILE_M = 128 * GROUP;
  static constexpr int NB = NMMA / 128;                  // scale tiles of B per 128 values of K
  static constexpr int OUT_N = EPI == EPI_SWIGLU ? NMMA / 2 : NMMA;
  static constexpr int B_ROWS = NMMA / GROUP;            // B columns this CTA loads
  static constexpr int B_BOX = B_ROWS < 128 ? B_ROWS : 128;  // of one TMA box
  static constexpr int OPERANDS = kBoxBytes + B_ROWS * 128;
  static constexpr int SCALES = (1 + NB) * 2 * kScaleTile;
  static constexpr int STAGE_BYTES = OPERANDS + SCALES;  // a multiple of 1024
  static constexpr int STAGES = 224 * 1024 / STAGE_BYTES < 8 ? 224 * 1024 / STAGE_BYTES : 8;
  static constexpr int ACC1 = NMMA == 256 ? 224 : 128;   // first column of the second accumulator
  static constexpr int SF_COL = 480;
  static constexpr int TMEM_COLS = 512;
  // epilogue warps: four lane quarters x PARTS of the columns. GELU: four warps
  // a scheduler hide the activation's latencies (d 1024, 64 experts of 128 rows
  // 78 -> 75 us); elsewhere they cost (Mixtral-shaped 574 -> 601 us: more warps
  // waiting on shared memory beside the MMAs).
  static constexpr int PARTS = EPI == EPI_GELU ? 4 : 2;
  static constexpr int EPI_WARPS = 4 * PARTS;
  static constexpr int SCHED_WARP = 2 + EPI_WARPS;
  static constexpr int THREADS = 32 * (SCHED_WARP + 1);
  static constexpr uint32_t UNIT_READERS = 1 + EPI_WARPS;  // producer, epilogue warps (and the even CTA's MMA warp)
  static constexpr size_t SMEM = static_cast<size_t>(STAGES) * STAGE_BYTES + 1024;
};

// 32 fp32 values (one block) of a row to 16 bytes of codes; returns the scale byte.
__device__ __forceinline__ uint32_t quantise_block(float (&h)[32], uint4& codes) {
  // two values an instruction; a NaN stays one
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; i += 2)
    asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(h[i]), "f"(h[i + 1]));
  const uint32_t top = __float_as_uint(m) & 0x7fffffffu;
  const uint32_t sb = mx_scale_byte(top);
  const float inv = mx_inv_scale(sb);
  uint32_t q[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 p = unpack2(mul2(pack2(h[8 * g + i], h[8 * g + i + 1]), pack2(inv, inv)));
      v[i] = p.x;
      v[i + 1] = p.y;
    }
    q[g] = sb == 255u ? 0u : e2m1x8(v);
  }
  codes = make_uint4(q[0], q[1], q[2], q[3]);
  return sb;
}

// Among four neighbouring lanes, p[i] of lane j becomes p[j] of lane i. A thread
// has a row of the accumulator; stores of 16 bytes in 32 rows take the load-store
// unit a cycle each, four lanes with 64 bytes of a row a quarter of that (d 2048,
// F 1408, 64 experts of 256 rows: 111 -> 100 us). The codes of h, half a line in
// all, gain nothing by it.
__device__ __forceinline__ void transpose_quad(uint4 (&p)[4], int lane) {
#pragma unroll
  for (int d = 1; d <= 2; d *= 2) {
    const bool hi = lane & d;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & d) continue;
      uint4& a = p[i];
      uint4& b = p[i + d];
      uint4 g = hi ? a : b;  // given away
      g.x = __shfl_xor_sync(0xffffffffu, g.x, d);
      g.y = __shfl_xor_sync(0xffffffffu, g.y, d);
      g.z = __shfl_xor_sync(0xffffffffu, g.z, d);
      g.w = __shfl_xor_sync(0xffffffffu, g.w, d);
      if (hi) a = g;
      else b = g;
    }
  }
}

// One warp's 32 rows (crow: the first in the tile) and the column groups [g0,
// g0 + G) of 32. reverse: the last group first; `free_overlap` is called once
// the first group's loads are done.
template <int EPI, int OUT_N, int G, typename Free>
__device__ __forceinline__ void epilogue(uint32_t tbase, const MxArgs& args, const MxTile& t, int crow, int lane,
                                         int g0, bool reverse, Free&& free_overlap) {
  const bool valid = crow + lane < t.rows;
  const size_t row = static_cast<size_t>(t.row0) + crow + lane;
  uint32_t sw = 0;
#pragma unroll 1
  for (int gi = 0; gi < G; ++gi) {
    const int gl = reverse ? G - 1 - gi : gi;
    const int g = g0 + gl;
    float h[32];
    uint32_t v[32];
    if constexpr (EPI == EPI_SWIGLU) {
      uint32_t u[32];
      tmem_ld_32x32b_x32(tbase + 32 * g, v);
      tmem_ld_32x32b_x32(tbase + OUT_N + 32 * g, u);
      tmem_ld_wait();
      if (gi == 0) free_overlap();
#pragma unroll
      for (int i = 0; i < 32; ++i) h[i] = silu_fast(__uint_as_float(v[i])) * __uint_as_float(u[i]);
    } else {
      tmem_ld_32x32b_x32(tbase + 32 * g, v);
      tmem_ld_wait();
      if (gi == 0) free_overlap();
      auto activate = [&](auto phi) {
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float2 r = gelu2<decltype(phi)>(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
          h[i] = r.x;
          h[i + 1] = r.y;
        }
      };
      if constexpr (EPI == EPI_GELU) {
        if (gelu_tail(v)) activate(PhiTail{});
        else activate(Phi{});
        __syncwarp();  // the next loads from tensor memory are the whole warp's
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) h[i] = __uint_as_float(v[i]);
      }
    }
    const int col = t.n0 + 32 * g;
    if constexpr (EPI == EPI_STORE) {
      uint4 p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        p[i] = make_uint4(pack_bf16(h[8 * i], h[8 * i + 1]), pack_bf16(h[8 * i + 2], h[8 * i + 3]),
                          pack_bf16(h[8 * i + 4], h[8 * i + 5]), pack_bf16(h[8 * i + 6], h[8 * i + 7]));
      transpose_quad(p, lane);
      const int quad = crow + (lane & ~3);
      __nv_bfloat16* dst = args.out + (static_cast<size_t>(t.row0) + quad) * args.N + col + 8 * (lane & 3);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (quad + i < t.rows) *reinterpret_cast<uint4*>(dst + static_cast<size_t>(i) * args.N) = p[i];
    } else {
      uint4 codes;
      const uint32_t sb = quantise_block(h, codes);
      if (valid) *reinterpret_cast<uint4*>(args.out_codes + row * (args.N / 2) + col / 2) = codes;
      sw |= sb << (8 * gl);
    }
  }
  if constexpr (EPI != EPI_STORE) {
    if (valid) {
      const int r = crow + lane;
      uint8_t* dst = args.out_scales + mx_scale_at(t.group + r / 128, args.N / 128, r & 127, t.n0 / 32 + g0);
      static_assert(G == 1 || G == 2, "a part of 128 or of 256 columns");
      if constexpr (G == 2) *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(sw);
      else *dst = static_cast<uint8_t>(sw);
    }
  }
}

template <int EPI, int NMMA, int GROUP>
__global__ void __launch_bounds__(Cfg<EPI, NMMA, GROUP>::THREADS, 1)
grouped_gemm_mxf4(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
                  const __grid_constant__ CUtensorMap tmB1, const __grid_constant__ CUtensorMap tmSA,
                  const __grid_constant__ CUtensorMap tmSB0, const __grid_constant__ CUtensorMap tmSB1, MxArgs args) {
  using C = Cfg<EPI, NMMA, GROUP>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[STAGES], empty_bar[STAGES];
  __shared__ __align__(8) uint64_t tfull_bar[2], tfree_bar[2], drain_bar;
  __shared__ __align__(8) uint64_t unit_full[kUnitSlots], unit_empty[kUnitSlots];
  __shared__ MxTile unit_ring[kUnitSlots];  // rows = 0: the end
  // the even CTA's scheduler to the odd one's: full in the odd, empty in the even CTA
  __shared__ __align__(8) uint64_t peer_full[kUnitSlots], peer_empty[kUnitSlots];
  __shared__ MxTile peer_ring[kUnitSlots];
  __shared__ Segments segments;
  __shared__ uint32_t tmem_base_s;
  __shared__ volatile int abort_s;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = GROUP == 2 ? cluster_ctarank() : 0u;  // 0: the CTA that issues the MMAs
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));

  // Set-up that needs nothing of the kernel before this one, so that it runs
  // under that kernel's tail.
  if (threadIdx.x == 0) {
    abort_s = 0;
    for (int s = 0; s < STAGES; ++s) { mbar_init(&full_bar[s], 1); mbar_init(&empty_bar[s], 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(&tfull_bar[b], 1); mbar_init(&tfree_bar[b], GROUP * C::EPI_WARPS); }
    for (int i = 0; i < kUnitSlots; ++i) {
      mbar_init(&unit_full[i], 1);
      mbar_init(&unit_empty[i], C::UNIT_READERS + (rank == 0 ? 1 : 0));
      mbar_init(&peer_full[i], 1);
      mbar_init(&peer_empty[i], 1);
    }
    mbar_init(&drain_bar, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (GROUP == 2) {
      tmem_alloc_pair(&tmem_base_s, C::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&tmem_base_s, C::TMEM_COLS);
      tmem_relinquish();
    }
  }
  if (warp == C::SCHED_WARP && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB0);
    prefetch_tmap(&tmB1);
    prefetch_tmap(&tmSA);
    prefetch_tmap(&tmSB0);
    prefetch_tmap(&tmSB1);
  }
  tc_fence_before();
  group_sync<GROUP>();  // barriers initialised and tensor memory allocated in every CTA of the group
  tc_fence_after();
  // The down projection follows the up projection, whose blocks all started
  // after the kernel before it was complete: its row segments can be read now,
  // and weights loaded, before the up projection is done.
  const bool early = args.early != 0;
  if (!early) pdl_begin();
  // All 512 columns are this CTA's, so they start at 0: addresses below are
  // constants (a loaded base would go through registers at every instruction).
  if (tmem_base_s != 0 && threadIdx.x == 0) {
    set_error(args.ctl, MOE_DEVERR_TIMEOUT);
    abort_s = 1;
  }
  constexpr uint32_t tmem_base = 0;
  const int W = gridDim.x / GROUP;  // groups
  const int katoms = args.K / 128;  // scale tiles along K
  const int nkb = (katoms + 1) / 2;
  // the even CTA's full and tfree barriers, as shared::cluster addresses
  // (GROUP 1: this CTA's)
  const uint32_t full0 = GROUP == 2 ? mapa_shared(smem_u32(&full_bar[0]), 0) : smem_u32(&full_bar[0]);
  const uint32_t tfree0 = GROUP == 2 ? mapa_shared(smem_u32(&tfree_bar[0]), 0) : smem_u32(&tfree_bar[0]);

  auto give_up = [&] {
    set_error(args.ctl, MOE_DEVERR_TIMEOUT);
    abort_s = 1;
  };
  // A wait of a whole converged warp: true in all lanes or false in all.
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    const bool ok = mbar_wait_bounded(bar, parity);
    if (__all_sync(0xffffffffu, ok)) return true;
    give_up();
    return false;
  };
  // A reader's next tile, by a whole converged warp: wait for its slot, read it
  // and free it (every reader frees every slot it reads, the end marker too).
  // False at the end, and once anything gave up.
  auto next_unit = [&](int& uslot, uint32_t& uphase, MxTile& t) -> bool {
    if (!warp_wait(&unit_full[uslot], uphase)) return false;
    t = unit_ring[uslot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&unit_empty[uslot]);
    if (++uslot == kUnitSlots) { uslot = 0; uphase ^= 1u; }
    return t.rows > 0;
  };

  if (warp == C::SCHED_WARP) {
    TileList<C::TILE_M> list;
    load_segments(segments, args, lane, 32);
    __syncwarp();
    list.build(args, segments, args.N / C::OUT_N, lane);
    const uint32_t pring1 = GROUP == 2 ? mapa_shared(smem_u32(&peer_ring[0]), 1) : 0u;
    const uint32_t pfull1 = GROUP == 2 ? mapa_shared(smem_u32(&peer_full[0]), 1) : 0u;
    const uint32_t pempty0 = GROUP == 2 ? mapa_shared(smem_u32(&peer_empty[0]), 0) : 0u;
    // Group g starts with tile g, which all of its CTAs know; the counter hands
    // out the tiles from W on.
    int u = static_cast<int>(blockIdx.x) / GROUP;
    int slot = 0, pslot = 0;
    uint32_t phase = 0, pphase = 0;
    for (bool first = true;; first = false) {
      MxTile t{};
      // a slot is free here once every role of this CTA has read it
      bool ok = warp_wait(&unit_empty[slot], phase ^ 1u);
      if (first || rank == 0) {
        if (ok && !abort_s && u < list.total) t = list.tile(u, C::OUT_N, lane);
      } else if (ok) {
        ok = __all_sync(0xffffffffu, mbar_wait_cluster_bounded(&peer_full[pslot], pphase));
        if (ok) t = *const_cast<const MxTile*>(&peer_ring[pslot]);
        else give_up();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive_cluster(pempty0 + pslot * 8u);
        if (++pslot == kUnitSlots) { pslot = 0; pphase ^= 1u; }
      }
      const bool end = !__all_sync(0xffffffffu, ok && !abort_s && t.rows > 0);
      if (end) t.rows = 0;
      if (lane == 0) {
        unit_ring[slot] = t;
        mbar_arrive(&unit_full[slot]);
      }
      if (rank == 0) {
        if (GROUP == 2 && !first) {
          // hand it over; the odd CTA frees the slot once it has taken it
          ok = __all_sync(0xffffffffu, mbar_wait_cluster_bounded(&peer_empty[pslot], pphase ^ 1u));
          if (!ok) {
            give_up();
          } else if (lane == 0) {
            const uint32_t dst = pring1 + pslot * static_cast<uint32_t>(sizeof(MxTile));
            st_shared_cluster_u32(dst, static_cast<uint32_t>(t.row0));
            st_shared_cluster_u32(dst + 4, static_cast<uint32_t>(t.rows));
            st_shared_cluster_u32(dst + 8, static_cast<uint32_t>(t.n0));
            st_shared_cluster_u32(dst + 12, static_cast<uint32_t>(t.group));
            st_shared_cluster_u32(dst + 16, static_cast<uint32_t>(t.e));
            mbar_arrive_cluster(pfull1 + pslot * 8u);
          }
          if (++pslot == kUnitSlots) { pslot = 0; pphase ^= 1u; }
        }
        if (first && early) {
          pdl_begin();  // the counter is the previous kernel's until it is done
        }
        if (!end) {
          int v = 0;
          if (lane == 0) v = static_cast<int>(min(atomicAdd(&args.ctl->gemm_next, 1u), static_cast<unsigned>(list.total)));
          u = W + __shfl_sync(0xffffffffu, v, 0);
        }
      }
      if (++slot == kUnitSlots) { slot = 0; phase ^= 1u; }
      if (end) break;
    }
    // The last pair to finish resets the tile counter for the next launch
    // (every pair's last take precedes its increment here).
    if (rank == 0 && lane == 0 && atomicAdd(&args.ctl->gemm_done, 1u) == static_cast<unsigned>(W) - 1u) {
      atomicExch(&args.ctl->gemm_next, 0u);
      atomicExch(&args.ctl->gemm_done, 0u);
    }
  } else if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0;
    uint32_t issued_mask = 0;  // stages that ever received a load
    uint32_t last_parity = 0;  // parity of that stage's latest load
    int uslot = 0;
    uint32_t uphase = 0;
    const int ngroups = args.N / 128;
    MxTile t;
    bool ok = true;
    // early: the first tile's weights go out before the wait for the previous
    // kernel (stages of a fresh ring are free), its rows after it
    int ahead = 0;
    for (bool first = early; ok; first = false) {
      if (!next_unit(uslot, uphase, t)) break;
      const int arow = t.row0 + 128 * static_cast<int>(rank);
      const int ga = (t.group + static_cast<int>(rank)) * katoms;
      const int gb = (t.e * ngroups + t.n0 / 128) * katoms;
      // SwiGLU: W_gate's columns, then W_up's; a pair's CTA r has the half r of
      // all columns
      const int brow = t.e * args.N + t.n0;
      auto load_weights = [&](int st, int kb) {
        uint8_t* sa = smem + st * C::STAGE_BYTES;
        uint8_t* ss = sa + C::OPERANDS;
        const uint32_t fb = full0 + st * 8u;
        if (rank == 0) mbar_arrive_expect_tx(&full_bar[st], GROUP * C::STAGE_BYTES);
#pragma unroll
        for (int j = 0; j < C::B_ROWS / C::B_BOX; ++j) {
          const int col = C::B_ROWS * static_cast<int>(rank) + j * C::B_BOX;  // in the MMA's N
          const bool up = EPI == EPI_SWIGLU && col >= C::OUT_N;
          load_box<GROUP>(sa + kBoxBytes + j * C::B_BOX * 128, up ? &tmB1 : &tmB0, fb, kb * 128,
                          brow + (up ? col - C::OUT_N : col));
        }
        // two scale tiles each (the second is not used where K ends after one)
        load_box<GROUP>(ss + 2 * kScaleTile, &tmSB0, fb, 0, gb + 2 * kb);
        if (C::NB == 2)
          load_box<GROUP>(ss + 4 * kScaleTile, EPI == EPI_SWIGLU ? &tmSB1 : &tmSB0, fb, 0,
                          (EPI == EPI_SWIGLU ? gb : gb + katoms) + 2 * kb);
      };
      if (first) {
        ahead = min(STAGES, nkb);
        if (elect_one())
          for (int kb = 0; kb < ahead; ++kb) load_weights(kb, kb);
        __syncwarp();
        pdl_begin();
      }
      for (int kb = 0; kb < nkb; ++kb) {
        if (!warp_wait(&empty_bar[stage], phase ^ 1u)) {
          ok = false;
          break;
        }
        uint8_t* sa = smem + stage * C::STAGE_BYTES;
        const uint32_t fb = full0 + stage * 8u;
        if (elect_one()) {
          if (kb >= ahead) load_weights(stage, kb);
          load_box<GROUP>(sa, &tmA, fb, kb * 128, arow);
          load_box<GROUP>(sa + C::OPERANDS, &tmSA, fb, 0, ga + 2 * kb);
        }
        __syncwarp();
        issued_mask |= 1u << stage;
        last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
      ahead = 0;
    }
    // Every load issued must have been consumed by the MMAs (so it landed)
    // before this CTA may leave: the MMA commit of each stage's last load
    // arrives on empty[s] in both CTAs.
    for (int s = 0; s < STAGES; ++s)
      if (issued_mask & (1u << s))
        if (!mbar_wait_bounded(&empty_bar[s], (last_parity >> s) & 1u)) set_error(args.ctl, MOE_DEVERR_TIMEOUT);
  } else if (warp == 1) {
    if (early) pdl_begin();
    if (rank == 0) {
      constexpr uint32_t kIdesc0 = make_idesc_mxf4(C::TILE_M, NMMA, 0);
      constexpr uint32_t kIdesc2 = make_idesc_mxf4(C::TILE_M, NMMA, 2);
      const uint32_t base = smem_u32(smem);
      const uint64_t adesc0 = make_sw128_desc(base, 16, 1024);
      const uint64_t bdesc0 = make_sw128_desc(base + kBoxBytes, 16, 1024);
      const uint64_t sdesc0 = make_scale_desc(base + C::OPERANDS);
      int stage = 0;
      uint32_t phase = 0;
      uint32_t set = 0;
      bool issued_any = false, dead = false;  // in the issuing thread
      int uslot = 0;
      uint32_t uphase = 0;
      for (int i = 0;; ++i) {  // i: tiles this pair has started
        MxTile t;
        if (!next_unit(uslot, uphase, t)) break;
        const uint32_t d_tmem = tmem_base + ((i & 1) ? C::ACC1 : 0);
        for (int kb = 0; kb < nkb; ++kb) {
          const uint32_t so = stage * (C::STAGE_BYTES >> 4);  // descriptors count 16 bytes
          const int atoms = min(2, katoms - 2 * kb);
          if (elect_one()) {
            if (!dead) dead = !mbar_wait_bounded(&full_bar[stage], phase);
            // the previous tile's epilogues have read the columns shared with
            // this tile's accumulator (and everything of the tile before it)
            if (kb == 0 && i > 0 && !dead) dead = !mbar_wait_bounded(&tfree_bar[(i - 1) & 1], ((i - 1) >> 1) & 1);
            if (!dead) {
              tc_fence_after();
#pragma unroll
              for (int at = 0; at < 2; ++at) {
                if (at < atoms) {
                  const uint32_t sfa = tmem_base + C::SF_COL + (set ^ at) * 16;
                  const uint32_t sfb = sfa + 4;
                  copy_scales<GROUP>(sfa, sdesc0 + so + at * (kScaleTile >> 4));
#pragma unroll
                  for (int j = 0; j < C::NB; ++j)
                    copy_scales<GROUP>(sfb + 4 * j, sdesc0 + so + ((1 + j) * 2 + at) * (kScaleTile >> 4));
#pragma unroll
                  for (int kk = 0; kk < 2; ++kk) {
                    const uint32_t off = so + (at * 2 + kk) * 2;
                    umma_mxf4<GROUP>(d_tmem, adesc0 + off, bdesc0 + off, kk == 0 ? kIdesc0 : kIdesc2, sfa, sfb,
                              (kb | at | kk) != 0 ? 1u : 0u);
                  }
                }
              }
              commit<GROUP>(&empty_bar[stage]);
              if (kb == nkb - 1) commit<GROUP>(&tfull_bar[i & 1]);
              issued_any = true;
            }
          }
          __syncwarp();
          set ^= atoms & 1;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (__any_sync(0xffffffffu, dead)) {
          give_up();
          break;
        }
      }
      if (__any_sync(0xffffffffu, issued_any)) {
        // Tensor memory is freed below: wait until every MMA issued is done.
        if (elect_one()) {
          if constexpr (GROUP == 2) umma_commit_pair_mc(&drain_bar, 0x1);
          else umma_commit(&drain_bar);
        }
        __syncwarp();
        (void)mbar_wait_bounded(&drain_bar, 0);
      }
    }
  } else {
    // epilogue warps: tensor-memory lane quarter = warp % 4 of this CTA's 128
    // rows, and a part of the column groups
    constexpr int G = C::OUT_N / 32 / C::PARTS;  // groups of 32 columns per warp
    if (early) pdl_begin();
    const int q = warp & 3, part = (warp - 2) >> 2;
    int uslot = 0;
    uint32_t uphase = 0;
    for (int i = 0;; ++i) {
      const int acc = i & 1;
      MxTile t;
      if (!next_unit(uslot, uphase, t) || !warp_wait(&tfull_bar[acc], (i >> 1) & 1)) break;
      tc_fence_after();
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + (acc ? C::ACC1 : 0);
      auto free_overlap = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (GROUP == 2) arrive_relaxed_cluster(tfree0 + acc * 8u);
          else mbar_arrive(&tfree_bar[acc]);
        }
      };
      const int crow = 128 * static_cast<int>(rank) + q * 32;
      // The shared columns are in the last group of the first accumulator
      // (last part's warps) and in the first group of the second. A warp
      // without rows leaves the others its issue slots (a skewed layer's last
      // tiles have few rows: 2% there).
      if (crow >= t.rows) free_overlap();
      else epilogue<EPI, C::OUT_N, G>(tbase, args, t, crow, lane, part * G, acc == 0,
                                 free_overlap);
    }
  }
  tc_fence_before();
  __syncthreads();
  group_sync<GROUP>();  // no peer still reads or signals this CTA; every MMA is done
  if (warp == 1) {
    tc_fence_after();
    if constexpr (GROUP == 2) tmem_dealloc_pair(tmem_base_s, C::TMEM_COLS);
    else tmem_dealloc(tmem_base_s, C::TMEM_COLS);
  }
}

template <int EPI, int NMMA, int GROUP>
cudaError_t run_group(const MxRows& a, const MxWeights& b0, const MxWeights& b1, const MxArgs& args, cudaStream_t s) {
  using C = Cfg<EPI, NMMA, GROUP>;
  CUtensorMap ta, tb0, tb1, sa, sb0, sb1;
  const uint64_t brows = static_cast<uint64_t>(args.E) * args.N, katoms = args.K / 128;
  const uint64_t atiles = (static_cast<uint64_t>(args.rows_max) / 128 + args.E) * katoms;
  const MxWeights& up = EPI == EPI_SWIGLU ? b1 : b0;
  if (!make_tma_codes(&ta, a.codes, static_cast<uint64_t>(args.rows_max), args.K / 2, 128) ||
      !make_tma_codes(&tb0, b0.codes, brows, args.K / 2, C::B_BOX) ||
      !make_tma_codes(&tb1, up.codes, brows, args.K / 2, C::B_BOX) ||
      !make_tma_scales(&sa, a.scales, atiles) || !make_tma_scales(&sb0, b0.scales, brows / 128 * katoms) ||
      !make_tma_scales(&sb1, up.scales, brows / 128 * katoms))
    return cudaErrorInvalidValue;
  auto kern = grouped_gemm_mxf4<EPI, NMMA, GROUP>;
  cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::SMEM));
  const int grid = num_sms() / GROUP * GROUP;
  if constexpr (GROUP == 2)
    return launch_pdl_cluster(kern, dim3(grid), dim3(C::THREADS), C::SMEM, s, 2, ta, tb0, tb1, sa, sb0, sb1, args);
  else
    return launch_pdl(kern, dim3(grid), dim3(C::THREADS), C::SMEM, s, false, ta, tb0, tb1, sa, sb0, sb1, args);
}

// A product runs on CTA pairs where experts have many rows on average (of the
// most that can be in use, which is all the host knows) and K is long; single
// CTAs' 128-row tiles fill better, and with short K a tile's turnaround counts,
// which the second CTA lengthens. Measured, whole FFN, single against pairs for
// both products, in short runs (back to back, under the power cap, the largest
// take a sixth longer): 8 experts, d 4096, F 14336: 32 rows
// an expert 131 / 154 us, 128 rows 166 / 159, 256 rows 229 / 220, 512 rows 377 /
// 350, 1024 rows 659 / 570; 64 experts, d 4096, F 2048, skewed, 128 rows 182 /
// 208, 512 rows 469 / 457; d 2048, F 1408: 256 rows 116 / 115, 512 rows 189 /
// 181. With d 1024, F 4096, 512 rows: singles 195, pairs for the down projection
// alone 191, for both 195; if a capacity leaves 173 of the 512: 91, 92, 102.
constexpr int64_t kPairRows = 256;
constexpr int kPairK = 2048;

template <int EPI, int NMMA>
cudaError_t run_gemm(const MxRows& a, const MxWeights& b0, const MxWeights& b1, const MxArgs& args, int64_t rows,
                     cudaStream_t s) {
  if (rows >= kPairRows * args.E && args.K >= kPairK) return run_group<EPI, NMMA, 2>(a, b0, b1, args, s);
  return run_group<EPI, NMMA, 1>(a, b0, b1, args, s);
}

}  // namespace

cudaError_t launch_ffn_mxfp4(const MxRows& x, const MxWeights& w1, const MxWeights& w3, const MxWeights& w2,
                             moe_act_t act, int64_t rows_max, int d, int F, int E, const int32_t* seg,
                             const int32_t* kept, const MxRows& h, void* y, float* partials, Control* ctl,
                             cudaStream_t s, cudaEvent_t after_up, bool early_up, int64_t slots) {
  if (rows_max <= 0) {
    if (after_up) cudaEventRecord(after_up, s);
    return cudaSuccess;
  }
  MxArgs a{};
  a.seg = seg;
  a.kept = kept;
  a.E = E;
  a.d = d;
  a.F = F;
  a.rows_max = rows_max;
  a.ctl = ctl;
  a.early = early_up ? 1 : 0;
  a.out_codes = h.codes;
  a.out_scales = h.scales;
  a.out = static_cast<__nv_bfloat16*>(y);
  const int64_t rows = mxfp4_rows(rows_max, slots);
  // A decode step's rows (32 at most, so no expert has more) go through the
  // weight stream: one token of a Mixtral-shaped layer takes 44 us there,
  // 57 us here.
  if (rows <= kMxStreamRows) {
    a.partials = partials;
    const cudaError_t err = launch_stream_ffn_mxfp4(x, w1, w3, w2, act, h, a, s);
    if (after_up) cudaEventRecord(after_up, s);
    return err;
  }
  a.K = d;
  a.N = F;
  cudaError_t err;
  if (act == MOE_ACT_SWIGLU)
    err = run_gemm<EPI_SWIGLU, 256>(x, w1, w3, a, rows, s);
  else if (F % 256 == 0)
    err = run_gemm<EPI_GELU, 256>(x, w1, w1, a, rows, s);
  else
    err = run_gemm<EPI_GELU, 128>(x, w1, w1, a, rows, s);
  if (err != cudaSuccess) return err;
  if (after_up) cudaEventRecord(after_up, s);
  a.early = 1;
  a.K = F;
  a.N = d;
  if (d % 256 == 0) return run_gemm<EPI_STORE, 256>(h, w2, w2, a, rows, s);
  return run_gemm<EPI_STORE, 128>(h, w2, w2, a, rows, s);
}

}  // namespace moe
