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
// CTA = 6 warps, one CTA per SM, persistent over tiles:
//   warp 0   producer: per stage (256 values of K) the 128-row A box and the B
//            boxes by TMA (128 bytes = 256 codes a row, 128-byte swizzle), and
//            the scales of both by bulk copies (1 KB per 128 rows)
//   warp 1   MMA issuer: per 128 values of K one thread copies the scale tiles
//            to tensor memory (tcgen05.cp, replicated to the four lane
//            quarters) and issues two MMAs of K = 64 with them
//   warps 2-5 epilogue: a thread per row, 32 columns (one block) at a time
//
// Tensor memory: two accumulators of 256 columns and the scales do not fit in
// 512 columns, so the accumulators overlap by 32 columns (columns 0-255 and
// 224-479) and the scales use 480-511 (two sets of 12, taken in turn). The
// epilogue reads the overlapping columns first and frees them at once; the
// next tile's MMAs start then, while the rest of the tile is still read.
// Every wait is bounded; a time-out sets MOE_DEVERR_TIMEOUT and unwinds.
#include "gemm_common.cuh"
#include "mxfp4.cuh"
#include "ptx.cuh"
#include <cudaTypedefs.h>

namespace moe {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

namespace {

constexpr int kTileM = 128;
constexpr int kBoxBytes = 128 * 128;  // 128 rows x 128 bytes (256 values of K)
constexpr int kThreads = 192;
constexpr int kStages = 4;
constexpr int kEpiWarps = 4;

enum { EPI_SWIGLU = 0, EPI_GELU = 1, EPI_STORE = 2 };

struct MxArgs {
  const int32_t* seg;    // [E+1] row segment offsets
  const int32_t* kept;   // [E] rows of each expert from seg[e] (binned layout), or null
  const uint8_t* sa;     // scales of A
  const uint8_t* sb0;    // scales of B (W_gate / W1 / W2)
  const uint8_t* sb1;    // scales of W_up (SwiGLU)
  uint8_t* out_codes;    // up projection: h codes [rows_max, N/2]
  uint8_t* out_scales;   // up projection: h scales
  __nv_bfloat16* out;    // down projection: [rows_max, N]
  int E;
  int K;
  int N;  // output columns
  long long rows_max;
  Control* ctl;
};

// ------------------------------------------------------------ tcgen05, mxf4
// Instruction descriptor of kind::mxf4: E2M1 operands (1 at bits 7 and 10),
// both K-major, N / 8 at bit 17, scales UE8M0 (bit 23), M / 128 at bit 27; the
// ids of the scale bytes to use (0 or 2) go to bits 4 (B) and 29 (A).
__host__ __device__ constexpr uint32_t make_idesc_mxf4(int M, int N, uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(M >> 7) << 27) | (sf_id << 29);
}

__device__ __forceinline__ void umma_mxf4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
      ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
      : "memory");
}

// One 512-byte scale tile (32 rows of 16 bytes, 8-row groups 128 bytes apart)
// to 4 columns of tensor memory, replicated to the four 32-lane quarters.
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint32_t smem_addr) {
  const uint64_t desc = static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(128 >> 4) << 32) |
                        (static_cast<uint64_t>(1u) << 46);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

template <int EPI, int NMMA>
struct Cfg {
  static constexpr int NB = NMMA / 128;  // 128-column B boxes
  static constexpr int OUT_N = EPI == EPI_SWIGLU ? NMMA / 2 : NMMA;
  static constexpr int OPERANDS = (1 + NB) * kBoxBytes;
  static constexpr int SCALES = (1 + NB) * 2 * kScaleTile;
  static constexpr int STAGE_BYTES = OPERANDS + SCALES;  // a multiple of 1024
  static constexpr int ACC1 = NMMA == 256 ? 224 : 128;   // first column of the second accumulator
  static constexpr int SF_COL = 480;
  static constexpr int TMEM_COLS = 512;
  static constexpr size_t SMEM = static_cast<size_t>(kStages) * STAGE_BYTES + 1024;
};

struct MxTile {
  int e, mt, row0, rows, n0;
};

// Tile u of the list: expert-major, then N tile, M tile fastest.
__device__ __forceinline__ MxTile decode_tile(int u, const int* tile_start, const int* seg, const int* cnt,
                                              int E, int out_n) {
  int lo = 0, hi = E - 1;  // last e with tile_start[e] <= u
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tile_start[mid] <= u) lo = mid; else hi = mid - 1;
  }
  MxTile t;
  t.e = lo;
  const int mt_e = (cnt[lo] + kTileM - 1) / kTileM;
  const int local = u - tile_start[lo];
  const int nt = local / mt_e;
  t.mt = local - nt * mt_e;
  t.row0 = seg[lo] + t.mt * kTileM;
  t.rows = min(kTileM, cnt[lo] - t.mt * kTileM);
  t.n0 = nt * out_n;
  return t;
}

// 32 fp32 values (one block) of a row to 16 bytes of codes; returns the scale byte.
__device__ __forceinline__ uint32_t quantise_block(float (&h)[32], uint4& codes) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) top = max(top, __float_as_uint(h[i]) & 0x7fffffffu);
  const uint32_t sb = mx_scale_byte(top);
  const float inv = mx_inv_scale(sb);
  uint32_t q[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = h[8 * g + i] * inv;
    q[g] = sb == 255u ? 0u : e2m1x8(v);
  }
  codes = make_uint4(q[0], q[1], q[2], q[3]);
  return sb;
}

// One warp's 32 rows of a tile. first: the 32-column group to read first (it
// holds the columns that overlap the other accumulator); `free_overlap` is
// called once its loads are done.
template <int EPI, int OUT_N, typename Free>
__device__ __forceinline__ void epilogue(uint32_t tbase, const MxArgs& args, const MxTile& t, int wrow, int lane,
                                         int first, Free&& free_overlap) {
  constexpr int G = OUT_N / 32;
  const int r = wrow + lane;  // row in the tile
  const bool valid = r < t.rows;
  const size_t row = static_cast<size_t>(t.row0) + r;
  uint32_t sw[G / 4] = {};
#pragma unroll 1
  for (int gi = 0; gi < G; ++gi) {
    const int g = first == 0 ? gi : (gi == 0 ? G - 1 : gi - 1);
    float h[32];
    uint32_t v[32];
    if constexpr (EPI == EPI_SWIGLU) {
      uint32_t u[32];
      tmem_ld_32x32b_x32(tbase + 32 * g, v);
      tmem_ld_32x32b_x32(tbase + OUT_N + 32 * g, u);
      tmem_ld_wait();
      if (gi == 0) free_overlap();
#pragma unroll
      for (int i = 0; i < 32; ++i) h[i] = silu(__uint_as_float(v[i])) * __uint_as_float(u[i]);
    } else {
      tmem_ld_32x32b_x32(tbase + 32 * g, v);
      tmem_ld_wait();
      if (gi == 0) free_overlap();
#pragma unroll
      for (int i = 0; i < 32; ++i)
        h[i] = EPI == EPI_GELU ? gelu_erf(__uint_as_float(v[i])) : __uint_as_float(v[i]);
    }
    const int col = t.n0 + 32 * g;
    if constexpr (EPI == EPI_STORE) {
      if (valid) {
        uint4* dst = reinterpret_cast<uint4*>(args.out + row * args.N + col);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          dst[i] = make_uint4(pack_bf16(h[8 * i], h[8 * i + 1]), pack_bf16(h[8 * i + 2], h[8 * i + 3]),
                              pack_bf16(h[8 * i + 4], h[8 * i + 5]), pack_bf16(h[8 * i + 6], h[8 * i + 7]));
      }
    } else {
      uint4 codes;
      const uint32_t sb = quantise_block(h, codes);
      if (valid) *reinterpret_cast<uint4*>(args.out_codes + row * (args.N / 2) + col / 2) = codes;
#pragma unroll
      for (int w = 0; w < G / 4; ++w)
        if (w == (g >> 2)) sw[w] |= sb << (8 * (g & 3));
    }
  }
  if constexpr (EPI != EPI_STORE) {
    if (valid) {
      const long long group = t.row0 - t.mt * kTileM;  // seg[e]
#pragma unroll
      for (int w = 0; w < G / 4; ++w)
        *reinterpret_cast<uint32_t*>(args.out_scales + mx_scale_at(group / 128 + t.e + t.mt, args.N / 128, r,
                                                                   t.n0 / 32 + 4 * w)) = sw[w];
    }
  }
}

template <int EPI, int NMMA>
__global__ void __launch_bounds__(kThreads, 1)
grouped_gemm_mxf4(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
                  const __grid_constant__ CUtensorMap tmB1, MxArgs args) {
  pdl_begin();
  using C = Cfg<EPI, NMMA>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[kStages], empty_bar[kStages];
  __shared__ __align__(8) uint64_t tfull_bar[2], tfree_bar[2], drain_bar;
  __shared__ uint32_t tmem_base_s;
  __shared__ int seg_s[kMaxE + 1];
  __shared__ int cnt_s[kMaxE];
  __shared__ int tile_start_s[kMaxE + 1];
  __shared__ volatile int abort_s;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = args.E;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));

  for (int i = threadIdx.x; i <= E; i += kThreads) {
    seg_s[i] = __ldg(args.seg + i);
    if (i < E)
      cnt_s[i] = args.kept != nullptr ? __ldg(args.kept + i) : __ldg(args.seg + i + 1) - __ldg(args.seg + i);
  }
  if (threadIdx.x == 0) abort_s = 0;
  __syncthreads();
  if (warp == 0) build_schedule<kTileM>(args, args.N / C::OUT_N, seg_s, cnt_s, tile_start_s, lane);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) { mbar_init(&full_bar[s], 1); mbar_init(&empty_bar[s], 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(&tfull_bar[b], 1); mbar_init(&tfree_bar[b], kEpiWarps); }
    mbar_init(&drain_bar, 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&tmem_base_s, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_base_s;
  const int total = tile_start_s[E];
  const int W = gridDim.x;
  const int katoms = args.K / 128;  // scale tiles along K
  const int nkb = (katoms + 1) / 2;

  if (warp == 0) {
    if (lane == 0) {
      prefetch_tmap(&tmA);
      prefetch_tmap(&tmB0);
      prefetch_tmap(&tmB1);
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued_mask = 0;  // stages that ever received a load
      uint32_t last_parity = 0;  // parity of that stage's latest load
      const int ngroups = args.N / 128;
      for (int u = blockIdx.x; u < total && !abort_s; u += W) {
        const MxTile t = decode_tile(u, tile_start_s, seg_s, cnt_s, E, C::OUT_N);
        const size_t ga = static_cast<size_t>(seg_s[t.e] / 128 + t.e + t.mt) * katoms;
        const size_t gb = (static_cast<size_t>(t.e) * ngroups + t.n0 / 128) * katoms;
        const int brow = t.e * args.N + t.n0;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait_bounded(&empty_bar[stage], phase ^ 1u)) {
            set_error(args.ctl, MOE_DEVERR_TIMEOUT);
            abort_s = 1;
            break;
          }
          uint8_t* sa = smem + stage * C::STAGE_BYTES;
          uint8_t* ss = sa + C::OPERANDS;
          uint64_t* fb = &full_bar[stage];
          const uint32_t sbytes = min(2, katoms - 2 * kb) * kScaleTile;
          mbar_arrive_expect_tx(fb, C::OPERANDS + (1 + C::NB) * sbytes);
          tma_load_2d(sa, &tmA, fb, kb * 128, t.row0);
          bulk_load(ss, args.sa + (ga + 2 * kb) * kScaleTile, sbytes, fb);
#pragma unroll
          for (int j = 0; j < C::NB; ++j) {
            uint8_t* sb = sa + (1 + j) * kBoxBytes;
            uint8_t* sj = ss + (1 + j) * 2 * kScaleTile;
            if (EPI == EPI_SWIGLU) {
              tma_load_2d(sb, j == 0 ? &tmB0 : &tmB1, fb, kb * 128, brow);
              bulk_load(sj, (j == 0 ? args.sb0 : args.sb1) + (gb + 2 * kb) * kScaleTile, sbytes, fb);
            } else {
              tma_load_2d(sb, &tmB0, fb, kb * 128, brow + 128 * j);
              bulk_load(sj, args.sb0 + (gb + static_cast<size_t>(j) * katoms + 2 * kb) * kScaleTile, sbytes, fb);
            }
          }
          issued_mask |= 1u << stage;
          last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
      }
      // Every load issued must have landed before the CTA may exit.
      for (int s = 0; s < kStages; ++s)
        if (issued_mask & (1u << s)) if (!mbar_wait_bounded(&full_bar[s], (last_parity >> s) & 1u)) set_error(args.ctl, MOE_DEVERR_TIMEOUT);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t kIdesc0 = make_idesc_mxf4(kTileM, NMMA, 0);
      constexpr uint32_t kIdesc2 = make_idesc_mxf4(kTileM, NMMA, 2);
      int stage = 0;
      uint32_t phase = 0;
      uint32_t set = 0;
      int i = 0;  // tiles this CTA has started
      bool issued_any = false;
      for (int u = blockIdx.x; u < total && !abort_s; u += W, ++i) {
        // the previous tile's epilogue has read the columns shared with this
        // tile's accumulator (and everything of the tile before it)
        if (i > 0 && !mbar_wait_bounded(&tfree_bar[(i - 1) & 1], ((i - 1) >> 1) & 1)) {
          set_error(args.ctl, MOE_DEVERR_TIMEOUT);
          abort_s = 1;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + ((i & 1) ? C::ACC1 : 0);
        bool ok = true;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait_bounded(&full_bar[stage], phase)) {
            set_error(args.ctl, MOE_DEVERR_TIMEOUT);
            abort_s = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(smem + stage * C::STAGE_BYTES);
          const uint32_t b_addr = a_addr + kBoxBytes;
          const uint32_t s_addr = a_addr + C::OPERANDS;
          const int atoms = min(2, katoms - 2 * kb);
          for (int at = 0; at < atoms; ++at) {
            const uint32_t sfa = tmem_base + C::SF_COL + set * 16;
            const uint32_t sfb = sfa + 4;
            copy_scales(sfa, s_addr + at * kScaleTile);
#pragma unroll
            for (int j = 0; j < C::NB; ++j)
              copy_scales(sfb + 4 * j, s_addr + ((1 + j) * 2 + at) * kScaleTile);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
              const uint32_t off = (at * 2 + kk) * 32;
              umma_mxf4(d_tmem, make_sw128_desc(a_addr + off, 16, 1024), make_sw128_desc(b_addr + off, 16, 1024),
                        kk == 0 ? kIdesc0 : kIdesc2, sfa, sfb, (kb | at | kk) != 0 ? 1u : 0u);
            }
            set ^= 1u;
          }
          issued_any = true;
          umma_commit(&empty_bar[stage]);
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        umma_commit(&tfull_bar[i & 1]);
      }
      if (issued_any) {
        // Tensor memory is freed below: wait until every MMA issued is done.
        umma_commit(&drain_bar);
        (void)mbar_wait_bounded(&drain_bar, 0);
      }
    }
  } else {
    // epilogue warps 2..5: tensor-memory lane quarter = warp % 4
    const int q = warp & 3;
    int i = 0;
    for (int u = blockIdx.x; u < total; u += W, ++i) {
      const int acc = i & 1;
      // Lane 0 polls and decides for the whole warp, so the warp-wide
      // tcgen05.ld below always runs converged.
      int ok = 0;
      if (lane == 0) {
        ok = !abort_s && mbar_wait_bounded(&tfull_bar[acc], (i >> 1) & 1);
        if (!ok && !abort_s) {
          set_error(args.ctl, MOE_DEVERR_TIMEOUT);
          abort_s = 1;
        }
      }
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      tc_fence_after();
      const MxTile t = decode_tile(u, tile_start_s, seg_s, cnt_s, E, C::OUT_N);
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + (acc ? C::ACC1 : 0);
      epilogue<EPI, C::OUT_N>(tbase, args, t, q * 32, lane, acc == 0 ? 1 : 0, [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tfree_bar[acc]);
      });
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// Codes [rows, cols / 2 bytes], box 128 bytes x box_rows, 128-byte swizzle.
bool make_tma_codes(CUtensorMap* m, const void* base, uint64_t rows, uint64_t row_bytes, uint32_t box_rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {row_bytes, rows};
  cuuint64_t strides[1] = {row_bytes};
  cuuint32_t box[2] = {128, box_rows};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

template <int EPI, int NMMA>
cudaError_t run_gemm(const uint8_t* a, const uint8_t* b0, const uint8_t* b1, const MxArgs& args, cudaStream_t s) {
  using C = Cfg<EPI, NMMA>;
  CUtensorMap ta, tb0, tb1;
  const uint64_t brows = static_cast<uint64_t>(args.E) * args.N;
  if (!make_tma_codes(&ta, a, static_cast<uint64_t>(args.rows_max), args.K / 2, 128) ||
      !make_tma_codes(&tb0, b0, brows, args.K / 2, 128) ||
      !make_tma_codes(&tb1, b1 != nullptr ? b1 : b0, brows, args.K / 2, 128))
    return cudaErrorInvalidValue;
  auto kern = grouped_gemm_mxf4<EPI, NMMA>;
  cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::SMEM));
  return launch_pdl(kern, dim3(num_sms()), dim3(kThreads), C::SMEM, s, false, ta, tb0, tb1, args);
}

}  // namespace

cudaError_t launch_ffn_mxfp4(const MxRows& x, const MxWeights& w1, const MxWeights& w3, const MxWeights& w2,
                             moe_act_t act, int64_t rows_max, int d, int F, int E, const int32_t* seg,
                             const int32_t* kept, const MxRows& h, void* y, Control* ctl, cudaStream_t s,
                             cudaEvent_t after_up) {
  if (rows_max <= 0) {
    if (after_up) cudaEventRecord(after_up, s);
    return cudaSuccess;
  }
  MxArgs a{};
  a.seg = seg;
  a.kept = kept;
  a.E = E;
  a.rows_max = rows_max;
  a.ctl = ctl;
  a.sa = x.scales;
  a.sb0 = w1.scales;
  a.sb1 = w3.scales;
  a.out_codes = h.codes;
  a.out_scales = h.scales;
  a.K = d;
  a.N = F;
  cudaError_t err;
  if (act == MOE_ACT_SWIGLU)
    err = run_gemm<EPI_SWIGLU, 256>(x.codes, w1.codes, w3.codes, a, s);
  else if (F % 256 == 0)
    err = run_gemm<EPI_GELU, 256>(x.codes, w1.codes, nullptr, a, s);
  else
    err = run_gemm<EPI_GELU, 128>(x.codes, w1.codes, nullptr, a, s);
  if (err != cudaSuccess) return err;
  if (after_up) cudaEventRecord(after_up, s);
  a.sa = h.scales;
  a.sb0 = w2.scales;
  a.sb1 = nullptr;
  a.out = static_cast<__nv_bfloat16*>(y);
  a.K = F;
  a.N = d;
  if (d % 256 == 0) return run_gemm<EPI_STORE, 256>(h.codes, w2.codes, nullptr, a, s);
  return run_gemm<EPI_STORE, 128>(h.codes, w2.codes, nullptr, a, s);
}

}  // namespace moe
