// Shared by the grouped GEMM kernels: the activations, the device-side list of
// row tiles over the experts' segments and its work units.
#pragma once
#include "common.cuh"

namespace moe {

namespace {

constexpr int kMaxE = 256;

// silu(g) = g / (1 + e^-g) with the hardware exponential and reciprocal
// (CUDA's __expf and __fdividef intrinsics, a few ulp of fp32): the result is
// rounded to bf16 (2^-9 relative), so their error never shows, and the
// epilogue of the up projection runs in the tensor cores' shadow. For
// g < -88 the exponential overflows and __fdividef returns 0, the limit.
__device__ __forceinline__ float silu(float g) { return __fdividef(g, 1.0f + __expf(-g)); }
__device__ __forceinline__ float gelu_erf(float z) {
  return 0.5f * z * (1.0f + erff(z * 0.70710678118654752440f));
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ------------------------------------------------------------------ schedule
// Warp 0: tile_start[e] = exclusive prefix of the per-expert unit counts
// ceil(m_e / TILE_M) * ntn (m_e = cnt[e] rows from seg[e]); tile_start[E] =
// total. Lane l owns experts [8l, 8l + 8). A segment whose rows are out of
// range is reported and gets zero tiles.
template <int TILE_M, typename Args>
__device__ __forceinline__ void build_schedule(const Args& args, int ntn, const int* seg_s,
                                               const int* cnt_s, int* tile_start_s, int lane) {
  const int E = args.E;
  int loc[8];
  int sum = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = lane * 8 + i;
    int m = 0;
    if (e < E) {
      m = cnt_s[e];
      if (m < 0 || seg_s[e] < 0 || static_cast<long long>(seg_s[e]) + m > args.rows_max ||
          seg_s[e] + m > seg_s[e + 1]) {
        set_error(args.ctl, MOE_DEVERR_ROW_RANGE);
        m = 0;
      }
    }
    loc[i] = ((m + TILE_M - 1) / TILE_M) * ntn;
    sum += loc[i];
  }
  int incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += n;
  }
  int run = incl - sum;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = lane * 8 + i;
    if (e < E) tile_start_s[e] = run;
    run += loc[i];
  }
  // The lanes cover experts 0..255 only; the total goes to entry E (which is
  // 256 when E = 256). Experts >= E contributed 0 tiles to the sum.
  if (lane == 31) tile_start_s[E] = incl;
}

// Tile -> (expert, first row, valid rows, first output column, half width).
struct Tile {
  int e, row0, rows, n0;
  bool half;
};

// Work units: tiles ordered expert-major, then N tile, M tile fastest, dealt
// round-robin to W persistent workers. When the last wave would leave workers
// idle (total % W = r tiles, 2r <= W), those r tiles become 2r half-width
// units (N/2 columns each), so the tail takes half a tile's time.
__device__ __forceinline__ bool split_tail(int total, int W) {
  const int r = total % W;
  return r != 0 && 2 * r <= W;
}

__device__ __forceinline__ int num_units(int total, int W) {
  return split_tail(total, W) ? total + total % W : total;
}

template <int TILE_M, int OUT_N>
__device__ __forceinline__ Tile decode_unit(int u, int total, int W, const int* tile_start,
                                            const int* seg, const int* cnt, int E) {
  int tau = u, half = -1;
  if (split_tail(total, W)) {
    const int r = total % W;
    if (u >= total - r) {
      const int h = u - (total - r);
      tau = total - r + (h >> 1);
      half = h & 1;
    }
  }
  int lo = 0, hi = E - 1;  // last e with tile_start[e] <= tau
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tile_start[mid] <= tau) lo = mid; else hi = mid - 1;
  }
  const int e = lo;
  const int m_e = cnt[e];
  const int mt_e = (m_e + TILE_M - 1) / TILE_M;
  const int local = tau - tile_start[e];
  const int nt = local / mt_e, mt = local - nt * mt_e;
  Tile t;
  t.e = e;
  t.row0 = seg[e] + mt * TILE_M;
  t.rows = min(TILE_M, m_e - mt * TILE_M);
  t.n0 = nt * OUT_N + (half > 0 ? OUT_N / 2 : 0);
  t.half = half >= 0;
  return t;
}

}  // namespace

}  // namespace moe
