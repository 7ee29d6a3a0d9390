// Shared by the MXFP4 grouped GEMMs: activations, the kind::mxf4 instructions
// and their descriptors, the list of tiles, tensor maps.
#pragma once
#include "gemm_common.cuh"
#include "mxfp4.cuh"
#include "ptx.cuh"
#include <cudaTypedefs.h>

namespace moe {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

struct MxArgs {
  const int32_t* seg;    // [E+1] row segment offsets
  const int32_t* kept;   // [E] rows of each expert from seg[e] (binned layout), or null
  uint8_t* out_codes;    // up projection: h codes [rows_max, N/2]
  uint8_t* out_scales;   // up projection: h scales
  __nv_bfloat16* out;    // down projection: [rows_max, N]
  int E;
  int d, F;  // the layer's
  int K;     // of one projection: what is summed over
  int N;     // of one projection: output columns
  int early;  // seg, kept and the weights were complete before the previous kernel on the stream began
  long long rows_max;
  float* partials;  // decode kernel: mxfp4_stream_partials_bytes()
  Control* ctl;
};

namespace {

constexpr int kBoxBytes = 128 * 128;  // 128 rows x 128 bytes (256 values of K)

enum { EPI_SWIGLU = 0, EPI_GELU = 1, EPI_STORE = 2 };

// Hardware exponential (base 2) and reciprocal, subnormals flushed: one
// instruction each, within a few ulp.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The up projection's activations. Their result is rounded to E2M1 with a scale
// of its block's own, so what counts is the error relative to the largest value
// of the block. A tile has up to 32768 of them, and they bound the kernel where K
// is short (with erff the epilogue of a 128 x 256 tile took 11500 cycles, the
// MMAs of K = 1024 2400).
//
// silu(g) = g / (1 + e^-g): for g < -126 ln 2 the reciprocal is subnormal or 0
// and the result -0 (its value is below 2^-119).
__device__ __forceinline__ float silu_fast(float g) { return g * rcp(1.0f + ex2(-1.44269504f * g)); }

// Two fp32 values in one 64-bit register pair, for the packed instructions (two
// results an issue slot).
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// gelu(z) = z Phi(z) = max(z, 0) - |z| Phi(-|z|). log2 Phi(-a) is nearly a
// parabola, and 2^p(a) with a polynomial p gives Phi(-a); its coefficients were
// found by linear programming, and both leave 0 beyond a = 13. Two values at a
// time.
//
// Phi, degree 5: the smallest largest error of Phi on [0, 6.5], 2.9e-7; in fp32
// gelu is within 3.7e-7 |z|. One special function (8 cycles) and six
// multiply-adds a value: with a reciprocal and eleven (Abramowitz and Stegun
// 7.1.28, 1.1e-6 |z|) an epilogue of 128 x 256 values took 5000 cycles, with both
// special functions (7.1.26) 6300. Relative to Phi(-a) it is within 8e-6 for a up
// to 2, 3e-5 to 2.5, 6e-5 to 3, but 6e-3 to 4 and 5e-2 to 5.
//
// PhiTail, degree 12: relative to Phi(-a), in fp32, within 1.7e-6 for a up to 3,
// 5.5e-6 to 6, 1.2e-5 to 8, 3.5e-5 to 10, 2.2e-4 to 13. For blocks of h that lie
// in the tail altogether. In all others (a value of at least 0.3, whose gelu is
// 0.18, or none below -2.5) what is below -2.9 has the code 0, since |gelu| is
// less than a 32nd of the block's largest: Phi is within 6e-5 of the rest.
struct Phi {
  static constexpr int N = 6;
  static __device__ __forceinline__ constexpr float c(int i) {
    constexpr float v[N] = {-1.0000008f, -1.1510831f, -0.45927668f, -0.052538015f, 0.0073872f, -0.0005188585f};
    return v[i];
  }
};
struct PhiTail {
  static constexpr int N = 13;
  static __device__ __forceinline__ constexpr float c(int i) {
    constexpr float v[N] = {-0.999998033f,    -1.15117109f,     -0.458849788f,   -0.0532412268f,  0.0078255767f,
                            -0.000555978215f, -6.54001778e-05f, 2.56033727e-05f, -3.80394295e-06f, 3.34066243e-07f,
                            -1.79620532e-08f, 5.47664081e-10f,  -7.26788898e-12f};
    return v[i];
  }
};

template <typename P>
__device__ __forceinline__ float2 gelu2(float z0, float z1) {
  const float a0 = fabsf(z0), a1 = fabsf(z1);
  const uint64_t a = pack2(a0, a1);
  uint64_t p = pack2(P::c(P::N - 1), P::c(P::N - 1));
#pragma unroll
  for (int i = P::N - 2; i >= 0; --i) p = fma2(p, a, pack2(P::c(i), P::c(i)));
  const float2 q = unpack2(p);
  return make_float2(fmaf(-a0, ex2(q.x), fmaxf(z0, 0.0f)), fmaf(-a1, ex2(q.y), fmaxf(z1, 0.0f)));
}

// Whether a block of h (32 values z of one row) needs PhiTail. Its second half
// is rarely reached.
__device__ __forceinline__ bool gelu_tail(const uint32_t (&z)[32]) {
  float low = __uint_as_float(z[0]);
#pragma unroll
  for (int i = 1; i < 31; i += 2)
    asm("min.f32 %0, %0, %1, %2;" : "+f"(low) : "f"(__uint_as_float(z[i])), "f"(__uint_as_float(z[i + 1])));
  if (fminf(low, __uint_as_float(z[31])) >= -2.5f) return false;
  float high = __uint_as_float(z[0]);
#pragma unroll
  for (int i = 1; i < 32; ++i) high = fmaxf(high, __uint_as_float(z[i]));
  return high < 0.3f;
}

// ------------------------------------------------------------ tcgen05, mxf4
// Instruction descriptor of kind::mxf4: E2M1 operands (1 at bits 7 and 10),
// both K-major, N / 8 at bit 17, scales UE8M0 (bit 23), M / 128 at bit 27; the
// ids of the scale bytes to use (0 or 2) go to bits 4 (B) and 29 (A).
// GROUP below: CTAs that issue together (cta_group).
__host__ __device__ constexpr uint32_t make_idesc_mxf4(int M, int N, uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(M >> 7) << 27) | (sf_id << 29);
}

// True in one thread of a converged warp, the same one every time. The tensor
// core's and TMA's instructions take warp-uniform operands: issued under this
// predicate from code that the whole warp runs they cost a few cycles each,
// from a branch that one lane took (lane == 0) about 80 (measured: a stage's
// eleven took 885 cycles, more than the MMAs themselves).
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}

template <int GROUP>
__device__ __forceinline__ void umma_mxf4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
  if constexpr (GROUP == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
}

// Descriptor of scale tiles at a shared-memory address: no swizzle, 32 rows of
// 16 bytes, 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t make_scale_desc(uint32_t smem_addr) {
  return static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(128 >> 4) << 32) |
         (static_cast<uint64_t>(1u) << 46);
}

// One 512-byte scale tile to 4 columns of tensor memory, replicated to the four
// 32-lane quarters (GROUP 2: of each CTA of the pair to its own).
template <int GROUP>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
  if constexpr (GROUP == 2)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

struct __align__(16) MxTile {
  int row0, rows, n0;
  int group;  // row group (of 128) of its first row's scales
  int e;
  int pad[3];
};

// The experts' row segments in shared memory, read once per block: every block
// wants the same few lines at the same time, and one L2 slice serves them (a
// read by every lane of every warp that needs them cost 3 us).
struct Segments {
  int seg[kMaxE + 1], kept[kMaxE];
};

// By `threads` threads; the caller orders the writes before the reads.
__device__ __forceinline__ void load_segments(Segments& s, const MxArgs& args, int thread, int threads) {
  for (int i = thread; i <= args.E; i += threads) {
    s.seg[i] = __ldcg(args.seg + i);
    if (args.kept != nullptr && i < args.E) s.kept[i] = __ldcg(args.kept + i);
  }
}

// The list of tiles, held by one warp: lane l has experts [8 l, 8 l + 8) with
// their first rows, row counts and first tiles. Tiles are ordered
// expert-major, then N tile, M tile fastest.
template <int TILE_M>
struct TileList {
  int seg[8], cnt[8], start[8];
  int total;

  // From the segment list in shared memory (see load_segments).
  __device__ __forceinline__ void build(const MxArgs& args, const Segments& in, int ntn, int lane) {
    int sum = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane * 8 + i;
      const bool there = e < args.E;
      seg[i] = there ? in.seg[e] : 0;
      const int end = there ? in.seg[e + 1] : 0;
      cnt[i] = !there ? 0 : args.kept != nullptr ? in.kept[e] : end - seg[i];
      // rows out of range are reported and their expert gets no tiles
      if (cnt[i] < 0 || seg[i] < 0 || static_cast<long long>(seg[i]) + cnt[i] > min(args.rows_max, static_cast<long long>(end))) {
        bad = true;
        cnt[i] = 0;
      }
      start[i] = ((cnt[i] + TILE_M - 1) / TILE_M) * ntn;
      sum += start[i];
    }
    if (bad) set_error(args.ctl, MOE_DEVERR_ROW_RANGE);
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += n;
    }
    total = __shfl_sync(0xffffffffu, incl, 31);
    int run = incl - sum;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int n = start[i];
      start[i] = run;
      run += n;
    }
  }

  // Tile u < total, by the whole warp.
  __device__ __forceinline__ MxTile tile(int u, int out_n, int lane) const {
    int s = -1, c = 0, st = 0, e = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (start[i] <= u) { s = seg[i]; c = cnt[i]; st = start[i]; e = lane * 8 + i; }
    // the last lane with an expert that starts at or before u
    const int src = 31 - __clz(__ballot_sync(0xffffffffu, s >= 0));
    s = __shfl_sync(0xffffffffu, s, src);
    c = __shfl_sync(0xffffffffu, c, src);
    st = __shfl_sync(0xffffffffu, st, src);
    MxTile t;
    t.e = __shfl_sync(0xffffffffu, e, src);
    const int mt_e = (c + TILE_M - 1) / TILE_M;
    const int local = u - st;
    const int nt = local / mt_e, mt = local - nt * mt_e;
    t.row0 = s + mt * TILE_M;
    t.rows = min(TILE_M, c - mt * TILE_M);
    t.n0 = nt * out_n;
    t.group = s / 128 + t.e + mt * (TILE_M / 128);
    return t;
  }
};

// Codes [rows, cols / 2 bytes], box 128 bytes x box_rows, 128-byte swizzle.
inline bool make_tma_codes(CUtensorMap* m, const void* base, uint64_t rows, uint64_t row_bytes, uint32_t box_rows) {
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

// Scale tiles [tiles, 512 bytes], box two tiles.
inline bool make_tma_scales(CUtensorMap* m, const void* base, uint64_t tiles) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {kScaleTile / 4, tiles};
  cuuint64_t strides[1] = {kScaleTile};
  cuuint32_t box[2] = {kScaleTile / 4, 2};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace

// Both projections for at most kMxStreamRows rows (gemm_mxfp4_stream.cu).
cudaError_t launch_stream_ffn_mxfp4(const MxRows& x, const MxWeights& w1, const MxWeights& w3, const MxWeights& w2,
                                    moe_act_t act, const MxRows& h, const MxArgs& args, cudaStream_t s);

}  // namespace moe
