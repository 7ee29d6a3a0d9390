// Quantising to MXFP4 and reading back: expert weights, and token rows on
// their way to the experts (see mxfp4.cuh for the format and the layout of
// the scales).
//
// Weights [E, K, N] are stored along N but their blocks run along K, the
// dimension the products sum over, and the tensor cores want K contiguous:
// quantising transposes. Both directions stream the matrix once through
// registers, a 128 x 128 tile per block of threads, and are bound by DRAM.
#include "mxfp4.cuh"
#include <algorithm>
#include <type_traits>

namespace moe {

namespace {

template <typename T> struct Pair;  // two neighbouring columns
template <> struct Pair<__nv_bfloat16> {
  using Raw = uint32_t;
  static __device__ __forceinline__ float2 f32(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t raw(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <> struct Pair<float> {
  using Raw = float2;
  static __device__ __forceinline__ float2 f32(float2 v) { return v; }
  static __device__ __forceinline__ float2 raw(float a, float b) { return make_float2(a, b); }
};

constexpr int kWTile = 128;     // tile of K and of N
constexpr int kWThreads = 256;  // 64 column pairs x 4 blocks of 32 along K

// One 128 (K) x 128 (N) tile: a thread holds 32 k of two neighbouring columns,
// exactly one block of each, so that amax and codes need no other thread; a
// warp's loads are 64 columns of one k row. Codes and scales go through shared
// memory to leave as 64-byte row pieces and one 512-byte tile.
template <typename T>
__global__ void __launch_bounds__(kWThreads)
quantize_weights(const T* __restrict__ w, int K, int N, uint8_t* __restrict__ codes,
                 uint8_t* __restrict__ scales) {
  pdl_begin();
  __shared__ uint4 code_s[kWTile][5];  // 64 bytes a column, one vector of padding
  __shared__ __align__(16) uint8_t scale_s[kScaleTile];
  const int c = threadIdx.x & 63, kb = threadIdx.x >> 6;
  const int n0 = blockIdx.x * kWTile, k0 = blockIdx.y * kWTile;
  const long long e = blockIdx.z;
  const T* src = w + (static_cast<size_t>(e) * K + k0 + kb * 32) * N + n0 + 2 * c;
  typename Pair<T>::Raw raw[32];
#pragma unroll
  for (int i = 0; i < 32; ++i)
    raw[i] = __ldg(reinterpret_cast<const typename Pair<T>::Raw*>(src + static_cast<size_t>(i) * N));
  uint32_t top[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const float2 v = Pair<T>::f32(raw[i]);
    top[0] = max(top[0], __float_as_uint(v.x) & 0x7fffffffu);
    top[1] = max(top[1], __float_as_uint(v.y) & 0x7fffffffu);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = 2 * c + h;
    const uint32_t sb = mx_scale_byte(top[h]);
    const float inv = mx_inv_scale(sb);
    uint32_t q[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 p = Pair<T>::f32(raw[8 * g + i]);
        v[i] = (h == 0 ? p.x : p.y) * inv;
      }
      q[g] = sb == 255u ? 0u : e2m1x8(v);
    }
    code_s[n][kb] = make_uint4(q[0], q[1], q[2], q[3]);
    scale_s[(n & 31) * 16 + (n >> 5) * 4 + kb] = static_cast<uint8_t>(sb);
  }
  __syncthreads();
  uint8_t* dst = codes + (static_cast<size_t>(e) * N + n0) * (K / 2) + k0 / 2;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int u = threadIdx.x + i * kWThreads;  // 128 columns x 4 vectors
    *reinterpret_cast<uint4*>(dst + static_cast<size_t>(u >> 2) * (K / 2) + (u & 3) * 16) = code_s[u >> 2][u & 3];
  }
  if (threadIdx.x < kScaleTile / 16) {
    const long long group = e * (N / 128) + blockIdx.x;
    *reinterpret_cast<uint4*>(scales + mx_scale_at(group, K / 128, 0, 4 * blockIdx.y) + threadIdx.x * 16) =
        *reinterpret_cast<const uint4*>(scale_s + threadIdx.x * 16);
  }
}

template <typename T>
__global__ void __launch_bounds__(kWThreads)
dequantize_weights(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int K, int N,
                   T* __restrict__ w) {
  pdl_begin();
  __shared__ uint4 code_s[kWTile][5];
  __shared__ uint4 scale_s[kScaleTile / 16];
  const int c = threadIdx.x & 63, kb = threadIdx.x >> 6;
  const int n0 = blockIdx.x * kWTile, k0 = blockIdx.y * kWTile;
  const long long e = blockIdx.z;
  const uint8_t* src = codes + (static_cast<size_t>(e) * N + n0) * (K / 2) + k0 / 2;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int u = threadIdx.x + i * kWThreads;
    code_s[u >> 2][u & 3] =
        __ldg(reinterpret_cast<const uint4*>(src + static_cast<size_t>(u >> 2) * (K / 2) + (u & 3) * 16));
  }
  if (threadIdx.x < kScaleTile / 16) {
    const long long group = e * (N / 128) + blockIdx.x;
    scale_s[threadIdx.x] = __ldg(reinterpret_cast<const uint4*>(
        scales + mx_scale_at(group, K / 128, 0, 4 * blockIdx.y) + threadIdx.x * 16));
  }
  __syncthreads();
  float f[2];
  uint32_t q[2][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = 2 * c + h;
    f[h] = mx_scale(reinterpret_cast<const uint8_t*>(scale_s)[(n & 31) * 16 + (n >> 5) * 4 + kb]);
    const uint4 v = code_s[n][kb];
    q[h][0] = v.x; q[h][1] = v.y; q[h][2] = v.z; q[h][3] = v.w;
  }
  T* dst = w + (static_cast<size_t>(e) * K + k0 + kb * 32) * N + n0 + 2 * c;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    float a[8], b[8];
    e2m1x8_values(q[0][g], f[0], a);
    e2m1x8_values(q[1][g], f[1], b);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<typename Pair<T>::Raw*>(dst + static_cast<size_t>(8 * g + i) * N) = Pair<T>::raw(a[i], b[i]);
  }
}

// Eight consecutive values of a row: as loaded, as fp32, the fp32 bits of the
// largest magnitude.
template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
  struct Raw { uint4 u; };
  static __device__ __forceinline__ Raw load(const __nv_bfloat16* p) { return {__ldg(reinterpret_cast<const uint4*>(p))}; }
  static __device__ __forceinline__ Raw zero() { return {make_uint4(0, 0, 0, 0)}; }
  static __device__ __forceinline__ void f32(const Raw& r, float (&v)[8]) {
    const uint32_t x[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(x[i] << 16);
      v[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint32_t top(const Raw& r) {
    constexpr uint32_t m = 0x7fff7fffu;
    const uint32_t t = __vmaxu2(__vmaxu2(r.u.x & m, r.u.y & m), __vmaxu2(r.u.z & m, r.u.w & m));
    return max(t & 0xffff0000u, t << 16);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[8]) {
    using P = Pair<__nv_bfloat16>;
    *reinterpret_cast<uint4*>(p) = make_uint4(P::raw(v[0], v[1]), P::raw(v[2], v[3]), P::raw(v[4], v[5]), P::raw(v[6], v[7]));
  }
};
template <> struct Eight<float> {
  struct Raw { float4 a, b; };
  static __device__ __forceinline__ Raw load(const float* p) {
    return {__ldg(reinterpret_cast<const float4*>(p)), __ldg(reinterpret_cast<const float4*>(p) + 1)};
  }
  static __device__ __forceinline__ Raw zero() { return {make_float4(0, 0, 0, 0), make_float4(0, 0, 0, 0)}; }
  static __device__ __forceinline__ void f32(const Raw& r, float (&v)[8]) {
    v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
    v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
  }
  static __device__ __forceinline__ uint32_t top(const Raw& r) {
    float v[8];
    f32(r, v);
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = max(t, __float_as_uint(v[i]) & 0x7fffffffu);
    return t;
  }
  static __device__ __forceinline__ void store(float* p, const float (&v)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *(reinterpret_cast<float4*>(p) + 1) = make_float4(v[4], v[5], v[6], v[7]);
  }
};

constexpr int kRowWarps = 8;
constexpr int kRowIter = 8;                  // a unit: 8 x 256 values of one row (4: 8% slower at d = 4096, 2: 35%)
constexpr int kRowChunk = kRowIter * 256;
constexpr int kRowMaxE = 256;
constexpr int kGatherBlocksPerSm = 3;        // by registers

// Expert of row r: the last e with seg[e] <= r (empty experts share a start
// with the one that has the row). Valid for seg[0] <= r < seg[E].
__device__ __forceinline__ int row_expert(const int* seg, int E, int r) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (seg[mid] <= r) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The rows on their way to the experts: a warp takes 2048 values of one token,
// quantises them once and writes them to each of the token's rows. Four lanes
// hold a block (8 values a lane), so a block's largest magnitude is two
// shuffles away, and a lane's codes are one 4-byte store of a 128-byte run.
template <typename T>
__global__ void __launch_bounds__(kRowWarps * 32, kGatherBlocksPerSm)
gather_mxfp4(const T* __restrict__ x, int T_, int d, int k, const int32_t* __restrict__ slot_to_row,
             const int32_t* __restrict__ seg, int E, long long rows_max, uint8_t* __restrict__ codes,
             uint8_t* __restrict__ scales, Control* ctl) {
  pdl_begin();
  __shared__ int seg_s[kRowMaxE + 1];
  for (int i = threadIdx.x; i <= E; i += blockDim.x) seg_s[i] = __ldg(seg + i);
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const long long R = min(static_cast<long long>(seg_s[E]), rows_max);
  const int chunks = (d + kRowChunk - 1) / kRowChunk;
  const long long units = static_cast<long long>(T_) * chunks;
  const long long step = static_cast<long long>(gridDim.x) * kRowWarps;
  for (long long u = static_cast<long long>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5); u < units; u += step) {
    const long long t = u / chunks;
    const int c0 = static_cast<int>(u - t * chunks) * kRowChunk;
    // lane j: the token's j-th row
    const int row = lane < k ? __ldg(slot_to_row + t * k + lane) : -1;
    typename Eight<T>::Raw raw[kRowIter];  // all loads of the unit before the first use
#pragma unroll
    for (int i = 0; i < kRowIter; ++i) {
      const int col = c0 + i * 256 + lane * 8;
      raw[i] = col < d ? Eight<T>::load(x + static_cast<size_t>(t) * d + col) : Eight<T>::zero();
    }
    // where that row's codes and scales begin; -1: none
    long long code_at = -1, scale_at = 0;
    if (row >= 0) {
      const int e = row_expert(seg_s, E, row);
      const int rank = row - seg_s[e];
      if (row >= R || rank < 0 || seg_s[e] < 0) {  // out of range, or seg is not an ascending list from 0
        set_error(ctl, MOE_DEVERR_ROW_RANGE);
      } else {
        code_at = static_cast<long long>(row) * (d / 2);
        scale_at = static_cast<long long>(mx_scale_at(seg_s[e] / 128 + e + rank / 128, d / 128, rank & 127, 0));
      }
    }
    uint32_t q[kRowIter], sw[kRowIter];  // codes; scale bytes of the lane's four neighbouring blocks
#pragma unroll
    for (int i = 0; i < kRowIter; ++i) {
      uint32_t top = Eight<T>::top(raw[i]);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t sb = mx_scale_byte(top);
      const float inv = mx_inv_scale(sb);
      float v[8];
      Eight<T>::f32(raw[i], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= inv;
      q[i] = sb == 255u ? 0u : e2m1x8(v);
      sw[i] = sb << (8 * ((lane >> 2) & 3));
      sw[i] |= __shfl_xor_sync(0xffffffffu, sw[i], 4);
      sw[i] |= __shfl_xor_sync(0xffffffffu, sw[i], 8);
    }
    for (int j = 0; j < k; ++j) {
      const long long cj = __shfl_sync(0xffffffffu, code_at, j), sj = __shfl_sync(0xffffffffu, scale_at, j);
      if (cj < 0) continue;
      uint8_t* cdst = codes + cj + c0 / 2 + lane * 4;
      uint8_t* sdst = scales + sj + (c0 / 128 + (lane >> 4)) * kScaleTile;
#pragma unroll
      for (int i = 0; i < kRowIter; ++i) {
        if (c0 + i * 256 + lane * 8 >= d) continue;
        *reinterpret_cast<uint32_t*>(cdst + i * 128) = q[i];
        if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(sdst + i * 2 * kScaleTile) = sw[i];
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kRowWarps * 32)
dequantize_rows(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                const int32_t* __restrict__ seg, int E, long long rows_max, int K, T* __restrict__ out,
                Control* ctl) {
  pdl_begin();
  __shared__ int seg_s[kRowMaxE + 1];
  for (int i = threadIdx.x; i <= E; i += blockDim.x) seg_s[i] = __ldg(seg + i);
  __syncthreads();
  const int lane = threadIdx.x & 31;
  long long R = seg_s[E];
  if (R > rows_max || R < 0) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_error(ctl, MOE_DEVERR_ROW_RANGE);
    R = R < 0 ? 0 : rows_max;
  }
  const int chunks = (K + kRowChunk - 1) / kRowChunk;
  const long long units = R * chunks;
  const long long step = static_cast<long long>(gridDim.x) * kRowWarps;
  for (long long u = static_cast<long long>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5); u < units; u += step) {
    const int row = static_cast<int>(u / chunks);
    const int c0 = static_cast<int>(u - static_cast<long long>(row) * chunks) * kRowChunk;
    const int e = row_expert(seg_s, E, row);
    const int rank = row - seg_s[e];
    if (rank < 0 || seg_s[e] < 0) {
      if (lane == 0) set_error(ctl, MOE_DEVERR_ROW_RANGE);
      continue;
    }
    const long long group = seg_s[e] / 128 + e + rank / 128;
    uint32_t q[kRowIter], sb[kRowIter];
#pragma unroll
    for (int i = 0; i < kRowIter; ++i) {
      const int col = c0 + i * 256 + lane * 8;
      q[i] = sb[i] = 0;
      if (col < K) {
        q[i] = __ldg(reinterpret_cast<const uint32_t*>(codes + static_cast<size_t>(row) * (K / 2) + col / 2));
        sb[i] = __ldg(scales + mx_scale_at(group, K / 128, rank & 127, col / 32));
      }
    }
#pragma unroll
    for (int i = 0; i < kRowIter; ++i) {
      const int col = c0 + i * 256 + lane * 8;
      if (col >= K) continue;
      float v[8];
      e2m1x8_values(q[i], mx_scale(sb[i]), v);
      Eight<T>::store(out + static_cast<size_t>(row) * K + col, v);
    }
  }
}

// Blocks for so many units (a warp each): at most what is resident at once,
// since every block takes an equal share.
int row_grid(long long units, int per_sm) {
  return static_cast<int>(
      std::max<long long>(1, std::min<long long>((units + kRowWarps - 1) / kRowWarps, static_cast<long long>(per_sm) * num_sms())));
}

}  // namespace

cudaError_t launch_mxfp4_quantize_weights(const void* w, moe_dtype_t dt, int E, int K, int N,
                                          uint8_t* codes, uint8_t* scales, cudaStream_t s) {
  const dim3 grid(N / kWTile, K / kWTile, E);
  if (dt == MOE_BF16)
    return launch_pdl(quantize_weights<__nv_bfloat16>, grid, dim3(kWThreads), 0, s, false,
                      static_cast<const __nv_bfloat16*>(w), K, N, codes, scales);
  return launch_pdl(quantize_weights<float>, grid, dim3(kWThreads), 0, s, false,
                    static_cast<const float*>(w), K, N, codes, scales);
}

cudaError_t launch_mxfp4_dequantize_weights(const uint8_t* codes, const uint8_t* scales, moe_dtype_t dt,
                                            int E, int K, int N, void* w, cudaStream_t s) {
  const dim3 grid(N / kWTile, K / kWTile, E);
  if (dt == MOE_BF16)
    return launch_pdl(dequantize_weights<__nv_bfloat16>, grid, dim3(kWThreads), 0, s, false, codes, scales,
                      K, N, static_cast<__nv_bfloat16*>(w));
  return launch_pdl(dequantize_weights<float>, grid, dim3(kWThreads), 0, s, false, codes, scales, K, N,
                    static_cast<float*>(w));
}

cudaError_t launch_gather_mxfp4(const void* x, moe_dtype_t dt, int T, int d, int k,
                                const int32_t* slot_to_row, const int32_t* seg, int E, int64_t rows_max,
                                uint8_t* codes, uint8_t* scales, Control* ctl, cudaStream_t s) {
  if (T <= 0 || rows_max <= 0) return cudaSuccess;
  const int grid = row_grid(static_cast<long long>(T) * ((d + kRowChunk - 1) / kRowChunk), kGatherBlocksPerSm);
  if (dt == MOE_BF16)
    return launch_pdl(gather_mxfp4<__nv_bfloat16>, dim3(grid), dim3(kRowWarps * 32), 0, s, false,
                      static_cast<const __nv_bfloat16*>(x), T, d, k, slot_to_row, seg, E, rows_max, codes,
                      scales, ctl);
  return launch_pdl(gather_mxfp4<float>, dim3(grid), dim3(kRowWarps * 32), 0, s, false,
                    static_cast<const float*>(x), T, d, k, slot_to_row, seg, E, rows_max, codes, scales, ctl);
}

cudaError_t launch_mxfp4_dequantize_rows(const uint8_t* codes, const uint8_t* scales, const int32_t* seg,
                                         int E, int64_t rows_max, int K, moe_dtype_t dt, void* out,
                                         Control* ctl, cudaStream_t s) {
  if (rows_max <= 0) return cudaSuccess;
  const int grid = row_grid(rows_max * ((K + kRowChunk - 1) / kRowChunk), 8);
  if (dt == MOE_BF16)
    return launch_pdl(dequantize_rows<__nv_bfloat16>, dim3(grid), dim3(kRowWarps * 32), 0, s, false, codes,
                      scales, seg, E, rows_max, K, static_cast<__nv_bfloat16*>(out), ctl);
  return launch_pdl(dequantize_rows<float>, dim3(grid), dim3(kRowWarps * 32), 0, s, false, codes, scales, seg,
                    E, rows_max, K, static_cast<float*>(out), ctl);
}

}  // namespace moe
