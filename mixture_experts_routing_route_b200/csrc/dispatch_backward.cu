// Backward passes of the combine and of the gather: the gradients of the
// rows' way to the experts and back.
//
// combine: out[t] = sum_j w[t,j] y[row(t,j)] over the kept slots, so
//   dy[row(t,j)] = w[t,j] dout[t]
//   dw[t,j]      = <dout[t], y[row(t,j)]>   (0 for a dropped slot)
// gather: x_perm[r] = x[token of r], so
//   dx[t] = dx_in[t] + sum_j dx_perm[row(t,j)]
//
// Every output element is written once, by one thread, and every sum runs in
// fp32 in a fixed order (no atomics): the results are the same bit for bit
// from call to call.
#include "common.cuh"
#include <algorithm>

namespace moe {

namespace {

// 16-byte vectors as fp32 values, and back (rounded to nearest).
template <typename T>
struct Vec;
template <> struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&a)[N]) {
    const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[2 * i] = __uint_as_float(v[i] << 16);
      a[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&a)[N]) {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(a[2 * i], a[2 * i + 1]);
      v[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
  }
};
template <> struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&a)[N]) {
    a[0] = __uint_as_float(u.x);
    a[1] = __uint_as_float(u.y);
    a[2] = __uint_as_float(u.z);
    a[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&a)[N]) {
    return make_uint4(__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(a[2]),
                      __float_as_uint(a[3]));
  }
};

__device__ __forceinline__ float warp_sum_f32(float v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// A warp per slot: it reads the slot's expert row and its token's gradient
// row, writes the row's gradient and reduces the dot product. The k slots of
// a token are neighbouring warps, so the token's gradient row comes from DRAM
// once and from L1/L2 for the others.
constexpr int kSlotWarps = 8;
constexpr int kSlotVec = 4;  // vectors of each row in flight per lane

template <typename T>
__global__ void __launch_bounds__(kSlotWarps * 32)
combine_bwd(const T* __restrict__ dout, const T* __restrict__ y, const float* __restrict__ w,
            const int32_t* __restrict__ slot_to_row, long long slots, int d, int k,
            long long rows_max, T* __restrict__ dy, float* __restrict__ dw, Control* ctl) {
  pdl_begin();
  using V = Vec<T>;
  const int lane = threadIdx.x & 31;
  const int nvec = d / V::N;
  const long long step = static_cast<long long>(gridDim.x) * kSlotWarps;
  for (long long s = static_cast<long long>(blockIdx.x) * kSlotWarps + (threadIdx.x >> 5); s < slots;
       s += step) {
    const int row = __ldg(slot_to_row + s);
    if (row < 0 || row >= rows_max) {
      if (lane == 0) {
        if (row >= rows_max) set_error(ctl, MOE_DEVERR_ROW_RANGE);
        if (dw != nullptr) dw[s] = 0.f;
      }
      continue;
    }
    const float ws = dy != nullptr ? __ldg(w + s) : 0.f;
    const uint4* g = reinterpret_cast<const uint4*>(dout + static_cast<size_t>(s / k) * d);
    const uint4* src = reinterpret_cast<const uint4*>(y + static_cast<size_t>(row) * d);
    uint4* dst = reinterpret_cast<uint4*>(dy + static_cast<size_t>(row) * d);
    float dot = 0.f;
    for (int base = 0; base < nvec; base += 32 * kSlotVec) {
      uint4 gv[kSlotVec], yv[kSlotVec];
#pragma unroll
      for (int i = 0; i < kSlotVec; ++i) {
        const int j = base + i * 32 + lane;
        gv[i] = j < nvec ? __ldg(g + j) : make_uint4(0, 0, 0, 0);
        yv[i] = dw != nullptr && j < nvec ? __ldg(src + j) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < kSlotVec; ++i) {
        const int j = base + i * 32 + lane;
        float ga[V::N], ya[V::N];
        V::unpack(gv[i], ga);
        V::unpack(yv[i], ya);
#pragma unroll
        for (int c = 0; c < V::N; ++c) {
          dot = fmaf(ga[c], ya[c], dot);
          ga[c] *= ws;
        }
        if (dy != nullptr && j < nvec) dst[j] = V::pack(ga);
      }
    }
    if (dw != nullptr) {
      dot = warp_sum_f32(dot);
      if (lane == 0) dw[s] = dot;
    }
  }
}

// A thread owns two 16-byte column vectors of one token and requests its K
// rows of both before it adds them (dx_in first, then j ascending; dx may be
// dx_in: a thread reads what it writes before it writes it). A token
// takes tpt threads; a block takes whole tokens when tpt fits it, otherwise a
// token spreads over grid.y.
constexpr int kSumThreads = 128;

template <typename T, int K>
__global__ void __launch_bounds__(kSumThreads)
gather_bwd(const T* __restrict__ rows_g, const int32_t* __restrict__ slot_to_row,
           const T* dx_in, int T_, int d, int tpt, long long rows_max, T* dx, Control* ctl) {
  pdl_begin();
  using V = Vec<T>;
  constexpr int NV = 2;
  int t, v0, vstride;
  if (tpt <= kSumThreads) {
    const int tpb = kSumThreads / tpt;
    const int local = threadIdx.x / tpt;
    if (local >= tpb) return;
    t = blockIdx.x * tpb + local;
    v0 = threadIdx.x - local * tpt;
    vstride = tpt;
  } else {
    t = blockIdx.x;
    v0 = blockIdx.y * kSumThreads * NV + threadIdx.x;
    vstride = kSumThreads;
  }
  const int nvec = d / V::N;
  if (t >= T_ || v0 >= nvec) return;
  int rows[K];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    rows[j] = __ldg(slot_to_row + static_cast<size_t>(t) * K + j);
    if (rows[j] >= rows_max) {
      if (v0 == 0) set_error(ctl, MOE_DEVERR_ROW_RANGE);
      rows[j] = -1;
    }
  }
  uint4 in[NV], u[K][NV];
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int v = v0 + c * vstride;
    in[c] = make_uint4(0, 0, 0, 0);
    if (dx_in != nullptr && v < nvec)
      in[c] = *(reinterpret_cast<const uint4*>(dx_in + static_cast<size_t>(t) * d) + v);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      u[j][c] = make_uint4(0, 0, 0, 0);
      if (rows[j] >= 0 && v < nvec)
        u[j][c] = __ldg(reinterpret_cast<const uint4*>(rows_g + static_cast<size_t>(rows[j]) * d) + v);
    }
  }
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int v = v0 + c * vstride;
    if (v >= nvec) continue;
    float acc[V::N];
    V::unpack(in[c], acc);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (rows[j] < 0) continue;
      float a[V::N];
      V::unpack(u[j][c], a);
#pragma unroll
      for (int i = 0; i < V::N; ++i) acc[i] += a[i];
    }
    *(reinterpret_cast<uint4*>(dx + static_cast<size_t>(t) * d) + v) = V::pack(acc);
  }
}

template <typename T>
cudaError_t launch_combine_bwd_t(const void* dout, const void* y, const float* w, const int32_t* s2r,
                                 int T_, int d, int k, long long rows_max, void* dy, float* dw,
                                 Control* ctl, cudaStream_t s) {
  const long long slots = static_cast<long long>(T_) * k;
  const int grid = static_cast<int>(
      std::min<long long>((slots + kSlotWarps - 1) / kSlotWarps, 8LL * num_sms()));
  return launch_pdl(combine_bwd<T>, dim3(grid), dim3(kSlotWarps * 32), 0, s, false,
                    static_cast<const T*>(dout), static_cast<const T*>(y), w, s2r, slots, d, k,
                    rows_max, static_cast<T*>(dy), dw, ctl);
}

template <typename T>
cudaError_t launch_gather_bwd_t(const void* rows_g, const int32_t* s2r, const void* dx_in, int T_,
                                int d, int k, long long rows_max, void* dx, Control* ctl,
                                cudaStream_t s) {
  const int nvec = d / Vec<T>::N;
  const int tpt = (nvec + 1) / 2;  // threads per token, two vectors each
  const dim3 grid = tpt <= kSumThreads
                        ? dim3((T_ + kSumThreads / tpt - 1) / (kSumThreads / tpt), 1)
                        : dim3(T_, (nvec + kSumThreads * 2 - 1) / (kSumThreads * 2));
  auto kern = gather_bwd<T, 1>;
  switch (k) {
    case 2: kern = gather_bwd<T, 2>; break;
    case 3: kern = gather_bwd<T, 3>; break;
    case 4: kern = gather_bwd<T, 4>; break;
    case 5: kern = gather_bwd<T, 5>; break;
    case 6: kern = gather_bwd<T, 6>; break;
    case 7: kern = gather_bwd<T, 7>; break;
    case 8: kern = gather_bwd<T, 8>; break;
    default: break;
  }
  return launch_pdl(kern, grid, dim3(kSumThreads), 0, s, false, static_cast<const T*>(rows_g), s2r,
                    static_cast<const T*>(dx_in), T_, d, tpt, rows_max, static_cast<T*>(dx), ctl);
}

}  // namespace

cudaError_t launch_combine_backward(const void* dout, const void* y, const float* w,
                                    const int32_t* slot_to_row, size_t elem, int T, int d, int k,
                                    int64_t rows_max, void* dy, float* dw, Control* ctl,
                                    cudaStream_t s) {
  if (T <= 0 || (dy == nullptr && dw == nullptr)) return cudaSuccess;
  if (elem == 2)
    return launch_combine_bwd_t<__nv_bfloat16>(dout, y, w, slot_to_row, T, d, k, rows_max, dy, dw,
                                               ctl, s);
  return launch_combine_bwd_t<float>(dout, y, w, slot_to_row, T, d, k, rows_max, dy, dw, ctl, s);
}

cudaError_t launch_gather_backward(const void* dx_perm, const int32_t* slot_to_row,
                                   const void* dx_in, size_t elem, int T, int d, int k,
                                   int64_t rows_max, void* dx, Control* ctl, cudaStream_t s) {
  if (T <= 0) return cudaSuccess;
  if (elem == 2)
    return launch_gather_bwd_t<__nv_bfloat16>(dx_perm, slot_to_row, dx_in, T, d, k, rows_max, dx, ctl, s);
  return launch_gather_bwd_t<float>(dx_perm, slot_to_row, dx_in, T, d, k, rows_max, dx, ctl, s);
}

}  // namespace moe
