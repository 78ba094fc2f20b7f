// rows.cuh -- one warp's access to a row of E fp32 logits, shared by the
// kernels with which the router learns (balance.cu).
//
// Lane l owns elements 4 l + 128 i + c (i < NV, c < 4): with E % 4 == 0 (all
// rows then start on 16 bytes) a row is read and written as 16-byte vectors,
// 512 contiguous bytes per warp instruction; otherwise element by element
// with the same ownership.
#pragma once

#include <cfloat>
#include <cstdint>
#include <cuda_bf16.h>

namespace moezc {

constexpr int ROW_MAX_NV = 8;   // 128 * 8 = 1024 logits

template <int NV>
struct Row {
  float v[NV][4];
};

template <int NV, bool VEC>
__device__ __forceinline__ void row_load(Row<NV>& r, const float* __restrict__ src, int E,
                                         int lane, float fill) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = 4 * lane + 128 * i;
    if (VEC) {
      float4 q = make_float4(fill, fill, fill, fill);
      if (j < E) q = *reinterpret_cast<const float4*>(src + j);
      r.v[i][0] = q.x; r.v[i][1] = q.y; r.v[i][2] = q.z; r.v[i][3] = q.w;
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) r.v[i][c] = j + c < E ? src[j + c] : fill;
    }
  }
}

template <int NV, bool VEC>
__device__ __forceinline__ void row_store(const Row<NV>& r, float* __restrict__ dst, int E,
                                          int lane) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = 4 * lane + 128 * i;
    if (VEC) {
      if (j < E)
        *reinterpret_cast<float4*>(dst + j) =
            make_float4(r.v[i][0], r.v[i][1], r.v[i][2], r.v[i][3]);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (j + c < E) dst[j + c] = r.v[i][c];
    }
  }
}

// Rounded once to bf16 (nearest, ties to even).
template <int NV, bool VEC>
__device__ __forceinline__ void row_store(const Row<NV>& r, __nv_bfloat16* __restrict__ dst,
                                          int E, int lane) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = 4 * lane + 128 * i;
    if (VEC) {
      if (j < E) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(r.v[i][0], r.v[i][1]);
        const __nv_bfloat162 b = __floats2bfloat162_rn(r.v[i][2], r.v[i][3]);
        uint2 q;
        q.x = *reinterpret_cast<const uint32_t*>(&a);
        q.y = *reinterpret_cast<const uint32_t*>(&b);
        *reinterpret_cast<uint2*>(dst + j) = q;
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (j + c < E) dst[j + c] = __float2bfloat16_rn(r.v[i][c]);
    }
  }
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Softmax of the row in place (absent elements, loaded as -FLT_MAX, get 0):
// p = exp(l - max) / sum, fp32.  offset (or nullptr) is added first.
template <int NV, bool VEC>
__device__ __forceinline__ void row_softmax(Row<NV>& r, const float* __restrict__ offset, int E,
                                            int lane) {
  if (offset) {
    Row<NV> o;
    row_load<NV, VEC>(o, offset, E, lane, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) r.v[i][c] += o.v[i][c];
  }
  float mx = -FLT_MAX;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) mx = fmaxf(mx, r.v[i][c]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int j = 4 * lane + 128 * i + c;
      r.v[i][c] = j < E ? expf(r.v[i][c] - mx) : 0.f;
      sum += r.v[i][c];
    }
  const float inv = 1.0f / warp_sum(sum);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) r.v[i][c] *= inv;
}

// Calls f with integral constants (vectors per lane, whether rows are read as
// 16-byte vectors) for rows of E elements.
template <int V>
struct IntC {
  static constexpr int value = V;
};
template <typename F>
inline auto with_row_shape(int E, F&& f) {
  const bool vec = E % 4 == 0;
#define MOEZC_ROW(NV)                          \
  if (E <= 128 * (NV))                         \
    return vec ? f(IntC<NV>{}, IntC<1>{}) : f(IntC<NV>{}, IntC<0>{});
  MOEZC_ROW(1)
  MOEZC_ROW(2)
  MOEZC_ROW(3)
  MOEZC_ROW(4)
  MOEZC_ROW(6)
#undef MOEZC_ROW
  return vec ? f(IntC<8>{}, IntC<1>{}) : f(IntC<8>{}, IntC<0>{});
}

}  // namespace moezc
