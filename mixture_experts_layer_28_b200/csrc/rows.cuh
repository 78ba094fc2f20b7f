// rows.cuh -- one warp's access to a row of E fp32 logits, shared by the
// kernels with which the router learns (balance.cu).
//
// Lane l owns elements 4 l + 128 i + c (i < NV, c < 4), held as pairs: with
// E % 4 == 0 (all rows then start on 16 bytes) a row is read and written as
// 16-byte vectors, 512 contiguous bytes per warp instruction; otherwise element
// by element with the same ownership.
#pragma once

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>

#include "packed.cuh"
#include "ptx.cuh"

namespace moezc {

template <int NV>
struct Row {
  F2 v[NV][2];
  __device__ __forceinline__ void fill(float x) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i][0] = v[i][1] = both(x);
  }
};

// Elements past E read as `fill`.
template <int NV, bool VEC>
__device__ __forceinline__ void row_load(Row<NV>& r, const float* src, int E,
                                         int lane, float fill) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = 4 * lane + 128 * i;
    if (VEC) {
      float4 q = make_float4(fill, fill, fill, fill);
      if (j < E) q = *reinterpret_cast<const float4*>(src + j);
      r.v[i][0] = pk(q.x, q.y);
      r.v[i][1] = pk(q.z, q.w);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        r.v[i][h] = pk(j + 2 * h < E ? src[j + 2 * h] : fill,
                       j + 2 * h + 1 < E ? src[j + 2 * h + 1] : fill);
    }
  }
}

template <int NV, bool VEC>
__device__ __forceinline__ void row_store(const Row<NV>& r, float* __restrict__ dst, int E,
                                          int lane) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = 4 * lane + 128 * i;
    const float2 a = up(r.v[i][0]), b = up(r.v[i][1]);
    if (VEC) {
      if (j < E) __stcs(reinterpret_cast<float4*>(dst + j), make_float4(a.x, a.y, b.x, b.y));
    } else {
      if (j < E) dst[j] = a.x;
      if (j + 1 < E) dst[j + 1] = a.y;
      if (j + 2 < E) dst[j + 2] = b.x;
      if (j + 3 < E) dst[j + 3] = b.y;
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
    const __nv_bfloat162 a = __float22bfloat162_rn(up(r.v[i][0]));
    const __nv_bfloat162 b = __float22bfloat162_rn(up(r.v[i][1]));
    if (VEC) {
      if (j < E)
        __stcs(reinterpret_cast<uint2*>(dst + j), make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                                            *reinterpret_cast<const uint32_t*>(&b)));
    } else {
      if (j < E) dst[j] = a.x;
      if (j + 1 < E) dst[j + 1] = a.y;
      if (j + 2 < E) dst[j + 2] = b.x;
      if (j + 3 < E) dst[j + 3] = b.y;
    }
  }
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// Two sums at once.
__device__ __forceinline__ F2 warp_sum2(F2 x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = add2(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float warp_max(float x) {   // (a NaN is passed over)
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float ex2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The row's exponentials exp(l + offset - max), in place; offset may be
// nullptr.  Absent elements, loaded as -inf, and logits of -inf become 0; a row
// of nothing but -inf, or with a NaN or +inf, becomes NaN.  (2 to the power of
// (l - max) log2 e: 2^-22 and |l - max| 2^-24 relative, far inside the error of
// the sums taken of them.)
template <int NV, bool VEC>
__device__ __forceinline__ void row_exp(Row<NV>& r, const float* __restrict__ offset, int E,
                                        int lane) {
  if (offset) {
    Row<NV> o;
    row_load<NV, VEC>(o, offset, E, lane, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) r.v[i][h] = add2(r.v[i][h], o.v[i][h]);
  }
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 a = up(r.v[i][h]);
      mx = fmaxf(mx, fmaxf(a.x, a.y));
    }
  const F2 neg = both(-warp_max(mx)), log2e = both(1.4426950408889634f);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 x = up(mul2(add2(r.v[i][h], neg), log2e));
      r.v[i][h] = pk(ex2_approx(x.x), ex2_approx(x.y));
    }
}

// This lane's part of a row's sum.
template <int NV>
__device__ __forceinline__ float row_lane_sum(const Row<NV>& r) {
  F2 s = add2(r.v[0][0], r.v[0][1]);
#pragma unroll
  for (int i = 1; i < NV; ++i) s = add2(s, add2(r.v[i][0], r.v[i][1]));
  const float2 a = up(s);
  return a.x + a.y;
}

// A warp's rows on their way to it: a ring of DEPTH stages in shared memory,
// each a row and two arrays of up to 32 words, filled by asynchronous copies.
// Each lane reads back only what it copied itself, so waiting for its own
// copies is all the ordering there is, and DEPTH - 1 tokens are in flight
// without holding registers (a single row ahead in registers left each token
// waiting for most of a memory latency).
template <int NV, bool VEC>
struct RowRing {
  static constexpr int WORDS = NV * 128 + 64;       // of a stage
  static constexpr int DEPTH = NV >= 8 ? 2 : NV >= 6 ? 3 : NV >= 4 ? 4 : NV >= 3 ? 5 : 6;
  static constexpr int BYTES = DEPTH * WORDS * 4;   // per warp
  float* base;
  int put = 0, got = 0;   // stages of the next fetch and the next wait

  static __device__ __forceinline__ void copy4(float* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src)
                 : "memory");
  }
  // The row at src and, per lane < K, words of a and b (nullptr: none).  One
  // call a token (or `none`), in order.
  __device__ __forceinline__ void fetch(const float* src, const int* a, const float* b, int E,
                                        int K, int lane) {
    float* st = base + put * WORDS;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = 4 * lane + 128 * i;
      if (VEC) {
        if (j < E)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(st + j)),
                       "l"(src + j)
                       : "memory");
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (j + c < E) copy4(st + j + c, src + j + c);
      }
    }
    if (lane < K) {
      if (a) copy4(st + NV * 128 + lane, a + lane);
      if (b) copy4(st + NV * 128 + 32 + lane, b + lane);
    }
    none();
  }
  __device__ __forceinline__ void none() {
    asm volatile("cp.async.commit_group;" ::: "memory");
    put = put + 1 == DEPTH ? 0 : put + 1;
  }
  // Waits for the oldest token fetched, DEPTH - 1 others staying in flight, and
  // takes it: its row, and this lane's words.
  __device__ __forceinline__ void take(Row<NV>& r, int& a, float& b, int E, int lane) {
    asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
    const float* st = base + got * WORDS;
    row_load<NV, true>(r, st, VEC ? E : NV * 128, lane, -INFINITY);
    if (!VEC) row_cut(r, E, lane);
    a = reinterpret_cast<const int*>(st)[NV * 128 + lane];
    b = st[NV * 128 + 32 + lane];
    got = got + 1 == DEPTH ? 0 : got + 1;
  }
  // -inf past E, where a vector of four may cross it
  static __device__ __forceinline__ void row_cut(Row<NV>& r, int E, int lane) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = 4 * lane + 128 * i + 2 * h;
        const float2 a = up(r.v[i][h]);
        r.v[i][h] = pk(j < E ? a.x : -INFINITY, j + 1 < E ? a.y : -INFINITY);
      }
  }
};

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
