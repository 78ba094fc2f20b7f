// adamw.cu -- one AdamW step over many tensors.
//
// Per element, with g the gradient times the caller's scale and n the step:
//   m = b1 m + (1 - b1) g          v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr (m / (1 - b1^n)) / (sqrt(v / (1 - b2^n)) + eps)
// in fp32; the bias corrections (1 - b^n cancels for b near 1) in fp64, once
// per block.
//
// States are fp32 (m, v) or 8 bits: m and r = sqrt(v) as E4M3 codes, one fp32
// scale amax / 448 per 256 elements of the tensor, the step itself taken from
// the fp32 values before they are rounded.  r rather than v is kept because
// E4M3 spans 2^17.8: v spans twice the binades that r does.  A positive r
// never gets the code of zero, so that no m is divided by eps alone.  Codes
// are rounded to nearest (at most 2^-4 relative); the scale is not a power of
// two, so that a block whose gradients stop decays by b every step although
// its codes stand still.
//
// Bound by the bytes of weights, gradients and states.  The tensors' addresses
// travel in the launch's parameters (no copy to the device, so a captured step
// replays as it is), a block takes units of ADAM_UNIT elements of the
// concatenated tensors, and the step count lives on the device: the last block
// to have read it moves it on.
#include "kernels.cuh"
#include "ptx.cuh"

#include <cuda_fp8.h>

namespace moezc {
namespace {

constexpr int ADAM_THREADS = 256;
constexpr int ADAM_WARPS = ADAM_THREADS / 32;
constexpr int ADAM_UNIT = ADAM_WARPS * ADAM_BLOCK;   // elements a block takes at a time

template <int MAXT>
struct AdamArgs {
  AdamTensor t[MAXT];
  int unit_end[MAXT];       // prefix sum of units, tensor by tensor
  int nt;
  int advance;              // 1: this launch moves the step count on
  AdamHyper h;
  int* step;                // [0] steps done, [1] blocks that have read it (zero between steps)
  const float* lr_scale;    // or nullptr
  const float* grad_scale;  // or nullptr
};

// 1 - b^n, in fp64 (repeated squaring).
__device__ __forceinline__ double one_minus_pow(double b, int n) {
  double r = 1.0;
  for (; n > 0; n >>= 1) {
    if (n & 1) r *= b;
    b *= b;
  }
  return 1.0 - r;
}

__device__ __forceinline__ void load8(float (&v)[8], const float* p) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(float (&v)[8], const __nv_bfloat16* p) {
  const uint4 q = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ void store8(const float (&v)[8], float* p) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(const float (&v)[8], __nv_bfloat16* p) {
  uint4 q;
  uint32_t* w = reinterpret_cast<uint32_t*>(&q);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = q;
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float x, float* p) { *p = x; }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16* p) { *p = __float2bfloat16_rn(x); }

// Eight consecutive elements at p, of which n (1..8) exist; the rest read 0.
template <typename E>
__device__ __forceinline__ void load_n(float (&v)[8], const E* p, int n) {
  if (n == 8) {
    load8(v, p);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f(p[i]) : 0.f;
  }
}
template <typename E>
__device__ __forceinline__ void store_n(const float (&v)[8], E* p, int n) {
  if (n == 8) {
    store8(v, p);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) from_f(v[i], p + i);
  }
}

// Eight E4M3 codes <-> values in units of their scale.
__device__ __forceinline__ void decode8(float (&v)[8], const uint2& q) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ uint2 encode8(const float (&v)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(
        make_float2(v[4 * i] * inv, v[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(v[4 * i + 2] * inv, v[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int n) {
  if (n == 8) return *reinterpret_cast<const uint2*>(p);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) w[i >> 2] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(const uint2& q, uint8_t* p, int n) {
  if (n == 8) {
    *reinterpret_cast<uint2*>(p) = q;
  } else {
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
  }
}

// Scale of a block from its largest magnitude (bits of a non-negative float,
// or of an infinity or NaN), and the factor to units of it.  A block holding
// an infinity or a NaN gets scale 1 (a NaN keeps the NaN code, an infinity
// saturates); the floor keeps 448 / amax finite.
__device__ __forceinline__ float block_scale(uint32_t amax_bits, float& inv) {
  if (amax_bits >= 0x7F800000u) {
    inv = 1.0f;
    return 1.0f;
  }
  const float a = fmaxf(__uint_as_float(amax_bits), 0x1p-100f);
  inv = __fdiv_rn(448.0f, a);
  return __fdiv_rn(a, 448.0f);
}

struct Coef {
  float b1, omb1, b2, omb2, eps, decay, step_size, rs, gscale;
};

__device__ __forceinline__ void adam8(float (&p)[8], const float (&g)[8], float (&m)[8],
                                      float (&v)[8], float (&r)[8], const Coef& c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float gi = g[i] * c.gscale;
    m[i] = fmaf(c.b1, m[i], c.omb1 * gi);
    v[i] = fmaf(c.b2, v[i], c.omb2 * (gi * gi));
    r[i] = sqrtf(v[i]);
    const float den = fmaf(r[i], c.rs, c.eps);
    p[i] = fmaf(p[i], c.decay, -c.step_size * (m[i] / den));
  }
}

template <typename PT, typename GT, bool MASTER, bool BITS8, int MAXT>
__global__ void __launch_bounds__(ADAM_THREADS)
adamw_kernel(const __grid_constant__ AdamArgs<MAXT> a) {
  __shared__ Coef coef_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  if (threadIdx.x == 0) {
    const int n = *reinterpret_cast<volatile int*>(a.step) + 1;
    const double lr = static_cast<double>(a.h.lr) * (a.lr_scale ? *a.lr_scale : 1.0f);
    Coef c;
    c.b1 = static_cast<float>(a.h.beta1);
    c.omb1 = static_cast<float>(1.0 - a.h.beta1);
    c.b2 = static_cast<float>(a.h.beta2);
    c.omb2 = static_cast<float>(1.0 - a.h.beta2);
    c.eps = static_cast<float>(a.h.eps);
    c.decay = static_cast<float>(1.0 - lr * a.h.weight_decay);
    c.step_size = static_cast<float>(lr / one_minus_pow(a.h.beta1, n));
    c.rs = static_cast<float>(rsqrt(one_minus_pow(a.h.beta2, n)));
    c.gscale = a.grad_scale ? *a.grad_scale : 1.0f;
    coef_s = c;
    if (a.advance) {
      __threadfence();   // the step count is read before this block counts itself
      if (atomicAdd(a.step + 1, 1) == static_cast<int>(gridDim.x) - 1) {
        a.step[1] = 0;
        a.step[0] = n;
      }
    }
  }
  __syncthreads();
  const Coef c = coef_s;
  const int units = a.unit_end[a.nt - 1];
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    int ti = 0;   // the first tensor whose units end after u
    for (int hi = a.nt - 1; ti < hi;) {
      const int mid = (ti + hi) >> 1;
      if (a.unit_end[mid] > u) hi = mid; else ti = mid + 1;
    }
    const AdamTensor& T = a.t[ti];
    const int u0 = ti ? a.unit_end[ti - 1] : 0;
    const int64_t blk = static_cast<int64_t>(u - u0) * ADAM_WARPS + warp;
    const int64_t e = blk * ADAM_BLOCK + lane * 8;
    const int64_t left = T.n - e;
    if (blk * ADAM_BLOCK >= T.n) continue;   // (whole warp)
    const int n = left >= 8 ? 8 : (left > 0 ? static_cast<int>(left) : 0);
    float p[8], g[8], m[8], v[8], r[8];
    PT* pp = static_cast<PT*>(T.p) + e;
    float* mp = T.master + e;
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = g[i] = m[i] = v[i] = 0.f;
    if (n > 0) {
      if (MASTER) load_n(p, mp, n); else load_n(p, pp, n);
      load_n(g, static_cast<const GT*>(T.g) + e, n);
      if (!BITS8) {
        load_n(m, static_cast<const float*>(T.m) + e, n);
        load_n(v, static_cast<const float*>(T.v) + e, n);
      } else {
        decode8(m, load_codes(static_cast<const uint8_t*>(T.m) + e, n));
        decode8(v, load_codes(static_cast<const uint8_t*>(T.v) + e, n));
        const float sm = T.ms[blk], sv = T.vs[blk];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          m[i] *= sm;
          v[i] *= sv;
          v[i] *= v[i];
        }
      }
    }
    adam8(p, g, m, v, r, c);
    if (n > 0) {
      if (MASTER) store_n(p, mp, n);
      store_n(p, pp, n);
      if (!BITS8) {
        store_n(m, static_cast<float*>(T.m) + e, n);
        store_n(v, static_cast<float*>(T.v) + e, n);
      }
    }
    if (BITS8) {
      uint32_t am = 0, ar = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) {
          am = max(am, __float_as_uint(m[i]) & 0x7FFFFFFFu);
          ar = max(ar, __float_as_uint(r[i]) & 0x7FFFFFFFu);
        }
      am = __reduce_max_sync(0xffffffffu, am);
      ar = __reduce_max_sync(0xffffffffu, ar);
      float im, ir;
      const float sm = block_scale(am, im), sr = block_scale(ar, ir);
      if (n > 0) {
        store_codes(encode8(m, im), static_cast<uint8_t*>(T.m) + e, n);
        uint2 q = encode8(r, ir);
        // a positive root never gets the code of zero
        uint32_t w[2] = {q.x, q.y};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (r[i] > 0.f && ((w[i >> 2] >> (8 * (i & 3))) & 0xFFu) == 0u)
            w[i >> 2] |= 1u << (8 * (i & 3));
        q = make_uint2(w[0], w[1]);
        store_codes(q, static_cast<uint8_t*>(T.v) + e, n);
      }
      if (lane == 0) {
        T.ms[blk] = sm;
        T.vs[blk] = sr;
      }
    }
  }
  griddep_launch_dependents();
}

template <typename PT, typename GT, bool MASTER, bool BITS8, int MAXT>
cudaError_t launch_some(const AdamTensor* t, int nt, bool advance, const AdamHyper& h, int* step,
                        const float* lr_scale, const float* grad_scale, cudaStream_t stream) {
  AdamArgs<MAXT> a;
  int64_t units = 0;
  for (int i = 0; i < nt; ++i) {
    a.t[i] = t[i];
    units += (t[i].n + ADAM_UNIT - 1) / ADAM_UNIT;
    if (units > 0x7fffffff) return cudaErrorInvalidValue;
    a.unit_end[i] = static_cast<int>(units);
  }
  a.nt = nt;
  a.advance = advance ? 1 : 0;
  a.h = h;
  a.step = step;
  a.lr_scale = lr_scale;
  a.grad_scale = grad_scale;
  constexpr auto kern = adamw_kernel<PT, GT, MASTER, BITS8, MAXT>;
  const int64_t cap = static_cast<int64_t>(device_sms()) * blocks_per_sm<kern>(ADAM_THREADS, 0);
  const int64_t grid = units < cap ? (units > 0 ? units : 1) : cap;
  return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(ADAM_THREADS), 0, stream, a);
}

// Tensors of one launch: as many as its parameters (32764 bytes at most) hold.
constexpr int ADAM_FEW = 16, ADAM_MANY = 448;
static_assert(sizeof(AdamArgs<ADAM_MANY>) <= 32764, "kernel parameters");

template <typename PT, typename GT, bool MASTER, bool BITS8>
cudaError_t launch_all(const AdamTensor* t, int nt, const AdamHyper& h, int* step,
                       const float* lr_scale, const float* grad_scale, cudaStream_t stream) {
  if (nt <= ADAM_FEW)
    return launch_some<PT, GT, MASTER, BITS8, ADAM_FEW>(t, nt, true, h, step, lr_scale, grad_scale,
                                                        stream);
  for (int i = 0; i < nt; i += ADAM_MANY) {
    const int k = nt - i < ADAM_MANY ? nt - i : ADAM_MANY;
    const cudaError_t e = launch_some<PT, GT, MASTER, BITS8, ADAM_MANY>(
        t + i, k, i + k == nt, h, step, lr_scale, grad_scale, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename PT, bool MASTER>
cudaError_t launch_typed(const AdamTensor* t, int nt, bool g_bf16, bool bits8, const AdamHyper& h,
                         int* step, const float* lr_scale, const float* grad_scale,
                         cudaStream_t stream) {
  if (g_bf16)
    return bits8 ? launch_all<PT, __nv_bfloat16, MASTER, true>(t, nt, h, step, lr_scale,
                                                               grad_scale, stream)
                 : launch_all<PT, __nv_bfloat16, MASTER, false>(t, nt, h, step, lr_scale,
                                                                grad_scale, stream);
  return bits8 ? launch_all<PT, float, MASTER, true>(t, nt, h, step, lr_scale, grad_scale, stream)
               : launch_all<PT, float, MASTER, false>(t, nt, h, step, lr_scale, grad_scale, stream);
}

}  // namespace

cudaError_t launch_adamw(const AdamTensor* t, int nt, bool p_bf16, bool g_bf16, bool master,
                         bool bits8, const AdamHyper& h, int* step, const float* lr_scale,
                         const float* grad_scale, cudaStream_t stream) {
  if (nt <= 0) return cudaSuccess;
  if (!p_bf16)
    return launch_typed<float, false>(t, nt, g_bf16, bits8, h, step, lr_scale, grad_scale, stream);
  if (master)
    return launch_typed<__nv_bfloat16, true>(t, nt, g_bf16, bits8, h, step, lr_scale, grad_scale,
                                             stream);
  return launch_typed<__nv_bfloat16, false>(t, nt, g_bf16, bits8, h, step, lr_scale, grad_scale,
                                            stream);
}

}  // namespace moezc
