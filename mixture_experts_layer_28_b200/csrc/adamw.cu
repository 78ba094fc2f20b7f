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

#include <type_traits>

namespace moezc {
namespace {

constexpr int ADAM_THREADS = 256;
constexpr int ADAM_WARPS = ADAM_THREADS / 32;
constexpr int ADAM_GROUPS = 2;   // 256-element groups (8 a lane) a warp has in flight
constexpr int ADAM_WARP_ELEMS = ADAM_GROUPS * ADAM_BLOCK;
constexpr int ADAM_UNIT = ADAM_WARPS * ADAM_WARP_ELEMS;   // elements a block takes at a time
static_assert(ADAM_BLOCK == 256, "one scale per 8 elements of each lane of a warp");

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

// Pairs of fp32 values in one 64-bit register: the packed instructions round
// each half like their scalar forms and take one issue slot for both, which is
// what the 8-bit step is short of (DRAM feeds 2.3 elements per clock and SM,
// 55 scalar issue slots each).
using F2 = unsigned long long;
__device__ __forceinline__ F2 pk(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 up(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// 1 / x to about an ulp, for normal x.
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Maximum that keeps a NaN (as the largest bits).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Eight consecutive elements as they sit in memory, loaded (the first n of
// them, the rest zero; FULL: all eight) before anything is computed from them.
template <typename E>
struct Raw8;
template <>
struct Raw8<float> {
  float4 a, b;
  template <bool FULL>
  __device__ __forceinline__ void load(const float* p, int n) {
    if (FULL) {
      a = __ldcs(reinterpret_cast<const float4*>(p));
      b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    } else {
      a = make_float4(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f,
                      n > 3 ? p[3] : 0.f);
      b = make_float4(n > 4 ? p[4] : 0.f, n > 5 ? p[5] : 0.f, n > 6 ? p[6] : 0.f,
                      n > 7 ? p[7] : 0.f);
    }
  }
  __device__ __forceinline__ void get(F2 (&v)[4]) const {
    v[0] = pk(a.x, a.y); v[1] = pk(a.z, a.w);
    v[2] = pk(b.x, b.y); v[3] = pk(b.z, b.w);
  }
};
template <>
struct Raw8<__nv_bfloat16> {
  uint4 q;
  template <bool FULL>
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int n) {
    if (FULL) {
      q = __ldcs(reinterpret_cast<const uint4*>(p));
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) w[i >> 1] |= static_cast<uint32_t>(h[i]) << (16 * (i & 1));
      q = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  __device__ __forceinline__ void get(F2 (&v)[4]) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pk(bf16_lo(w[i]), bf16_hi(w[i]));
  }
};
// Eight E4M3 codes (get: in units of their scale).
template <>
struct Raw8<uint8_t> {
  uint2 q;
  template <bool FULL>
  __device__ __forceinline__ void load(const uint8_t* p, int n) {
    if (FULL) {
      q = __ldcs(reinterpret_cast<const uint2*>(p));
    } else {
      uint32_t w[2] = {0u, 0u};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) w[i >> 2] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
      q = make_uint2(w[0], w[1]);
    }
  }
  __device__ __forceinline__ void get(F2 (&v)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = i < 2 ? q.x : q.y;
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
          static_cast<__nv_fp8x2_storage_t>(w >> (16 * (i & 1))), __NV_E4M3);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      v[i] = pk(f.x, f.y);
    }
  }
};

template <bool FULL>
__device__ __forceinline__ void put8(const F2 (&v)[4], float* p, int n) {
  const float2 a = up(v[0]), b = up(v[1]), c = up(v[2]), d = up(v[3]);
  if (FULL) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(a.x, a.y, b.x, b.y));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(c.x, c.y, d.x, d.y));
  } else {
    const float f[8] = {a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = f[i];
  }
}
template <bool FULL>
__device__ __forceinline__ void put8(const F2 (&v)[4], __nv_bfloat16* p, int n) {
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __float22bfloat162_rn(up(v[i]));
  if (FULL) {
    __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(h));
  } else {
    const __nv_bfloat16* e = reinterpret_cast<const __nv_bfloat16*>(h);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = e[i];
  }
}
// Codes of values in units of their scale (|v| <= 448 up to rounding).
template <bool FULL>
__device__ __forceinline__ void put8(const F2 (&v)[4], uint8_t* p, int n) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(up(v[2 * i]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(up(v[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  if (FULL) {
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
  } else {
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
  const bool finite = amax_bits < 0x7F800000u;
  const float a = finite ? fmaxf(__uint_as_float(amax_bits), 0x1p-100f) : 448.0f;
  inv = finite ? __fmul_rn(__frcp_rn(a), 448.0f) : 1.0f;
  return finite ? __fmul_rn(a, 1.0f / 448.0f) : 1.0f;
}

struct Coef {
  F2 b1, omb1, b2, omb2, eps, decay, neg_step, rs, gscale;
};

// m, v and p of eight elements; r = sqrt(v).  m and v are rounded product by
// product (no contraction): they decide codes, which a reference in plain
// fp32 operations then shares.  The step's quotient is an approximation to an
// ulp or two: the weight moves by a small part of itself.
__device__ __forceinline__ void adam8(F2 (&p)[4], const F2 (&g)[4], F2 (&m)[4], F2 (&v)[4],
                                      F2 (&r)[4], const Coef& c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const F2 gi = mul2(g[i], c.gscale);
    m[i] = add2(mul2(m[i], c.b1), mul2(gi, c.omb1));
    v[i] = add2(mul2(v[i], c.b2), mul2(mul2(gi, gi), c.omb2));
    const float2 vi = up(v[i]);
    r[i] = pk(__fsqrt_rn(vi.x), __fsqrt_rn(vi.y));
    const float2 den = up(fma2(r[i], c.rs, c.eps));
    const F2 q = mul2(m[i], pk(rcp_approx(den.x), rcp_approx(den.y)));
    p[i] = fma2(q, c.neg_step, mul2(p[i], c.decay));
  }
}

// One warp's ADAM_GROUPS groups of a tensor from element e0 (a multiple of
// ADAM_BLOCK) on.  FULL: all of them lie inside the tensor.
template <typename PT, typename GT, bool MASTER, bool BITS8, bool FULL>
__device__ __forceinline__ void adam_warp(const AdamTensor& T, int64_t e0, int lane,
                                          const Coef& c) {
  using WT = typename std::conditional<MASTER, float, PT>::type;   // the weight stepped on
  using ST = typename std::conditional<BITS8, uint8_t, float>::type;
  WT* w = (MASTER ? reinterpret_cast<WT*>(T.master) : static_cast<WT*>(T.p)) + e0 + 8 * lane;
  PT* pp = static_cast<PT*>(T.p) + e0 + 8 * lane;
  const GT* gp = static_cast<const GT*>(T.g) + e0 + 8 * lane;
  ST* mp = static_cast<ST*>(T.m) + e0 + 8 * lane;
  ST* vp = static_cast<ST*>(T.v) + e0 + 8 * lane;
  const int64_t b0 = e0 / ADAM_BLOCK;
  Raw8<WT> rp[ADAM_GROUPS];
  Raw8<GT> rg[ADAM_GROUPS];
  Raw8<ST> rm[ADAM_GROUPS], rv[ADAM_GROUPS];
  float sm[ADAM_GROUPS], sv[ADAM_GROUPS];
  int n[ADAM_GROUPS];        // this lane's elements of the group
  bool there[ADAM_GROUPS];   // the group has any (uniform)
#pragma unroll
  for (int k = 0; k < ADAM_GROUPS; ++k) {
    const int o = k * ADAM_BLOCK;
    const int64_t left = FULL ? 8 : T.n - (e0 + o + 8 * lane);
    n[k] = left >= 8 ? 8 : (left > 0 ? static_cast<int>(left) : 0);
    there[k] = FULL || e0 + o < T.n;
    rp[k].template load<FULL>(w + o, n[k]);
    rg[k].template load<FULL>(gp + o, n[k]);
    rm[k].template load<FULL>(mp + o, n[k]);
    rv[k].template load<FULL>(vp + o, n[k]);
    if (BITS8) {
      sm[k] = there[k] ? T.ms[b0 + k] : 0.f;
      sv[k] = there[k] ? T.vs[b0 + k] : 0.f;
    }
  }
#pragma unroll
  for (int k = 0; k < ADAM_GROUPS; ++k) {
    const int o = k * ADAM_BLOCK;
    if (!there[k]) break;
    F2 p[4], g[4], m[4], v[4], r[4];
    rp[k].get(p);
    rg[k].get(g);
    rm[k].get(m);
    rv[k].get(v);
    if (BITS8) {
      const F2 s2 = pk(sm[k], sm[k]), t2 = pk(sv[k], sv[k]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[i] = mul2(m[i], s2);
        v[i] = mul2(v[i], t2);
        v[i] = mul2(v[i], v[i]);
      }
    }
    adam8(p, g, m, v, r, c);
    if (MASTER) put8<FULL>(p, w + o, n[k]);
    put8<FULL>(p, pp + o, n[k]);
    if constexpr (!BITS8) {
      put8<FULL>(m, mp + o, n[k]);
      put8<FULL>(v, vp + o, n[k]);
    } else {
      // (elements past the tensor's end are zero: their m and r stay zero)
      float fm = 0.f, fr = 0.f, low = 0x1p+120f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 a = up(m[i]), b = up(r[i]);
        fm = max_nan(max_nan(fm, fabsf(a.x)), fabsf(a.y));
        fr = max_nan(max_nan(fr, b.x), b.y);
        low = fminf(fminf(low, b.x), b.y);
      }
      float im, ir;
      const float nm = block_scale(__reduce_max_sync(0xffffffffu, __float_as_uint(fm)), im);
      const float nr = block_scale(__reduce_max_sync(0xffffffffu, __float_as_uint(fr)), ir);
      const F2 im2 = pk(im, im), ir2 = pk(ir, ir);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[i] = mul2(m[i], im2);
        r[i] = mul2(r[i], ir2);
      }
      // a positive root never gets the code of zero (few blocks span that much)
      if (low * ir < 0x1p-9f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 b = up(r[i]);
          b.x = b.x > 0.f ? fmaxf(b.x, 0x1p-9f) : b.x;
          b.y = b.y > 0.f ? fmaxf(b.y, 0x1p-9f) : b.y;
          r[i] = pk(b.x, b.y);
        }
      }
      put8<FULL>(m, mp + o, n[k]);
      put8<FULL>(r, vp + o, n[k]);
      if (lane == 0) {
        T.ms[b0 + k] = nm;
        T.vs[b0 + k] = nr;
      }
    }
  }
}

__device__ __forceinline__ F2 both(double x) {
  const float f = static_cast<float>(x);
  return pk(f, f);
}

template <typename PT, typename GT, bool MASTER, bool BITS8, int MAXT>
__global__ void __launch_bounds__(ADAM_THREADS)
adamw_kernel(const __grid_constant__ AdamArgs<MAXT> a) {
  __shared__ Coef coef_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  if (threadIdx.x == 0) {
    const int n = *reinterpret_cast<volatile int*>(a.step) + 1;
    const double lr = a.h.lr * (a.lr_scale ? *a.lr_scale : 1.0f);
    Coef c;
    c.b1 = both(a.h.beta1);
    c.omb1 = both(1.0 - a.h.beta1);
    c.b2 = both(a.h.beta2);
    c.omb2 = both(1.0 - a.h.beta2);
    c.eps = both(a.h.eps);
    c.decay = both(1.0 - lr * a.h.weight_decay);
    c.neg_step = both(-lr / one_minus_pow(a.h.beta1, n));
    c.rs = both(rsqrt(one_minus_pow(a.h.beta2, n)));
    c.gscale = both(a.grad_scale ? *a.grad_scale : 1.0f);
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
    const int64_t e0 = static_cast<int64_t>(u - u0) * ADAM_UNIT + warp * ADAM_WARP_ELEMS;
    if (e0 + ADAM_WARP_ELEMS <= T.n)
      adam_warp<PT, GT, MASTER, BITS8, true>(T, e0, lane, c);
    else if (e0 < T.n)
      adam_warp<PT, GT, MASTER, BITS8, false>(T, e0, lane, c);
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
