// combine_backward.cu -- gradient of the weighted combine with respect to the
// gates and the experts' rows.
//
// The combine is out_t = zsum_t x_t + sum_{k: slot >= 0} gate_{t,k} Y[slot],
// zsum_t the sum of the gates of zero-expert picks (slot -1), so with dout
//   dgate_{t,k} = dout_t . Y[slot_{t,k}]    FFN pick
//               = dout_t . x_t              zero-expert pick
//   dY[slot_{t,k}] = gate_{t,k} dout_t      FFN pick, rounded once to bf16
// One pass: a block holds one token; each thread takes 8 features at a time,
// reads dout once, streams the rows of Y and of dY, and keeps one fp32 partial
// dot per pick, added over the block in a fixed order.  Bound by the rows' bytes.
#include "kernels.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace moezc {
namespace {

constexpr int CB_THREADS = 256;
constexpr int CB_WARPS = CB_THREADS / 32;
constexpr int CB_GROUP = 4;   // rows of Y whose loads are in flight together

__device__ __forceinline__ float dot8(const float (&d)[8], const uint4& v, float acc) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc = fmaf(d[2 * i], bf16_lo(w[i]), acc);
    acc = fmaf(d[2 * i + 1], bf16_hi(w[i]), acc);
  }
  return acc;
}

__device__ __forceinline__ uint4 scale8(const float (&d)[8], float g) {
  uint4 o;
  uint32_t* ow = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(d[2 * i] * g, d[2 * i + 1] * g);
    ow[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return o;
}

// KM: picks at most; ROWS: dY is wanted.
template <int KM, bool ROWS>
__global__ void __launch_bounds__(CB_THREADS)
combine_backward_kernel(const uint4* __restrict__ dout, const uint4* __restrict__ x,
                        const uint4* __restrict__ Y, const int* __restrict__ slot,
                        const float* __restrict__ gate, int d8, int K, int64_t rows,
                        float* __restrict__ dgate, uint4* __restrict__ dY) {
  __shared__ int sl[KM];
  __shared__ float gt[KM];
  __shared__ int pk[KM];
  __shared__ int nffn;
  __shared__ float red[CB_WARPS][KM + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = blockIdx.x;
  griddep_wait();
  int s = -1;   // (warp 0) this lane's pick
  if (warp == 0) {
    // the FFN picks, in k order
    if (lane < K) s = slot[t * K + lane];
    const bool ffn = s >= 0 && s < rows;
    const unsigned m = __ballot_sync(0xffffffffu, ffn);
    if (ffn) {
      const int at = __popc(m & ((1u << lane) - 1u));
      sl[at] = s;
      gt[at] = ROWS ? gate[t * K + lane] : 0.f;
      pk[at] = lane;
    }
    if (lane == 0) nffn = __popc(m);
  }
  __syncthreads();
  const int n = nffn;
  const bool zero = n < K;
  float acc[KM];
  float accz = 0.f;
#pragma unroll
  for (int k = 0; k < KM; ++k) acc[k] = 0.f;
  for (int c = threadIdx.x; c < d8; c += CB_THREADS) {
    const uint4 dv = dout[t * d8 + c];
    const float d[8] = {bf16_lo(dv.x), bf16_hi(dv.x), bf16_lo(dv.y), bf16_hi(dv.y),
                        bf16_lo(dv.z), bf16_hi(dv.z), bf16_lo(dv.w), bf16_hi(dv.w)};
    if (zero) accz = dot8(d, x[t * d8 + c], accz);
#pragma unroll
    for (int k0 = 0; k0 < KM; k0 += CB_GROUP) {
      if (k0 >= n) break;
      uint4 v[CB_GROUP];
#pragma unroll
      for (int u = 0; u < CB_GROUP; ++u)
        if (k0 + u < n) v[u] = Y[static_cast<int64_t>(sl[k0 + u]) * d8 + c];
#pragma unroll
      for (int u = 0; u < CB_GROUP; ++u)
        if (k0 + u < n) {
          acc[k0 + u] = dot8(d, v[u], acc[k0 + u]);
          if (ROWS) dY[static_cast<int64_t>(sl[k0 + u]) * d8 + c] = scale8(d, gt[k0 + u]);
        }
    }
  }
#pragma unroll
  for (int k = 0; k < KM; ++k) {
    if (k >= n) break;
    const float v = warp_sum(acc[k]);
    if (lane == 0) red[warp][k] = v;
  }
  if (zero) {
    const float v = warp_sum(accz);
    if (lane == 0) red[warp][KM] = v;
  }
  __syncthreads();
  if (warp == 0) {
    if (lane < K) {
      // this lane's pick: the FFN pick it was compacted to, or a zero expert
      int at = KM;
      for (int k = 0; k < n; ++k)
        if (pk[k] == lane) at = k;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < CB_WARPS; ++w) sum += red[w][at];
      dgate[t * K + lane] = s < rows ? sum : 0.f;   // (a slot past the rows has no gradient)
    }
  }
  griddep_launch_dependents();
}

template <int KM>
cudaError_t launch_km(const __nv_bfloat16* dout, const __nv_bfloat16* x, const __nv_bfloat16* Y,
                      const int* slot, const float* gate, int64_t T, int d, int K, int64_t rows,
                      float* dgate, __nv_bfloat16* dY, cudaStream_t stream) {
  const uint4* d4 = reinterpret_cast<const uint4*>(dout);
  const uint4* x4 = reinterpret_cast<const uint4*>(x);
  const uint4* y4 = reinterpret_cast<const uint4*>(Y);
  const dim3 grid(static_cast<unsigned>(T)), block(CB_THREADS);
  if (dY)
    return launch_pdl(combine_backward_kernel<KM, true>, grid, block, 0, stream, d4, x4, y4, slot,
                      gate, d / 8, K, rows, dgate, reinterpret_cast<uint4*>(dY));
  return launch_pdl(combine_backward_kernel<KM, false>, grid, block, 0, stream, d4, x4, y4, slot,
                    gate, d / 8, K, rows, dgate, static_cast<uint4*>(nullptr));
}

}  // namespace

cudaError_t launch_combine_backward(const __nv_bfloat16* dout, const __nv_bfloat16* x,
                                    const __nv_bfloat16* Y, const int* slot, const float* gate,
                                    int64_t T, int d, int K, int64_t rows, float* dgate,
                                    __nv_bfloat16* dY, cudaStream_t stream) {
  if (T <= 0) return cudaSuccess;
#define MOEZC_CB(KM) \
  if (K <= (KM)) return launch_km<KM>(dout, x, Y, slot, gate, T, d, K, rows, dgate, dY, stream);
  MOEZC_CB(4)
  MOEZC_CB(8)
  MOEZC_CB(12)
  MOEZC_CB(16)
#undef MOEZC_CB
  return launch_km<32>(dout, x, Y, slot, gate, T, d, K, rows, dgate, dY, stream);
}

}  // namespace moezc
