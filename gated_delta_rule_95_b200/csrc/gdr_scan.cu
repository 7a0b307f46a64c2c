// The gated delta rule with scalar gates over a prompt, token by token in fp32 on the CUDA
// cores (the recurrence of gdr_decode.cu with the state held on chip):
//
//     S <- alpha_t S,   u_t = beta_t (v_t - S^T k_t),   S <- S + k_t u_t^T,   o_t = scale S^T q_t
//
// Value columns never mix, so a CTA takes (sequence, value head, 128 / G columns): G threads
// to a column, each with d_k / G rows of it in registers; a token costs two sums over the G
// lanes of a column (shuffles).  Tokens come in blocks of TB through shared memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn2_internal.h"

namespace gdn2 {
namespace {

__device__ __forceinline__ float tok(const float* p) { return __ldg(p); }
__device__ __forceinline__ float tok(const __nv_bfloat16* p) { return __bfloat162float(__ldg(p)); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

constexpr int THREADS = 128;
constexpr int TB = 16;

template <typename T, int DK, int DV, int G>
__global__ void __launch_bounds__(THREADS) gdr_scan_kernel(const T* __restrict__ q, const T* __restrict__ k,
                                                           const T* __restrict__ v, const float* __restrict__ g,
                                                           const float* __restrict__ beta, const int* cu,
                                                           const float* S0, T* __restrict__ o, float* S_T, int T_seq,
                                                           int Hk, int Hv, float scale, unsigned* err) {
  constexpr int COLS = THREADS / G, RPT = DK / G, SLICES = DV / COLS;
  __shared__ float s_q[TB][DK], s_k[TB][DK], s_v[TB][COLS];
  __shared__ float s_a[TB], s_b[TB];
  const int unit = blockIdx.x / SLICES, slice = blockIdx.x % SLICES;
  const int n = unit / Hv, hv = unit % Hv, hk = hv / (Hv / Hk);
  const int tid = threadIdx.x, part = tid % G, col = tid / G;
  long long t0 = (long long)n * T_seq;
  int len = T_seq;
  if (cu) {
    const int lo = cu[n], hi = cu[n + 1];
    if (lo < 0 || hi < lo || hi > T_seq) {  // (T_seq: tokens of the packed batch)
      if (tid == 0 && err) atomicOr(err, kErrBadSeqlens);
      return;
    }
    t0 = lo;
    len = hi - lo;
  }
  // row i of this thread: key channel 4 (part + G (i / 4)) + i % 4
  const size_t st = (size_t)unit * DK * DV + slice * COLS + col;
  float s[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = 4 * (part + G * (i / 4)) + i % 4;
    s[i] = S0 ? S0[st + (size_t)r * DV] : 0.f;
  }
  for (int b0 = 0; b0 < len; b0 += TB) {
    const int m = min(TB, len - b0);
    __syncthreads();
    for (int i = tid; i < m * DK; i += THREADS) {
      const size_t at = ((size_t)(t0 + b0 + i / DK) * Hk + hk) * DK + i % DK;
      s_q[i / DK][i % DK] = tok(q + at);
      s_k[i / DK][i % DK] = tok(k + at);
    }
    for (int i = tid; i < m * COLS; i += THREADS)
      s_v[i / COLS][i % COLS] = tok(v + ((size_t)(t0 + b0 + i / COLS) * Hv + hv) * DV + slice * COLS + i % COLS);
    if (tid < m) {
      const size_t at = (size_t)(t0 + b0 + tid) * Hv + hv;
      s_a[tid] = expf(__ldg(g + at));
      s_b[tid] = __ldg(beta + at);
    }
    __syncthreads();
    for (int t = 0; t < m; ++t) {
      const float a = s_a[t];
      float kk[RPT], e = 0.f, r = 0.f;
#pragma unroll
      for (int i = 0; i < RPT; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(&s_k[t][4 * (part + G * (i / 4))]);
        kk[i] = x.x, kk[i + 1] = x.y, kk[i + 2] = x.z, kk[i + 3] = x.w;
      }
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        s[i] *= a;
        e = fmaf(kk[i], s[i], e);
      }
#pragma unroll
      for (int off = 1; off < G; off <<= 1) e += __shfl_xor_sync(0xffffffffu, e, off);
      const float u = s_b[t] * (s_v[t][col] - e);
#pragma unroll
      for (int i = 0; i < RPT; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(&s_q[t][4 * (part + G * (i / 4))]);
        const float qq[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          s[i + c] = fmaf(kk[i + c], u, s[i + c]);
          r = fmaf(qq[c], s[i + c], r);
        }
      }
#pragma unroll
      for (int off = 1; off < G; off <<= 1) r += __shfl_xor_sync(0xffffffffu, r, off);
      if (part == 0) put(o + ((size_t)(t0 + b0 + t) * Hv + hv) * DV + slice * COLS + col, scale * r);
    }
  }
  if (S_T) {
#pragma unroll
    for (int i = 0; i < RPT; ++i) S_T[st + (size_t)(4 * (part + G * (i / 4)) + i % 4) * DV] = s[i];
  }
}

template <typename T, int DK, int DV>
cudaError_t launch_dims(const GdrArgs& a, cudaStream_t st) {
  constexpr int G = 8;
  const long long blocks = (long long)a.B * a.Hv * (DV * G / THREADS);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  gdr_scan_kernel<T, DK, DV, G><<<(unsigned)blocks, THREADS, 0, st>>>(
      static_cast<const T*>(a.q), static_cast<const T*>(a.k), static_cast<const T*>(a.v), a.g, a.beta, a.cu_seqlens,
      a.S0, static_cast<T*>(a.o), a.S_T, a.T, a.Hk, a.Hv, a.scale, device_error_word());
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(const GdrArgs& a, cudaStream_t st) {
  if (a.dk == 128) return a.dv == 128 ? launch_dims<T, 128, 128>(a, st) : launch_dims<T, 128, 64>(a, st);
  return a.dv == 128 ? launch_dims<T, 64, 128>(a, st) : launch_dims<T, 64, 64>(a, st);
}

}  // namespace

cudaError_t launch_gdr_scan(const GdrArgs& a, cudaStream_t st) {
  return a.bf16 ? launch_typed<__nv_bfloat16>(a, st) : launch_typed<float>(a, st);
}

}  // namespace gdn2
