// The gated delta rule with scalar gates over a prompt for fp32 inputs, on the CUDA cores (the
// recurrence of gdr_decode.cu with the state held on chip), four tokens at a time.  With the
// state S before the four, A_j = alpha_0 .. alpha_j and c_ji = alpha_{i+1} .. alpha_j:
//
//     u_j = beta_j (v_j - A_j S^T k_j - sum_{i < j} c_ji (k_j . k_i) u_i)
//     o_j = scale (A_j S^T q_j + sum_{i <= j} c_ji (q_j . k_i) u_i)
//     S' = A_3 S + sum_i c_3i k_i u_i^T
//
// so that the eight sums over the key axis are of the same S, and their latency (the shuffles, not
// the arithmetic, is what a token waits for) is paid once for four tokens.
//
// Value columns never mix: a CTA takes (sequence, value head, 16 columns), 8 lanes to a column,
// each with d_k / 8 rows of it in registers.  Tokens come in batches of 16 through two
// shared-memory buffers by asynchronous copies; the dot products among the tokens of a group are
// formed per batch, two threads each.
// Measured on one head of 256 tokens at d = 64: 35 us (one token at a time 86; eight at a time with 16
// lanes to a column 31, but 412 us instead of 309 for 32 heads of 1000 tokens at d = 128).
#include <cuda_runtime.h>

#include "gdn2_internal.h"
#include "ptx.cuh"

namespace gdn2 {
namespace {

constexpr int THREADS = 128;
constexpr int TB = 16, NB = 4;  // tokens of a batch and of a group
constexpr int G = 8;            // lanes of a column
constexpr int COLS = THREADS / G;

// The dot products of a group: k_i . k_j at (i, j < i), q_i . k_j at (i, j <= i).
__device__ __forceinline__ constexpr int kk(int i, int j) { return i * (i - 1) / 2 + j; }
__device__ __forceinline__ constexpr int qk(int i, int j) { return 6 + i * (i + 1) / 2 + j; }

template <int DK>
struct Batch {
  static constexpr int LD = DK + 4;  // rows 4 banks apart
  alignas(16) float q[TB][LD], k[TB][LD], v[TB][COLS];
  alignas(16) float a[TB], b[TB];
};

template <int DK, int DV>
__global__ void __launch_bounds__(THREADS) gdr_scan_kernel(const float* __restrict__ q, const float* __restrict__ k,
                                                           const float* __restrict__ v, const float* __restrict__ g,
                                                           const float* __restrict__ beta, const int* cu,
                                                           const float* S0, float* __restrict__ o, float* S_T, int T_seq,
                                                           int Hk, int Hv, float scale, unsigned* err) {
  constexpr int RPT = DK / G, SLICES = DV / COLS;
  __shared__ Batch<DK> buf[2];
  __shared__ __align__(16) float dots[TB / NB][16];
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
  // a batch's copies; tokens past the end are zeros with alpha = 1, beta = 0
  auto fetch = [&](int b0, Batch<DK>& w) {
    for (int i = tid; i < TB * DK / 4; i += THREADS) {
      const int t = i / (DK / 4), c = 4 * (i % (DK / 4));
      const bool there = b0 + t < len;
      const size_t at = ((size_t)(t0 + (there ? b0 + t : 0)) * Hk + hk) * DK + c;
      cp_async16(&w.q[t][c], q + at, there);
      cp_async16(&w.k[t][c], k + at, there);
    }
    if (tid < TB * COLS / 4) {
      const int t = tid / (COLS / 4), c = 4 * (tid % (COLS / 4));
      const bool there = b0 + t < len;
      cp_async16(&w.v[t][c], v + ((size_t)(t0 + (there ? b0 + t : 0)) * Hv + hv) * DV + slice * COLS + c, there);
    }
  };
  auto gate = [&](int b0, float& ga, float& be) {  // token tid of the batch
    const bool there = tid < TB && b0 + tid < len;
    const size_t at = (size_t)(t0 + (there ? b0 + tid : 0)) * Hv + hv;
    ga = there ? __ldg(g + at) : 0.f;
    be = there ? __ldg(beta + at) : 0.f;
  };
  // row i of this thread: key channel 4 (part + G (i / 4)) + i % 4
  const size_t st = (size_t)unit * DK * DV + slice * COLS + col;
  float s[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = 4 * (part + G * (i / 4)) + i % 4;
    s[i] = S0 ? S0[st + (size_t)r * DV] : 0.f;
  }
  float ga = 0.f, be = 0.f;
  if (len > 0) {
    fetch(0, buf[0]);
    gate(0, ga, be);
  }
#pragma unroll 1
  for (int b0 = 0, turn = 0; b0 < len; b0 += TB, turn ^= 1) {
    Batch<DK>& w = buf[turn];
    if (tid < TB) w.a[tid] = expf(ga), w.b[tid] = be;
    cp_async_wait_all();
    __syncthreads();  // this batch is there, and the other buffer is free
    if (b0 + TB < len) {
      fetch(b0 + TB, buf[turn ^ 1]);
      gate(b0 + TB, ga, be);
    }
    {  // the dot products among each group's tokens
      const int d = (tid >> 1) & 15, grp = tid >> 5, half = tid & 1;
      int i, j;
      if (d < 6) {
        i = d < 1 ? 1 : d < 3 ? 2 : 3;
        j = d - i * (i - 1) / 2;
      } else {
        i = d < 7 ? 0 : d < 9 ? 1 : d < 12 ? 2 : 3;
        j = d - 6 - i * (i + 1) / 2;
      }
      const float* x = (d < 6 ? w.k : w.q)[NB * grp + i];
      const float* y = w.k[NB * grp + j];
      float r[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int c = 4 * half; c < DK; c += 8) {
        const float4 a = *reinterpret_cast<const float4*>(x + c), b = *reinterpret_cast<const float4*>(y + c);
        r[0] = fmaf(a.x, b.x, r[0]), r[1] = fmaf(a.y, b.y, r[1]), r[2] = fmaf(a.z, b.z, r[2]), r[3] = fmaf(a.w, b.w, r[3]);
      }
      float t = (r[0] + r[1]) + (r[2] + r[3]);
      t += __shfl_xor_sync(0xffffffffu, t, 1);
      if (half == 0) dots[grp][d] = t;
    }
    __syncthreads();
    const int groups = (min(TB, len - b0) + NB - 1) / NB;
#pragma unroll 1
    for (int grp = 0; grp < groups; ++grp) {
      // S^T k_j (sum[j]) and S^T q_j (sum[4 + j]): this thread's rows, then over the column's lanes
      float sum[8];
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const float *kr = w.k[NB * grp + j], *qr = w.q[NB * grp + j];
        float e0 = 0.f, e1 = 0.f, r0 = 0.f, r1 = 0.f;
#pragma unroll
        for (int i = 0; i < RPT; i += 4) {
          const float4 x = *reinterpret_cast<const float4*>(kr + 4 * (part + G * (i / 4)));
          const float4 y = *reinterpret_cast<const float4*>(qr + 4 * (part + G * (i / 4)));
          e0 = fmaf(x.x, s[i], fmaf(x.y, s[i + 1], e0)), e1 = fmaf(x.z, s[i + 2], fmaf(x.w, s[i + 3], e1));
          r0 = fmaf(y.x, s[i], fmaf(y.y, s[i + 1], r0)), r1 = fmaf(y.z, s[i + 2], fmaf(y.w, s[i + 3], r1));
        }
        sum[j] = e0 + e1;
        sum[4 + j] = r0 + r1;
      }
      // halving exchange: lane `part` ends up with the whole of sum[part's bits reversed]
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool up = part & 4;
        const float send = up ? sum[i] : sum[i + 4], keep = up ? sum[i + 4] : sum[i];
        sum[i] = keep + __shfl_xor_sync(0xffffffffu, send, 4);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool up = part & 2;
        const float send = up ? sum[i] : sum[i + 2], keep = up ? sum[i + 2] : sum[i];
        sum[i] = keep + __shfl_xor_sync(0xffffffffu, send, 2);
      }
      {
        const bool up = part & 1;
        const float send = up ? sum[0] : sum[1], keep = up ? sum[1] : sum[0];
        sum[0] = keep + __shfl_xor_sync(0xffffffffu, send, 1);
      }
      float e[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) e[j] = __shfl_sync(0xffffffffu, sum[0], j, G);  // lane j < 4: S^T k_j; lane 4 + j: S^T q_j
      // the group's tokens one after the other
      const float4 av = *reinterpret_cast<const float4*>(&w.a[NB * grp]), bv = *reinterpret_cast<const float4*>(&w.b[NB * grp]);
      const float a[NB] = {av.x, av.y, av.z, av.w}, b[NB] = {bv.x, bv.y, bv.z, bv.w};
      float d[16];
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(&dots[grp][i]);
        d[i] = x.x, d[i + 1] = x.y, d[i + 2] = x.z, d[i + 3] = x.w;
      }
      float u[NB], A = 1.f;  // u_i carries c_ji after token j
      float mine = 0.f;      // lane 4 + j: token j's output
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        A *= a[j];
        float x = fmaf(-A, e[j], w.v[NB * grp + j][col]), y = 0.f;
#pragma unroll
        for (int i = 0; i < j; ++i) {
          u[i] *= a[j];
          x = fmaf(-d[kk(j, i)], u[i], x);
          y = fmaf(d[qk(j, i)], u[i], y);
        }
        u[j] = b[j] * x;
        y = fmaf(d[qk(j, j)], u[j], y);
        if (part == 4 + j) mine = scale * fmaf(A, sum[0], y);
      }
      const int t = b0 + NB * grp + part - 4;
      if (part >= 4 && t < len) o[((size_t)(t0 + t) * Hv + hv) * DV + slice * COLS + col] = mine;
#pragma unroll
      for (int i = 0; i < RPT; ++i) s[i] *= A;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const float* kr = w.k[NB * grp + j];
#pragma unroll
        for (int i = 0; i < RPT; i += 4) {
          const float4 x = *reinterpret_cast<const float4*>(kr + 4 * (part + G * (i / 4)));
          s[i] = fmaf(x.x, u[j], s[i]), s[i + 1] = fmaf(x.y, u[j], s[i + 1]);
          s[i + 2] = fmaf(x.z, u[j], s[i + 2]), s[i + 3] = fmaf(x.w, u[j], s[i + 3]);
        }
      }
    }
  }
  if (S_T) {
#pragma unroll
    for (int i = 0; i < RPT; ++i) S_T[st + (size_t)(4 * (part + G * (i / 4)) + i % 4) * DV] = s[i];
  }
}

template <int DK, int DV>
cudaError_t launch_dims(const GdrArgs& a, cudaStream_t st) {
  const long long blocks = (long long)a.B * a.Hv * (DV / COLS);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  gdr_scan_kernel<DK, DV><<<(unsigned)blocks, THREADS, 0, st>>>(
      static_cast<const float*>(a.q), static_cast<const float*>(a.k), static_cast<const float*>(a.v), a.g, a.beta,
      a.cu_seqlens, a.S0, static_cast<float*>(a.o), a.S_T, a.T, a.Hk, a.Hv, a.scale, device_error_word());
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gdr_scan(const GdrArgs& a, cudaStream_t st) {
  // (bf16 only without tokens, where no input is read: the states are copied)
  if (a.bf16 && a.T != 0) return cudaErrorInvalidValue;
  if (a.dk == 128) return a.dv == 128 ? launch_dims<128, 128>(a, st) : launch_dims<128, 64>(a, st);
  return a.dv == 128 ? launch_dims<64, 128>(a, st) : launch_dims<64, 64>(a, st);
}

}  // namespace gdn2
