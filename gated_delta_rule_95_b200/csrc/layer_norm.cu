// Layer norm over the last axis and its backward pass: the end of the layer, LayerNorm(x +
// out_proj(y)) (Gated DeltaNet-2 guide, "End-to-End PyTorch Implementation").
//
//     s = round(x + r)              (the residual sum, in the storage type; s = x without r)
//     mu = mean(s),  rho = (mean((s - mu)^2) + eps)^-1/2
//     y = (s - mu) rho w + b
//
// and, with h = dy w and xh = (s - mu) rho,
//
//     dx = rho (h - mean(h) - xh mean(h xh)) + ds       (the gradient of x and of r alike)
//     dw = sum over rows of dy xh,   db = sum over rows of dy
//
// Both passes are bound by memory: every tensor is read or written once.  A row stays in
// registers between its statistics and its outputs; mean and variance are two sums in fp32,
// the second over (s - mu)^2, so nothing cancels.
//
// Work split.  A row is held by G threads: a power of two up to a warp for rows of at most
// 2 x 32 vectors of 16 bytes or 8 x 32 single elements (shuffles only, several rows to a warp when
// they are narrow), whole blocks above that; rows past what a block's registers hold are read
// again for each pass (the second and third reading come from the caches).  A vector is 16 bytes
// when a row's bytes divide by 16 and one element otherwise.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gdn2_internal.h"
#include "ptx.cuh"  // pairs of fp32 operations

namespace gdn2 {
namespace {

// VE adjacent elements: one 16-byte access (VE = 16 / sizeof(T)) or one element, as stored (Raw)
// and as floats.
template <typename T, int VE>
struct Vec;
template <>
struct Vec<float, 4> {
  using Raw = float4;
  static __device__ __forceinline__ void cvt(const Raw& u, float (&f)[4]) { f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w; }
  static __device__ __forceinline__ Raw pack(const float (&f)[4]) { return make_float4(f[0], f[1], f[2], f[3]); }
};
template <>
struct Vec<__nv_bfloat16, 8> {
  using Raw = uint4;
  static __device__ __forceinline__ void cvt(const Raw& u, float (&f)[8]) {
    const uint32_t r[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(r[i] << 16);
      f[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ Raw pack(const float (&f)[8]) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      r[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
  }
};
template <>
struct Vec<float, 1> {
  using Raw = float;
  static __device__ __forceinline__ void cvt(const Raw& u, float (&f)[1]) { f[0] = u; }
  static __device__ __forceinline__ Raw pack(const float (&f)[1]) { return f[0]; }
};
template <>
struct Vec<__nv_bfloat16, 1> {
  using Raw = __nv_bfloat16;
  static __device__ __forceinline__ void cvt(const Raw& u, float (&f)[1]) { f[0] = __bfloat162float(u); }
  static __device__ __forceinline__ Raw pack(const float (&f)[1]) { return __float2bfloat16_rn(f[0]); }
};
// Vector j of a row.  (Plain loads: the sum may be written over x or the residual.)
template <typename T, int VE>
__device__ __forceinline__ typename Vec<T, VE>::Raw load_raw(const T* row, int j) {
  return reinterpret_cast<const typename Vec<T, VE>::Raw*>(row)[j];
}
// As pairs; a lone element is (x, 0).
template <typename T, int VE>
__device__ __forceinline__ void cvt_pairs(const typename Vec<T, VE>::Raw& u, float2 (&f)[(VE + 1) / 2]) {
  float e[VE];
  Vec<T, VE>::cvt(u, e);
#pragma unroll
  for (int i = 0; i < (VE + 1) / 2; ++i) f[i] = make_float2(e[2 * i], VE > 1 ? e[2 * i + (VE > 1)] : 0.f);
}
template <typename T, int VE>
__device__ __forceinline__ void load_vec(const T* row, int j, float (&f)[VE]) {
  Vec<T, VE>::cvt(load_raw<T, VE>(row, j), f);
}
template <typename T, int VE>
__device__ __forceinline__ void store_vec(T* row, int j, const float (&f)[VE]) {
  reinterpret_cast<typename Vec<T, VE>::Raw*>(row)[j] = Vec<T, VE>::pack(f);
}
// VE adjacent fp32 values (weight, bias).
template <int VE>
__device__ __forceinline__ void load_f32(const float* p, float (&f)[VE]) {
  if constexpr (VE == 1) {
    f[0] = __ldg(p);
  } else {
#pragma unroll
    for (int i = 0; i < VE; i += 4) {
      const float4 u = __ldg(reinterpret_cast<const float4*>(p + i));
      f[i] = u.x, f[i + 1] = u.y, f[i + 2] = u.z, f[i + 3] = u.w;
    }
  }
}
__device__ __forceinline__ float round_to(float x, float) { return x; }
__device__ __forceinline__ float round_to(float x, __nv_bfloat16) { return __bfloat162float(__float2bfloat16_rn(x)); }

constexpr int MAX_WARPS = 32;
constexpr int MAX_STAGES = 8;

// Sums of N values (a power of two) over the G threads of a row (G a power of two up to 32:
// lanes that differ in their low bits; G = 0: the whole block), the results in each of them.
// One barrier: the caller passes a buffer that no thread may still be reading.
//
// In a block, the lanes of a warp halve the values as they halve the lanes (N = 4: 6 shuffles
// instead of 20) until lane l holds the warp's sum of value l / (32 / N); then every warp adds
// up all warps' sums, value l % N in lane l.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], int G, float (*red)[N]) {
  const int lane = threadIdx.x & 31;
  if (G) {
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      if (off < G) {
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], off);
      }
    }
    return;
  }
  float t[N];
#pragma unroll
  for (int n = 0; n < N; ++n) t[n] = v[n];
  int left = N;
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    if (left > 1) {
      left /= 2;
#pragma unroll
      for (int n = 0; n < N / 2; ++n) {
        if (n < left) {
          const float send = (lane & off) ? t[n] : t[n + left], keep = (lane & off) ? t[n + left] : t[n];
          t[n] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
      }
    } else {
      t[0] += __shfl_xor_sync(0xffffffffu, t[0], off);
    }
  }
  if (lane % (32 / N) == 0) red[threadIdx.x >> 5][lane / (32 / N)] = t[0];
  __syncthreads();
  const int nw = blockDim.x >> 5;
  float u = 0.f;
  for (int w = lane / N; w < nw; w += 32 / N) u += red[w][lane % N];
#pragma unroll
  for (int off = 16; off >= N; off >>= 1) u += __shfl_xor_sync(0xffffffffu, u, off);
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = __shfl_sync(0xffffffffu, u, n);
}

// ---------------------------------------------------------------------------- forward

// A row's vectors in registers, NV to a thread (all loads in flight before any is used).  G: threads of
// a row (0 = the block); nv = vectors of a row.  32768 x 2048 bf16 with a residual: 87 us, 537 MB at 6.2
// TB/s (two rows at once to a block were no faster, 87 us, and 2048 rows took 8.8 us instead of 7.6).
template <typename T, int VE, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_fwd_kernel(const T* x, const T* r, const float* __restrict__ w,
                                                        const float* __restrict__ b, T* y, T* s,
                                                        float* __restrict__ mean, float* __restrict__ rstd, int rows,
                                                        int nv, int G, float eps) {
  __shared__ float red[2][MAX_WARPS][1];
  using V = Vec<T, VE>;
  const int gw = G ? G : blockDim.x;  // threads of a row
  const int per = blockDim.x / gw;    // rows of a block
  const int jt = G ? (threadIdx.x & (gw - 1)) : threadIdx.x;
  const long long row = (long long)blockIdx.x * per + (G ? threadIdx.x / gw : 0);
  const bool there = row < rows;
  const size_t base = (size_t)(there ? row : 0) * nv * VE;
  const float cols = (float)nv * VE;  // (at most 2^24: exact; divided by, so that a constant row has no variance)
  float f[NV][VE], sum[1] = {0.f}, sq[1] = {0.f};
  {
    typename V::Raw xr[NV], rr[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      if (there && jt + n * gw < nv) {
        xr[n] = load_raw<T, VE>(x + base, jt + n * gw);
        if (r) rr[n] = load_raw<T, VE>(r + base, jt + n * gw);
      }
    }
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      if (there && jt + n * gw < nv) {
        V::cvt(xr[n], f[n]);
        if (r) {
          float e[VE];
          V::cvt(rr[n], e);
#pragma unroll
          for (int i = 0; i < VE; ++i) f[n][i] = round_to(f[n][i] + e[i], T());
        }
      } else {
#pragma unroll
        for (int i = 0; i < VE; ++i) f[n][i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < VE; ++i) sum[0] += f[n][i];
    }
  }
  group_sum<1>(sum, G, red[0]);
  const float mu = sum[0] / cols;
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    if (jt + n * gw < nv) {
#pragma unroll
      for (int i = 0; i < VE; ++i) sq[0] = fmaf(f[n][i] - mu, f[n][i] - mu, sq[0]);
    }
  }
  group_sum<1>(sq, G, red[1]);
  const float rho = rsqrtf(sq[0] / cols + eps);
  if (!there) return;
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int j = jt + n * gw;
    if (j < nv) {
      float wv[VE], bv[VE], o[VE];
      load_f32<VE>(w + (size_t)j * VE, wv);
      if (b) load_f32<VE>(b + (size_t)j * VE, bv);
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float t = (f[n][i] - mu) * rho;
        o[i] = b ? fmaf(t, wv[i], bv[i]) : t * wv[i];
      }
      store_vec<T, VE>(y + base, j, o);
      if (s) store_vec<T, VE>(s + base, j, f[n]);
    }
  }
  if (jt == 0) {
    if (mean) mean[row] = mu;
    if (rstd) rstd[row] = rho;
  }
}

// Rows of any length, a block each: read once for the mean, once for the variance and once
// for the outputs.
template <typename T, int VE>
__global__ void __launch_bounds__(512) norm_fwd_long_kernel(const T* x, const T* r, const float* __restrict__ w,
                                                            const float* __restrict__ b, T* y, T* s,
                                                            float* __restrict__ mean, float* __restrict__ rstd, int nv,
                                                            float eps) {
  __shared__ float red[2][MAX_WARPS][1];
  const size_t base = (size_t)blockIdx.x * nv * VE;
  const float cols = (float)nv * VE;
  float sum[1] = {0.f}, sq[1] = {0.f}, f[VE];
  auto load_sum = [&](int j) {
    load_vec<T, VE>(x + base, j, f);
    if (r) {
      float e[VE];
      load_vec<T, VE>(r + base, j, e);
#pragma unroll
      for (int i = 0; i < VE; ++i) f[i] = round_to(f[i] + e[i], T());
    }
  };
  for (int j = threadIdx.x; j < nv; j += blockDim.x) {
    load_sum(j);
#pragma unroll
    for (int i = 0; i < VE; ++i) sum[0] += f[i];
  }
  group_sum<1>(sum, 0, red[0]);
  const float mu = sum[0] / cols;
  for (int j = threadIdx.x; j < nv; j += blockDim.x) {
    load_sum(j);
#pragma unroll
    for (int i = 0; i < VE; ++i) sq[0] = fmaf(f[i] - mu, f[i] - mu, sq[0]);
  }
  group_sum<1>(sq, 0, red[1]);
  const float rho = rsqrtf(sq[0] / cols + eps);
  for (int j = threadIdx.x; j < nv; j += blockDim.x) {
    float wv[VE], bv[VE], o[VE];
    load_sum(j);
    load_f32<VE>(w + (size_t)j * VE, wv);
    if (b) load_f32<VE>(b + (size_t)j * VE, bv);
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const float t = (f[i] - mu) * rho;
      o[i] = b ? fmaf(t, wv[i], bv[i]) : t * wv[i];
    }
    store_vec<T, VE>(y + base, j, o);
    if (s) store_vec<T, VE>(s + base, j, f);
  }
  if (threadIdx.x == 0) {
    if (mean) mean[blockIdx.x] = mu;
    if (rstd) rstd[blockIdx.x] = rho;
  }
}

// --------------------------------------------------------------------------- backward

// A block's partial row [dw | db]: the row groups' sums added up through acc ([per][cols]).
template <int VE, int NV>
__device__ __forceinline__ void write_partials(const float2 (&dw)[NV][(VE + 1) / 2], const float2 (&db)[NV][(VE + 1) / 2],
                                               float* acc, float* out, int jt, int grp, int gw, int per, int nv) {
  const int cols = nv * VE;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (per > 1) __syncthreads();
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int j = jt + n * gw;
      if (j < nv) {
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          const float2 t = half ? db[n][i / 2] : dw[n][i / 2];
          const float v = i % 2 ? t.y : t.x;
          if (per > 1)
            acc[grp * cols + j * VE + i] = v;
          else
            out[half * cols + j * VE + i] = v;
        }
      }
    }
    if (per > 1) {
      __syncthreads();
      for (int c = threadIdx.x; c < cols; c += blockDim.x) {
        float t = 0.f;
        for (int q = 0; q < per; ++q) t += acc[q * cols + c];
        out[half * cols + c] = t;
      }
    }
  }
}

// A block walks rows blockIdx.x * per + i * gridDim.x * per with its columns fixed to its
// threads (NV vectors each), so dw and db accumulate in registers; at the end the block's
// row groups are added up in shared memory and one partial row [dw | db] is written.
// R rows at once: their loads are all in flight before any is used, and one barrier serves
// their sums.
template <typename T, int VE, int NV, int R, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_bwd_kernel(const T* dy, const T* s, const float* __restrict__ w,
                                                              const float* __restrict__ mean,
                                                              const float* __restrict__ rstd, const T* ds, T* dx,
                                                              float* __restrict__ part, int rows, int nv, int G) {
  __shared__ float red[2][MAX_WARPS][2 * R];
  extern __shared__ float acc[];  // [per][cols] of one sum at a time (G > 0)
  using V = Vec<T, VE>;
  const int gw = G ? G : blockDim.x, per = blockDim.x / gw;
  const int jt = G ? (threadIdx.x & (gw - 1)) : threadIdx.x, grp = G ? threadIdx.x / gw : 0;
  const int cols = nv * VE;
  const float inv = 1.f / (float)cols;
  constexpr int NP = (VE + 1) / 2;  // pairs of a vector
  float2 dw[NV][NP], db[NV][NP], wv[NV][NP];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    float e[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) e[i] = 0.f;
    if (jt + n * gw < nv) load_f32<VE>(w + (size_t)(jt + n * gw) * VE, e);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      dw[n][i] = db[n][i] = make_float2(0.f, 0.f);
      wv[n][i] = make_float2(e[2 * i], VE > 1 ? e[2 * i + (VE > 1)] : 0.f);
    }
  }
  int turn = 0;  // of the two buffers of the sums
  for (long long row0 = (long long)blockIdx.x * per * R; row0 < rows; row0 += (long long)gridDim.x * per * R, turn ^= 1) {
    typename V::Raw qy[R][NV], qs[R][NV], qd[R][NV];
    float mu[R], rho[R], sums[2 * R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const long long row = row0 + k * per + grp;
      if (row < rows) {
        const size_t base = (size_t)row * cols;
        mu[k] = __ldg(mean + row), rho[k] = __ldg(rstd + row);
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          const int j = jt + n * gw;
          if (j < nv) {
            qy[k][n] = load_raw<T, VE>(dy + base, j);
            qs[k][n] = load_raw<T, VE>(s + base, j);
            if (ds) qd[k][n] = load_raw<T, VE>(ds + base, j);
          }
        }
      }
    }
    const float2 one = make_float2(1.f, 1.f);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      float2 s0 = make_float2(0.f, 0.f), s1 = s0;
      if (row0 + k * per + grp < rows) {
        const float2 mm = make_float2(mu[k], mu[k]), rr = make_float2(rho[k], rho[k]);
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          if (jt + n * gw < nv) {
            float2 g[NP], x[NP];
            cvt_pairs<T, VE>(qy[k][n], g);
            cvt_pairs<T, VE>(qs[k][n], x);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
              x[i] = mul2(sub2(x[i], mm), rr);
              db[n][i] = fma2(g[i], one, db[n][i]);
              dw[n][i] = fma2(g[i], x[i], dw[n][i]);
              g[i] = mul2(g[i], wv[n][i]);
              s0 = fma2(g[i], one, s0);
              s1 = fma2(g[i], x[i], s1);
            }
          }
        }
      }
      sums[2 * k] = s0.x + s0.y;
      sums[2 * k + 1] = s1.x + s1.y;
    }
    group_sum<2 * R>(sums, G, red[turn]);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const long long row = row0 + k * per + grp;
      if (row < rows) {
        // dx = rho h + (-rho mean(h) + ds) - rho mean(h xh) xh
        const float c0 = -rho[k] * (sums[2 * k] * inv), c1 = -rho[k] * (sums[2 * k + 1] * inv);
        const float2 mm = make_float2(mu[k], mu[k]), rr = make_float2(rho[k], rho[k]);
        const float2 cc0 = make_float2(c0, c0), cc1 = make_float2(c1, c1);
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          const int j = jt + n * gw;
          if (j < nv) {
            float2 g[NP], x[NP], e[NP];
            float o[VE];
            cvt_pairs<T, VE>(qy[k][n], g);
            cvt_pairs<T, VE>(qs[k][n], x);
            if (ds) cvt_pairs<T, VE>(qd[k][n], e);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
              x[i] = mul2(sub2(x[i], mm), rr);
              g[i] = mul2(g[i], wv[n][i]);
              const float2 t = fma2(g[i], rr, fma2(x[i], cc1, ds ? fma2(e[i], one, cc0) : cc0));
              o[2 * i] = t.x;
              if (VE > 1) o[2 * i + (VE > 1)] = t.y;
            }
            store_vec<T, VE>(dx + (size_t)row * cols, j, o);
          }
        }
      }
    }
  }
  write_partials<VE, NV>(dw, db, acc, part + (size_t)blockIdx.x * 2 * cols, jt, grp, gw, per, nv);
}

// The same where a row's bytes divide by 16: the rows of dy, s and ds come through a ring of
// shared-memory stages by 1-D bulk copies (a stage: the `per` rows that the block works on next),
// so that the loads of the following rows never wait for this one's sums.  Measured at
// 32768 x 2048 bf16 with ds: 98 us, 537 MB at 5.5 TB/s (116 us with plain loads of two rows at once),
// and 3 us for the blocks' sums.
constexpr int NORM_WAIT_TRIES = 2000;  // suspensions of 1 ms
template <typename T, int VE, int NV, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_bwd_bulk_kernel(const T* __restrict__ dy, const T* __restrict__ s,
                                                                   const float* __restrict__ w,
                                                                   const float* __restrict__ mean,
                                                                   const float* __restrict__ rstd,
                                                                   const T* __restrict__ ds, T* __restrict__ dx,
                                                                   float* __restrict__ part, int rows, int nv, int G,
                                                                   int stages, unsigned* err) {
  __shared__ float red[2][MAX_WARPS][2];
  __shared__ uint64_t full[MAX_STAGES];
  extern __shared__ __align__(16) unsigned char ring[];  // [stage][dy | s | ds][per * cols]
  using V = Vec<T, VE>;
  using Raw = typename V::Raw;
  constexpr int NP = VE / 2;
  const int gw = G ? G : blockDim.x, per = blockDim.x / gw;
  const int jt = G ? (threadIdx.x & (gw - 1)) : threadIdx.x, grp = G ? threadIdx.x / gw : 0;
  const int cols = nv * VE;
  const float inv = 1.f / (float)cols;
  const uint32_t piece = (uint32_t)per * cols * sizeof(T);  // bytes of one tensor's rows in a stage
  const long long step = (long long)gridDim.x * per;
  const int count = (int)(((long long)rows - (long long)blockIdx.x * per + step - 1) / step);  // of this block (>= 1)
  auto first_row = [&](int i) { return (long long)blockIdx.x * per + i * step; };
  auto issue = [&](int i) {
    const long long row = first_row(i);
    const int live = (int)min((long long)per, rows - row);
    const uint32_t bytes = (uint32_t)live * cols * sizeof(T);
    uint64_t* bar = &full[i % stages];
    unsigned char* at = ring + (size_t)(i % stages) * 3 * piece;
    mbar_arrive_expect_tx(bar, bytes * (ds ? 3 : 2));
    bulk_load_1d(at, dy + (size_t)row * cols, bytes, bar);
    bulk_load_1d(at + piece, s + (size_t)row * cols, bytes, bar);
    if (ds) bulk_load_1d(at + 2 * piece, ds + (size_t)row * cols, bytes, bar);
  };
  grid_release();
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
    for (int i = 0; i < stages && i < count; ++i) issue(i);
  }
  float2 dw[NV][NP], db[NV][NP], wv[NV][NP];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    float e[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) e[i] = 0.f;
    if (jt + n * gw < nv) load_f32<VE>(w + (size_t)(jt + n * gw) * VE, e);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      dw[n][i] = db[n][i] = make_float2(0.f, 0.f);
      wv[n][i] = make_float2(e[2 * i], e[2 * i + 1]);
    }
  }
  __syncthreads();
  const float2 one = make_float2(1.f, 1.f);
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    const long long row = first_row(i) + grp;
    const bool live = row < rows;
    const float mu = live ? __ldg(mean + row) : 0.f, rho = live ? __ldg(rstd + row) : 0.f;
    const float2 mm = make_float2(mu, mu), rr = make_float2(rho, rho);
    // (a copy that does not land is reported; it is waited for once more, so that it is not in
    // flight when the block ends)
    if (!mbar_wait_short(&full[i % stages], (uint32_t)((i / stages) & 1), NORM_WAIT_TRIES)) {
      if (err) atomicOr(err, kErrWaitTimeout);
      mbar_wait_short(&full[i % stages], (uint32_t)((i / stages) & 1), NORM_WAIT_TRIES);
    }
    const unsigned char* at = ring + (size_t)(i % stages) * 3 * piece + (size_t)grp * cols * sizeof(T);
    float2 g[NV][NP], x[NV][NP], s0 = make_float2(0.f, 0.f), s1 = s0;
    Raw e[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int j = jt + n * gw;
      if (live && j < nv) {
        cvt_pairs<T, VE>(reinterpret_cast<const Raw*>(at)[j], g[n]);
        cvt_pairs<T, VE>(reinterpret_cast<const Raw*>(at + piece)[j], x[n]);
        if (ds) e[n] = reinterpret_cast<const Raw*>(at + 2 * piece)[j];
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          x[n][k] = mul2(sub2(x[n][k], mm), rr);
          db[n][k] = fma2(g[n][k], one, db[n][k]);
          dw[n][k] = fma2(g[n][k], x[n][k], dw[n][k]);
          g[n][k] = mul2(g[n][k], wv[n][k]);
          s0 = fma2(g[n][k], one, s0);
          s1 = fma2(g[n][k], x[n][k], s1);
        }
      }
    }
    float sums[2] = {s0.x + s0.y, s1.x + s1.y};
    group_sum<2>(sums, G, red[i & 1]);
    if (G) __syncthreads();  // (a block-wide sum has one)
    // every thread has read the stage
    if (threadIdx.x == 0 && i + stages < count) issue(i + stages);
    // dx = rho h + (-rho mean(h) + ds) - rho mean(h xh) xh
    const float c0 = -rho * (sums[0] * inv), c1 = -rho * (sums[1] * inv);
    const float2 cc0 = make_float2(c0, c0), cc1 = make_float2(c1, c1);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int j = jt + n * gw;
      if (live && j < nv) {
        float o[VE];
        float2 ep[NP];
        if (ds) cvt_pairs<T, VE>(e[n], ep);
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          const float2 t = fma2(g[n][k], rr, fma2(x[n][k], cc1, ds ? fma2(ep[k], one, cc0) : cc0));
          o[2 * k] = t.x, o[2 * k + 1] = t.y;
        }
        store_vec<T, VE>(dx + (size_t)row * cols, j, o);
      }
    }
  }
  float* acc = reinterpret_cast<float*>(ring);  // (every copy has landed and been read)
  write_partials<VE, NV>(dw, db, acc, part + (size_t)blockIdx.x * 2 * cols, jt, grp, gw, per, nv);
}

// Rows of any length: dx alone, the row read twice (the second time from the caches).
template <typename T, int VE>
__global__ void __launch_bounds__(1024) norm_bwd_long_kernel(const T* dy, const T* s, const float* __restrict__ w,
                                                             const float* __restrict__ mean,
                                                             const float* __restrict__ rstd, const T* ds, T* dx,
                                                             int nv) {
  __shared__ float red[MAX_WARPS][2];
  const size_t base = (size_t)blockIdx.x * nv * VE;
  const float mu = __ldg(mean + blockIdx.x), rho = __ldg(rstd + blockIdx.x), inv = 1.f / ((float)nv * VE);
  float sums[2] = {0.f, 0.f}, g[VE], xh[VE], wv[VE];
  auto load = [&](int j) {
    load_vec<T, VE>(dy + base, j, g);
    load_vec<T, VE>(s + base, j, xh);
    load_f32<VE>(w + (size_t)j * VE, wv);
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      g[i] *= wv[i];
      xh[i] = (xh[i] - mu) * rho;
    }
  };
  for (int j = threadIdx.x; j < nv; j += blockDim.x) {
    load(j);
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      sums[0] += g[i];
      sums[1] = fmaf(g[i], xh[i], sums[1]);
    }
  }
  group_sum<2>(sums, 0, red);
  const float m0 = sums[0] * inv, m1 = sums[1] * inv;
  for (int j = threadIdx.x; j < nv; j += blockDim.x) {
    load(j);
    float o[VE], e[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) o[i] = rho * (g[i] - m0 - xh[i] * m1);
    if (ds) {
      load_vec<T, VE>(ds + base, j, e);
#pragma unroll
      for (int i = 0; i < VE; ++i) o[i] += e[i];
    }
    store_vec<T, VE>(dx + base, j, o);
  }
}
// Its dw and db: a thread per column over a stretch of rows (partials as norm_bwd_kernel's).
template <typename T>
__global__ void norm_bwd_columns_kernel(const T* dy, const T* s, const float* __restrict__ mean,
                                        const float* __restrict__ rstd, float* __restrict__ part, int rows, int cols,
                                        int stretch) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= cols) return;
  const long long r0 = (long long)blockIdx.y * stretch, r1 = min((long long)rows, r0 + stretch);
  float dw = 0.f, db = 0.f;
  for (long long r = r0; r < r1; ++r) {
    float g[1], x[1];
    load_vec<T, 1>(dy + (size_t)r * cols, c, g);
    load_vec<T, 1>(s + (size_t)r * cols, c, x);
    db += g[0];
    dw = fmaf(g[0], (x[0] - __ldg(mean + r)) * __ldg(rstd + r), dw);
  }
  part[(size_t)blockIdx.y * 2 * cols + c] = dw;
  part[(size_t)blockIdx.y * 2 * cols + cols + c] = db;
}

// out[c] = sum over the P partial rows, in the order of the rows (the same result every
// time): 32 row walkers to a column, added up at the end.  (part without __restrict__: it may be written while
// this grid waits, so its loads stay behind the wait and on the coherent path.)
__global__ void __launch_bounds__(1024) norm_partials_kernel(const float* part, float* __restrict__ dw,
                                                             float* __restrict__ db, int P, int cols) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, wk = threadIdx.x >> 5;
  long long c = (long long)blockIdx.x * 32 + lane;  // over [dw | db]
  grid_wait();
  float t = 0.f;
  if (c < 2ll * cols) {
#pragma unroll 16
    for (int p = wk; p < P; p += 32) t += part[(size_t)p * 2 * cols + c];
  }
  red[wk][lane] = t;
  __syncthreads();
  t = red[lane][wk];  // warp wk adds up column wk of the block's 32
#pragma unroll
  for (int off = 16; off; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
  c = (long long)blockIdx.x * 32 + wk;
  if (lane == 0 && c < 2ll * cols) {
    if (c < cols)
      dw[c] = t;
    else if (db)
      db[c - cols] = t;
  }
}

int pow2_at_least(int n) {
  int p = 1;
  while (p < n) p <<= 1;
  return p;
}

// How a row of nv vectors is held: NV vectors to a thread, G threads to a row (a power of two
// up to 32, blocks of ROW_THREADS), or a whole block of `threads` (G = 0); NV = 0 when a
// block's registers do not hold the row.  A warp takes rows of up to two 16-byte vectors a lane: at
// 32768 x 512 bf16 the forward takes 25.0 us with warps and 24.6 with blocks, the backward 34 and 82
// (4 vectors a lane would hold dw and db of 64 columns a lane).
constexpr int ROW_THREADS = 128;
struct RowPlan {
  int NV, G, threads;
};
RowPlan plan_row(int nv, int warp_nv, int first_nv, int block_nv, int block_threads) {
  if (nv <= 32 * warp_nv) {
    const int G = nv >= 32 ? 32 : pow2_at_least(nv);
    return {pow2_at_least((nv + G - 1) / G), G, ROW_THREADS};
  }
  for (int n = first_nv; n <= block_nv; n *= 2) {
    const int most = n == block_nv ? block_threads : 256;  // small blocks while more vectors a thread are left
    if (nv <= most * n) return {n, 0, ((nv + n - 1) / n + 31) / 32 * 32};
  }
  return {0, 0, block_threads};
}

template <typename T, int VE>
cudaError_t fwd_typed(const LayerNormArgs& a, cudaStream_t st) {
  const int nv = a.cols / VE;
  constexpr int WNV = VE == 1 ? 8 : 2, BT = VE == 8 ? 512 : 1024;
  // (single elements: eight to a thread, so that fewer warps share a row's sums; 32768 x 1001 bf16: 87 us,
  // four to a thread 107)
  const RowPlan p = plan_row(nv, WNV, VE == 1 ? 8 : 2, 8, BT);
  const T *x = static_cast<const T*>(a.x), *r = static_cast<const T*>(a.r);
  T *y = static_cast<T*>(a.y), *s = static_cast<T*>(a.s);
  if (p.NV == 0) {
    norm_fwd_long_kernel<T, VE><<<a.rows, 512, 0, st>>>(x, r, a.w, a.b, y, s, a.mean, a.rstd, nv, a.eps);
    return cudaGetLastError();
  }
  const int per = p.G ? p.threads / p.G : 1;
  auto go = [&](auto kernel) {
    kernel<<<(unsigned)(((long long)a.rows + per - 1) / per), p.threads, 0, st>>>(x, r, a.w, a.b, y, s, a.mean, a.rstd,
                                                                                   a.rows, nv, p.G, a.eps);
    return cudaGetLastError();
  };
  const int held = p.G ? p.NV : 16 + p.NV;  // every plan has a case of its own
  if (held == 1) return go(norm_fwd_kernel<T, VE, 1, ROW_THREADS>);
  if (held == 2) return go(norm_fwd_kernel<T, VE, 2, ROW_THREADS>);
  if constexpr (VE == 1) {
    if (held == 4) return go(norm_fwd_kernel<T, VE, 4, ROW_THREADS>);
    if (held == 8) return go(norm_fwd_kernel<T, VE, 8, ROW_THREADS>);
    if (held == 16 + 8 && p.threads <= 128) return go(norm_fwd_kernel<T, VE, 8, 128>);
  } else {
    if (held == 16 + 2) return go(norm_fwd_kernel<T, VE, 2, 256>);
    if (held == 16 + 4) return go(norm_fwd_kernel<T, VE, 4, 256>);
  }
  return held == 16 + 8 ? go(norm_fwd_kernel<T, VE, 8, BT>) : cudaErrorInvalidValue;
}

// Blocks of the backward's row walk, and so partial rows of the workspace: four to an SM, which keep
// enough copies in flight, fewer when there are few rows.  Measured with 2, 4, 6 and 8 to an SM, 32768 rows of bf16
// without ds, us: 512 columns 43, 32, 42 and 38; 768 128, 73, 60 and 79; 1024 134, 79, 104 and 88; 1536 140, 86,
// 111 and 96; 2048 146, 96, 120 and 107; 16384 x 4096 99, 109, 120 and 127; fp32 4096 x 8192 142, 146, 156
// and 151.
constexpr int BWD_BLOCKS = 148 * 4;
int bwd_blocks(int rows) { return rows < BWD_BLOCKS ? (rows > 0 ? rows : 1) : BWD_BLOCKS; }

// the widest row that a block holds has 1024 vectors of 16 bytes: two stages of three rows
constexpr int BWD_SMEM_MOST = 2 * 3 * 1024 * 16;
template <typename T, int VE>
cudaError_t bwd_typed(const LayerNormBwdArgs& a, cudaStream_t st) {
  const int nv = a.cols / VE;
  constexpr int WNV = VE == 1 ? 8 : 2, BNV = VE == 1 ? 8 : 2;
  const RowPlan p = plan_row(nv, WNV, 2, BNV, 512);
  const T *dy = static_cast<const T*>(a.dy), *s = static_cast<const T*>(a.s), *ds = static_cast<const T*>(a.ds);
  T* dx = static_cast<T*>(a.dx);
  int P = bwd_blocks(a.rows);
  cudaError_t e;
  if (p.NV) {
    const int per = p.G ? p.threads / p.G : 1;
    if constexpr (VE > 1) {
      const long long need = ((long long)a.rows + per - 1) / per;
      if (need < P) P = (int)need;
      // stages: 48 KB a block where 2 to 8 of them fit (four blocks of 128 threads to an SM)
      const size_t stage = 3 * (size_t)per * a.cols * sizeof(T);
      int stages = (int)(49152 / stage);
      stages = stages < 2 ? 2 : stages > MAX_STAGES ? MAX_STAGES : stages;
      // (the row groups' sums go through the ring at the end: per x cols floats)
      const size_t acc = (size_t)per * a.cols * sizeof(float), smem = stage * stages > acc ? stage * stages : acc;
      auto go = [&](auto kernel, std::atomic<unsigned long long>& done) {
        cudaError_t e2 = smem_limit_once(kernel, BWD_SMEM_MOST, done);
        if (e2 != cudaSuccess) return e2;
        kernel<<<P, p.threads, smem, st>>>(dy, s, a.w, a.mean, a.rstd, ds, dx, a.part, a.rows, nv, p.G, stages,
                                           device_error_word());
        return cudaGetLastError();
      };
      static std::atomic<unsigned long long> done[4] = {};  // per kernel, a bit per device
      switch (p.G ? p.NV : 16 + p.NV) {
        case 1: e = go(norm_bwd_bulk_kernel<T, VE, 1, ROW_THREADS, 6>, done[0]); break;
        case 2: e = go(norm_bwd_bulk_kernel<T, VE, 2, ROW_THREADS, 4>, done[1]); break;
        default:  // (16 + 2)
          e = p.threads <= 128 ? go(norm_bwd_bulk_kernel<T, VE, 2, 128, 4>, done[2])
                               : go(norm_bwd_bulk_kernel<T, VE, 2, 512, 1>, done[3]);
      }
    } else {
      // rows at once: two where a thread has one element of each (262144 x 31 fp32: 71 us, one by one 104)
      const int R = p.NV == 1 ? 2 : 1;
      const long long need = ((long long)a.rows + per * R - 1) / (per * R);
      if (need < P) P = (int)need;
      const size_t smem = per > 1 ? (size_t)per * a.cols * sizeof(float) : 0;
      // four elements to a thread: bf16 fits 64 registers, and with them all of the blocks at once (32768 x
      // 1001: 136 us, with two to an SM 184); fp32 spills there (221 us, with two to an SM 182)
      constexpr int B4 = sizeof(T) == 2 ? 4 : 2;
      auto go = [&](auto kernel) {
        kernel<<<P, p.threads, smem, st>>>(dy, s, a.w, a.mean, a.rstd, ds, dx, a.part, a.rows, nv, p.G);
        return cudaGetLastError();
      };
      switch (p.G ? p.NV : 16 + p.NV) {
        case 1: e = go(norm_bwd_kernel<T, 1, 1, 2, ROW_THREADS, 6>); break;
        case 2: e = go(norm_bwd_kernel<T, 1, 2, 1, ROW_THREADS, 4>); break;
        case 4: e = go(norm_bwd_kernel<T, 1, 4, 1, ROW_THREADS, 4>); break;
        case 8: e = go(norm_bwd_kernel<T, 1, 8, 1, ROW_THREADS, 4>); break;
        case 16 + 2: e = go(norm_bwd_kernel<T, 1, 2, 1, 256, 4>); break;
        case 16 + 4: e = go(norm_bwd_kernel<T, 1, 4, 1, 256, B4>); break;
        default: e = go(norm_bwd_kernel<T, 1, 8, 1, 512, 1>); break;  // (16 + 8)
      }
    }
  } else {
    const int stretch = (a.rows + P - 1) / P;
    P = (int)(((long long)a.rows + stretch - 1) / stretch);
    norm_bwd_columns_kernel<T><<<dim3((a.cols + 255) / 256, P), 256, 0, st>>>(dy, s, a.mean, a.rstd, a.part, a.rows,
                                                                             a.cols, stretch);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    norm_bwd_long_kernel<T, VE><<<a.rows, 1024, 0, st>>>(dy, s, a.w, a.mean, a.rstd, ds, dx, nv);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)((2ll * a.cols + 31) / 32);
  return launch_after(norm_partials_kernel, grid, 1024, 0, st, a.part, a.dw, a.db, P, a.cols);
}

}  // namespace

size_t layer_norm_bwd_workspace_bytes(int rows, int cols) {
  return (size_t)bwd_blocks(rows) * 2 * (size_t)cols * sizeof(float);
}

cudaError_t launch_layer_norm_fwd(const LayerNormArgs& a, cudaStream_t st) {
  if (a.bf16) return a.cols % 8 == 0 ? fwd_typed<__nv_bfloat16, 8>(a, st) : fwd_typed<__nv_bfloat16, 1>(a, st);
  return a.cols % 4 == 0 ? fwd_typed<float, 4>(a, st) : fwd_typed<float, 1>(a, st);
}

cudaError_t launch_layer_norm_bwd(const LayerNormBwdArgs& a, cudaStream_t st) {
  if (a.rows == 0) {  // no rows: the parameters' gradients are zero
    cudaError_t e = cudaMemsetAsync(a.dw, 0, (size_t)a.cols * sizeof(float), st);
    if (e == cudaSuccess && a.db) e = cudaMemsetAsync(a.db, 0, (size_t)a.cols * sizeof(float), st);
    return e;
  }
  if (a.bf16) return a.cols % 8 == 0 ? bwd_typed<__nv_bfloat16, 8>(a, st) : bwd_typed<__nv_bfloat16, 1>(a, st);
  return a.cols % 4 == 0 ? bwd_typed<float, 4>(a, st) : bwd_typed<float, 1>(a, st);
}

}  // namespace gdn2
