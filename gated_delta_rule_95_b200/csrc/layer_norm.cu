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
// 8 x 32 vectors (shuffles only, several rows to a warp when they are narrow), whole blocks
// above that; rows past what a block's registers hold are read again for each pass (the
// second and third reading come from the caches).  A vector is 16 bytes when a row's bytes
// divide by 16 and one element otherwise.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gdn2_internal.h"

namespace gdn2 {
namespace {

// VE adjacent elements as floats: one 16-byte access (VE = 16 / sizeof(T)) or one element.
template <typename T, int VE>
struct Vec;
template <>
struct Vec<float, 4> {
  static __device__ __forceinline__ void load(const float* p, float (&f)[4]) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&f)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <>
struct Vec<__nv_bfloat16, 8> {
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&f)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t r[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(r[i] << 16);
      f[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[8]) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      r[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(r[0], r[1], r[2], r[3]);
  }
};
template <>
struct Vec<float, 1> {
  static __device__ __forceinline__ void load(const float* p, float (&f)[1]) { f[0] = *p; }
  static __device__ __forceinline__ void store(float* p, const float (&f)[1]) { *p = f[0]; }
};
template <>
struct Vec<__nv_bfloat16, 1> {
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&f)[1]) { f[0] = __bfloat162float(*p); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[1]) { *p = __float2bfloat16_rn(f[0]); }
};
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

// Sum of N values over the G threads of a row (G a power of two up to 32: lanes that differ
// in their low bits; G = 0: the whole block), the result in each of them.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], int G, float (*red)[MAX_WARPS]) {
  const int width = G ? G : 32;
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    if (off < width) {
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], off);
    }
  }
  if (G) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  __syncthreads();  // the previous sum's readers are done with red
  if (lane == 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) red[n][warp] = v[n];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float x = lane < nw ? red[n][lane] : 0.f;
#pragma unroll
    for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    v[n] = x;
  }
}

// ---------------------------------------------------------------------------- forward

// NV > 0: a row's vectors in registers, NV to a thread.  NV = 0: rows of any length, read
// once for the mean, once for the variance and once for the outputs.
// G: threads of a row (0 = the block, one row at a time); nv = vectors of a row.
template <typename T, int VE, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_fwd_kernel(const T* x, const T* r, const float* __restrict__ w,
                                                        const float* __restrict__ b, T* y, T* s,
                                                        float* __restrict__ mean, float* __restrict__ rstd, int rows,
                                                        int nv, int G, float eps) {
  __shared__ float red[1][MAX_WARPS];
  using V = Vec<T, VE>;
  const int gw = G ? G : blockDim.x;             // threads of a row
  const int per = blockDim.x / gw;               // rows of a block
  const int j0 = threadIdx.x & (gw - 1);         // (G is a power of two; per == 1 otherwise)
  const int jt = G ? j0 : (int)threadIdx.x;
  const long long row = (long long)blockIdx.x * per + (G ? threadIdx.x / gw : 0);
  const bool live = row < rows;                  // every thread stays for the shuffles
  const size_t base = (size_t)(live ? row : 0) * nv * VE;
  const float cols = (float)nv * VE;  // (at most 2^24: exact; divided by, so that a constant row has no variance)
  auto load_sum = [&](int j, float (&f)[VE]) {
    V::load(x + base + (size_t)j * VE, f);
    if (r) {
      float e[VE];
      V::load(r + base + (size_t)j * VE, e);
#pragma unroll
      for (int i = 0; i < VE; ++i) f[i] = round_to(f[i] + e[i], T());
    }
  };
  auto store_out = [&](int j, const float (&f)[VE], float mu, float rho) {
    float wv[VE], bv[VE], o[VE];
    load_f32<VE>(w + (size_t)j * VE, wv);
    if (b) load_f32<VE>(b + (size_t)j * VE, bv);
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const float t = (f[i] - mu) * rho;
      o[i] = b ? fmaf(t, wv[i], bv[i]) : t * wv[i];
    }
    V::store(y + base + (size_t)j * VE, o);
    if (s) V::store(s + base + (size_t)j * VE, f);
  };
  float mu, rho;
  if constexpr (NV > 0) {
    float f[NV][VE];
    float sum[1] = {0.f};
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int j = jt + n * gw;
      if (live && j < nv) {
        load_sum(j, f[n]);
      } else {
#pragma unroll
        for (int i = 0; i < VE; ++i) f[n][i] = 0.f;
      }
    }
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int i = 0; i < VE; ++i) sum[0] += f[n][i];
    group_sum<1>(sum, G, red);
    mu = sum[0] / cols;
    float sq[1] = {0.f};
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      if (jt + n * gw < nv) {
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          const float d = f[n][i] - mu;
          sq[0] = fmaf(d, d, sq[0]);
        }
      }
    }
    group_sum<1>(sq, G, red);
    rho = rsqrtf(sq[0] / cols + eps);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int j = jt + n * gw;
      if (live && j < nv) store_out(j, f[n], mu, rho);
    }
  } else {
    float sum[1] = {0.f}, sq[1] = {0.f}, f[VE];
    for (int j = jt; j < nv; j += gw) {
      load_sum(j, f);
#pragma unroll
      for (int i = 0; i < VE; ++i) sum[0] += f[i];
    }
    group_sum<1>(sum, G, red);
    mu = sum[0] / cols;
    for (int j = jt; j < nv; j += gw) {
      load_sum(j, f);
#pragma unroll
      for (int i = 0; i < VE; ++i) sq[0] = fmaf(f[i] - mu, f[i] - mu, sq[0]);
    }
    group_sum<1>(sq, G, red);
    rho = rsqrtf(sq[0] / cols + eps);
    for (int j = jt; j < nv; j += gw) {
      load_sum(j, f);
      store_out(j, f, mu, rho);
    }
  }
  if (live && jt == 0) {
    if (mean) mean[row] = mu;
    if (rstd) rstd[row] = rho;
  }
}

// --------------------------------------------------------------------------- backward

// A block walks rows blockIdx.x * per + i * gridDim.x * per with its columns fixed to its
// threads (NV vectors each), so dw and db accumulate in registers; at the end the block's
// row groups are added up in shared memory and one partial row [dw | db] is written.
template <typename T, int VE, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_bwd_kernel(const T* dy, const T* s, const float* __restrict__ w,
                                                        const float* __restrict__ mean,
                                                        const float* __restrict__ rstd, const T* ds, T* dx,
                                                        float* __restrict__ part, int rows, int nv, int G) {
  __shared__ float red[2][MAX_WARPS];
  extern __shared__ float acc[];  // [per][cols] of one sum at a time (G > 0)
  using V = Vec<T, VE>;
  const int gw = G ? G : blockDim.x, per = blockDim.x / gw;
  const int jt = G ? (threadIdx.x & (gw - 1)) : threadIdx.x, grp = G ? threadIdx.x / gw : 0;
  const int cols = nv * VE;
  const float inv = 1.f / (float)cols;
  float dw[NV][VE], db[NV][VE], wv[NV][VE];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int j = jt + n * gw;
#pragma unroll
    for (int i = 0; i < VE; ++i) dw[n][i] = db[n][i] = wv[n][i] = 0.f;
    if (j < nv) load_f32<VE>(w + (size_t)j * VE, wv[n]);
  }
  for (long long row0 = (long long)blockIdx.x * per; row0 < rows; row0 += (long long)gridDim.x * per) {
    const long long row = row0 + grp;
    const bool live = row < rows;
    const size_t base = (size_t)(live ? row : 0) * cols;
    const float mu = live ? __ldg(mean + row) : 0.f, rho = live ? __ldg(rstd + row) : 0.f;
    float g[NV][VE], xh[NV][VE];
    float sums[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int j = jt + n * gw;
      if (live && j < nv) {
        V::load(dy + base + (size_t)j * VE, g[n]);
        V::load(s + base + (size_t)j * VE, xh[n]);
      } else {
#pragma unroll
        for (int i = 0; i < VE; ++i) g[n][i] = 0.f, xh[n][i] = mu;
      }
    }
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        xh[n][i] = (xh[n][i] - mu) * rho;
        db[n][i] += g[n][i];
        dw[n][i] = fmaf(g[n][i], xh[n][i], dw[n][i]);
        g[n][i] *= wv[n][i];
        sums[0] += g[n][i];
        sums[1] = fmaf(g[n][i], xh[n][i], sums[1]);
      }
    group_sum<2>(sums, G, red);
    const float m0 = sums[0] * inv, m1 = sums[1] * inv;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int j = jt + n * gw;
      if (live && j < nv) {
        float o[VE], e[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i) o[i] = rho * (g[n][i] - m0 - xh[n][i] * m1);
        if (ds) {
          V::load(ds + base + (size_t)j * VE, e);
#pragma unroll
          for (int i = 0; i < VE; ++i) o[i] += e[i];
        }
        V::store(dx + base + (size_t)j * VE, o);
      }
    }
  }
  float* out = part + (size_t)blockIdx.x * 2 * cols;
  if (per == 1) {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int j = jt + n * gw;
      if (j < nv) {
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          out[(size_t)j * VE + i] = dw[n][i];
          out[cols + (size_t)j * VE + i] = db[n][i];
        }
      }
    }
    return;
  }
  for (int half = 0; half < 2; ++half) {
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int j = jt + n * gw;
      if (j < nv) {
#pragma unroll
        for (int i = 0; i < VE; ++i) acc[grp * cols + j * VE + i] = half ? db[n][i] : dw[n][i];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += blockDim.x) {
      float t = 0.f;
      for (int q = 0; q < per; ++q) t += acc[q * cols + c];
      out[half * cols + c] = t;
    }
  }
}

// Rows of any length: dx alone, the row read twice (the second time from the caches).
template <typename T, int VE>
__global__ void __launch_bounds__(1024) norm_bwd_long_kernel(const T* dy, const T* s, const float* __restrict__ w,
                                                             const float* __restrict__ mean,
                                                             const float* __restrict__ rstd, const T* ds, T* dx,
                                                             int nv) {
  __shared__ float red[2][MAX_WARPS];
  using V = Vec<T, VE>;
  const size_t base = (size_t)blockIdx.x * nv * VE;
  const float mu = __ldg(mean + blockIdx.x), rho = __ldg(rstd + blockIdx.x), inv = 1.f / ((float)nv * VE);
  float sums[2] = {0.f, 0.f}, g[VE], xh[VE], wv[VE];
  auto load = [&](int j) {
    V::load(dy + base + (size_t)j * VE, g);
    V::load(s + base + (size_t)j * VE, xh);
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
      V::load(ds + base + (size_t)j * VE, e);
#pragma unroll
      for (int i = 0; i < VE; ++i) o[i] += e[i];
    }
    V::store(dx + base + (size_t)j * VE, o);
  }
}
// Its dw and db: a thread per column over a stretch of rows (partials as norm_bwd_kernel's).
// Runs before dx is written, so dx may alias dy or ds.
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
    Vec<T, 1>::load(dy + (size_t)r * cols + c, g);
    Vec<T, 1>::load(s + (size_t)r * cols + c, x);
    db += g[0];
    dw = fmaf(g[0], (x[0] - __ldg(mean + r)) * __ldg(rstd + r), dw);
  }
  part[(size_t)blockIdx.y * 2 * cols + c] = dw;
  part[(size_t)blockIdx.y * 2 * cols + cols + c] = db;
}

// out[c] = sum over the P partial rows, in the order of the rows (the same result every
// time): 8 row walkers to a column, added up at the end.
__global__ void __launch_bounds__(256) norm_partials_kernel(const float* __restrict__ part, float* __restrict__ dw,
                                                            float* __restrict__ db, int P, int cols) {
  __shared__ float red[8][33];
  const int lane = threadIdx.x & 31, wk = threadIdx.x >> 5;
  const long long c = (long long)blockIdx.x * 32 + lane;  // over [dw | db]
  float t = 0.f;
  if (c < 2ll * cols)
    for (int p = wk; p < P; p += 8) t += part[(size_t)p * 2 * cols + c];
  red[wk][lane] = t;
  __syncthreads();
  if (wk == 0 && c < 2ll * cols) {
#pragma unroll
    for (int q = 1; q < 8; ++q) t += red[q][lane];
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
// block's registers do not hold the row.
constexpr int ROW_THREADS = 128;
struct RowPlan {
  int NV, G, threads;
};
RowPlan plan_row(int nv, int warp_nv, int block_nv, int block_threads) {
  if (nv <= 32 * warp_nv) {
    const int G = nv >= 32 ? 32 : pow2_at_least(nv);
    return {pow2_at_least((nv + G - 1) / G), G, ROW_THREADS};
  }
  for (int n = 1; n <= block_nv; n *= 2) {
    const int most = n == block_nv ? block_threads : 256;  // small blocks while more vectors a thread are left
    if (nv <= most * n) return {n, 0, ((nv + n - 1) / n + 31) / 32 * 32};
  }
  return {0, 0, block_threads};
}

template <typename T, int VE>
cudaError_t fwd_typed(const LayerNormArgs& a, cudaStream_t st) {
  const int nv = a.cols / VE;
  const RowPlan p = plan_row(nv, 8, 8, VE == 8 ? 512 : 1024);
  const int per = p.G ? p.threads / p.G : 1;
  const unsigned grid = (unsigned)(((long long)a.rows + per - 1) / per);
  auto go = [&](auto kernel) {
    kernel<<<grid, p.threads, 0, st>>>(static_cast<const T*>(a.x), static_cast<const T*>(a.r), a.w, a.b,
                                       static_cast<T*>(a.y), static_cast<T*>(a.s), a.mean, a.rstd, a.rows, nv, p.G,
                                       a.eps);
    return cudaGetLastError();
  };
  constexpr int BT = VE == 8 ? 512 : 1024;
  switch (p.G ? p.NV : 16 + p.NV) {
    case 1: return go(norm_fwd_kernel<T, VE, 1, ROW_THREADS>);
    case 2: return go(norm_fwd_kernel<T, VE, 2, ROW_THREADS>);
    case 4: return go(norm_fwd_kernel<T, VE, 4, ROW_THREADS>);
    case 8: return go(norm_fwd_kernel<T, VE, 8, ROW_THREADS>);
    case 16 + 2: return go(norm_fwd_kernel<T, VE, 2, BT>);
    case 16 + 4: return go(norm_fwd_kernel<T, VE, 4, BT>);
    case 16 + 8: return go(norm_fwd_kernel<T, VE, 8, BT>);
    default: return go(norm_fwd_kernel<T, VE, 0, BT>);
  }
}

// Blocks of the backward's row walk, and so partial rows of the workspace: enough to fill
// 148 SMs several times over, fewer when there are few rows.
constexpr int BWD_BLOCKS = 148 * 4;
int bwd_blocks(int rows) { return rows < BWD_BLOCKS ? (rows > 0 ? rows : 1) : BWD_BLOCKS; }

template <typename T, int VE>
cudaError_t bwd_typed(const LayerNormBwdArgs& a, cudaStream_t st) {
  const int nv = a.cols / VE;
  constexpr int WNV = VE == 1 ? 8 : 2, BNV = VE == 1 ? 8 : 2;
  const RowPlan p = plan_row(nv, WNV, BNV, 512);
  const T *dy = static_cast<const T*>(a.dy), *s = static_cast<const T*>(a.s), *ds = static_cast<const T*>(a.ds);
  T* dx = static_cast<T*>(a.dx);
  int P = bwd_blocks(a.rows);
  cudaError_t e;
  if (p.NV) {
    const int per = p.G ? p.threads / p.G : 1;
    const long long need = ((long long)a.rows + per - 1) / per;
    if (need < P) P = (int)need;
    const size_t smem = per > 1 ? (size_t)per * a.cols * sizeof(float) : 0;
    auto go = [&](auto kernel) {
      kernel<<<P, p.threads, smem, st>>>(dy, s, a.w, a.mean, a.rstd, ds, dx, a.part, a.rows, nv, p.G);
      return cudaGetLastError();
    };
    switch (p.G ? p.NV : 16 + p.NV) {
      case 1: e = go(norm_bwd_kernel<T, VE, 1, ROW_THREADS>); break;
      case 2: e = go(norm_bwd_kernel<T, VE, 2, ROW_THREADS>); break;
      case 4: e = go(norm_bwd_kernel<T, VE, WNV == 8 ? 4 : 2, ROW_THREADS>); break;
      case 8: e = go(norm_bwd_kernel<T, VE, WNV == 8 ? 8 : 2, ROW_THREADS>); break;
      case 16 + 1: e = go(norm_bwd_kernel<T, VE, 1, 512>); break;
      case 16 + 2: e = go(norm_bwd_kernel<T, VE, 2, 512>); break;
      case 16 + 4: e = go(norm_bwd_kernel<T, VE, BNV == 8 ? 4 : 2, 512>); break;
      default: e = go(norm_bwd_kernel<T, VE, BNV == 8 ? 8 : 2, 512>); break;
    }
  } else {
    const int stretch = (a.rows + P - 1) / P;
    P = (a.rows + stretch - 1) / stretch;
    norm_bwd_columns_kernel<T><<<dim3((a.cols + 255) / 256, P), 256, 0, st>>>(dy, s, a.mean, a.rstd, a.part, a.rows,
                                                                             a.cols, stretch);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    norm_bwd_long_kernel<T, VE><<<a.rows, 1024, 0, st>>>(dy, s, a.w, a.mean, a.rstd, ds, dx, nv);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)((2ll * a.cols + 31) / 32);
  norm_partials_kernel<<<grid, 256, 0, st>>>(a.part, a.dw, a.db, P, a.cols);
  return cudaGetLastError();
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
