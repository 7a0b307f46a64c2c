// Backward of the short causal depthwise convolution (4 taps over the token axis; the forward
// is short_conv.cu).  With e = token + 3 indexing [history (3) | tokens] of a sequence,
//
//     y[t] = bias + sum_j w[j] x[t - 3 + j]
//     dx[t] = sum_j w[j] dy[t + 3 - j]  (+ dhist_out[i] where token t is history slot i handed on)
//     dw[j] = sum over sequences and t of dy[t] x[t - 3 + j],    dbias = sum of dy
//     dhist_in[m] = sum_{j <= m} w[j] dy[m - j]  (+ dhist_out where a slot is handed on again)
//
// Bound by memory: x and dy are read once and dx is written once.  A thread walks a strip of
// tokens for four adjacent channels with the last three inputs and the next three gradients
// in registers; the next tokens of both tensors are being loaded while it works.  The sums over
// tokens stay in fp32 registers over the strip; each strip writes one partial row, and a
// second kernel adds the strips in order (the same result every time, no atomics).  A strip
// may cross sequences: inside a sequence no token is tested, at its ends each one is.
//
// 8 x 4096 x 2048 bf16: 71 us for the strips (403 MB at 5.7 TB/s) and 6 for the sums over them.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gdn2_internal.h"
#include "ptx.cuh"  // pairs of fp32 operations

namespace gdn2 {
namespace {

constexpr int THREADS = 128;
constexpr int END_THREADS = 512;  // of the kernel after it
constexpr int BLOCKS_PER_SM = 4;  // of the main kernel: at most 128 registers a thread

template <typename T>
struct Four;  // four adjacent channels as stored
template <>
struct Four<float> {
  using Raw = float4;
  static __device__ __forceinline__ float4 cvt(Raw v) { return v; }
};
template <>
struct Four<__nv_bfloat16> {
  using Raw = uint2;
  static __device__ __forceinline__ float4 cvt(Raw v) {
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xFFFF0000u));
  }
};
// (volatile: a strip's loads stay together, ahead of their uses)
__device__ __forceinline__ uint2 raw4(const __nv_bfloat16* p) {
  uint2 v;
  asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ float4 raw4(const float* p) {
  float4 v;
  asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
  return v;
}
template <typename T>
__device__ __forceinline__ float4 load4(const T* p) { return Four<T>::cvt(raw4(p)); }
// Of what this kernel also writes: not by the read-only path.
template <typename T>
__device__ __forceinline__ float4 plain4(const T* p) {
  return Four<T>::cvt(*reinterpret_cast<const typename Four<T>::Raw*>(p));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ float4 fma4(float4 a, float4 b, float4 c) {
  const float2 x = fma2(make_float2(a.x, a.y), make_float2(b.x, b.y), make_float2(c.x, c.y));
  const float2 y = fma2(make_float2(a.z, a.w), make_float2(b.z, b.w), make_float2(c.z, c.w));
  return make_float4(x.x, x.y, y.x, y.y);
}
__device__ __forceinline__ float4 add4(float4 a, float4 b) { return fma4(a, make_float4(1.f, 1.f, 1.f, 1.f), b); }
__device__ __forceinline__ float4 mul4(float4 a, float4 b) {
  const float2 x = mul2(make_float2(a.x, a.y), make_float2(b.x, b.y)), y = mul2(make_float2(a.z, a.w), make_float2(b.z, b.w));
  return make_float4(x.x, x.y, y.x, y.y);
}
__device__ __forceinline__ float4 zero4() { return make_float4(0.f, 0.f, 0.f, 0.f); }
// taps of four channels: t[j] = (w[c][j], w[c + 1][j], w[c + 2][j], w[c + 3][j])
__device__ __forceinline__ void load_taps(const float* w, float4 (&t)[4]) {
  const float4 a = load4(w), b = load4(w + 4), c = load4(w + 8), d = load4(w + 12);
  t[0] = make_float4(a.x, b.x, c.x, d.x);
  t[1] = make_float4(a.y, b.y, c.y, d.y);
  t[2] = make_float4(a.z, b.z, c.z, d.z);
  t[3] = make_float4(a.w, b.w, c.w, d.w);
}

// Sequence of flat token g: fixed length T, or the packed offsets cu[0..nseq].
__device__ __forceinline__ int seq_at(int g, const int* cu, int nseq, int T) {
  if (!cu) return g / T;
  int lo = 0, hi = nseq;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= g) lo = mid; else hi = mid;
  }
  return lo;
}

// part: [strip][5][C] (the four taps, then the bias).  blockIdx.x = strip * ncb + channel block.
template <typename T>
__global__ void __launch_bounds__(THREADS, BLOCKS_PER_SM) short_conv_bwd_kernel(const T* __restrict__ dy, const T* __restrict__ x,
                                                                const float* __restrict__ w, const int* cu, int nseq,
                                                                const T* __restrict__ hist,
                                                                const T* __restrict__ dhist_out, T* __restrict__ dx,
                                                                float* __restrict__ part, int ntok, int T_seq, int C,
                                                                int ncb, int strip_len, unsigned* err) {
  constexpr int U = 16 / (int)sizeof(T);  // tokens loaded at once: 64 bytes of each tensor a thread
  const int cb = blockIdx.x % ncb, strip = blockIdx.x / ncb;
  const int c = 4 * (cb * THREADS + threadIdx.x);
  if (c >= C) return;
  grid_release();
  const int g0 = strip * strip_len, g1 = (int)min((long long)g0 + strip_len, (long long)ntok);
  float4 acc[5] = {zero4(), zero4(), zero4(), zero4(), zero4()};
  int n = seq_at(g0, cu, nseq, T_seq);
  int start = cu ? cu[n] : n * T_seq;
  int next = cu ? cu[n + 1] : start + T_seq;
  // packed offsets are checked where they are used: what they lead to stays inside the tensors
  bool ok = !cu || (cu[0] == 0 && cu[nseq] == ntok && start >= 0 && start <= g0 && next > g0 && next <= ntok);
  if (ok) {
    float4 wt[4];
    load_taps(w + 4 * (size_t)c, wt);
    const T* xc = x + c;
    const T* dc = dy + c;
    float4 h[3];  // x at g - 3, g - 2, g - 1
    float4 d[3];  // dy at g, g + 1, g + 2 (what lies in the strip's sequence)
    auto hist_at = [&](int slot) { return hist ? load4(hist + ((size_t)n * 3 + slot) * C + c) : zero4(); };
    auto window = [&](int g) {  // both windows at token g of sequence n
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        const int p = g - 3 + j;
        h[j] = p >= start ? load4(xc + (size_t)p * C) : hist_at(p - start + 3);
        d[j] = g + j < next ? load4(dc + (size_t)(g + j) * C) : zero4();
      }
    };
    auto token = [&](float4 xg, float4 d3) {  // x at g, dy at g + 3
      acc[0] = fma4(d[0], h[0], acc[0]);
      acc[1] = fma4(d[0], h[1], acc[1]);
      acc[2] = fma4(d[0], h[2], acc[2]);
      acc[3] = fma4(d[0], xg, acc[3]);
      acc[4] = add4(acc[4], d[0]);
      const float4 o = fma4(wt[0], d3, fma4(wt[1], d[2], fma4(wt[2], d[1], mul4(wt[3], d[0]))));
      h[0] = h[1], h[1] = h[2], h[2] = xg;
      d[0] = d[1], d[1] = d[2], d[2] = d3;
      return o;
    };
    window(g0);
    int g = g0;
    while (g < g1) {
      if (g >= next) {  // the next sequence that has tokens
        while (g >= next && n + 1 < nseq) {
          ++n;
          start = next;
          next = cu ? cu[n + 1] : start + T_seq;
        }
        if (start < 0 || g < start || g >= next || next > ntok) {  // offsets out of order
          ok = false;
          break;
        }
        window(g);
      }
      const int run = min(g1, next);
      // inside the sequence: dy up to g + U + 2 exists, and no token hands on its input
      const int fast = dhist_out ? min(run, next - 3) : run;
      if (g + U <= fast && g + U + 3 <= next) {
        typename Four<T>::Raw xs[U], ds[U], xn[U], dn[U];  // as stored (converted when used: fewer registers)
        auto fetch = [&](int at, typename Four<T>::Raw (&xr)[U], typename Four<T>::Raw (&dr)[U]) {
#pragma unroll
          for (int i = 0; i < U; ++i) {
            xr[i] = raw4(xc + (size_t)(at + i) * C);
            dr[i] = raw4(dc + (size_t)(at + 3 + i) * C);
          }
        };
        fetch(g, xs, ds);
        for (bool more = true; more;) {  // the next tokens' loads are in flight while these are used
          more = g + 2 * U <= fast && g + 2 * U + 3 <= next;
          if (more) fetch(g + U, xn, dn);
#pragma unroll
          for (int i = 0; i < U; ++i)
            store4(dx + (size_t)(g + i) * C + c, token(Four<T>::cvt(xs[i]), Four<T>::cvt(ds[i])));
#pragma unroll
          for (int i = 0; i < U; ++i) xs[i] = xn[i], ds[i] = dn[i];
          g += U;
        }
      }
      // the rest of the run token by token, up to where a fast run may start again
      const int stop = min(run, g + U);
      for (; g < stop; ++g) {
        const float4 xg = load4(xc + (size_t)g * C);
        const float4 d3 = g + 3 < next ? load4(dc + (size_t)(g + 3) * C) : zero4();
        float4 o = token(xg, d3);
        const int slot = g - (next - 3);  // >= 0: this token's input is handed on in that slot
        if (dhist_out && slot >= 0) o = add4(o, load4(dhist_out + ((size_t)n * 3 + slot) * C + c));
        store4(dx + (size_t)g * C + c, o);
      }
    }
  }
  if (!ok && threadIdx.x == 0 && err) atomicOr(err, kErrBadSeqlens);
  float* out = part + (size_t)strip * 5 * C + c;
#pragma unroll
  for (int j = 0; j < 5; ++j) store4(out + (size_t)j * C, acc[j]);
}

// What is left after the strips, in one launch: the first `sums` blocks add up the partial rows, the
// others form the gradient of the history that the sequences entered with.
//
// Sums of the strips' partial rows, in order (16 walkers to a column): dweight [C, 4], dbias [C].  (part without
// __restrict__: it may be written while this grid waits, so its loads stay behind the wait and on the coherent
// path.)
__device__ __forceinline__ void sum_partials(const float* part, float* __restrict__ dw, float* __restrict__ db,
                                             int strips, int C, float (*red)[33]) {
  const int lane = threadIdx.x & 31, wk = threadIdx.x >> 5;
  const long long n = 5ll * C;
  long long i = (long long)blockIdx.x * 32 + lane;
  float t = 0.f;
  if (i < n) {
#pragma unroll 10
    for (int s = wk; s < strips; s += 16) t += part[(size_t)s * n + i];
  }
  red[wk][lane] = t;
  __syncthreads();
#pragma unroll
  for (int half = 0; half < 2; ++half) {  // warp wk adds up columns wk and wk + 16 of the block's 32
    const int col = wk + 16 * half;
    t = red[lane & 15][col];
#pragma unroll
    for (int off = 8; off; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    i = (long long)blockIdx.x * 32 + col;
    if (lane == 0 && i < n) {
      const int j = (int)(i / C), c = (int)(i % C);
      if (j < 4)
        dw[4 * (size_t)c + j] = t;
      else if (db)
        db[c] = t;
    }
  }
}

// Gradient of the history a sequence entered with; a thread per (sequence, four channels).  dhist may be
// dhist_out, which is therefore read by plain loads.
template <typename T>
__device__ __forceinline__ void history_gradient(const T* __restrict__ dy, const float* __restrict__ w, const int* cu,
                                                 const T* dhist_out, T* dhist, int ntok, int T_seq, int C, long long at,
                                                 int N, unsigned* err) {
  const int n = (int)(at / (C / 4)), c = 4 * (int)(at % (C / 4));
  if (n >= N) return;
  const int start = cu ? cu[n] : n * T_seq, end = cu ? cu[n + 1] : start + T_seq;
  if (start < 0 || end < start || end > ntok) {
    if (err) atomicOr(err, kErrBadSeqlens);
    return;
  }
  const int len = end - start;
  float4 wt[4], d[3], o[3];
  load_taps(w + 4 * (size_t)c, wt);
#pragma unroll
  for (int i = 0; i < 3; ++i) d[i] = i < len ? load4(dy + (size_t)(start + i) * C + c) : zero4();
#pragma unroll
  for (int m = 0; m < 3; ++m) {
    o[m] = zero4();
#pragma unroll
    for (int j = 0; j <= m; ++j) o[m] = fma4(wt[j], d[m - j], o[m]);
    if (dhist_out && m >= len) o[m] = add4(o[m], plain4(dhist_out + ((size_t)n * 3 + m - len) * C + c));
  }
#pragma unroll
  for (int m = 0; m < 3; ++m) store4(dhist + ((size_t)n * 3 + m) * C + c, o[m]);
}

template <typename T>
__global__ void __launch_bounds__(END_THREADS)
    short_conv_bwd_end_kernel(const float* part, float* __restrict__ dw, float* __restrict__ db, int strips,
                              int sums, const T* __restrict__ dy, const float* __restrict__ w, const int* cu,
                              const T* dhist_out, T* dhist, int ntok, int T_seq, int C, int N, unsigned* err) {
  __shared__ float red[16][33];
  grid_wait();
  if ((int)blockIdx.x < sums)
    sum_partials(part, dw, db, strips, C, red);
  else
    history_gradient<T>(dy, w, cu, dhist_out, dhist, ntok, T_seq, C,
                        (long long)(blockIdx.x - sums) * END_THREADS + threadIdx.x, N, err);
}

// Tokens of a strip: as many strips as fill 148 SMs once with four blocks each (8 x 4096 x 2048 bf16:
// 77 us; with two blocks 95, in two turns 85), but 16 tokens at least (1024 x 2048 bf16: 9.2 us; with 64
// 11.5, with 4 10.6).  Each strip writes a partial row of 20 bytes a channel: at 200 tokens 2 to 5 % of
// its own traffic.
int strip_tokens(long long ntok, int C) {
  const long long ncb = (C / 4 + THREADS - 1) / THREADS;
  const long long strips = ncb < 148 * BLOCKS_PER_SM ? 148 * BLOCKS_PER_SM / ncb : 1;
  const long long len = (ntok + strips - 1) / strips;
  return len < 16 ? 16 : (int)len;
}

template <typename T>
cudaError_t launch_typed(const ShortConvBwdArgs& a, cudaStream_t st) {
  const int ntok = a.B == 0 ? 0 : a.cu_seqlens ? a.T : a.B * a.T;
  const int ncb = (a.C / 4 + THREADS - 1) / THREADS;
  const int len = strip_tokens(ntok, a.C), strips = (int)(((long long)ntok + len - 1) / len);
  const T *dy = static_cast<const T*>(a.dy), *x = static_cast<const T*>(a.x);
  const T *hist = static_cast<const T*>(a.hist_in), *dho = static_cast<const T*>(a.dhist_out);
  cudaError_t e;
  if (strips > 0) {
    const long long blocks = (long long)strips * ncb;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    short_conv_bwd_kernel<T><<<(unsigned)blocks, THREADS, 0, st>>>(dy, x, a.weight, a.cu_seqlens, a.B, hist, dho,
                                                                  static_cast<T*>(a.dx), a.part, ntok, a.T, a.C, ncb,
                                                                  len, device_error_word());
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  // (no tokens: no strips, and the sums over them are zero)
  const int sums = (int)((5ll * a.C + 31) / 32);
  const long long blocks = sums + (a.dhist ? ((long long)a.B * (a.C / 4) + END_THREADS - 1) / END_THREADS : 0);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_after(short_conv_bwd_end_kernel<T>, (unsigned)blocks, END_THREADS, 0, st, a.part, a.dweight, a.dbias, strips,
                      sums, dy, a.weight, a.cu_seqlens, dho, static_cast<T*>(a.dhist), ntok, a.T, a.C, a.B,
                      device_error_word());
}

}  // namespace

size_t short_conv_bwd_workspace_bytes(long long ntok, int C) {
  if (ntok <= 0 || C <= 0) return 0;
  const int len = strip_tokens(ntok, C);
  return (size_t)((ntok + len - 1) / len) * 5 * (size_t)C * sizeof(float);
}

cudaError_t launch_short_conv_bwd(const ShortConvBwdArgs& a, cudaStream_t st) {
  return a.bf16 ? launch_typed<__nv_bfloat16>(a, st) : launch_typed<float>(a, st);
}

}  // namespace gdn2
