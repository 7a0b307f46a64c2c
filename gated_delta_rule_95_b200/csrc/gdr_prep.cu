// Scalar-gate prefill, what does not depend on the state (gdr_chain.cu has the formulas): for every
// chunk of 64 tokens and value head the decays' factors, P, and T = (I + A)^-1 diag(beta) with
//
//     A_ts = beta_t e^(G_t - G_s) k_t . k_s  (s < t),    P_ts = scale e^(G_t - G_s) q_t . k_s  (s <= t)
//
// All chunks at once, a block of 128 threads each, six blocks to an SM (the chain of steps inside a
// chunk is long; what hides it is other chunks).  [K; Q] K^T is one tcgen05 product of 128 x 64, a
// row of it to a thread.  A and T are fp32 in shared memory: 8 x 8 diagonal blocks by substitution,
// then T_IJ = -T_II (A_IJ T_JJ) for blocks of 8 (FMA), 16 and 32 (warp-level tf32 products of split
// operands, 2^-21; they are too small for tcgen05).  Substitution in blocks is stable where powers
// of A are not (one key repeated: A is all ones).  The record leaves by two bulk stores, P's second part by
// plain ones to the rows of o (gdr_chain.cu).
//
// Bound by neither memory nor issue alone: 85 us for 8192 chunks at d = 128 (444 MB of q, k, records and second
// parts, 5.2 TB/s; without the second parts 80 us, shared memory 68 % busy, issue slots 44 %, a quarter of a
// warp's time at the block's barriers).
// Measured on the way: A and P on warp-level products and four blocks to an SM 112 us, records of
// whole 64 x 64 tiles (26 KB) 87 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn2_internal.h"
#include "gdr_chunk.cuh"
#include "ptx.cuh"

namespace gdn2 {
namespace {

constexpr int C = GDR_C;
constexpr int NT = 128;
constexpr int LDM = 68;  // row stride of M: rows 4 banks apart
constexpr uint32_t R64 = 64 * 128, R128 = 128 * 128;  // panels of 64 channels: rows of 128 bytes
constexpr int WAIT_TRIES = 2000;                      // suspensions of 1 ms

// shared memory (from a 1024-byte aligned base): [K; Q] tiles, whose place M (fp32 A and T), P and X
// take; and T's parts and the gates M's in the end; the factors
constexpr uint32_t OFF_P = 64 * LDM * 4;
constexpr uint32_t OFF_X = OFF_P + GDR_TRI;  // [32][LDX]
constexpr int LDX = 36;
static_assert(GDR_P <= OFF_P, "T and the gates in M's place");
__host__ __device__ constexpr uint32_t off_f(int dk) {
  return (uint32_t)(dk / 64) * R128 > OFF_X + 32 * LDX * 4 ? (uint32_t)(dk / 64) * R128 : OFF_X + 32 * LDX * 4;
}
struct Factors {
  alignas(16) double G[C];     // log2 decay summed up to t
  GdrGates out;
  alignas(16) float mid[C];    // e^(G_m - G_t), m = the chunk's middle (mild chunks)
  alignas(16) float rowA[C];   // beta e^(G_t - G_m); not mild: beta
  alignas(16) float rowP[C];   // scale e^(G_t - G_C); not mild: scale
  alignas(16) float beta[C];
  uint64_t full, done;         // the tiles landed; their product is there
  uint32_t tmem_base;
};
__host__ __device__ constexpr uint32_t smem_bytes(int dk) {
  return off_f(dk) + (uint32_t)sizeof(Factors) + 1024;
}

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
// x = hi + lo, hi its upper 10 mantissa bits.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xFFFFE000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}
struct PrepParams {
  const float *g, *beta;
  const int* cu;
  unsigned char* records;
  __nv_bfloat16* o;  // [.., T, Hv, dv]: the place of P's second part
  int N, T, Hk, Hv, dv;
  float scale;
  unsigned* err;
};

template <int DK>
__global__ void __launch_bounds__(NT, 6) gdr_prep_kernel(const __grid_constant__ CUtensorMap tmQ,
                                                         const __grid_constant__ CUtensorMap tmK, const PrepParams p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float* M = reinterpret_cast<float*>(sm);
  float* X = reinterpret_cast<float*>(sm + OFF_X);
  Factors& f = *reinterpret_cast<Factors*>(sm + off_f(DK));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g4 = lane >> 2, t4 = lane & 3;
  const int hv = blockIdx.x % p.Hv, hk = hv / (p.Hv / p.Hk);
  const long long slot = blockIdx.x / p.Hv;
  // this block's sequence and chunk
  long long first;  // flat token index of the chunk
  int live;         // its tokens
  int tb = 0, t0;   // tensor-map coordinates
  if (p.cu) {
    int lo = 0, hi = p.N;  // the last sequence that starts at or before the slot
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((long long)(p.cu[mid] >> 6) + mid <= slot) lo = mid; else hi = mid;
    }
    const int s0 = p.cu[lo], s1 = p.cu[lo + 1];
    const long long c = slot - ((s0 >> 6) + lo);
    if (s0 < 0 || s1 < s0 || s1 > p.T || c < 0 || c * C >= s1 - s0) return;  // (bad offsets: the chain reports them)
    first = s0 + c * C;
    live = (int)min((long long)C, s1 - first);
    t0 = (int)first;
  } else {
    const int nch = (p.T + C - 1) / C, c = (int)(slot % nch);
    tb = (int)(slot / nch);
    t0 = c * C;
    first = (long long)tb * p.T + t0;
    live = min(C, p.T - t0);
  }

  if (tid == 0) {
    mbar_init(&f.full, 1), mbar_init(&f.done, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(&f.full, (uint32_t)(DK / 64) * R128);
#pragma unroll
    for (int pn = 0; pn < DK / 64; ++pn) {
      tma_load_4d(sm + pn * R128, &tmK, &f.full, 64 * pn, hk, t0, tb);
      tma_load_4d(sm + pn * R128 + R64, &tmQ, &f.full, 64 * pn, hk, t0, tb);
    }
  }
  if (warp == 2) {
    tmem_alloc(&f.tmem_base, 64);
    tmem_relinquish();
  }
  const float beta = tid < live && tid < C ? __ldg(p.beta + (size_t)(first + tid) * p.Hv + hv) : 0.f;
  // the log decays' sums, two tokens a lane, in fp64 (rounded to fp32 they would show in
  // e^(G_t - G_s))
  if (warp == 1) {
    double x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = 2 * lane + e;
      const float v = t < live ? __ldg(p.g + (size_t)(first + t) * p.Hv + hv) : 0.f;
      // below e^-10000 every product of decays is zero in fp32 (and -inf stays comparable)
      x[e] = (double)(v < -1e4f ? -1e4f : v) * 1.4426950408889634;
    }
    double sum = x[0] + x[1];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += y;
    }
    f.G[2 * lane] = sum - x[1];
    f.G[2 * lane + 1] = sum;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = f.tmem_base;
  {  // the factors: a token and two of four kinds to a thread
    const int t = tid & 63;
    const double G = f.G[t], end = f.G[C - 1], mid = f.G[C / 2 - 1];
    const bool mild = end > -60.0;
    if (tid < 64) {
      const float eg = exp2f((float)G);
      f.out.neg[t] = -eg;
      f.out.out[t] = p.scale * eg;
      f.rowA[t] = mild ? beta * exp2f((float)(G - mid)) : beta;
      f.beta[t] = beta;
      if (t == 0) f.out.total = exp2f((float)end), f.out.mild = mild;
    } else {
      f.out.end[t] = exp2f((float)(end - G));
      f.rowP[t] = mild ? p.scale * exp2f((float)(G - end)) : p.scale;
      f.mid[t] = mild ? exp2f((float)(mid - G)) : 1.f;
    }
  }
  // (a wait that gives up is reported; and repeated once, so that nothing is in flight when the
  // block ends)
  auto wait = [&](uint64_t* bar) {
    if (mbar_wait_short(bar, 0, WAIT_TRIES)) return;
    if (p.err) atomicOr(p.err, kErrWaitTimeout);
    mbar_wait_short(bar, 0, WAIT_TRIES);
  };
  if (p.cu && live < C) {  // rows after the sequence's end: another's, or anything
    wait(&f.full);
    for (int i = tid; i < (C - live) * 8 * 2 * (DK / 64); i += NT) {
      const int part = i / ((C - live) * 8), j = i % ((C - live) * 8);
      *reinterpret_cast<uint4*>(sm + part * R64 + live * 128 + j * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
  }
  __syncthreads();
  if (__shfl_sync(0xffffffffu, warp, 0) == 0 && elect_one()) {  // [K; Q] K^T
    wait(&f.full);
    tc_fence_after();
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
      const uint64_t at = sdesc_sw128(smem_u32(sm) + (ks >> 2) * R128 + (ks & 3) * 32, 16, 1024);
      umma_f16_ss(tmem, at, at, idesc_bf16(128, 64, 0, 0), ks > 0);
    }
    umma_commit(&f.done);
  }
  __syncwarp();
  wait(&f.done);  // (the tiles are read: the record takes their place)
  tc_fence_after();

  // A (rows of K: threads 0-63) and P (rows of Q), a row to a thread.  In a mild chunk (its decay stays
  // above 2^-60) e^(G_t - G_s) = e^(G_t - G_m) e^(G_m - G_s) with the chunk's middle m, and P is kept
  // for the product with U_end; otherwise element by element.
  {
    const bool isA = warp < 2, mild = f.out.mild;
    const int t = tid & 63;
    const float own = isA ? f.rowA[t] : f.rowP[t];
    const uint32_t tl = tmem + ((uint32_t)(32 * warp) << 16);
#pragma unroll 1
    for (int s0 = 0; s0 < 32 + 32 * (warp & 1); s0 += 16) {
      float x[16];
      tmem_ld16(tl + s0, x);
      tmem_ld_wait();
      if (mild && isA) {
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 m = ld4(&f.mid[s0 + i]);
          x[i] *= own * m.x, x[i + 1] *= own * m.y, x[i + 2] *= own * m.z, x[i + 3] *= own * m.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] *= own;
        if (!mild) {
          const double G = f.G[t];
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] *= ex2_approx(fminf((float)(G - f.G[s0 + i]), 0.f));
        }
      }
      if (s0 >= 32 * (warp & 1)) {  // (the diagonal's 32 columns)
        const int lim = t - s0 + (isA ? 0 : 1);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = i < lim ? x[i] : 0.f;
      }
      if (isA) {
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<float4*>(M + t * LDM + s0 + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
      } else if (s0 <= t) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split2(x[8 * i + 2 * e], x[8 * i + 2 * e + 1], hi[e], lo[e]);
          *reinterpret_cast<uint4*>(sm + OFF_P + gdr_tri_off(t, s0 / 8 + i)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          if (t < live)
            *reinterpret_cast<uint4*>(p.o + ((size_t)(first + t) * p.Hv + hv) * p.dv + s0 + 8 * i) =
                make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 64);
  }

  if (warp < 2) {  // the diagonal blocks of 8: a column to a lane, four blocks to a warp
    const int r0 = 32 * warp + 8 * (lane >> 3), col = lane & 7;
    float x[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) x[r] = (r == col) ? 1.f : 0.f;
#pragma unroll
    for (int r = 1; r < 8; ++r) {
      const float4 a0 = ld4(M + (r0 + r) * LDM + r0), a1 = ld4(M + (r0 + r) * LDM + r0 + 4);
      const float ar[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < r; ++i) s = fmaf(ar[i], x[i], s);
      if (r > col) x[r] = -s;
    }
    __syncwarp();
#pragma unroll
    for (int r = 0; r < 8; ++r) M[(r0 + r) * LDM + r0 + col] = x[r];
    __syncwarp();
    // 16: the blocks below the diagonal of this warp's two merges, two rows and two columns to a lane
    const int J = 32 * warp + 16 * (lane >> 4), I = J + 8, r = (lane & 15) >> 2, c = 2 * (lane & 3);
    float2 z[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    float* Xw = X + J / 2 * LDX;  // 8 rows a merge
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const float2 b = *reinterpret_cast<const float2*>(M + (J + s) * LDM + J + c);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float a = M[(I + r + 4 * e) * LDM + J + s];
        z[e].x = fmaf(a, b.x, z[e].x), z[e].y = fmaf(a, b.y, z[e].y);
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) *reinterpret_cast<float2*>(Xw + (r + 4 * e) * LDX + c) = z[e], z[e] = make_float2(0.f, 0.f);
    __syncwarp();
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const float2 b = *reinterpret_cast<const float2*>(Xw + s * LDX + c);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float a = M[(I + r + 4 * e) * LDM + I + s];
        z[e].x = fmaf(a, b.x, z[e].x), z[e].y = fmaf(a, b.y, z[e].y);
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) *reinterpret_cast<float2*>(M + (I + r + 4 * e) * LDM + J + c) = make_float2(-z[e].x, -z[e].y);
    __syncwarp();
  }
  // D (16 x 16) = A (16 rows of M at Ar) B (8 KS rows at Bc), operands split in two tf32 parts:
  // hi hi, hi lo and lo hi
  auto mma3 = [&](const float* Ar, const float* Bc, int ldb, auto KS, float (&d)[2][4]) {
    float dl[2][4], dm[2][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i >> 2][i & 3] = dl[i >> 2][i & 3] = dm[i >> 2][i & 3] = 0.f;
    const float* a = Ar + ((lane & 7) + (lane & 8)) * LDM + ((lane & 16) >> 2);
    const float* b = Bc + t4 * ldb + g4;
#pragma unroll
    for (int ks = 0; ks < decltype(KS)::value; ++ks) {
      uint32_t ah[4], al[4];
      ldmatrix_x4(ah, a + 8 * ks);
#pragma unroll
      for (int i = 0; i < 4; ++i) split_tf32(__uint_as_float(ah[i]), ah[i], al[i]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t bh[2], bl[2];
        split_tf32(b[8 * ks * ldb + 8 * h], bh[0], bl[0]);
        split_tf32(b[(8 * ks + 4) * ldb + 8 * h], bh[1], bl[1]);
        mma_16x8x8_tf32(d[h], ah, bh);
        mma_16x8x8_tf32(dl[h], ah, bl);
        mma_16x8x8_tf32(dm[h], al, bh);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i >> 2][i & 3] += dl[i >> 2][i & 3] + dm[i >> 2][i & 3];
  };
  auto put = [&](float* at, int ld, const float (&d)[2][4], float sign) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      *reinterpret_cast<float2*>(at + g4 * ld + 8 * h + 2 * t4) = make_float2(sign * d[h][0], sign * d[h][1]);
      *reinterpret_cast<float2*>(at + (g4 + 8) * ld + 8 * h + 2 * t4) = make_float2(sign * d[h][2], sign * d[h][3]);
    }
  };
  constexpr std::integral_constant<int, 2> K16{};  // K steps of 8
  constexpr std::integral_constant<int, 4> K32{};
  float d[2][4];
  if (warp < 2) {  // 32: a merge of the warp's own two blocks of 16
    const int J = 32 * warp, I = J + 16;
    float* Xw = X + J / 2 * LDX;  // 16 rows
    mma3(M + I * LDM + J, M + J * LDM + J, LDM, K16, d);
    put(Xw, LDX, d, 1.f);
    __syncwarp();
    mma3(M + I * LDM + I, Xw, LDX, K16, d);
    put(M + I * LDM + J, LDM, d, -1.f);
  }
  __syncthreads();
  // 64: a 16 x 16 block of T_10 to a warp
  const int r0 = 16 * (warp >> 1), cc = 16 * (warp & 1);
  mma3(M + (32 + r0) * LDM, M + cc, LDM, K32, d);
  put(X + r0 * LDX + cc, LDX, d, 1.f);
  __syncthreads();
  if (r0 == 0)
    mma3(M + 32 * LDM + 32, X + cc, LDX, K16, d);  // (T_II is zero right of the diagonal)
  else
    mma3(M + 48 * LDM + 32, X + cc, LDX, K32, d);
  put(M + (32 + r0) * LDM + cc, LDM, d, -1.f);
  __syncthreads();
  {  // T's parts with their factors, in M's place: 8 columns of a row to a thread and turn
    uint4 h[3], l[3];
    uint32_t at[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int item = (tid >> 5) + 4 * k;  // block of 16 x 16
      const int rb = item >= 6 ? 3 : item >= 3 ? 2 : item >= 1 ? 1 : 0, cb = item - rb * (rb + 1) / 2;
      const int row = 16 * rb + (lane & 15), piece = 2 * cb + (lane >> 4);
      at[k] = gdr_tri_off(row, piece);
      if (item < 10) {
        const float end = f.out.mild ? f.out.end[row] : 1.f;
        const float2 ee = make_float2(end, end);
        uint32_t hh[4], ll[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 x = ld4(M + row * LDM + 8 * piece + 4 * e), be = ld4(&f.beta[8 * piece + 4 * e]);
          const float2 y = mul2(mul2(ee, make_float2(be.x, be.y)), make_float2(x.x, x.y));
          const float2 z = mul2(mul2(ee, make_float2(be.z, be.w)), make_float2(x.z, x.w));
          split2(y.x, y.y, hh[2 * e], ll[2 * e]);
          split2(z.x, z.y, hh[2 * e + 1], ll[2 * e + 1]);
        }
        h[k] = make_uint4(hh[0], hh[1], hh[2], hh[3]), l[k] = make_uint4(ll[0], ll[1], ll[2], ll[3]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if ((tid >> 5) + 4 * k < 10) {
        *reinterpret_cast<uint4*>(sm + GDR_T_HI + at[k]) = h[k];
        *reinterpret_cast<uint4*>(sm + GDR_T_LO + at[k]) = l[k];
      }
    }
    if (tid < (int)(sizeof(GdrGates) / 16))
      reinterpret_cast<uint4*>(sm + GDR_GATES)[tid] = reinterpret_cast<const uint4*>(&f.out)[tid];
  }
  fence_proxy_async_smem();
  __syncthreads();
  if (tid == 0) {
    unsigned char* record = p.records + (size_t)blockIdx.x * GDR_RECORD;
    bulk_store_1d(record, sm, GDR_P);
    bulk_store_1d(record + GDR_P, sm + OFF_P, GDR_TRI);
    bulk_commit();
    bulk_wait_read_all();  // (shared memory is read; the writes land by the kernel's end)
  }
}

template <int DK>
cudaError_t launch_dk(const GdrArgs& a, const CUtensorMap& mq, const CUtensorMap& mk, unsigned char* records,
                      long long slots, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = smem_limit_once(gdr_prep_kernel<DK>, (int)smem_bytes(DK), done);
  if (e != cudaSuccess) return e;
  const PrepParams p{a.g,  a.beta, a.cu_seqlens, records, static_cast<__nv_bfloat16*>(a.o), a.B, a.T, a.Hk, a.Hv,
                     a.dv, a.scale, device_error_word()};
  gdr_prep_kernel<DK><<<(unsigned)(slots * a.Hv), NT, smem_bytes(DK), st>>>(mq, mk, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gdr_prep(const GdrArgs& a, const CUtensorMap& mq, const CUtensorMap& mk, unsigned char* records,
                            cudaStream_t st) {
  const long long slots = gdr_slots(a.B, a.T, a.cu_seqlens != nullptr);
  if (slots * a.Hv > 0x7fffffffLL) return cudaErrorInvalidValue;
  return a.dk == 128 ? launch_dk<128>(a, mq, mk, records, slots, st) : launch_dk<64>(a, mq, mk, records, slots, st);
}

}  // namespace gdn2
