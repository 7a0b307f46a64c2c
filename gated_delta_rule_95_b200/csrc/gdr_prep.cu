// Scalar-gate prefill, what does not depend on the state (gdr_chain.cu has the formulas): for every
// chunk of 64 tokens and value head the decays' factors, P, and T = (I + A)^-1 with
//
//     A_ts = beta_t e^(G_t - G_s) k_t . k_s  (s < t),    P_ts = scale e^(G_t - G_s) q_t . k_s  (s <= t)
//
// All chunks at once, a block of 256 threads each, four blocks to an SM.  [K; Q] K^T runs on
// warp-level bf16 products (128 x 64 x 128: a tenth of the time, and T's merges need warp-level
// products anyway); A and T are fp32 in shared memory: 8 x 8 diagonal blocks by substitution, then
// T_IJ = -T_II (A_IJ T_JJ) for blocks of 8 (FMA), 16 and 32 (tf32 products of split operands, 2^-21).
// Substitution in blocks is stable where powers of A are not (one key repeated: A is all ones).
// The record leaves by one bulk store.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn2_internal.h"
#include "gdr_chunk.cuh"
#include "ptx.cuh"

namespace gdn2 {
namespace {

constexpr int C = GDR_C;
constexpr int NT = 256;
constexpr int LDM = 68;  // row stride of M: rows 4 banks apart
constexpr int LDW = 12;  // [32][LDW]: X of a merge, one per four warps
constexpr uint32_t R128 = 128 * 128;  // a panel of 64 channels: 128 rows of 128 bytes

struct PrepGates {
  GdrGates out;
  alignas(16) float2 G[C];   // log2 decay summed up to t, in two floats
  alignas(16) float mid[C];  // e^(G_m - G_t), m = the chunk's middle (mild chunks)
};
// shared memory: [K; Q] tiles, later the record; M; X; the gates
__host__ __device__ constexpr uint32_t kq_bytes(int dk) {
  return (uint32_t)(dk / 64) * R128 > GDR_RECORD ? (uint32_t)(dk / 64) * R128 : GDR_RECORD;
}
__host__ __device__ constexpr uint32_t smem_bytes(int dk) {
  return kq_bytes(dk) + 64 * LDM * 4 + 4 * 32 * LDW * 4 + (uint32_t)sizeof(PrepGates);
}

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
// x = hi + lo, hi its upper 10 mantissa bits.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xFFFFE000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}
// D += A B, A 16 x 16 (row-major), B 16 x 8, bf16 (fragments of mma_16x8x8_tf32 with pairs of
// adjacent k in a word).
__device__ __forceinline__ void mma_16x8x16_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

struct PrepParams {
  const __nv_bfloat16 *q, *k;
  const float *g, *beta;
  const int* cu;
  unsigned char* records;
  int N, T, Hk, Hv;
  float scale;
};

template <int DK>
__global__ void __launch_bounds__(NT, 3) gdr_prep_kernel(const PrepParams p) {
  extern __shared__ __align__(1024) unsigned char sm[];
  float* M = reinterpret_cast<float*>(sm + kq_bytes(DK));
  PrepGates& gt = *reinterpret_cast<PrepGates*>(sm + kq_bytes(DK) + 64 * LDM * 4 + 4 * 32 * LDW * 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g4 = lane >> 2, t4 = lane & 3;
  float* X = M + 64 * LDM + (warp & 3) * 32 * LDW;
  const int hv = blockIdx.x % p.Hv, hk = hv / (p.Hv / p.Hk);
  const long long slot = blockIdx.x / p.Hv;
  // this block's sequence and chunk
  long long first;  // flat token index of the chunk
  int live;         // its tokens
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
  } else {
    const int nch = (p.T + C - 1) / C, n = (int)(slot / nch), c = (int)(slot % nch);
    first = (long long)n * p.T + (long long)c * C;
    live = min(C, p.T - c * C);
  }

  // K and Q, absent rows zero
  {
    constexpr int CPR = DK / 8;
    const size_t row_elems = (size_t)p.Hk * DK;
#pragma unroll
    for (int i = tid; i < 2 * C * CPR; i += NT) {
      const int ch = i % CPR, row = i / CPR, t = row & (C - 1);
      const __nv_bfloat16* src = (row < C ? p.k : p.q) + (size_t)(first + (t < live ? t : 0)) * row_elems + (size_t)hk * DK + 8 * ch;
      cp_async16(sm + (ch >> 3) * R128 + sw128_off(row, ch & 7), src, t < live);
    }
  }
  // the decays' factors, two tokens a lane; sums in fp64 (a sum of 64 log decays rounded to fp32
  // would show in e^(G_t - G_s))
  if (warp == 0) {
    float gn[2], bn[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = 2 * lane + e;
      const size_t at = (size_t)(first + t) * p.Hv + hv;
      gn[e] = t < live ? __ldg(p.g + at) : 0.f;
      bn[e] = t < live ? __ldg(p.beta + at) : 0.f;
    }
    // below e^-10000 every product of decays is zero in fp32 (and -inf stays comparable)
    const double l2e = 1.4426950408889634;
    const double x0 = (double)(gn[0] < -1e4f ? -1e4f : gn[0]) * l2e, x1 = (double)(gn[1] < -1e4f ? -1e4f : gn[1]) * l2e;
    double sum = x0 + x1;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += y;
    }
    const double G[2] = {sum - x1, sum};
    const double end = __shfl_sync(0xffffffffu, sum, 31), mid = __shfl_sync(0xffffffffu, sum, 15);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = 2 * lane + e;
      const float hi = (float)G[e], eg = exp2f((float)G[e]);
      gt.G[t] = make_float2(hi, (float)(G[e] - (double)hi));
      gt.mid[t] = exp2f((float)(mid - G[e]));
      gt.out.r[t] = make_float2(bn[e], -bn[e] * eg);
      gt.out.end[t] = exp2f((float)(end - G[e]));
      gt.out.out[t] = p.scale * eg;
    }
    if (lane == 31) gt.out.total = exp2f((float)end), gt.out.mild = end > -60.0;
  }
  cp_async_wait_all();
  __syncthreads();

  // [K; Q] K^T: warp w has rows 16 w on (w < 4: A), columns up to its diagonal block
  const int rb = warp & 3;
  const bool isA = warp < 4;
  float acc[4][2][4];
#pragma unroll
  for (int pr = 0; pr < 4; ++pr)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[pr][h][i] = 0.f;
#pragma unroll
  for (int ks = 0; ks < DK / 16; ++ks) {
    uint32_t a[4];
    {
      const int row = 16 * warp + (lane & 15), ch = 2 * ks + (lane >> 4);
      ldmatrix_x4(a, sm + (ch >> 3) * R128 + sw128_off(row, ch & 7));
    }
#pragma unroll
    for (int pr = 0; pr < 4; ++pr) {
      if (pr <= rb) {
        uint32_t b[4];
        const int row = 16 * pr + (lane & 7) + ((lane & 16) >> 1), ch = 2 * ks + ((lane >> 3) & 1);
        ldmatrix_x4(b, sm + (ch >> 3) * R128 + sw128_off(row, ch & 7));
        mma_16x8x16_bf16(acc[pr][0], a, b[0], b[1]);
        mma_16x8x16_bf16(acc[pr][1], a, b[2], b[3]);
      }
    }
  }
  __syncthreads();  // the tiles are read: the record takes their place

  // A and P.  In a mild chunk (its decay stays above 2^-60) e^(G_t - G_s) = e^(G_t - G_m) e^(G_m - G_s)
  // with the chunk's middle m, and P is kept for the product with e^(G_C - G) U; otherwise
  // element by element.
  {
    const bool mild = gt.out.mild;
    float own[2];
    float2 Gt[2];
    int tr[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {  // rows g and g + 8
      tr[e] = 16 * rb + g4 + 8 * e;
      Gt[e] = gt.G[tr[e]];
      own[e] = isA ? gt.out.r[tr[e]].x : p.scale;
      const float2 Gr = gt.G[isA ? 31 : 63];
      if (mild) own[e] *= ex2_approx((Gt[e].x - Gr.x) + (Gt[e].y - Gr.y));
    }
#pragma unroll
    for (int pr = 0; pr < 4; ++pr) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int s = 16 * pr + 8 * h + 2 * t4;
        float2 f = make_float2(1.f, 1.f);
        if (isA && mild) f = *reinterpret_cast<const float2*>(&gt.mid[s]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x[2] = {acc[pr][h][2 * e] * own[e], acc[pr][h][2 * e + 1] * own[e]};
          if (mild) {
            x[0] *= f.x, x[1] *= f.y;
          } else if (pr <= rb) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float2 Gs = gt.G[s + i];
              x[i] *= ex2_approx(fminf((Gt[e].x - Gs.x) + (Gt[e].y - Gs.y), 0.f));
            }
          }
          const int lim = tr[e] + (isA ? 0 : 1);  // columns that count
#pragma unroll
          for (int i = 0; i < 2; ++i) x[i] = pr <= rb && s + i < lim ? x[i] : 0.f;
          if (isA)
            *reinterpret_cast<float2*>(M + tr[e] * LDM + s) = make_float2(x[0], x[1]);
          else
            *reinterpret_cast<uint32_t*>(sm + GDR_P + sw128_off(tr[e], s >> 3) + (s & 7) * 2) = pack_bf16(x[0], x[1]);
        }
      }
    }
  }
  for (int i = tid; i < (int)(sizeof(GdrGates) / 16); i += NT)
    reinterpret_cast<uint4*>(sm + GDR_GATES)[i] = reinterpret_cast<const uint4*>(&gt.out)[i];
  __syncthreads();

  // T: warps 0-3 take 16 rows each
  if (warp < 4) {
    {  // the diagonal blocks 2 warp (lanes 0-7) and 2 warp + 1 (lanes 8-15): a column to a lane
      const int r0 = 16 * warp + 8 * ((lane >> 3) & 1), col = lane & 7;
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
      if (lane < 16) {
#pragma unroll
        for (int r = 0; r < 8; ++r) M[(r0 + r) * LDM + r0 + col] = x[r];
      }
      __syncwarp();
    }
    {  // 16: the block below the diagonal, two columns to a lane
      const int J = 16 * warp, I = J + 8, c0 = 2 * t4;
      float2 z = make_float2(0.f, 0.f);
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const float a = M[(I + g4) * LDM + J + s];
        const float2 b = *reinterpret_cast<const float2*>(M + (J + s) * LDM + J + c0);
        z.x = fmaf(a, b.x, z.x), z.y = fmaf(a, b.y, z.y);
      }
      *reinterpret_cast<float2*>(X + g4 * LDW + c0) = z;
      __syncwarp();
      float2 y = make_float2(0.f, 0.f);
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const float a = M[(I + g4) * LDM + I + s];
        const float2 b = *reinterpret_cast<const float2*>(X + s * LDW + c0);
        y.x = fmaf(a, b.x, y.x), y.y = fmaf(a, b.y, y.y);
      }
      *reinterpret_cast<float2*>(M + (I + g4) * LDM + J + c0) = make_float2(-y.x, -y.y);
    }
  }
  // D (16 x 8) = A (16 rows of M at Ar) B (16 KS rows at Bc), operands split in two tf32 parts:
  // hi hi, hi lo and lo hi in chains of their own
  auto mma3 = [&](const float* Ar, const float* Bc, int ldb, int KS, float (&d)[4]) {
    float dl[4] = {0.f, 0.f, 0.f, 0.f}, dm[4] = {0.f, 0.f, 0.f, 0.f};
    d[0] = d[1] = d[2] = d[3] = 0.f;
    const float* a = Ar + ((lane & 7) + (lane & 8)) * LDM + ((lane & 16) >> 2);
    const float* b = Bc + t4 * ldb + g4;
#pragma unroll
    for (int k = 0; k < 2; ++k, a += 16, b += 16 * ldb) {
      if (k >= KS) break;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        uint32_t ah[4], al[4], bh[2], bl[2];
        ldmatrix_x4(ah, a + 8 * ks);
#pragma unroll
        for (int i = 0; i < 4; ++i) split_tf32(__uint_as_float(ah[i]), ah[i], al[i]);
        split_tf32(b[8 * ks * ldb], bh[0], bl[0]);
        split_tf32(b[(8 * ks + 4) * ldb], bh[1], bl[1]);
        mma_16x8x8_tf32(d, ah, bh);
        mma_16x8x8_tf32(dl, ah, bl);
        mma_16x8x8_tf32(dm, al, bh);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] += dl[i] + dm[i];
  };
  // Size 32: warps 2 j, 2 j + 1 (of 0-3) merge blocks 2 j and 2 j + 1, eight columns each.
  // Size 64: warps w and w + 4 take eight columns, sixteen rows each.
#pragma unroll 1
  for (int size = 32; size <= 64; size += 32) {
    const bool half = size == 32, mine = !half || warp < 4;
    const int J = half ? 32 * (warp >> 1) : 0, I = J + size / 2;  // T_IJ
    const int c0 = J + 8 * (half ? warp & 1 : warp & 3);          // its columns
    const int r0 = half ? 0 : 16 * (warp >> 2);                   // its rows I + r0 on
    float d[4];
    __syncthreads();  // the smaller blocks are there
    if (mine) {
      mma3(M + (I + r0) * LDM + J, M + J * LDM + c0, LDM, half ? 1 : 2, d);
      *reinterpret_cast<float2*>(X + (r0 + g4) * LDW + 2 * t4) = make_float2(d[0], d[1]);
      *reinterpret_cast<float2*>(X + (r0 + g4 + 8) * LDW + 2 * t4) = make_float2(d[2], d[3]);
    }
    __syncthreads();  // (two warps share A_IJ, or X)
    if (mine) {
      // (T_II is zero right of the diagonal: its first 16 rows need 16 of X's)
      mma3(M + (I + r0) * LDM + I, X, LDW, r0 ? 2 : 1, d);
      float* m = M + (I + r0 + g4) * LDM + c0 + 2 * t4;
      *reinterpret_cast<float2*>(m) = make_float2(-d[0], -d[1]);
      *reinterpret_cast<float2*>(m + 8 * LDM) = make_float2(-d[2], -d[3]);
    }
  }
  __syncthreads();
  {  // T's tiles: 16 columns of a row to a thread (M is not kept right of the diagonal's block)
    const int r = tid >> 2, s0 = 16 * (tid & 3);
#pragma unroll
    for (int s = s0; s < s0 + 16; s += 8) {
      const bool low = s0 <= r;
      const float4 z = make_float4(0.f, 0.f, 0.f, 0.f), a = low ? ld4(M + r * LDM + s) : z, b = low ? ld4(M + r * LDM + s + 4) : z;
      uint32_t h[4], l[4];
      split2(a.x, a.y, h[0], l[0]), split2(a.z, a.w, h[1], l[1]);
      split2(b.x, b.y, h[2], l[2]), split2(b.z, b.w, h[3], l[3]);
      const uint32_t at = sw128_off(r, s >> 3);
      *reinterpret_cast<uint4*>(sm + GDR_T_HI + at) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4*>(sm + GDR_T_LO + at) = make_uint4(l[0], l[1], l[2], l[3]);
    }
  }
  fence_proxy_async_smem();
  __syncthreads();
  if (tid == 0) {
    bulk_store_1d(p.records + (size_t)blockIdx.x * GDR_RECORD, sm, GDR_RECORD);
    bulk_commit();
    bulk_wait_all();
  }
}

template <int DK>
cudaError_t launch_dk(const GdrArgs& a, unsigned char* records, long long slots, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = smem_limit_once(gdr_prep_kernel<DK>, (int)smem_bytes(DK), done);
  if (e != cudaSuccess) return e;
  const PrepParams p{static_cast<const __nv_bfloat16*>(a.q), static_cast<const __nv_bfloat16*>(a.k), a.g, a.beta,
                     a.cu_seqlens, records, a.B, a.T, a.Hk, a.Hv, a.scale};
  gdr_prep_kernel<DK><<<(unsigned)(slots * a.Hv), NT, smem_bytes(DK), st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gdr_prep(const GdrArgs& a, unsigned char* records, cudaStream_t st) {
  const long long slots = gdr_slots(a.B, a.T, a.cu_seqlens != nullptr);
  if (slots * a.Hv > 0x7fffffffLL) return cudaErrorInvalidValue;
  return a.dk == 128 ? launch_dk<128>(a, records, slots, st) : launch_dk<64>(a, records, slots, st);
}

}  // namespace gdn2
