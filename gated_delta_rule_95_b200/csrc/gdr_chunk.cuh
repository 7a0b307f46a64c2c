// What the two kernels of the scalar-gate prefill share: the record that the preparation kernel
// (gdr_prep.cu) leaves in the workspace for every chunk and value head, and the chain kernel
// (gdr_chain.cu) loads as one bulk copy.
#pragma once
#include <cuda.h>

#include <cstdint>

#include "gdn2_internal.h"
#include "ptx.cuh"

namespace gdn2 {

constexpr int GDR_C = 64;  // tokens of a chunk

// Factors of a chunk's tokens; G_t = the sum of the log decays up to token t, G_C over the chunk.
struct GdrGates {
  alignas(16) float neg[GDR_C];  // -e^G
  alignas(16) float out[GDR_C];  // scale e^G
  alignas(16) float end[GDR_C];  // e^(G_C - G_t) (used where the chunk is not mild)
  float total;                   // e^(G_C)
  int mild;  // the chunk's decay stays above 2^-60: T's rows carry e^(G_C - G_t), and P is
             // scale e^(G_t - G_C) q_t k_s; otherwise T has no row factor, and P is
             // scale e^(G_t - G_s) q_t k_s (s <= t)
  int pad[2];
};
// T and P are lower triangular 64 x 64 matrices of bf16, operands of products over their columns in
// steps of 16.  Step ks holds the rows from 16 ks on, in blocks of 8 rows x 8 columns (128 bytes),
// two side by side: 5 KB instead of 8.
constexpr uint32_t GDR_TRI = 20 * 256;
__host__ __device__ constexpr uint32_t gdr_tri_step(int ks) { return 256u * (uint32_t)(ks * (9 - ks)); }
// Columns 8 piece to 8 piece + 7 of a row >= 16 (piece / 2).
__host__ __device__ constexpr uint32_t gdr_tri_off(int row, int piece) {
  return gdr_tri_step(piece >> 1) + 256u * (uint32_t)((row >> 3) - 2 * (piece >> 1)) + 128u * (uint32_t)(piece & 1) +
         16u * (uint32_t)(row & 7);
}
// T = (I + A)^-1 diag(beta) in two bf16 parts, the gates, P's first part.  (Its second part takes the place of the
// chunk's outputs, [token][64 channels], until they are written.)
constexpr uint32_t GDR_T_HI = 0, GDR_T_LO = GDR_TRI, GDR_GATES = 2 * GDR_TRI, GDR_P = GDR_GATES + 1024;
constexpr uint32_t GDR_RECORD = GDR_P + GDR_TRI;
static_assert(sizeof(GdrGates) <= GDR_P - GDR_GATES, "gates in their place");

// Records of a call: one per (chunk slot, value head), the heads innermost.  Sequence n's chunk c
// has slot n ceil(T / 64) + c, or in a packed batch floor(cu[n] / 64) + n + c: floor(a + b) >=
// floor(a) + ceil(b) - 1, so that no two sequences share one, and there are at most T / 64 + N.
__host__ __device__ inline long long gdr_slots(int B, int T, bool packed) {
  return packed ? (long long)T / GDR_C + B : (long long)B * (((long long)T + GDR_C - 1) / GDR_C);
}

// The records of all chunks; mq, mk: tensor maps of q and k, boxes of 64 tokens x 64 channels.
cudaError_t launch_gdr_prep(const GdrArgs& a, const CUtensorMap& mq, const CUtensorMap& mk, unsigned char* records,
                            cudaStream_t st);

// (x0, x1) -> packed bf16 hi parts and lo parts, x = hi + lo to 2^-16 |x|.
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16(x0, x1);
  const float2 d = sub2(make_float2(x0, x1), make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xFFFF0000u)));
  lo = pack_bf16(d.x, d.y);
}

}  // namespace gdn2
