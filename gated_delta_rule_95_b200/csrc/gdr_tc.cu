// Chunkwise prefill forward of the gated delta rule with scalar gates for bf16 inputs, on the
// 5th-generation tensor cores (tcgen05.mma kind::f16, accumulators in tensor memory, q, k, v
// tiles by TMA).
//
// The recurrence (snilld.dk, "Hvad Gated DeltaNet-2 aendrer": the rule left when both gates and
// the decay are scalars) in its WY form over chunks of 64 tokens (Gated DeltaNet-2 guide,
// "Chunkwise Parallel Algorithm for GPU Training").  With G_t the sum of the log decays of the
// chunk up to token t, e^G its exponential and K, Q, V the chunk's rows:
//
//     A_ts = beta_t e^(G_t - G_s) k_t . k_s  (s < t),      T = (I + A)^-1
//     P_ts = e^(G_t - G_s) q_t . k_s         (s <= t)
//     R  = beta (V - e^G K S),     U = T R
//     O  = scale (e^G Q S + P U),  S' = e^(G_C) S + K^T (e^(G_C - G) U)
//
// A scalar decay never has to be folded into K or Q, so the products take the raw bf16 tiles
// (exact operands) and every factor of a decay is e^(difference <= 0): nothing overflows, and
// there is no limit on the decay.
//
// Precision.  S, R, U and T are fp32 values; where one of them is an operand it is split into
// two bf16 parts, x = hi + lo (off by 2^-18 |x| at most), and a product of two split operands drops
// lo lo (2^-18): the state keeps 16 to 17 bits a step with the exact K on the other side, which
// leaves S_T a few 1e-6 off.  The output needs less: P enters P U as a single bf16.
//
// Layout.  One CTA per (sequence, value head).  Everything on the state's way through a chunk
// is held transposed, value channels on the 128 lanes of tensor memory, so that each
// product's result is the next one's A operand in place, thread by thread, and nothing but T
// and P goes through shared memory.  The 16 columns of one K step (two bf16 to a column) hold
// [hi (8) | lo (8)] where the 16 fp32 results were.
//   warps 0-15  the state: rows = value channel, quarters of the columns (S itself in registers);
//               R and U as product fragments (row and pair of tokens by lane), where the
//               factors of a token serve many rows and V comes by transposing loads
//   warps 16-23 two chunks ahead: A and P out of [K; Q] K^T, T by blocked substitution
//   warps 24-27 the outputs: Q S and P U to bf16 rows of o
//   warps 28-31 one thread issues the products and the TMA loads; one warp sums the decays
// d_v = 64 runs with the upper 64 lanes zero.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "gdn2_internal.h"
#include "ptx.cuh"

namespace gdn2 {
namespace {

constexpr int C = 64;
constexpr int NSTATE = 512, NSOLVE = 256, NOUT = 128;
constexpr int CTL = NSTATE + NSOLVE + NOUT;  // the issuing thread
constexpr int NT = CTL + 128;
// registers a thread of each warpgroup: four of the state (which holds S), two of the solve, the
// outputs and the issuing one share what NT threads are launched with, 64 each
constexpr int REG_LAUNCH = 64, REG_STATE = 72, REG_SOLVE = 72, REG_OUT = 40, REG_CTL = 40;
static_assert(4 * REG_STATE + 2 * REG_SOLVE + REG_OUT + REG_CTL <= NT / 128 * REG_LAUNCH, "the launch's registers");
constexpr int BAR_SOLVE = 1, BAR_OUT = 2, BAR_PAIR = 3;  // named barriers (BAR_PAIR + 0..3: two warps)
constexpr int WAIT_TRIES = 2000;                // suspensions of 1 ms: about 2 s per wait
constexpr int QK_STAGES = 3, V_STAGES = 2, GATE_SLOTS = 5;

// ---- shared memory (byte offsets from a 1024-byte aligned base) ---------------------------
constexpr uint32_t R64 = 64 * 128, R128 = 128 * 128;  // panels of 64 channels (128 bytes) by rows
constexpr uint32_t OFF_KQ = 0;                        // [K; Q]: stages x 2 panels x 128 rows
constexpr uint32_t KQ_STAGE = 2 * R128;
constexpr uint32_t OFF_V = OFF_KQ + QK_STAGES * KQ_STAGE;  // V: stages x 2 panels x 64 rows
constexpr uint32_t V_STAGE = 2 * R64;
constexpr uint32_t OFF_T = OFF_V + V_STAGES * V_STAGE;  // T: 2 buffers x [hi; lo] x 64 rows
constexpr uint32_t OFF_P = OFF_T + 2 * 2 * R64;         // P: 2 buffers x 64 rows
constexpr uint32_t OFF_O = OFF_P + 2 * R64;             // o staging [t][v] bf16
constexpr uint32_t OFF_M = OFF_O + 2 * R64;             // the solve's fp32 scratch [64][LDM]
constexpr int LDM = 68;                                 // (rows 4 banks apart)
constexpr int LDW = 12;                                 // per warp [32][LDW]: X of a merge
constexpr uint32_t OFF_X = OFF_M + 64 * LDM * 4;
constexpr uint32_t TILES = OFF_X + 4 * 32 * LDW * 4;

struct Gates {
  alignas(16) float2 r[C];   // (beta, -beta e^G)
  alignas(16) float end[C];  // e^(G_C - G_t)
  alignas(16) float out[C];  // scale e^G
  alignas(16) float2 G[C];   // log2 decay summed up to t, in two floats
  alignas(16) float mid[C];  // e^(G_m - G_t), m = the chunk's middle (mild chunks)
  float total;               // e^(G_C)
  int mild;                  // the chunk's decay stays above 2^-60
  float pad[2];
};
struct Misc {
  uint64_t kq[QK_STAGES], v[V_STAGES];           // TMA loads landed
  uint64_t ap, ks, u, s, o, drain;               // products done
  uint64_t sready, rready, uready, oread, apread;  // threads -> the issuing thread
  uint64_t g[2], t[2];                           // gates; gates, T and P of a chunk (its parity)
  uint64_t clean;                                // the last chunk's absent rows are zero
  uint32_t tmem_base;
  Gates gate[GATE_SLOTS];
};
constexpr uint32_t SMEM_BYTES = TILES + 1024 + sizeof(Misc);
static_assert(SMEM_BYTES <= 232448, "one CTA's shared memory");

// ---- tensor memory columns ------------------------------------------------------------------
constexpr uint32_t TM_S = 0;     // S^T in [hi | lo] blocks, then U_end^T K in its place (d_k)
constexpr uint32_t TM_R = 128;   // S^T K^T (64), then R^T in its place
constexpr uint32_t TM_Q = 192;   // S^T Q^T (64)
constexpr uint32_t TM_U = 256;   // U^T (64), then e^(G_C - G) U^T in [hi | lo] blocks in its place
constexpr uint32_t TM_UB = 320;  // U^T in [hi | lo] blocks (64)
constexpr uint32_t TM_AP = 384;  // [K; Q] K^T (64)
constexpr uint32_t TM_O = 448;   // U^T P^T (64)
constexpr uint32_t TM_COLS = 512;

struct TcParams {
  const float *g, *beta;
  const int* cu;
  const float* S0;
  __nv_bfloat16* o;
  float* S_T;
  int T, Hk, Hv;
  float scale;
  unsigned* err;
  unsigned long long* stamps = nullptr;  // instrumented build only: per-chunk clock stamps
};
#ifdef GDN2_STAMPS
// Instrumented build (GDN2_STAMPS): clock64 of the SM at fixed points of the first CTA's chunks.
#define STAMP(cc, slot)                                                                                    \
  do {                                                                                                     \
    if (p.stamps && blockIdx.x == 0 && (cc) < 64) p.stamps[(cc) * 32 + (slot)] = (unsigned long long)clock64(); \
  } while (0)
#else
#define STAMP(cc, slot) \
  do {                  \
  } while (0)
#endif

// (x0, x1) -> packed bf16 hi parts and lo parts.
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16(x0, x1);
  const float2 d = sub2(make_float2(x0, x1), make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xFFFF0000u)));
  lo = pack_bf16(d.x, d.y);
}
// A K step (two blocks of 8 tokens) of fragments, x as tmem_ld_frag32 gives it -> its 16
// columns [hi (8) | lo (8)] for tmem_st_frag16.
__device__ __forceinline__ void split_frag(const float* x, uint32_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) split2(x[2 * i], x[2 * i + 1], w[i], w[4 + i]);
}
// 16 values -> one K step's columns [hi (8) | lo (8)].
__device__ __forceinline__ void split16(const float* x, uint32_t (&w)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) split2(x[2 * i], x[2 * i + 1], w[i], w[8 + i]);
}
__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
// 3-pass tf32 product of fp32 operands: x = hi + lo with hi its upper 10 mantissa bits.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xFFFFE000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}
// Descriptor of the first K step of a K-major panel (the next one is 32 bytes on), and of an
// N-major tile in panels of 64 columns (the next one is 16 rows on).
__device__ __forceinline__ uint64_t kdesc(uint32_t base) { return sdesc_sw128(base, 16, 1024); }
__device__ __forceinline__ uint64_t ndesc(uint32_t base) { return sdesc_sw128(base, R128, 1024); }
constexpr uint32_t KSTEP = 32 >> 4, NSTEP = 2048 >> 4, PANEL = R128 >> 4;  // in descriptor units

// Four K steps of a product.  Out of line: the issuing thread runs through some seventy
// products a chunk, and unrolled they took the instruction cache from the other warps.
__device__ __forceinline__ void four_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t bstep, uint32_t idesc, uint32_t acc) {
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) umma_f16_ts(d, a + 16 * ks, b + bstep * ks, idesc, ks > 0 ? 1u : acc);
}
__device__ __forceinline__ void four_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) umma_f16_ss(d, a + KSTEP * ks, b + KSTEP * ks, idesc, ks > 0 ? 1u : acc);
}

template <int DK, int DV>
__global__ void __launch_bounds__(NT, 1)
    gdr_chunk_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const TcParams p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Misc& ms = *reinterpret_cast<Misc*>(sm + TILES);
  const uint32_t sbase = smem_u32(sm);
  constexpr uint32_t ID_AP = idesc_bf16(128, 64, 0, 0);  // also N = 64 of the others
  constexpr uint32_t ID_ST = idesc_bf16(128, DK, 0, 1);  // B = K as [token][channel]: N-major

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int wid = __shfl_sync(0xffffffffu, warp, 0);  // the same value, known to be uniform
  const int unit = blockIdx.x, n = unit / p.Hv, hv = unit % p.Hv, hk = hv / (p.Hv / p.Hk);
  long long first = (long long)n * p.T;  // flat token index of the sequence's start
  int len = p.T, tb = n, t0 = 0;         // tensor-map coordinates: sequence tb, token t0
  if (p.cu) {
    const int lo = p.cu[n], hi = p.cu[n + 1];
    if (lo < 0 || hi < lo || hi > p.T) {  // offsets out of order or range: nothing is touched
      if (tid == 0 && p.err) atomicOr(p.err, kErrBadSeqlens);
      return;
    }
    first = lo, len = hi - lo, tb = 0, t0 = lo;
  }
  const int nch = (len + C - 1) / C;
  const int tail = len - (nch - 1) * C;  // tokens of the last chunk

  if (tid == 0) {
    for (int i = 0; i < QK_STAGES; ++i) mbar_init(&ms.kq[i], 1);
    for (int i = 0; i < V_STAGES; ++i) mbar_init(&ms.v[i], 1);
    uint64_t* ones[] = {&ms.ap, &ms.ks, &ms.u, &ms.s, &ms.drain};
    for (uint64_t* b : ones) mbar_init(b, 1);
    mbar_init(&ms.o, 2);  // the products, and the issuing thread's own arrival
    mbar_init(&ms.sready, NSTATE / 32);
    mbar_init(&ms.rready, NSTATE / 32);
    mbar_init(&ms.uready, NSTATE / 32);
    mbar_init(&ms.oread, NOUT / 32);
    mbar_init(&ms.apread, NSOLVE / 32);
    mbar_init(&ms.g[0], 1), mbar_init(&ms.g[1], 1);
    mbar_init(&ms.t[0], NSOLVE / 32);
    mbar_init(&ms.t[1], NSOLVE / 32);
    mbar_init(&ms.clean, NSOLVE / 32);
    fence_mbar_init();
    tma_prefetch_desc(&tmQ), tma_prefetch_desc(&tmK), tma_prefetch_desc(&tmV);
  }
  // the blocks of T and P above the diagonal stay zero
  for (int i = tid; i < (int)((OFF_P + 2 * R64 - OFF_T) / 16); i += NT)
    *reinterpret_cast<uint4*>(sm + OFF_T + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  if (warp == 0) {
    tmem_alloc(&ms.tmem_base, TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms.tmem_base;
  const uint32_t tlane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);

  auto wait = [&](uint64_t* bar, int parity) -> bool {
    return mbar_wait_short(bar, (uint32_t)(parity & 1), WAIT_TRIES);
  };
  auto give_up = [&]() {  // a wait ran out: the host is told (and the other warps' waits run out too)
    if (p.err) atomicOr(p.err, kErrWaitTimeout);
  };
  auto warp_arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  if (tid >= CTL) {
    setmaxnreg_dec<REG_CTL>();
    // ============================== the issuing thread ======================================
    if (wid == CTL / 32 && elect_one()) {
      int n_kq = 0, n_v = 0;  // chunks whose loads were issued
      auto load_kq = [&](int c) {
        unsigned char* at = sm + OFF_KQ + (c % QK_STAGES) * KQ_STAGE;
        uint64_t* bar = &ms.kq[c % QK_STAGES];
        mbar_arrive_expect_tx(bar, (uint32_t)(DK / 64) * R128);
        for (int pn = 0; pn < DK / 64; ++pn) {
          tma_load_4d(at + pn * R128, &tmK, bar, 64 * pn, hk, t0 + C * c, tb);
          tma_load_4d(at + pn * R128 + R64, &tmQ, bar, 64 * pn, hk, t0 + C * c, tb);
        }
        ++n_kq;
      };
      auto load_v = [&](int c) {
        unsigned char* at = sm + OFF_V + (c % V_STAGES) * V_STAGE;
        uint64_t* bar = &ms.v[c % V_STAGES];
        mbar_arrive_expect_tx(bar, (uint32_t)(DV / 64) * R64);
        for (int pn = 0; pn < DV / 64; ++pn) tma_load_4d(at + pn * R64, &tmV, bar, 64 * pn, hv, t0 + C * c, tb);
        ++n_v;
      };
      // [K; Q] K^T of chunk c (its tile landed, its absent rows zero)
      auto issue_ap = [&](int c) -> bool {
        if (!wait(&ms.kq[c % QK_STAGES], c / QK_STAGES)) return false;
        if (c == nch - 1 && tail < C && !wait(&ms.clean, 0)) return false;
        tc_fence_after();
        const uint32_t kq = sbase + OFF_KQ + (c % QK_STAGES) * KQ_STAGE;
#pragma unroll 1
        for (int pn = 0; pn < DK / 64; ++pn)
          four_ss(tmem + TM_AP, kdesc(kq) + PANEL * pn, kdesc(kq) + PANEL * pn, ID_AP, pn > 0);
        umma_commit(&ms.ap);
        return true;
      };
      // S^T (hi, then lo) times the rows of K (at = 0) or Q (at = R64)
      auto issue_state = [&](uint32_t d, uint32_t kq) {
#pragma unroll 1
        for (int half = 0; half < 2; ++half)
#pragma unroll 1
          for (int pn = 0; pn < DK / 64; ++pn)
            four_ts(tmem + d, tmem + TM_S + 64 * pn + 8 * half, kdesc(kq) + PANEL * pn, KSTEP, ID_AP, half + pn > 0);
      };
      // The order of the products (they execute in it), and what it guarantees:
      //   [K; Q] K^T of chunk c + 2 comes after P U of chunk c, so when it is done T(c) and P(c)
      //   are free to be overwritten by those of c + 2; A and P of c + 1 were read by then, as
      //   T(c + 1) is announced after that and chunk c + 2 is solved after chunk c + 1;
      //   the state handed on for chunk c means that all products of chunk c - 1 but P U are done.
      auto run = [&]() -> bool {
        for (int c = 0; c < QK_STAGES && c < nch; ++c) load_kq(c);
        for (int c = 0; c < V_STAGES && c < nch; ++c) load_v(c);
        if (!issue_ap(0)) return false;
        if (nch > 1 && (!wait(&ms.apread, 0) || !issue_ap(1))) return false;
#pragma unroll 1
        for (int c = 0; c < nch; ++c) {
          const uint32_t kq = sbase + OFF_KQ + (c % QK_STAGES) * KQ_STAGE;
          const uint32_t tt = sbase + OFF_T + (c & 1) * 2 * R64, pp = sbase + OFF_P + (c & 1) * R64;
          if (!wait(&ms.sready, c)) return false;
          STAMP(c, 0);
          tc_fence_after();
          issue_state(TM_R, kq);
          umma_commit(&ms.ks);
          STAMP(c, 1);
          if (c > 0 && c + 2 < nch) load_kq(c + 2);  // into chunk c - 1's stage
          STAMP(c, 2);
          if (!wait(&ms.t[c & 1], c >> 1) || !wait(&ms.rready, c)) return false;
          STAMP(c, 3);
          tc_fence_after();
          // U^T = R^T T^T: hi hi + hi lo + lo hi
          four_ts(tmem + TM_U, tmem + TM_R, kdesc(tt), KSTEP, ID_AP, 0);
          four_ts(tmem + TM_U, tmem + TM_R, kdesc(tt + R64), KSTEP, ID_AP, 1);
          four_ts(tmem + TM_U, tmem + TM_R + 8, kdesc(tt), KSTEP, ID_AP, 1);
          umma_commit(&ms.u);
          STAMP(c, 6);
          if (c + 2 < nch) load_v(c + 2);  // (V of chunk c was read before R was)
          // Q S, off the state's way: while U is read
          if (c > 0 && !wait(&ms.oread, c - 1)) return false;
          tc_fence_after();
          issue_state(TM_Q, kq + R64);
          if (!wait(&ms.uready, c)) return false;
          STAMP(c, 4);
          tc_fence_after();
          four_ts(tmem + TM_S, tmem + TM_U, ndesc(kq), NSTEP, ID_ST, 0);
          four_ts(tmem + TM_S, tmem + TM_U + 8, ndesc(kq), NSTEP, ID_ST, 1);
          umma_commit(&ms.s);
          STAMP(c, 7);
          const uint32_t ub = tmem + (ms.gate[c % GATE_SLOTS].mild ? TM_U : TM_UB);
          four_ts(tmem + TM_O, ub, kdesc(pp), KSTEP, ID_AP, 0);
          four_ts(tmem + TM_O, ub + 8, kdesc(pp), KSTEP, ID_AP, 1);
          umma_commit(&ms.o);
          mbar_arrive(&ms.o);  // (hands on the gates, which this thread has seen)
          STAMP(c, 5);
          if (c + 2 < nch && (!wait(&ms.apread, c + 1) || !issue_ap(c + 2))) return false;
        }
        return true;
      };
      const bool done = nch == 0 || run();
      if (!done) give_up();
      // every product and copy issued lands before the block releases its memory
      umma_commit(&ms.drain);
      mbar_wait_short(&ms.drain, 0, WAIT_TRIES);
      if (!done) {
        for (int c = max(0, n_kq - QK_STAGES); c < n_kq; ++c)
          mbar_wait_short(&ms.kq[c % QK_STAGES], (uint32_t)((c / QK_STAGES) & 1), WAIT_TRIES);
        for (int c = max(0, n_v - V_STAGES); c < n_v; ++c)
          mbar_wait_short(&ms.v[c % V_STAGES], (uint32_t)((c / V_STAGES) & 1), WAIT_TRIES);
      }
    }
    __syncwarp();
    if (wid == CTL / 32 + 1) {
      // ============================ decays, two tokens a lane =================================
      // sums in fp64 (a sum of 64 log decays rounded to fp32 would show in e^(G_t - G_s))
      float gn[2], bn[2];
      auto fetch_gates = [&](int c) {
  #pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int tt = C * c + 2 * lane + e;
          const size_t at = (size_t)(first + tt) * p.Hv + hv;
          gn[e] = tt < len ? __ldg(p.g + at) : 0.f;
          bn[e] = tt < len ? __ldg(p.beta + at) : 0.f;
        }
      };
      auto make_gates = [&](int c) {
        Gates& gt = ms.gate[c % GATE_SLOTS];
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
        const bool mild = end > -60.0;
        auto e2 = [](double x) { return exp2f((float)x); };
  #pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int tt = 2 * lane + e;
          const float hi = (float)G[e], eg = e2(G[e]);
          gt.G[tt] = make_float2(hi, (float)(G[e] - (double)hi));
          gt.r[tt] = make_float2(bn[e], -bn[e] * eg);
          gt.end[tt] = e2(end - G[e]);
          gt.out[tt] = p.scale * eg;
          gt.mid[tt] = e2(mid - G[e]);
        }
        if (lane == 31) gt.total = e2(end), gt.mild = mild;
      };
      if (nch > 0) fetch_gates(0);
#pragma unroll 1
      for (int c = 0; c < nch; ++c) {
        // when U of chunk c - 2 is there every warp has seen the barrier's previous use (the
        // outputs' warps before chunk c - 3 was written out), and chunk c - 5, whose slot this
        // is, is written out
        if (c >= 2 && !wait(&ms.u, c - 2)) {
          give_up();
          break;
        }
        make_gates(c);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.g[c & 1]);
        if (c + 1 < nch) fetch_gates(c + 1);
      }
    }
  } else if (warp < NSTATE / 32) {
    setmaxnreg_inc<REG_STATE>();
    // ============================== the state ==============================================
    constexpr int DKQ = DK / 4;
    const int cq = warp >> 2, ch = 32 * (warp & 3) + lane, t4 = lane & 3;
    const bool vval = ch < DV;  // (the same for a warp's 32 channels)
    const uint32_t vtile = sbase + OFF_V + (uint32_t)(((warp & 3) >> 1) & (DV / 64 - 1)) * R64;
    const int v16 = 4 * (warp & 1);  // the warp's first 16-byte piece (8 channels) of a row of V
    const size_t st = (size_t)unit * DK * DV + (size_t)(DKQ * cq) * DV + ch;
    float S[DKQ];
#pragma unroll
    for (int i = 0; i < DKQ; ++i) S[i] = (p.S0 && vval) ? p.S0[st + (size_t)i * DV] : 0.f;
    bool ok = true;
    for (int c = 0; c < nch; ++c) {
      const Gates& gt = ms.gate[c % GATE_SLOTS];
      if (tid == 0) STAMP(c, 8);
#pragma unroll
      for (int b = 0; b < DKQ / 16; ++b) {
        uint32_t w[16];
        split16(S + 16 * b, w);
        tmem_st16u(tlane + TM_S + DKQ * cq + 16 * b, w);
      }
      tmem_st_wait();
      if (tid == 0) STAMP(c, 9);
      tc_fence_before();
      warp_arrive(&ms.sready);
      // (g[] alternates between two barriers: that of chunk c runs again for c + 2, whose gates
      // wait for the product that this warp's R of chunk c goes into)
      if (!(ok = wait(&ms.g[c & 1], c >> 1) && wait(&ms.v[c % V_STAGES], c / V_STAGES))) break;
      const int live = c == nch - 1 ? tail : C;
      if (tid == 0) STAMP(c, 11);
      if (!(ok = wait(&ms.ks, c))) break;
      if (tid == 0) STAMP(c, 12);
      tc_fence_after();
      const uint32_t at = tlane + 16 * cq;  // this warp's K step of R and U; its rows in halves of 16
      {  // R = beta V - beta e^G (S^T K^T), in place
        float x[2][8];
        uint32_t vr[2][4];  // V^T in the same places, pairs of tokens packed
#pragma unroll
        for (int h = 0; h < 2; ++h) tmem_ld_frag16(at + ((uint32_t)(16 * h) << 16) + TM_R, x[h]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (vval) {
            const int t = 16 * cq + (lane & 7) + ((lane & 16) >> 1);
            ldmatrix_x4_trans(vr[h], vtile + (c % V_STAGES) * V_STAGE + t * 128 +
                                         (((v16 + 2 * h + ((lane >> 3) & 1)) ^ (t & 7)) << 4));
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) vr[h][i] = 0u;
          }
        }
        if (live < C) {  // tokens past the end
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int t = 16 * cq + 8 * ((i >> 1) & 1) + 2 * t4;
            uint32_t& w = vr[i >> 2][i & 3];
            w = t + 1 < live ? w : t < live ? (w & 0xFFFFu) : 0u;
          }
        }
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 2; ++j) {  // blocks of 8 tokens: this lane's pair of them
          const float4 f = *reinterpret_cast<const float4*>(&gt.r[16 * cq + 8 * j + 2 * t4]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // rows g, g + 8 of both halves
            const uint32_t pr = vr[i >> 1][2 * j + (i & 1)];
            float* y = &x[i >> 1][4 * j + 2 * (i & 1)];
            const float2 bv = mul2(make_float2(f.x, f.z), make_float2(__uint_as_float(pr << 16), __uint_as_float(pr & 0xFFFF0000u)));
            const float2 r = fma2(make_float2(f.y, f.w), make_float2(y[0], y[1]), bv);
            y[0] = r.x, y[1] = r.y;
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[8];
          split_frag(x[h], w);
          tmem_st_frag16(at + ((uint32_t)(16 * h) << 16) + TM_R, w);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&ms.rready);
      if (tid == 0) STAMP(c, 13);
      if (!(ok = wait(&ms.u, c))) break;
      if (tid == 0) STAMP(c, 14);
      tc_fence_after();
      {  // e^(G_C - G) U in place; and U itself for P U, unless P takes the former (mild)
        float x[2][8];
        uint32_t w[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) tmem_ld_frag16(at + ((uint32_t)(16 * h) << 16) + TM_U, x[h]);
        tmem_ld_wait();
        if (!gt.mild) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            split_frag(x[h], w);
            tmem_st_frag16(at + ((uint32_t)(16 * h) << 16) + TM_UB, w);
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 f = *reinterpret_cast<const float2*>(&gt.end[16 * cq + 8 * j + 2 * t4]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float* y = &x[i >> 1][4 * j + 2 * (i & 1)];
            const float2 r = mul2(f, make_float2(y[0], y[1]));
            y[0] = r.x, y[1] = r.y;
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          split_frag(x[h], w);
          tmem_st_frag16(at + ((uint32_t)(16 * h) << 16) + TM_U, w);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&ms.uready);
      if (tid == 0) STAMP(c, 15);
      const float total = gt.total;
      if (!(ok = wait(&ms.s, c))) break;
      if (tid == 0) STAMP(c, 16);
      tc_fence_after();
#pragma unroll
      for (int b = 0; b < DKQ / 16; ++b) {
        float x[16];
        tmem_ld16(tlane + TM_S + DKQ * cq + 16 * b, x);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float2 y = fma2(make_float2(total, total), make_float2(S[16 * b + i], S[16 * b + i + 1]),
                                make_float2(x[i], x[i + 1]));
          S[16 * b + i] = y.x, S[16 * b + i + 1] = y.y;
        }
      }
    }
    if (!ok) give_up();
    if (ok && p.S_T && vval) {
#pragma unroll
      for (int i = 0; i < DKQ; ++i) p.S_T[st + (size_t)i * DV] = S[i];
    }
  } else if (warp < (NSTATE + NSOLVE) / 32) {
    setmaxnreg_inc<REG_SOLVE>();
    // ============================== decays, A, P and T, a chunk ahead ========================
    const int sw = warp - NSTATE / 32;        // this warp of the eight
    const int row = 32 * (sw & 3) + lane;     // of [K; Q]; blocks of 16 columns: 2 (sw / 4) and the next
    const int t = row & 63;                   // token of rows K (0-63) and Q (64-127)
    float* M = reinterpret_cast<float*>(sm + OFF_M);
    float* X = reinterpret_cast<float*>(sm + OFF_X) + (sw & 3) * 32 * LDW;
    const int g4 = lane >> 2, t4 = lane & 3;
    constexpr std::integral_constant<int, 2> K16{};  // K steps of 8
    constexpr std::integral_constant<int, 4> K32{};
    bool ok = true;
#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
      const Gates& gt = ms.gate[c % GATE_SLOTS];
      if (c == nch - 1 && tail < C) {  // rows after the sequence's end: another's, or anything
        ok = ok && wait(&ms.kq[c % QK_STAGES], c / QK_STAGES);
        unsigned char* kq = sm + OFF_KQ + (c % QK_STAGES) * KQ_STAGE;
        for (int i = tid - NSTATE; i < (C - tail) * 8; i += NSOLVE) {
#pragma unroll
          for (int pn = 0; pn < DK / 64; ++pn)
#pragma unroll
            for (int q = 0; q < 2; ++q)
              *reinterpret_cast<uint4*>(kq + pn * R128 + q * R64 + (tail + (i >> 3)) * 128 + (i & 7) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        warp_arrive(&ms.clean);
      }
      if (sw == 0 && lane == 0) STAMP(c, 20);
      ok = ok && wait(&ms.g[c & 1], c >> 1) && wait(&ms.ap, c);
      if (sw == 0 && lane == 0) STAMP(c, 21);
      tc_fence_after();
      unsigned char* pt = sm + OFF_P + (c & 1) * R64;
      // A_ts = beta e^(G_t - G_s) k_t k_s and P.  In a mild chunk (its decay stays above 2^-60)
      // e^(G_t - G_s) = e^(G_t - G_m) e^(G_m - G_s) with the chunk's middle m, and P is kept as
      // scale e^(G_t - G_C) q_t k_s, for the product with e^(G_C - G) U; otherwise element by
      // element.  (Columns 32-63 of rows 0-31 are above the diagonal: P's stay zero, A's unread.)
      const int w2 = sw & 1, ch2 = sw >> 2;  // rows 32-63 of the token range; columns 32-63
      if (w2 >= ch2) {
        const bool isA = row < 64, diag = w2 == ch2, mild = gt.mild;
        const float2 Gt = gt.G[t], Gr = gt.G[isA ? 31 : 63];
        float own = isA ? gt.r[t].x : p.scale;
        if (mild) own *= ex2_approx((Gt.x - Gr.x) + (Gt.y - Gr.y));
        float x[32];
        tmem_ld32(tlane + TM_AP + 32 * ch2, x);
        tmem_ld_wait();
        if (mild) {
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            float2 f = make_float2(own, own), h = f;
            if (isA) {
              const float4 m = ld4(&gt.mid[32 * ch2 + i]);
              f = mul2(f, make_float2(m.x, m.y)), h = mul2(h, make_float2(m.z, m.w));
            }
            const float2 u = mul2(f, make_float2(x[i], x[i + 1])), v = mul2(h, make_float2(x[i + 2], x[i + 3]));
            x[i] = u.x, x[i + 1] = u.y, x[i + 2] = v.x, x[i + 3] = v.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 Gs = gt.G[32 * ch2 + i];
            x[i] *= own * ex2_approx(fminf((Gt.x - Gs.x) + (Gt.y - Gs.y), 0.f));
          }
        }
        if (diag) {
          const int lim = (t & 31) + (isA ? 0 : 1);  // columns of these 32 that count
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = i < lim ? x[i] : 0.f;
        }
        if (isA) {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(M + t * LDM + 32 * ch2 + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(pt + sw128_off(t, 4 * ch2 + i)) =
                make_uint4(pack_bf16(x[8 * i], x[8 * i + 1]), pack_bf16(x[8 * i + 2], x[8 * i + 3]),
                           pack_bf16(x[8 * i + 4], x[8 * i + 5]), pack_bf16(x[8 * i + 6], x[8 * i + 7]));
        }
      }
      tc_fence_before();
      warp_arrive(&ms.apread);
      if (named_bar_or(BAR_SOLVE, NSOLVE, !ok)) break;  // a wait gave up: the warps leave together
      if (sw == 0 && lane == 0) STAMP(c, 22);
      // ---- T = (I + A)^-1, blocks of 8, then merges T_IJ = -T_II (A_IJ T_JJ) of 16, 32 and 64;
      // fp32 in M (A's blocks turn into T's), and T as hi and lo operand tiles
      unsigned char* tt = sm + OFF_T + (c & 1) * 2 * R64;
      auto put_t = [&](int r, int s, float x) {
        const uint32_t at = sw128_off(r, s >> 3) + (uint32_t)(s & 7) * 2;
        const __nv_bfloat16 hi = __float2bfloat16_rn(x);
        *reinterpret_cast<__nv_bfloat16*>(tt + at) = hi;
        *reinterpret_cast<__nv_bfloat16*>(tt + R64 + at) = __float2bfloat16_rn(x - __bfloat162float(hi));
      };
      auto put_t2 = [&](int r, int s, float x0, float x1) {  // columns s (even) and s + 1
        const uint32_t at = sw128_off(r, s >> 3) + (uint32_t)(s & 7) * 2;
        uint32_t hi, lo;
        split2(x0, x1, hi, lo);
        *reinterpret_cast<uint32_t*>(tt + at) = hi;
        *reinterpret_cast<uint32_t*>(tt + R64 + at) = lo;
      };
      if (sw < 4) {  // the diagonal blocks 2 sw (lanes 0-7) and 2 sw + 1 (lanes 8-15): a column to a lane
        const int r0 = 16 * sw + 8 * ((lane >> 3) & 1), col = lane & 7;
        float x[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) x[r] = (r == col) ? 1.f : 0.f;
#pragma unroll
        for (int r = 1; r < 8; ++r) {
          const float4 a0 = ld4(M + (r0 + r) * LDM + r0), a1 = ld4(M + (r0 + r) * LDM + r0 + 4);
          const float ar[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
          float acc = 0.f;
#pragma unroll
          for (int s = 0; s < r; ++s) acc = fmaf(ar[s], x[s], acc);
          if (r > col) x[r] = -acc;
        }
        __syncwarp();
        if (lane < 16) {
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            M[(r0 + r) * LDM + r0 + col] = x[r];
            put_t(r0 + r, r0 + col, x[r]);
          }
        }
        __syncwarp();
      }
      if (sw < 4) {  // 16: the block below the diagonal, two columns to a lane
        const int J = 16 * sw, I = J + 8, r = g4, c0 = 2 * t4;
        float z0 = 0.f, z1 = 0.f;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const float a = M[(I + r) * LDM + J + s];
          const float2 tb2 = *reinterpret_cast<const float2*>(M + (J + s) * LDM + J + c0);
          z0 = fmaf(a, tb2.x, z0);
          z1 = fmaf(a, tb2.y, z1);
        }
        *reinterpret_cast<float2*>(X + r * LDW + c0) = make_float2(z0, z1);
        __syncwarp();
        float y0 = 0.f, y1 = 0.f;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const float a = M[(I + r) * LDM + I + s];
          const float2 xb = *reinterpret_cast<const float2*>(X + s * LDW + c0);
          y0 = fmaf(a, xb.x, y0);
          y1 = fmaf(a, xb.y, y1);
        }
        *reinterpret_cast<float2*>(M + (I + r) * LDM + J + c0) = make_float2(-y0, -y1);
        put_t2(I + r, J + c0, -y0, -y1);
      }
      // D (16 x 8) = A (16 rows of M at Ar) B (8 KS rows at Bc), operands split in two tf32
      // parts: hi hi, hi lo and lo hi in chains of their own
      auto mma3 = [&](const float* Ar, const float* Bc, int ldb, auto KS, float (&d)[4]) {
        float dl[4] = {0.f, 0.f, 0.f, 0.f}, dm[4] = {0.f, 0.f, 0.f, 0.f};
        d[0] = d[1] = d[2] = d[3] = 0.f;
        const float* a = Ar + ((lane & 7) + (lane & 8)) * LDM + ((lane & 16) >> 2);
#pragma unroll
        for (int ks = 0; ks < decltype(KS)::value; ++ks) {
          const float* b = Bc + (8 * ks + t4) * ldb + g4;
          uint32_t ah[4], al[4], bh[2], bl[2];
          ldmatrix_x4(ah, a + 8 * ks);
#pragma unroll
          for (int i = 0; i < 4; ++i) split_tf32(__uint_as_float(ah[i]), ah[i], al[i]);
          split_tf32(b[0], bh[0], bl[0]);
          split_tf32(b[4 * ldb], bh[1], bl[1]);
          mma_16x8x8_tf32(d, ah, bh);
          mma_16x8x8_tf32(dl, ah, bl);
          mma_16x8x8_tf32(dm, al, bh);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] += dl[i] + dm[i];
      };
      auto put_x = [&](int r, const float (&d)[4]) {
        *reinterpret_cast<float2*>(X + (r + g4) * LDW + 2 * t4) = make_float2(d[0], d[1]);
        *reinterpret_cast<float2*>(X + (r + g4 + 8) * LDW + 2 * t4) = make_float2(d[2], d[3]);
      };
      named_bar_sync(BAR_SOLVE, NSOLVE);
      if (sw == 0 && lane == 0) STAMP(c, 23);
      if (sw < 4) {  // 32: warps 2 k, 2 k + 1 merge blocks 2 k and 2 k + 1, eight columns each
        const int J = 32 * (sw >> 1), I = J + 16, c0 = J + 8 * (sw & 1);
        float d[4], y[4];
        mma3(M + I * LDM + J, M + J * LDM + c0, LDM, K16, d);
        put_x(0, d);
        named_bar_sync(BAR_PAIR + (sw >> 1), 64);  // (both warps have read A_IJ)
        mma3(M + I * LDM + I, X, LDW, K16, y);
        *reinterpret_cast<float2*>(M + (I + g4) * LDM + c0 + 2 * t4) = make_float2(-y[0], -y[1]);
        *reinterpret_cast<float2*>(M + (I + g4 + 8) * LDM + c0 + 2 * t4) = make_float2(-y[2], -y[3]);
        put_t2(I + g4, c0 + 2 * t4, -y[0], -y[1]);
        put_t2(I + g4 + 8, c0 + 2 * t4, -y[2], -y[3]);
      }
      named_bar_sync(BAR_SOLVE, NSOLVE);
      if (sw == 0 && lane == 0) STAMP(c, 24);
      {  // 64: warps q and q + 4 take eight columns, sixteen rows each
        const int c0 = 8 * (sw & 3), r0 = 16 * (sw >> 2);
        float d[4];
        mma3(M + (32 + r0) * LDM, M + c0, LDM, K32, d);
        put_x(r0, d);
        named_bar_sync(BAR_PAIR + (sw & 3), 64);
        if (r0 == 0)
          mma3(M + 32 * LDM + 32, X, LDW, K16, d);  // (T_II's upper half is zero)
        else
          mma3(M + 48 * LDM + 32, X, LDW, K32, d);
        put_t2(32 + r0 + g4, c0 + 2 * t4, -d[0], -d[1]);
        put_t2(40 + r0 + g4, c0 + 2 * t4, -d[2], -d[3]);
      }
      fence_proxy_async_smem();
      warp_arrive(&ms.t[c & 1]);
      if (sw == 0 && lane == 0) STAMP(c, 25);
      named_bar_sync(BAR_SOLVE, NSOLVE);  // (M is free again)
    }
    if (!ok) give_up();
  } else {
    setmaxnreg_dec<REG_OUT>();
    // ============================== outputs ================================================
    const int ch = tid - NSTATE - NSOLVE;  // value channel = lane of tensor memory
    const int ow = ch;                     // thread of this group
    const uint32_t stage = sbase + OFF_O;  // rows of DV channels, 16-byte pieces swizzled by the row
    const int t4 = lane & 3;
    bool ok = true;
#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
      const Gates& gt = ms.gate[c % GATE_SLOTS];
      ok = ok && wait(&ms.o, c);
      if (ow == 0) STAMP(c, 28);
      tc_fence_after();
      if (32 * (warp & 3) < DV) {
#pragma unroll 1
        for (int part = 0; part < 4; ++part) {  // 16 rows (h) by 32 tokens (from t0)
          const int h = part & 1, tok = 32 * (part >> 1);
          const uint32_t at = tlane + ((uint32_t)(16 * h) << 16) + tok;
          float x[16], y[16];
          tmem_ld_frag32(at + TM_Q, x);
          tmem_ld_frag32(at + TM_O, y);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int i = 8 * e + 4 * j;
              const float2 f = *reinterpret_cast<const float2*>(&gt.out[tok + 16 * e + 8 * j + 2 * t4]);
              const float2 a = fma2(f, make_float2(x[i], x[i + 1]), make_float2(y[i], y[i + 1]));
              const float2 b = fma2(f, make_float2(x[i + 2], x[i + 3]), make_float2(y[i + 2], y[i + 3]));
              w[2 * j] = pack_bf16(a.x, a.y), w[2 * j + 1] = pack_bf16(b.x, b.y);
            }
            // matrix m of the four: channels 8 (m % 2) on, tokens 8 (m / 2) on
            const int t = tok + 16 * e + (lane & 7) + ((lane & 16) >> 1);
            const int piece = 4 * (warp & 3) + 2 * h + ((lane >> 3) & 1);
            stmatrix_x4_trans(stage + t * DV * 2 + ((piece ^ (t & 7)) << 4), w);
          }
        }
      }
      tc_fence_before();
      warp_arrive(&ms.oread);  // (this chunk's gates are read as well)
      if (named_bar_or(BAR_OUT, NOUT, !ok)) {
        give_up();
        break;
      }
      if (ow == 0) STAMP(c, 29);
      const int rows = c == nch - 1 ? tail : C;
      constexpr int CPR = DV / 8;  // 16-byte pieces of a row
      __nv_bfloat16* ob = p.o + ((size_t)(first + (long long)C * c) * p.Hv + hv) * DV;
      for (int i = ow; i < rows * CPR; i += NOUT)
        *reinterpret_cast<uint4*>(ob + (size_t)(i / CPR) * p.Hv * DV + (i % CPR) * 8) =
            *reinterpret_cast<const uint4*>(sm + OFF_O + (i / CPR) * DV * 2 + (((i % CPR) ^ ((i / CPR) & 7)) << 4));
      named_bar_sync(BAR_OUT, NOUT);
      if (ow == 0) STAMP(c, 30);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, TM_COLS);
}

// ---- host side ------------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult qres;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &qres) != cudaSuccess ||
        qres != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }();
  return fn;
}
// [B, T, H, D] bf16; one box = C tokens x 64 channels of one (sequence, head)
bool map_tokens(CUtensorMap* m, const void* base, int B, int T, int H, int D) {
  auto fn = encoder();
  if (!fn) return false;
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T, (cuuint64_t)B};
  cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)H * D * 2, (cuuint64_t)T * H * D * 2};
  cuuint32_t box[4] = {64, 1, (cuuint32_t)C, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int DV>
cudaError_t launch_dims(const GdrArgs& a, cudaStream_t st) {
  CUtensorMap mq, mk, mv;
  const int B = a.cu_seqlens ? 1 : a.B;
  if (!map_tokens(&mq, a.q, B, a.T, a.Hk, DK) || !map_tokens(&mk, a.k, B, a.T, a.Hk, DK) ||
      !map_tokens(&mv, a.v, B, a.T, a.Hv, DV))
    return cudaErrorInvalidValue;
  TcParams p{a.g, a.beta, a.cu_seqlens, a.S0, static_cast<__nv_bfloat16*>(a.o), a.S_T, a.T, a.Hk, a.Hv, a.scale,
             device_error_word(), stamp_buffer()};
  static std::atomic<unsigned long long> attr_done{0};
  cudaError_t e = smem_limit_once(gdr_chunk_tc_kernel<DK, DV>, (int)SMEM_BYTES, attr_done);
  if (e != cudaSuccess) return e;
  gdr_chunk_tc_kernel<DK, DV><<<a.B * a.Hv, NT, SMEM_BYTES, st>>>(mq, mk, mv, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gdr_chunk_tc(const GdrArgs& a, cudaStream_t st) {
  if (!a.bf16 || a.T == 0) return cudaErrorInvalidValue;
  if (a.dk == 128) return a.dv == 128 ? launch_dims<128, 128>(a, st) : launch_dims<128, 64>(a, st);
  return a.dv == 128 ? launch_dims<64, 128>(a, st) : launch_dims<64, 64>(a, st);
}

}  // namespace gdn2
