// Chunkwise prefill forward of the gated delta rule with scalar gates for bf16 inputs, the state's
// way through the chunks on the 5th-generation tensor cores (tcgen05.mma kind::f16, accumulators in
// tensor memory, tiles by TMA), and the split of long sequences.
//
// The recurrence (snilld.dk, "Hvad Gated DeltaNet-2 aendrer": the rule left when both gates and
// the decay are scalars) in its WY form over chunks of 64 tokens (Gated DeltaNet-2 guide,
// "Chunkwise Parallel Algorithm for GPU Training").  With G_t the sum of the log decays of the
// chunk up to token t, e^G its exponential and K, Q, V the chunk's rows:
//
//     A_ts = beta_t e^(G_t - G_s) k_t . k_s  (s < t),      T = (I + A)^-1 diag(beta)
//     P_ts = e^(G_t - G_s) q_t . k_s         (s <= t)
//     R  = -e^G K S,               U = T V + T R
//     O  = scale (e^G Q S + P U),  S' = e^(G_C) S + K^T (e^(G_C - G) U)
//
// T, P and the factors of G come from gdr_prep.cu, which does all chunks at once; this kernel is
// what is left in sequence.  In a chunk whose decay stays above 2^-60 ("mild": all but the
// steepest) T's rows carry e^(G_C - G) already and P the inverse, so that the product leaves
// U_end = e^(G_C - G) U, which both of U's products take.  A scalar decay never has to be folded
// into K or Q, so the products take the raw bf16 tiles (exact operands) and every factor of a
// decay is e^(difference <= 0): nothing overflows, and there is no limit on the decay.
//
// Precision.  S, R, U, T and P are fp32 values; where one of them is an operand it is split into
// two bf16 parts, x = hi + lo (off by 2^-16 |x| at most), and a product of two split operands drops
// lo lo (2^-16).  Measured in the 2-norm with beta <= 1 or some decay, S_T is 3 to 5e-6 off for
// independent keys, 0.5 to 1e-5 for correlated ones, 1 to 6e-5 for one key all over; without decay at
// beta = 1.99, 3e-5, 1e-4 and (1500 times that key) 1.6e-3.  o is off by its rounding, 1.7e-3, in all of these
// but the last.  (Third parts, for 2^-24, would be one of T as well, 5 KB more a record.)  With P as a
// single bf16 the products of correlated keys, which cancel, left o 0.6 to 1.2e-2 off; its second part
// costs 4 % (B8 H16 T4096 262 -> 272 us).
//
// That second part is written by gdr_prep.cu where the chunk's outputs will be, row t of it to token t's first
// 64 channels, and loaded as a tile before they are: no room in the records, and none in the workspace.
// Rows past a sequence's end hold anything; they are columns of O^T past the last token, never stored.
//
// Layout.  One CTA per (sequence, value head).  Everything on the state's way through a chunk
// is held transposed, value channels on the 128 lanes of tensor memory, so that each
// product's result is the next one's A operand in place, thread by thread.  The 16 columns of one K
// step (two bf16 to a column) hold [hi (8) | lo (8)] where the 16 fp32 results were.
//   warps 0-15 (0-7 in the split's first launch): the state, rows = value channel, quarters (halves)
//               of the columns, S itself in registers; R and U as product fragments (row and pair
//               of tokens by lane), where the factors of a token serve many rows
//   four warps: the outputs, Q S and P U to bf16 rows of o (not in the split's first launch)
//   four warps: one thread issues the products and the loads
// d_v = 64 runs with the upper 64 lanes zero.  T and P are lower triangular: K step ks of their
// products takes the columns from 16 ks on only (B8 H16 T4096 274 -> 269 us in all).
//
// What bounds it: the latency of a chunk's chain, 5.1 thousand cycles (2.7 us) at d = 128: three products
// (0.73, 0.49 and 0.86 thousand cycles from the last operand seen to the result seen) with the state's
// warps between them, which split 32, 16 and 16 values a thread (1.31, 0.84 and 0.89 thousand).  The
// tensor pipe is busy 38 % of the time, the issue slots 36 %.  8192 chunks of 128 (sequence, head) pairs
// take 189 us, their preparation 85.  Slower, measured: the preparation in this kernel, on warps of its own
// (3.6 us a chunk) or in the waits of the state's (4.2 us); W = -T e^G K formed ahead, so that two
// products are left in the chain (6.1 thousand cycles a chunk: forming W and splitting it takes longer
// than the R it saves); a product's K steps issued as the warps of each quarter hand them on
// (275 to 285 us for all of it instead of 269: each wait costs the issuing thread more than it gains).
//
// Long sequences with few heads: the recurrence is linear in (S, V), so the state after a segment
// of chunks is M S + N, M from S = I without V and N from S = 0.  A first launch runs both for
// every segment (no outputs), gdr_join_kernel chains the segments' first states, and a second
// launch runs all segments at once (B1 H16 T65536: 2.9 ms in whole sequences, 0.90 in
// 9 segments: 171 us of preparation, 400, 26 and 356 of the three; the first launch's chunks take
// 3.5 us with two blocks to an SM and 2.65 alone).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "gdn2_internal.h"
#include "gdr_chunk.cuh"
#include "ptx.cuh"

namespace gdn2 {
namespace {

constexpr int C = GDR_C;
constexpr int BAR_OUT = 1;        // named barrier of the outputs' warps
constexpr int WAIT_TRIES = 2000;  // suspensions of 1 ms: about 2 s per wait
constexpr int KQ_STAGES_MOST = 3, V_STAGES = 2, REC_STAGES = 3;
constexpr uint32_t R64 = 64 * 128, R128 = 128 * 128;  // panels of 64 channels (128 bytes) by rows

// The kernel's two forms.  The split's first launch (FIRSTS) has states only, no Q and no outputs: half of the
// state's warps, of the shared and of the tensor memory, so that two blocks share an SM and one's
// products run beside the other's splits.
template <bool FIRSTS>
struct Form {
  static constexpr int NSTATE = FIRSTS ? 256 : 512, NOUT = FIRSTS ? 0 : 128;
  static constexpr int CTL = NSTATE + NOUT;  // the issuing thread's warp
  static constexpr int NT = CTL + 128, BLOCKS = FIRSTS ? 2 : 1;
  // registers a thread of each warpgroup: those of the state (which holds S), the outputs and the
  // issuing one share what NT threads are launched with, 80 each
  static constexpr int REG_LAUNCH = 80, REG_STATE = FIRSTS ? 104 : 96, REG_OUT = 56, REG_CTL = FIRSTS ? 32 : 40;
  static_assert(NSTATE / 128 * REG_STATE + NOUT / 128 * REG_OUT + REG_CTL <= NT / 128 * REG_LAUNCH, "the launch's registers");
  static constexpr int NQ = NSTATE / 128;  // parts of the columns that the state's warps share
  // ---- shared memory (byte offsets from a 1024-byte aligned base)
  static constexpr int KQ_STAGES = FIRSTS ? 2 : 3;
  static constexpr uint32_t KROWS = FIRSTS ? R64 : R128;  // a panel of [K; Q], or of K
  static constexpr uint32_t KQ_STAGE = 2 * KROWS, V_STAGE = 2 * R64;
  static constexpr uint32_t RECORD = FIRSTS ? GDR_P : GDR_RECORD;  // without P
  static constexpr uint32_t REC_STAGE = (RECORD + 1023) / 1024 * 1024;
  static constexpr uint32_t OFF_V = KQ_STAGES * KQ_STAGE;
  static constexpr uint32_t OFF_O = OFF_V + V_STAGES * V_STAGE;        // o staging [t][v] bf16
  static constexpr uint32_t OFF_REC = OFF_O + (FIRSTS ? 0 : 2 * R64);  // records: T, gates, P
  static constexpr uint32_t OFF_P2 = OFF_REC + REC_STAGES * REC_STAGE;  // P's second parts [t][s], a stage a record
  static constexpr uint32_t TILES = OFF_P2 + (FIRSTS ? 0 : REC_STAGES * R64);
  // ---- tensor memory columns
  static constexpr uint32_t TM_S = 0;     // S^T in [hi | lo] blocks, then U_end^T K in its place (d_k)
  static constexpr uint32_t TM_R = 128;   // S^T K^T (64), then R^T in its place
  static constexpr uint32_t TM_U = 192;   // U_end^T, not mild: U^T (64), then U_end^T in [hi | lo] blocks in its place
  static constexpr uint32_t TM_Q = 256;   // S^T Q^T (64)
  static constexpr uint32_t TM_UB = 320;  // U^T in [hi | lo] blocks (64), for chunks that are not mild
  static constexpr uint32_t TM_O = 384;   // U^T P^T (64)
  static constexpr uint32_t TM_COLS = FIRSTS ? 256 : 512;
};

struct Misc {
  uint64_t kq[KQ_STAGES_MOST], v[V_STAGES], rec[REC_STAGES];  // loads landed
  uint64_t ks, u, s, o, drain;                           // products done
  uint64_t sready, rready, uready, oread;                // threads -> the issuing thread
  uint32_t tmem_base;
};
template <bool FIRSTS>
constexpr uint32_t smem_bytes() {
  return Form<FIRSTS>::TILES + 1024 + (uint32_t)sizeof(Misc);
}
static_assert(smem_bytes<false>() <= 232448 && 2 * (smem_bytes<true>() + 1024) <= 233472, "shared memory of the SM's blocks");

struct ChainParams {
  const int* cu;
  const unsigned char* records;
  const float* S0;       // entering states, or NULL
  __nv_bfloat16* o;
  float* S_T;            // or NULL
  int T, Hv, Hk;
  // split: every sequence's chunks in segs segments of the same length (segs = 1: whole sequences).
  // First launch (FIRSTS): jobs 0 .. segs - 2 of a unit are N of those segments (segment 0 from
  // S0), then M of segments 1 .. segs - 2, into states [job][unit].  Second: jobs are segments,
  // entering states starts [segment][unit].
  int segs;
  float* states;
  const float* starts;
  unsigned* err;
  unsigned long long* stamps = nullptr;  // instrumented build only: per-chunk clock stamps
};
#ifdef GDN2_STAMPS
// Instrumented build (GDN2_STAMPS): clock64 of the SM at fixed points of the first CTA's chunks.
#define STAMP(cc, slot)                                                                                    \
  do {                                                                                                     \
    if (p.stamps && blockIdx.x == 0 && (cc) >= 0 && (cc) < 64)                                             \
      p.stamps[(cc) * 32 + (slot)] = (unsigned long long)clock64();                                        \
  } while (0)
#else
#define STAMP(cc, slot) \
  do {                  \
  } while (0)
#endif

// A K step (two blocks of 8 tokens) of fragments, x as tmem_ld_frag16 gives it -> its 16
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
// Descriptor of the first K step of a K-major panel (the next one is 32 bytes on), and of an
// N-major tile in panels of 64 columns (the next one is 16 rows on).
__device__ __forceinline__ uint64_t kdesc(uint32_t base) { return sdesc_sw128(base, 16, 1024); }
__device__ __forceinline__ uint64_t ndesc(uint32_t base, uint32_t panel) { return sdesc_sw128(base, panel, 1024); }
constexpr uint32_t KSTEP = 32 >> 4, NSTEP = 2048 >> 4;  // in descriptor units

// n K steps of a product, a (tensor memory, 16 columns a step) by b in panels of four steps, `panel` apart.
// (Unrolled by a panel: one by one, the issue of a product takes longer than the product; all
// unrolled, the code of a chunk outgrows the instruction cache.)
__device__ __forceinline__ void steps_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t bstep, uint32_t panel, int n,
                                         uint32_t idesc, uint32_t acc) {
#pragma unroll 1
  for (int pn = 0; pn < n / 4; ++pn, a += 64, b += panel, acc = 1) {
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) umma_f16_ts(d, a + 16 * ks, b + bstep * ks, idesc, ks > 0 ? 1u : acc);
  }
}

// T and P are lower triangular: step ks of a product with them meets columns 16 ks on only.  tdesc: its
// descriptor.
__device__ __forceinline__ uint64_t tdesc(uint32_t base, int ks) { return sdesc_plain(base, 128, 256) + (gdr_tri_step(ks) >> 4); }
__device__ __forceinline__ void steps_tri(uint32_t d, uint32_t a, uint32_t b, uint32_t acc) {
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
    umma_f16_ts(d + 16 * ks, a + 16 * ks, tdesc(b, ks), idesc_bf16(128, 64 - 16 * ks, 0, 0), ks > 0 ? 1u : acc);
}

// FIRSTS: the split's first launch (states only: no Q, no outputs).
template <int DK, int DV, bool FIRSTS>
__global__ void __launch_bounds__(Form<FIRSTS>::NT, Form<FIRSTS>::BLOCKS)
    gdr_chain_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmP, const ChainParams p) {
  using F = Form<FIRSTS>;
  constexpr int NSTATE = F::NSTATE, NOUT = F::NOUT, CTL = F::CTL, KQ_STAGES = F::KQ_STAGES;
  constexpr uint32_t KROWS = F::KROWS, KQ_STAGE = F::KQ_STAGE, V_STAGE = F::V_STAGE, REC_STAGE = F::REC_STAGE;
  constexpr uint32_t OFF_KQ = 0, OFF_V = F::OFF_V, OFF_O = F::OFF_O, OFF_REC = F::OFF_REC, OFF_P2 = F::OFF_P2, TILES = F::TILES;
  constexpr uint32_t TM_S = F::TM_S, TM_R = F::TM_R, TM_Q = F::TM_Q, TM_U = F::TM_U, TM_UB = F::TM_UB, TM_O = F::TM_O;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Misc& ms = *reinterpret_cast<Misc*>(sm + TILES);
  const uint32_t sbase = smem_u32(sm);
  constexpr uint32_t ID_64 = idesc_bf16(128, 64, 0, 0);
  constexpr uint32_t ID_ST = idesc_bf16(128, DK, 0, 1);  // B = K as [token][channel]: N-major

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int wid = __shfl_sync(0xffffffffu, warp, 0);  // the same value, known to be uniform
  const int jobs = FIRSTS ? 2 * p.segs - 3 : p.segs;
  const int unit = blockIdx.x / jobs, job = blockIdx.x % jobs;
  const int n = unit / p.Hv, hv = unit % p.Hv, hk = hv / (p.Hv / p.Hk);
  long long first = (long long)n * p.T;  // flat token index of the first chunk
  int len = p.T, tb = n, t0 = 0;         // tensor-map coordinates: sequence tb, token t0
  long long slot = (long long)n * ((p.T + C - 1) / C);  // of the first chunk's records
  if (p.cu) {
    const int lo = p.cu[n], hi = p.cu[n + 1];
    if (lo < 0 || hi < lo || hi > p.T) {  // offsets out of order or range: nothing is touched
      if (tid == 0 && p.err) atomicOr(p.err, kErrBadSeqlens);
      grid_wait();  // (so that this grid is done only when the one in front is)
      return;
    }
    first = lo, len = hi - lo, tb = 0, t0 = lo, slot = (lo >> 6) + n;
  }
  bool transition = false, last = true;  // M of a segment; the sequence's last segment
  int seg = 0;
  if (p.segs > 1) {
    transition = FIRSTS && job >= p.segs - 1;
    seg = transition ? job - (p.segs - 1) + 1 : job;
    const long long per = (((long long)len + C - 1) / C + p.segs - 1) / p.segs * C;
    const int begin = (int)min((long long)len, seg * per), end = (int)min((long long)len, (seg + 1) * per);
    last = seg == p.segs - 1;
    first += begin, t0 += begin, slot += begin / C, len = (last ? len : end) - begin;
  }
  const int nch = (len + C - 1) / C;
  const int tail = len - (nch - 1) * C;  // tokens of the last chunk

  if (tid == 0) {
    for (int i = 0; i < KQ_STAGES; ++i) mbar_init(&ms.kq[i], 1);
    for (int i = 0; i < V_STAGES; ++i) mbar_init(&ms.v[i], 1);
    for (int i = 0; i < REC_STAGES; ++i) mbar_init(&ms.rec[i], 1);
    uint64_t* ones[] = {&ms.ks, &ms.u, &ms.s, &ms.drain};
    for (uint64_t* b : ones) mbar_init(b, 1);
    mbar_init(&ms.o, 2);  // the products, and the issuing thread's own arrival
    mbar_init(&ms.sready, NSTATE / 32);
    mbar_init(&ms.rready, NSTATE / 32);
    mbar_init(&ms.uready, NSTATE / 32);
    mbar_init(&ms.oread, 4);
    fence_mbar_init();
    tma_prefetch_desc(&tmK), tma_prefetch_desc(&tmV);
    if (!FIRSTS) tma_prefetch_desc(&tmQ), tma_prefetch_desc(&tmP);
  }
  if (warp == 0) {
    tmem_alloc(&ms.tmem_base, F::TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (FIRSTS) grid_release();
  grid_wait();  // the records, and in the split's second launch the segments' first states
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
  auto gates = [&](int c) -> const GdrGates& {
    return *reinterpret_cast<const GdrGates*>(sm + OFF_REC + (c % REC_STAGES) * REC_STAGE + GDR_GATES);
  };

  if (tid >= CTL) {
    setmaxnreg_dec<F::REG_CTL>();
    // ============================== the issuing thread ======================================
    if (wid == CTL / 32 && elect_one()) {
      int n_kq = 0, n_v = 0, n_rec = 0;  // chunks whose loads were issued
      auto load_kq = [&](int c) {
        unsigned char* at = sm + OFF_KQ + (c % KQ_STAGES) * KQ_STAGE;
        uint64_t* bar = &ms.kq[c % KQ_STAGES];
        mbar_arrive_expect_tx(bar, (uint32_t)(DK / 64) * KROWS);
#pragma unroll 1
        for (int pn = 0; pn < DK / 64; ++pn) {
          tma_load_4d(at + pn * KROWS, &tmK, bar, 64 * pn, hk, t0 + C * c, tb);
          if (!FIRSTS) tma_load_4d(at + pn * KROWS + R64, &tmQ, bar, 64 * pn, hk, t0 + C * c, tb);
        }
        ++n_kq;
      };
      auto load_v = [&](int c) {
        if (transition) return;
        unsigned char* at = sm + OFF_V + (c % V_STAGES) * V_STAGE;
        uint64_t* bar = &ms.v[c % V_STAGES];
        mbar_arrive_expect_tx(bar, (uint32_t)(DV / 64) * R64);
#pragma unroll 1
        for (int pn = 0; pn < DV / 64; ++pn) tma_load_4d(at + pn * R64, &tmV, bar, 64 * pn, hv, t0 + C * c, tb);
        ++n_v;
      };
      auto load_rec = [&](int c) {
        uint64_t* bar = &ms.rec[c % REC_STAGES];
        mbar_arrive_expect_tx(bar, F::RECORD + (FIRSTS ? 0 : R64));
        bulk_load_1d(sm + OFF_REC + (c % REC_STAGES) * REC_STAGE,
                     p.records + (size_t)((slot + c) * p.Hv + hv) * GDR_RECORD, F::RECORD, bar);
        if (!FIRSTS) tma_load_4d(sm + OFF_P2 + (c % REC_STAGES) * R64, &tmP, bar, 0, hv, t0 + C * c, tb);
        ++n_rec;
      };
      // S^T (hi, then lo) times the rows of K (kq) or Q (kq + R64)
      auto issue_state = [&](uint32_t d, uint32_t kq) {
#pragma unroll 1
        for (int half = 0; half < 2; ++half)
          steps_ts(tmem + d, tmem + TM_S + 8 * half, kdesc(kq), KSTEP, KROWS >> 4, DK / 16, ID_64, half);
      };
      // The products execute in the order of their issue.  The state handed on for chunk c
      // means that all products of chunk c - 1 but P U are done, so its K, Q stage is free;
      // its record is when the outputs' warps have read its P U.
      auto run = [&]() -> bool {
#pragma unroll 1
        for (int c = -3; c < nch; ++c) {  // (-3 to -1: the first chunks' loads)
          const uint32_t kq = sbase + OFF_KQ + (c % KQ_STAGES) * KQ_STAGE;
          const uint32_t rec = sbase + OFF_REC + (c % REC_STAGES) * REC_STAGE;
          const bool chain = c >= 0;
          if (chain && (!wait(&ms.sready, c) || !wait(&ms.kq[c % KQ_STAGES], c / KQ_STAGES))) return false;
          tc_fence_after();
          if (chain) {
            STAMP(c, 0);
            issue_state(TM_R, kq);
            umma_commit(&ms.ks);
            STAMP(c, 1);
          }
          if (c >= 1 - KQ_STAGES && c + KQ_STAGES - 1 < nch) load_kq(c + KQ_STAGES - 1);  // into chunk c - 1's stage
          if (chain) {
            if (!wait(&ms.rec[c % REC_STAGES], c / REC_STAGES)) return false;
            if (!transition) {  // U^T = V^T T^T, while R is formed (the lanes past d_v read on: never used)
              if (!wait(&ms.v[c % V_STAGES], c / V_STAGES)) return false;
              tc_fence_after();
              const uint64_t v = ndesc(sbase + OFF_V + (c % V_STAGES) * V_STAGE, R64);
#pragma unroll 1
              for (int i = 0; i < 2; ++i) {
                const uint32_t t = rec + (i ? GDR_T_LO : GDR_T_HI);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                  umma_f16_ss(tmem + TM_U + 16 * ks, v + NSTEP * ks, tdesc(t, ks), idesc_bf16(128, 64 - 16 * ks, 1, 0),
                              i + ks > 0);
              }
            }
            if (!wait(&ms.rready, c)) return false;
            STAMP(c, 3);
            tc_fence_after();
#pragma unroll 1
            for (int i = 0; i < 3; ++i)  // U^T += R^T T^T: hi hi + hi lo + lo hi
              steps_tri(tmem + TM_U, tmem + TM_R + (i == 2 ? 8 : 0), rec + (i == 1 ? GDR_T_LO : GDR_T_HI),
                        !transition || i > 0);
            umma_commit(&ms.u);
            STAMP(c, 6);
            if (!FIRSTS && c > 0 && !wait(&ms.oread, c - 1)) return false;
          }
          // into chunk c - 1's stage: read by its products, the state's warps and the outputs'
          if (chain ? c >= 1 && c + 2 < nch : c + 3 < nch) load_rec(chain ? c + 2 : c + 3);
          if (c == -2 || c == -1) {
            if (c + 2 < nch) load_v(c + 2);
          }
          if (!chain) continue;
          if (!FIRSTS) {  // Q S, off the state's way: while U is read
            tc_fence_after();
            issue_state(TM_Q, kq + R64);
            STAMP(c, 2);
          }
          if (!wait(&ms.uready, c)) return false;
          STAMP(c, 4);
          tc_fence_after();
#pragma unroll 1
          for (int i = 0; i < 2; ++i) steps_ts(tmem + TM_S, tmem + TM_U + 8 * i, ndesc(kq, KROWS), NSTEP, 0, 4, ID_ST, i);
          umma_commit(&ms.s);
          STAMP(c, 7);
          if (c + 2 < nch) load_v(c + 2);  // (U is there: V of chunk c is read)
          if (!FIRSTS) {
            const uint32_t ub = tmem + (gates(c).mild ? TM_U : TM_UB);
#pragma unroll 1
            for (int i = 0; i < 2; ++i) steps_tri(tmem + TM_O, ub + 8 * i, rec + GDR_P, i);
            const uint32_t p2 = sbase + OFF_P2 + (c % REC_STAGES) * R64;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              umma_f16_ts(tmem + TM_O + 16 * ks, ub + 16 * ks, kdesc(p2 + 16 * ks * 128) + KSTEP * ks,
                          idesc_bf16(128, 64 - 16 * ks, 0, 0), 1);
            umma_commit(&ms.o);
            mbar_arrive(&ms.o);  // (hands on the record, which this thread has seen)
            STAMP(c, 5);
          }
        }
        return true;
      };
      const bool done = run();
      if (!done) give_up();
      // every product and copy issued lands before the block releases its memory
      umma_commit(&ms.drain);
      mbar_wait_short(&ms.drain, 0, WAIT_TRIES);
      if (!done) {
        for (int c = max(0, n_kq - KQ_STAGES); c < n_kq; ++c)
          mbar_wait_short(&ms.kq[c % KQ_STAGES], (uint32_t)((c / KQ_STAGES) & 1), WAIT_TRIES);
        for (int c = max(0, n_v - V_STAGES); c < n_v; ++c)
          mbar_wait_short(&ms.v[c % V_STAGES], (uint32_t)((c / V_STAGES) & 1), WAIT_TRIES);
        for (int c = max(0, n_rec - REC_STAGES); c < n_rec; ++c)
          mbar_wait_short(&ms.rec[c % REC_STAGES], (uint32_t)((c / REC_STAGES) & 1), WAIT_TRIES);
      }
    }
    __syncwarp();
  } else if (warp < NSTATE / 32) {
    setmaxnreg_inc<F::REG_STATE>();
    // ============================== the state ==============================================
    constexpr int DKQ = DK / F::NQ, STEPS = 4 / F::NQ;  // this warp's columns of S, and K steps of R and U
    const int cq = warp >> 2, ch = 32 * (warp & 3) + lane, t4 = lane & 3;
    const bool vval = ch < DV;  // (the same for a warp's 32 channels)
    const size_t sz = (size_t)DK * DV, units = gridDim.x / jobs, at_state = (size_t)(DKQ * cq) * DV + ch;
    const float* from = p.S0 ? p.S0 + unit * sz : nullptr;
    float* to = p.S_T ? p.S_T + unit * sz : nullptr;
    if (p.segs > 1) {
      if (FIRSTS) to = p.states + ((size_t)job * units + unit) * sz;
      else if (!last) to = nullptr;
      // (the second launch reads no S0: its last segments may write S_T over it)
      if (!FIRSTS) from = p.starts + ((size_t)seg * units + unit) * sz;
      else if (seg > 0) from = nullptr;
    }
    float S[DKQ];
#pragma unroll
    for (int i = 0; i < DKQ; ++i)
      S[i] = (from && vval) ? from[at_state + (size_t)i * DV] : (transition && DKQ * cq + i == ch) ? 1.f : 0.f;
    bool ok = true;
#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
      if (tid == 0) STAMP(c, 8);
#pragma unroll
      for (int b = 0; b < DKQ / 16; ++b) {
        uint32_t w[16];
        split16(S + 16 * b, w);
        tmem_st16u(tlane + TM_S + DKQ * cq + 16 * b, w);
      }
      if (p.cu && c == nch - 1 && tail < C) {  // K's and V's rows after the sequence's end: another's, or anything
        // (a transition has no V; its segment ends the sequence where the segments after it are empty)
        if (!(ok = wait(&ms.kq[c % KQ_STAGES], c / KQ_STAGES) && (transition || wait(&ms.v[c % V_STAGES], c / V_STAGES)))) break;
        for (int i = tid; i < (C - tail) * 8; i += NSTATE) {
          const uint32_t at = tail * 128 + i * 16;
#pragma unroll
          for (int pn = 0; pn < DK / 64; ++pn)
            *reinterpret_cast<uint4*>(sm + OFF_KQ + (c % KQ_STAGES) * KQ_STAGE + pn * KROWS + at) = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int pn = 0; pn < DV / 64; ++pn)
            *reinterpret_cast<uint4*>(sm + OFF_V + (c % V_STAGES) * V_STAGE + pn * R64 + at) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      tmem_st_wait();
      if (tid == 0) STAMP(c, 9);
      tc_fence_before();
      warp_arrive(&ms.sready);
      const GdrGates& gt = gates(c);
      if (!(ok = wait(&ms.rec[c % REC_STAGES], c / REC_STAGES))) break;
      if (tid == 0) STAMP(c, 11);
      const uint32_t at = tlane + 16 * STEPS * cq;  // this warp's K steps of R and U; their rows in halves of 16
      if (!(ok = wait(&ms.ks, c))) break;
      if (tid == 0) STAMP(c, 12);
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < STEPS; ++k) {  // R = -e^G (S^T K^T), in place
        float x[2][8];
        uint32_t w[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) tmem_ld_frag16(at + 16 * k + ((uint32_t)(16 * h) << 16) + TM_R, x[h]);
        float2 neg[2];  // of this lane's pair of tokens in the step's blocks of 8
#pragma unroll
        for (int j = 0; j < 2; ++j) neg[j] = *reinterpret_cast<const float2*>(&gt.neg[16 * (STEPS * cq + k) + 8 * j + 2 * t4]);
        tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // blocks i / 2, rows g and g + 8
            const float2 r = mul2(neg[i >> 1], make_float2(x[h][2 * i], x[h][2 * i + 1]));
            x[h][2 * i] = r.x, x[h][2 * i + 1] = r.y;
          }
          split_frag(x[h], w);
          tmem_st_frag16(at + 16 * k + ((uint32_t)(16 * h) << 16) + TM_R, w);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&ms.rready);
      if (tid == 0) STAMP(c, 13);
      if (!(ok = wait(&ms.u, c))) break;
      if (tid == 0) STAMP(c, 14);
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < STEPS; ++k) {  // U_end in place; where the product left U, that as well, for P U
        float x[2][8];
        uint32_t w[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) tmem_ld_frag16(at + 16 * k + ((uint32_t)(16 * h) << 16) + TM_U, x[h]);
        tmem_ld_wait();
        if (!gt.mild) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!FIRSTS) {
              split_frag(x[h], w);
              tmem_st_frag16(at + 16 * k + ((uint32_t)(16 * h) << 16) + TM_UB, w);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 f = *reinterpret_cast<const float2*>(&gt.end[16 * (STEPS * cq + k) + 8 * (i >> 1) + 2 * t4]);
              x[h][2 * i] *= f.x, x[h][2 * i + 1] *= f.y;
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          split_frag(x[h], w);
          tmem_st_frag16(at + 16 * k + ((uint32_t)(16 * h) << 16) + TM_U, w);
        }
      }
      const float total = gt.total;
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&ms.uready);
      if (tid == 0) STAMP(c, 15);
      if (!(ok = wait(&ms.s, c))) break;
      if (tid == 0) STAMP(c, 16);
      tc_fence_after();
      constexpr int AT_ONCE = DKQ < 32 ? DKQ : 32;  // columns (registers)
#pragma unroll
      for (int part = 0; part < DKQ; part += AT_ONCE) {
        float x[AT_ONCE / 16][16];
#pragma unroll
        for (int b = 0; b < AT_ONCE / 16; ++b) tmem_ld16(tlane + TM_S + DKQ * cq + part + 16 * b, x[b]);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < AT_ONCE; i += 2) {
          const float2 y = fma2(make_float2(total, total), make_float2(S[part + i], S[part + i + 1]),
                                make_float2(x[i / 16][i % 16], x[i / 16][i % 16 + 1]));
          S[part + i] = y.x, S[part + i + 1] = y.y;
        }
      }
    }
    if (!ok) give_up();
    if (ok && to && vval) {
#pragma unroll
      for (int i = 0; i < DKQ; ++i) to[at_state + (size_t)i * DV] = S[i];
    }
  } else if constexpr (!FIRSTS) {
    setmaxnreg_dec<F::REG_OUT>();
    // ============================== outputs ================================================
    const int ow = tid - NSTATE;           // thread of this group
    const uint32_t stage = sbase + OFF_O;  // rows of DV channels, 16-byte pieces swizzled by the row
    const int t4 = lane & 3;
    bool ok = true;
#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
      const GdrGates& gt = gates(c);
      ok = ok && wait(&ms.o, c);
      if (ow == 0) STAMP(c, 28);
      tc_fence_after();
      if (32 * (warp & 3) < DV) {
#pragma unroll 1
        for (int part = 0; part < 4; ++part) {  // 16 rows (h) by 32 tokens (from tok)
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
      warp_arrive(&ms.oread);  // (this chunk's record is read as well)
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
  if (warp == 0) tmem_dealloc(tmem, F::TM_COLS);
}

// The segments' first states: starts[0] = S0 (or zero), starts[1] = N_0, starts[s + 1] = M_s starts[s] + N_s,
// in fp32.  A block takes a unit's 16 value columns, a thread two rows, eight of the columns and half of
// the sum (pairs of operations; what M and S cost to read from shared memory is what bounds a step).  M
// comes a row to a thread by bulk copies into padded rows (16-byte reads of a column of rows without
// conflicts), the next segment's while this one's product runs.  3.1 us a segment at d = 128 (a row and the whole
// sum to a thread 4.2; three buffers instead of two 3.4).  (states without __restrict__: they may be written
// while this grid waits, so their loads stay behind the wait and on the coherent path.)
template <int D>
__global__ void __launch_bounds__(2 * D) gdr_join_kernel(const float* states, const float* __restrict__ S0,
                                                         float* __restrict__ starts, int segs, int units, unsigned* err) {
  constexpr int LD = D + 4, LS = 20;
  extern __shared__ __align__(16) float s_M[];  // [2][D][LD]
  __shared__ __align__(16) float s_S[D][LS], s_P[D][LS];
  __shared__ uint64_t full[2];
  const int unit = blockIdx.x / (D / 16), c0 = 16 * (blockIdx.x % (D / 16));
  const int tid = threadIdx.x, row = tid % (D / 2), ch = 8 * (tid / (D / 2) % 2), jh = tid / D;  // rows row, row + D / 2
  const size_t sz = (size_t)D * D;
  if (tid == 0) {
    mbar_init(&full[0], 1), mbar_init(&full[1], 1);
    fence_mbar_init();
  }
  __syncthreads();
  grid_release();
  grid_wait();
  auto fetch = [&](int s) {  // M of segment s >= 1
    if (tid == 0) mbar_arrive_expect_tx(&full[s & 1], D * D * 4);
    __syncthreads();
    if (tid < D)
      bulk_load_1d(s_M + ((s & 1) * D + tid) * LD, states + ((size_t)(segs - 1 + s - 1) * units + unit) * sz + (size_t)tid * D,
                   D * 4, &full[s & 1]);
  };
  auto at = [&](int r, int e) { return (size_t)(row + r * (D / 2)) * D + c0 + ch + 4 * e; };
  if (segs > 2) fetch(1);
  if (jh == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const size_t k = (size_t)unit * sz + at(i >> 1, i & 1);
      *reinterpret_cast<float4*>(starts + k) = S0 ? *reinterpret_cast<const float4*>(S0 + k) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  for (int s = 0; s < segs - 1; ++s) {
    float4 n[4] = {};  // N, of the threads with the sums' first half
    if (jh == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        n[i] = *reinterpret_cast<const float4*>(states + ((size_t)s * units + unit) * sz + at(i >> 1, i & 1));
    }
    if (s > 0) {
      if (s + 1 < segs - 1) fetch(s + 1);  // (all have left segment s - 1's M)
      if (!mbar_wait_short(&full[s & 1], (uint32_t)(((s - 1) >> 1) & 1), WAIT_TRIES)) {
        if (err) atomicOr(err, kErrWaitTimeout);
        mbar_wait_short(&full[s & 1], (uint32_t)(((s - 1) >> 1) & 1), WAIT_TRIES);
      }
      const float* m = s_M + ((s & 1) * D + row) * LD;
      float2 d[2][4] = {};
#pragma unroll 4
      for (int j = jh * (D / 2); j < (jh + 1) * (D / 2); j += 4) {
        const float4 a0 = *reinterpret_cast<const float4*>(m + j), a1 = *reinterpret_cast<const float4*>(m + D / 2 * LD + j);
        const float as[2][4] = {{a0.x, a0.y, a0.z, a0.w}, {a1.x, a1.y, a1.z, a1.w}};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 x = *reinterpret_cast<const float4*>(&s_S[j + i][ch]), y = *reinterpret_cast<const float4*>(&s_S[j + i][ch + 4]);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float2 t = make_float2(as[r][i], as[r][i]);
            d[r][0] = fma2(t, make_float2(x.x, x.y), d[r][0]), d[r][1] = fma2(t, make_float2(x.z, x.w), d[r][1]);
            d[r][2] = fma2(t, make_float2(y.x, y.y), d[r][2]), d[r][3] = fma2(t, make_float2(y.z, y.w), d[r][3]);
          }
        }
      }
      if (jh == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(&s_P[row + (i >> 1) * (D / 2)][ch + 4 * (i & 1)]) =
              make_float4(d[i >> 1][2 * (i & 1)].x, d[i >> 1][2 * (i & 1)].y, d[i >> 1][2 * (i & 1) + 1].x, d[i >> 1][2 * (i & 1) + 1].y);
      }
      __syncthreads();  // (and all have read S)
      if (jh == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 o = *reinterpret_cast<const float4*>(&s_P[row + (i >> 1) * (D / 2)][ch + 4 * (i & 1)]);
          const float2 u = d[i >> 1][2 * (i & 1)], v = d[i >> 1][2 * (i & 1) + 1];
          n[i].x += u.x + o.x, n[i].y += u.y + o.y, n[i].z += v.x + o.z, n[i].w += v.y + o.w;
        }
      }
    }
    if (jh == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        *reinterpret_cast<float4*>(&s_S[row + (i >> 1) * (D / 2)][ch + 4 * (i & 1)]) = n[i];
        *reinterpret_cast<float4*>(starts + ((size_t)(s + 1) * units + unit) * sz + at(i >> 1, i & 1)) = n[i];
      }
    }
    __syncthreads();
  }
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
// [B, T, H, D] bf16; one box = C tokens x 64 channels of one (sequence, head); ahead: what L2 fetches of a row at once
bool map_tokens(CUtensorMap* m, const void* base, int B, int T, int H, int D,
                CUtensorMapL2promotion ahead = CU_TENSOR_MAP_L2_PROMOTION_L2_256B) {
  auto fn = encoder();
  if (!fn) return false;
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T, (cuuint64_t)B};
  cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)H * D * 2, (cuuint64_t)T * H * D * 2};
  cuuint32_t box[4] = {64, 1, (cuuint32_t)C, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, ahead,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int DV, bool FIRSTS>
cudaError_t launch_chain(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mp,
                         const ChainParams& p, long long blocks, cudaStream_t st) {
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  static std::atomic<unsigned long long> done{0};
  constexpr uint32_t smem = smem_bytes<FIRSTS>();
  cudaError_t e = smem_limit_once(gdr_chain_kernel<DK, DV, FIRSTS>, (int)smem, done);
  if (e != cudaSuccess) return e;
  return launch_after(gdr_chain_kernel<DK, DV, FIRSTS>, (unsigned)blocks, Form<FIRSTS>::NT, smem, st, mq, mk, mv, mp, p);
}

// Segments of the sequences, of nch chunks each, for `units` (sequence, value head) pairs on 148 SMs: the
// count with the least time in chunks of the second launch (2.9 us each).  A chunk of the first launch is
// 0.9 of one with a block to an SM and 1.2 with two, a segment's step of the join 1.05, and the two launches
// more are 3.
// Measured with 1, 6, 12 and as many segments as this gives: B1 H16 T65536 2869, 1033, 1118 and 867 us (9),
// B1 H4 T16384 694, 254, 168 and 152 (20), B1 H16 T16384 725, 284, 330 and 266 (9), B2 H32 T8192 430, 485,
// 601 and 427 (2).  (P as a single bf16 then; its second part is 2 to 4 % more of each.)
int split_segments(long long units, long long nch) {
  auto first = [](long long blocks) {  // the first launch's chunks: turns of 296 blocks, the last one maybe of 148
    const long long rest = blocks % 296;
    return 1.2 * (double)(blocks / 296) + (rest > 148 ? 1.2 : rest > 0 ? 0.9 : 0.0);
  };
  auto second = [](long long blocks) { return (double)((blocks + 147) / 148); };
  double best = second(units) * (double)nch;
  int best_p = 1;
  for (int P = 2; P <= 64 && P * 4 <= nch; ++P) {
    const double len = (double)((nch + P - 1) / P);
    const double est = first(units * (2 * P - 3)) * len + second(units * P) * len + 1.05 * (P - 1) + 3.0;
    if (est < best) best = est, best_p = P;
  }
  return best_p;
}

struct Plan {
  int segs;
  long long slots;
  size_t records, states, starts;  // bytes of the workspace's parts
};
Plan plan(int B, int T, int Hv, int dk, int dv, bool packed) {
  Plan pl;
  const long long units = (long long)B * Hv;
  // (packed: a long sequence among short ones is not split; B1 H4 T65536 353 us alone, 2860 beside 23 of 64 tokens)
  const long long each = packed ? ((long long)T + B - 1) / (B > 0 ? B : 1) : T;  // (packed: the mean; lengths are on the device)
  pl.segs = dk != dv ? 1 : split_segments(units, (each + C - 1) / C);
  pl.slots = gdr_slots(B, T, packed);
  pl.records = (size_t)(pl.slots * Hv) * GDR_RECORD;
  const size_t state = (size_t)units * dk * dv * sizeof(float);
  pl.states = pl.segs > 1 ? (size_t)(2 * pl.segs - 3) * state : 0;
  pl.starts = pl.segs > 1 ? (size_t)pl.segs * state : 0;
  return pl;
}

template <int DK, int DV>
cudaError_t launch_dims(const GdrArgs& a, const Plan& pl, cudaStream_t st) {
  CUtensorMap mq, mk, mv, mp;  // (mp: the first 64 channels of o, where P's second parts are; nothing else of a row)
  const int B = a.cu_seqlens ? 1 : a.B;
  if (!map_tokens(&mq, a.q, B, a.T, a.Hk, DK) || !map_tokens(&mk, a.k, B, a.T, a.Hk, DK) ||
      !map_tokens(&mv, a.v, B, a.T, a.Hv, DV) || !map_tokens(&mp, a.o, B, a.T, a.Hv, DV, CU_TENSOR_MAP_L2_PROMOTION_NONE))
    return cudaErrorInvalidValue;
  unsigned char* ws = static_cast<unsigned char*>(a.workspace);
  cudaError_t e = launch_gdr_prep(a, mq, mk, ws, st);
  if (e != cudaSuccess) return e;
  ChainParams p{a.cu_seqlens, ws, a.S0, static_cast<__nv_bfloat16*>(a.o), a.S_T, a.T, a.Hv, a.Hk, 1, nullptr, nullptr,
                device_error_word(), stamp_buffer()};
  const long long units = (long long)a.B * a.Hv;
  if constexpr (DK == DV) {
    if (pl.segs > 1) {
      float* states = reinterpret_cast<float*>(ws + pl.records);
      float* starts = reinterpret_cast<float*>(ws + pl.records + pl.states);
      p.segs = pl.segs;
      p.states = states;
      e = launch_chain<DK, DV, true>(mq, mk, mv, mp, p, units * (2 * pl.segs - 3), st);
      if (e != cudaSuccess) return e;
      constexpr int JOIN_SMEM = 2 * DK * (DK + 4) * (int)sizeof(float);
      static std::atomic<unsigned long long> done{0};
      e = smem_limit_once(gdr_join_kernel<DK>, JOIN_SMEM, done);
      if (e != cudaSuccess) return e;
      e = launch_after(gdr_join_kernel<DK>, (unsigned)(units * (DK / 16)), 2 * DK, JOIN_SMEM, st, states, a.S0, starts, pl.segs,
                       (int)units, p.err);
      if (e != cudaSuccess) return e;
      p.starts = starts;
      return launch_chain<DK, DV, false>(mq, mk, mv, mp, p, units * pl.segs, st);
    }
  }
  return launch_chain<DK, DV, false>(mq, mk, mv, mp, p, units, st);
}

}  // namespace

size_t gdr_chunk_workspace_bytes(int B, int T, int Hv, int dk, int dv, bool packed) {
  const Plan pl = plan(B, T, Hv, dk, dv, packed);
  return pl.records + pl.states + pl.starts;
}

cudaError_t launch_gdr_chunk_tc(const GdrArgs& a, cudaStream_t st) {
  if (!a.bf16 || a.T == 0) return cudaErrorInvalidValue;
  const Plan pl = plan(a.B, a.T, a.Hv, a.dk, a.dv, a.cu_seqlens != nullptr);
  if (a.dk == 128) return a.dv == 128 ? launch_dims<128, 128>(a, pl, st) : launch_dims<128, 64>(a, pl, st);
  return a.dv == 128 ? launch_dims<64, 128>(a, pl, st) : launch_dims<64, 64>(a, pl, st);
}

}  // namespace gdn2
