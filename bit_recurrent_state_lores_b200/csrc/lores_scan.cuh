// lores_scan.cuh -- device side of the state scan and its backward pass (sm_100a).
//
// The scan runs the decode step's recurrence, without its quantizer, over packed sequences:
//   S'  = a_t S_{t-1},  E_t = v_t - d S' k_t,  S_t = S' + b_t E_t k_t^T,  o_t = S_t q_t
// (General recurrence form; a_t = exp(log_alpha_t), d = delta).  Sequences are cut into
// chunks of kChunk = 64 tokens.  With G_t the sum of log_alpha over the chunk up to t, S0 the
// state at its start, rows t of Q, K, V, E its tokens and dec_ts = exp(G_t - G_s):
//   A_ts = k_t.k_s b_s (s < t)         P_ts = dec_ts q_t.k_s b_s (s <= t)
//   T    = (I + d A)^-1                Tm_ts = dec_ts T_ts
//   E    = Tm V - d diag(e^G) T K S0^T
//   O    = diag(e^G) Q S0^T + P E      S_C = e^{G_C} S0 + (diag(w) E)^T K,  w = b e^{G_C - G}
// Only S0 -> S_C is sequential, so the work is split in two:
//   scan_prep     all chunks at once: gates, Tm, P, Kt = -d T K (and, for the backward pass,
//                 Z = P Tm and Kb = T^T diag(b) K).  (With Gam = diag(e^G), (I + L diag(b))^-1
//                 for L_ts = dec_ts k_t.k_s is Gam T Gam^-1: the decays leave the inverse,
//                 whose entries stay of size one, and come back as factors of its rows.)
//   scan_walk     per (sequence, head, block of value rows): E^T = S0 Kt^T diag(e^G) +
//                 (Tm V)^T, O^T and S_C, chunk after chunk.  Value rows are independent (as in the decode
//                 step), so one or two warps own 16 of them, keep S [16][d_k] in their
//                 accumulators and feed it back as the next product's left operand
//                 without leaving registers; two more warps per 16 rows do what the
//                 next chunk does not wait for.
// Backward, D = dL/dS_C:
//   R   = Z^T dO + diag(e^{G_C - G}) Kb D^T (= dV)
//   D0  = e^{G_C} D + (diag(e^G) dO)^T Q - d (diag(e^G) R)^T K
//   scan_walk     the same backwards over R and D;
//   scan_grads    all chunks at once: dQ, dK and the gates' gradients from S0, D, E, R.
//
// Tensor cores.  The products are mma.sync m16n8k16: a walk's blocks have 16 rows, because 32 heads
// of 128 value rows must spread over 148 SMs, and the state has to be an accumulator and the next
// product's left operand within a few hundred cycles; tcgen05 wants 64 rows at least and keeps
// accumulators in TMEM, so that every chunk would pay two trips through it on the critical path.
// Nothing here is bound by the rate of the products: mma.sync measured 555 TFLOP/s on this card, and
// the walk keeps the tensor cores busy for 2300 of a chunk's 5140 cycles.
// (Comparisons below between variants of a walk were measured when 16-bit outputs had one plane of S0, P and E: 286 us
// then for one sequence of 8192 tokens and 32 heads of 128 x 128, 335 with two.)
//
// Precision.  Sums and states are fp32; the tensor cores multiply fp16.  An fp32 operand x is given
// as two fp16 planes, hi = fp16(x) and lo = fp16(x - hi): 22 bits of significand, or an absolute
// 2^-25 where lo is subnormal.  A product is hi hi + hi lo + lo hi.  fp16's range is met by powers of two that leave the
// result exactly: K and Q are divided by one scale per chunk and head and so are the betas in Z, Kb, dP' and
// dL', P by one per row, the walks' operands by one per 16 value rows and chunk, so that the largest entries are near
// fp16's end (kUp below).  16-bit inputs are exact as one plane down to 2^-31 of that largest entry (bf16; keys 2^-25),
// fp32 ones keep 22 bits down to 2^-16 of it (keys 2^-10) and are off by at most 2^-39 of it (keys 2^-33) below.
// States, gradients and outputs before their rounding are 3e-7 to 8e-7 from exact (fp32 sums leave 1e-7 to 3e-7); two
// bf16 planes left 3e-6 to 1e-5, one fp16 plane 2e-4.  One plane of S0, P and E where they only reach a 16-bit o is not
// enough either: entries of o came out 1e-3 from the rounded exact value in bf16 (1.68e-3 from exact, where the rounding
// leaves 1.66e-3), and 1.6 times as far as the rounding in fp16.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "lores_device.cuh"

namespace lores {
namespace scan {

constexpr int kChunk = 64;
// Largest entries of the planes: 2^kUp .. 2^(kUp + 1) of S, D, V, dO, E and R and of Q, as large as fp16 allows, so that
// smaller entries beside them keep their digits; less for K, whose planes' products with T (Kt, Kb: up to sqrt(d_k)
// times as large) are planes too.  Products of K and Q come back into range by 2^kDownZ (d_k 2^15 2^9 2 = 2^32).
constexpr int kUp = 14, kUpK = 8, kDownZ = -17;
constexpr int kPrepThreads = 128;
constexpr unsigned kFlagOffsets = 1u;  // a sequence's offsets were not 0 <= a <= b <= total
constexpr unsigned kFlagWait = 2u;     // a wait for a kernel's own copies ran out

enum ScaleOf { kScaleS, kScaleE, kScaleD, kScaleR, kScaleO, kScales };

struct ScanParams {
  int n_seq, H, share, d_v, dvp, dtype, n_slots, max_len, stages;
  int rb;                              // walks: blocks of 16 value rows per CTA
  int early;                           // walks: may start beside the kernel before
  int hpc;                             // scan_prep: heads per CTA (a divisor of share)
  int qk16, v16, o16;                  // 16-byte accesses to q and k, v (and dv), o (or d_o) rows
  long long total;
  const int *offsets;
  const void *q, *k, *v;               // the caller's tensors
  long long q_stride, k_stride, v_stride, o_stride;
  const float *log_alpha, *beta;       // [total][H]
  const float *state_in;               // [n_seq][H][d_v][d_k] or null
  float *state_out;                    // likewise or null
  void *o;                             // forward: o; backward: d_o (read)
  unsigned *flag;
  // workspace
  longlong2 *seqs;                     // [n_seq] first token, tokens (written by scan_prep or scan_sequences)
  longlong2 *slot_tokens;              // [n_slots] first token, tokens (written by scan_prep for the backward pass)
  // records of one (slot, head); khat, qhat of one (slot, q/k head)
  float *gates;                        // kGateFloats
  __half *khat, *qhat;                 // [NP][64][d_k], divided by their scales
  __half *kt, *kb;                     // [2][64][d_k]
  __half *tm, *pp, *z;                 // [2], ten blocks of [16][16] (see tri)
  __half *s0, *dd;                     // [2][dvp][d_k]
  __half *et, *rt;                     // [2][dvp][64]
  float *scales[kScales];              // of s0, et, dd, rt and of d_o: [dvp/16]
  // backward
  const float *d_state_out;
  float *d_state_in;
  void *dv, *dq, *dk;                  // dq, dk: the caller's, or fp32 parts [total][H][d_k]
  int parts;                           // dq, dk are parts
  float *dlog_alpha, *dbeta;
};

// Record of a chunk and head, kChunk entries each: e^(G_C - G); e^G; w times 2^kUpK of the scale of K (that is, what
// multiplies 2^-kUpK of a row of khat); e^G likewise; what multiplies a row of P's planes (forward); w; b; G / ln 2 as a
// pair of floats.  Then
// the scales of K, Q and b.
enum GateRow { kGateC, kGateE, kGateWk, kGateEk, kGateP, kGateW, kGateB, kGateG };   // kGateG: two rows' worth of pairs
constexpr int kGateScales = (kGateG + 2) * kChunk;
constexpr int kGateFloats = kGateScales + 8;
constexpr int kGateStage = 4 * kChunk + 8;     // what a walk takes of it: four rows, the scales

// -------------------------------------------------------------------------------------
// sequences and chunk slots
// -------------------------------------------------------------------------------------
// Tokens [start, start + len) of sequence i; a sequence whose offsets do not fit is empty.
__device__ __forceinline__ bool seq_range(const ScanParams &p, int i, long long &start, int &len) {
  if (!p.offsets) {
    len = (int)(p.total / p.n_seq);
    start = (long long)i * len;
    return true;
  }
  const long long a = __ldg(p.offsets + i), b = __ldg(p.offsets + i + 1);
  if (a < 0 || b < a || b > p.total || b - a > p.max_len) {
    start = 0;
    len = 0;
    return false;
  }
  start = a;
  len = (int)(b - a);
  return true;
}
// Sequence i's chunks take slots floor(start / 64) + i onwards: since floor(b/64) -
// floor(a/64) + 1 >= ceil((b - a)/64), no two sequences share a slot, and no prefix sum over
// the sequences is needed.
__device__ __forceinline__ int slot_base(long long start, int i) { return (int)(start / kChunk) + i; }

// Where some offsets do not fit, the sequences that do need not lie in order.  One that starts before the end of an
// earlier one that fits is taken as empty, since its slots could be another's.
//
// Up to kFewSeqs sequences every block of scan_prep looks them all over for its slot (a bisection would trust offsets that
// do not fit); more are put in order first, by scan_sequences, and scan_prep bisects what that leaves.  (16384 sequences of
// 64 tokens, 2 heads of 32 x 32: looked over by every block 4345 us; 2048 of them, 4 heads: 476.)
constexpr int kFewSeqs = 256, kSeqThreads = 1024;

// Whether sequence i starts behind the ends of all earlier ones that fit.  All threads of a block.
__device__ __forceinline__ bool in_order(const ScanParams &p, int i, long long start) {
  int over = 0;
  for (int j = threadIdx.x; j < i; j += blockDim.x) {
    long long s;
    int n;
    if (seq_range(p, j, s, n)) over |= s + n > start;
  }
  return !__syncthreads_or(over);
}

// The first token of a slot's chunk and its number of tokens (0: the slot is not used).  All threads of a block.
// `bad`: some offsets do not fit (few sequences only).  part: one word per warp.
__device__ __forceinline__ int slot_tokens(const ScanParams &p, int slot, long long &token0, bool &bad, unsigned *part) {
  bad = false;
  if (!p.offsets || p.n_seq > kFewSeqs) {
    const long long each = p.total / p.n_seq;
    int lo = 0, hi = p.n_seq - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (slot_base(p.offsets ? __ldg(&p.seqs[mid].x) : each * mid, mid) <= slot) lo = mid; else hi = mid - 1;
    }
    const long long start = p.offsets ? __ldg(&p.seqs[lo].x) : each * lo, len = p.offsets ? __ldg(&p.seqs[lo].y) : each;
    const long long first = (long long)(slot - slot_base(start, lo)) * kChunk;
    if (first < 0 || first >= len) return 0;
    token0 = start + first;
    return (int)min((long long)kChunk, len - first);
  }
  constexpr unsigned NONE = 0xFFFFFFFFu;
  for (int lo = 0;;) {
    unsigned mine = NONE;
    int wrong = 0;
    for (int i = lo + (int)threadIdx.x; i < p.n_seq; i += blockDim.x) {
      long long s;
      int n;
      wrong |= !seq_range(p, i, s, n);
      const long long first = (long long)(slot - slot_base(s, i)) * kChunk;
      if (first >= 0 && first < n) mine = min(mine, (unsigned)i);
    }
    mine = __reduce_min_sync(0xFFFFFFFFu, mine);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = mine;
    bad |= __syncthreads_or(wrong) != 0;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) mine = min(mine, part[w]);
    if (mine == NONE) return 0;
    long long start;
    int len;
    seq_range(p, (int)mine, start, len);
    if (bad && !in_order(p, (int)mine, start)) {
      lo = (int)mine + 1;
      continue;
    }
    const long long first = (long long)(slot - slot_base(start, (int)mine)) * kChunk;
    token0 = start + first;
    return (int)min((long long)kChunk, len - first);
  }
}

// One block of scan_prep leaves few sequences as they are taken and the verdict in the workspace.
__device__ __forceinline__ void keep_sequences(const ScanParams &p, bool bad) {
  if (bad) {
    for (int i = 0; i < p.n_seq; ++i) {
      long long s;
      int n;
      seq_range(p, i, s, n);
      if (!in_order(p, i, s)) n = 0;
      if (threadIdx.x == 0) p.seqs[i] = make_longlong2(s, n);
    }
  } else {
    for (int i = threadIdx.x; i < p.n_seq; i += blockDim.x) {
      long long s;
      int n;
      seq_range(p, i, s, n);
      p.seqs[i] = make_longlong2(s, n);
    }
  }
  if (threadIdx.x == 0) *p.flag = bad ? kFlagOffsets : 0u;
}

// The same for many, by one block before scan_prep: a running maximum of the ends.  An empty sequence that does not fit
// starts there, so that the slots of all begin in order.
static __global__ void __launch_bounds__(kSeqThreads) scan_sequences_kernel(const ScanParams p) {
  __shared__ long long tops[kSeqThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long before = 0;                  // the largest end of the sequences of the rounds before
  int bad = 0;
  for (int i0 = 0; i0 < p.n_seq; i0 += kSeqThreads) {
    const int i = i0 + tid;
    long long start = 0;
    int len = 0;
    const bool fits = i < p.n_seq && seq_range(p, i, start, len);
    bad |= i < p.n_seq && !fits;
    long long top = fits ? start + len : 0;      // of this warp's sequences up to this one
    for (int d = 1; d < 32; d <<= 1) {
      const long long up = __shfl_up_sync(0xFFFFFFFFu, top, d);
      if (lane >= d) top = max(top, up);
    }
    if (lane == 31) tops[warp] = top;
    long long behind = __shfl_up_sync(0xFFFFFFFFu, top, 1);
    if (lane == 0) behind = 0;
    __syncthreads();
    long long all = before;
    for (int w = 0; w < kSeqThreads / 32; ++w) {
      if (w == warp) behind = max(behind, all);
      all = max(all, tops[w]);
    }
    __syncthreads();
    before = all;
    if (i < p.n_seq) p.seqs[i] = fits && start >= behind ? make_longlong2(start, len) : make_longlong2(behind, 0);
  }
  bad = __syncthreads_or(bad);
  if (tid == 0) *p.flag = bad ? kFlagOffsets : 0u;
}

// One block of a launch looks every sequence over and leaves the verdict in the workspace.
__device__ __forceinline__ void check_offsets(const ScanParams &p) {
  int bad = 0;
  for (int i = threadIdx.x; i < p.n_seq; i += blockDim.x) {
    long long s;
    int n;
    bad |= !seq_range(p, i, s, n);
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *p.flag = bad ? kFlagOffsets : 0u;
}

// -------------------------------------------------------------------------------------
// launches that overlap
// -------------------------------------------------------------------------------------
// A call's kernels are launched so that each may start once every CTA of the one before it has
// started and called launch_next(); what reads the other's results calls wait_before() first, which
// returns when the kernels before this one are complete and their writes visible.  The first kernel
// is launched the ordinary way, and every kernel waits before it ends, so that a call is
// ordered as a whole.
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// -------------------------------------------------------------------------------------
// fragments
// -------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_addr(const void *x) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(x));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t row) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(row));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t row) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(row));
}
__device__ __forceinline__ void stsm4t(uint32_t row, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(row), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
// Fragment loads of 16x16 blocks of a tiled matrix with COLS columns.
//   right operand, two column tiles (r[0], r[1]: columns n0..n0+7; r[2], r[3]: n0+8..):
//     b_rows:  stored [n][k]      b_cols: stored [k][n]
//   left operand:
//     a_rows:  stored [m][k]      a_cols: stored [k][m]
// ldmatrix's four tiles are (0, 0), (0, 1), (1, 0), (1, 1) of the block in the order of the registers, or with the
// middle two exchanged; `Lane` holds a lane's part of the address for both orders.
template <int COLS>
struct Lane {
  uint32_t down, across;
  __device__ __forceinline__ explicit Lane(int lane) {
    const int i = lane >> 3, r = (lane & 7) * 16;
    down = ((i >> 1) * (COLS / 8) + (i & 1)) * 128 + r;
    across = ((i & 1) * (COLS / 8) + (i >> 1)) * 128 + r;
  }
  __device__ __forceinline__ static uint32_t at(int row, int col) {
    return ((row >> 3) * (COLS / 8) + (col >> 3)) * 128;
  }
  __device__ __forceinline__ void b_rows(uint32_t (&r)[4], uint32_t x, int n0, int k0) const {
    ldsm4(r, x + down + at(n0, k0));
  }
  __device__ __forceinline__ void b_cols(uint32_t (&r)[4], uint32_t x, int k0, int n0) const {
    ldsm4t(r, x + across + at(k0, n0));
  }
  __device__ __forceinline__ void a_rows(uint32_t (&r)[4], uint32_t x, int m0, int k0) const {
    ldsm4(r, x + across + at(m0, k0));
  }
  __device__ __forceinline__ void a_cols(uint32_t (&r)[4], uint32_t x, int k0, int m0) const {
    ldsm4t(r, x + down + at(k0, m0));
  }
};
// The caller's token rows, in plain rows of ld elements.
__device__ __forceinline__ void a_rows_plain(uint32_t (&r)[4], uint32_t x, int ld, int m0, int k0, int lane) {
  ldsm4(r, x + 2 * ((m0 + (((lane >> 3) & 1) << 3) + (lane & 7)) * ld + k0 + ((lane >> 4) << 3)));
}
// Element (row, col) of a tiled matrix.
template <int COLS>
__device__ __forceinline__ int tiled(int row, int col) {
  return ((row >> 3) * (COLS / 8) + (col >> 3)) * 64 + (row & 7) * 8 + (col & 7);
}

// Tm, P and Z are zero above the diagonal: their planes hold the ten 16x16 blocks (i, k), k <= i, one behind the other,
// each as a tiled matrix of 16 columns.  The first entry of a block:
constexpr int kTri = 10 * 256;
__host__ __device__ constexpr int tri(int i, int k) { return (i * (i + 1) / 2 + k) * 256; }

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two column tiles at once (b as the loads above leave it).
__device__ __forceinline__ void mma2(float (&c0)[4], float (&c1)[4], const uint32_t (&a)[4],
                                     const uint32_t (&b)[4]) {
  mma(c0, a, b[0], b[1]);
  mma(c1, a, b[2], b[3]);
}

// x, y -> packed fp16 (x low).
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}
// ... and the packed rest: hi - x in one mixed-precision subtraction, rounded with its sign turned.
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
  hi = pack2(x, y);
  float rx, ry;
  asm("{\n\t.reg .f16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "sub.rn.f32.f16 %0, l, %3;\n\t"
      "sub.rn.f32.f16 %1, h, %4;\n\t}"
      : "=f"(rx), "=f"(ry)
      : "r"(hi), "f"(x), "f"(y));
  lo = pack2(-rx, -ry);
}
__device__ __forceinline__ float2 half2_of(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ float2 bf162_of(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// A packed pair of the caller's 16-bit type.
__device__ __forceinline__ float2 pair_of(uint32_t w, int dtype) {
  return dtype == 1 ? bf162_of(w) : half2_of(w);
}
// Accumulator tiles 2j, 2j+1 (16 columns) as a left operand's planes: the layouts agree.
__device__ __forceinline__ void split_tiles(const float (&c0)[4], const float (&c1)[4], uint32_t (&hi)[4],
                                            uint32_t (&lo)[4]) {
  split2(c0[0], c0[1], hi[0], lo[0]);
  split2(c0[2], c0[3], hi[1], lo[1]);
  split2(c1[0], c1[1], hi[2], lo[2]);
  split2(c1[2], c1[3], hi[3], lo[3]);
}
__device__ __forceinline__ void split_tiles(const float (&c0)[4], const float (&c1)[4], float by,
                                            uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  split2(c0[0] * by, c0[1] * by, hi[0], lo[0]);
  split2(c0[2] * by, c0[3] * by, hi[1], lo[1]);
  split2(c1[0] * by, c1[1] * by, hi[2], lo[2]);
  split2(c1[2] * by, c1[3] * by, hi[3], lo[3]);
}

// Scales: the power of two c with m / c in [2^up, 2^(up+1)) for the magnitude m with the given
// bits (limits at the ends of the range), and its inverse.  For zero: 1, or with LEAST the smallest, so that a
// part that holds zeros alone does not count where parts are brought to their largest unit.
template <bool LEAST = false>
__device__ __forceinline__ float scale_of(unsigned bits, int up, float &inv) {
  int e = max(1, min(253, (int)(bits >> 23) - up));
  if (!LEAST && bits == 0u) e = 127;
  inv = __uint_as_float((unsigned)(254 - e) << 23);
  return __uint_as_float((unsigned)e << 23);
}
__device__ __forceinline__ float pow2(int e) {
  return e < -126 ? 0.0f : __uint_as_float((unsigned)(127 + min(e, 127)) << 23);
}
// dec_ts = 2^(g_t - g_s), g a pair of floats (48 bits, so that the difference keeps its digits behind a
// strong decay).
__device__ __forceinline__ float decay(float2 gt, float2 gs) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(__fsub_rn(gt.x, gs.x), __fsub_rn(gt.y, gs.y))));
  return r;
}
// |x|, and NaN where x is not finite (fmaxf then passes it over).
__device__ __forceinline__ float finite_abs(float x) { return fabsf(__fmaf_rn(x, 0.0f, x)); }
constexpr unsigned kInf = 0x7F800000u;
__device__ __forceinline__ unsigned abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// -------------------------------------------------------------------------------------
// copies
// -------------------------------------------------------------------------------------
__device__ __forceinline__ void cp16(void *dst, const void *src, bool there) {
  const int n = there ? 16 : 0;        // 0: sixteen zero bytes
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp8(void *dst, const void *src, bool there) {
  const int n = there ? 8 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp4(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// `cols` columns (a multiple of 16) of 64 token rows of the caller's tensor: rows >= n and
// columns >= have (a multiple of 4) are zeros.  ld in elements.
template <int SIZE>
__device__ __forceinline__ void copy_tokens(uint8_t *dst, int ld, const uint8_t *src, long long stride, int cols,
                                            int n, int have, bool by16, int tid, int threads) {
  const int step = by16 ? 16 / SIZE : 8 / SIZE, per = cols / step;
  for (int i = tid; i < kChunk * per; i += threads) {
    const int r = i / per, c = (i % per) * step;
    const bool in = r < n && c < have;
    const uint8_t *s = in ? src + (r * stride + c) * SIZE : src;
    if (by16) cp16(dst + (r * ld + c) * SIZE, s, in);
    else cp8(dst + (r * ld + c) * SIZE, s, in);
  }
}

// Two values of a 16-bit type, x low.
__device__ __forceinline__ uint32_t pack_as(int dtype, float x, float y) {
  if (dtype != 1) return pack2(x, y);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}
__device__ __forceinline__ void store_pair(void *base, int dtype, long long i, float x, float y) {
  if (dtype == 0) *reinterpret_cast<float2 *>(static_cast<float *>(base) + i) = make_float2(x, y);
  else *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(base) + i) = pack_as(dtype, x, y);
}
__device__ __forceinline__ void load4(const void *src, int dtype, long long i, float (&x)[4]) {
  if (dtype == 0) {
    const float4 f = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(src) + i));
    x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
    return;
  }
  const uint2 w = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(src) + i));
  const float2 a = pair_of(w.x, dtype), b = pair_of(w.y, dtype);
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}
// -------------------------------------------------------------------------------------
// scan_prep
// -------------------------------------------------------------------------------------
// Grid (slot, group of p.hpc heads that share K and Q), 4 warps; warp w owns rows 16w .. 16w+15 of every [64][.]
// result, and only blocks on and below the diagonal are formed.  K and Q are fetched and converted
// once for the group.  Bound by latency: a chain of short products with four CTAs per SM to hide it.
// 8192 tokens, 32 heads, d_k = 128, bf16 (4096 items, 362 MB of matrices written): 154 us, 2.4 TB/s;
// without the delta rule and with 16 heads on one pair of Q and K (7897 tokens, 128 heads): 96 us (76 with one plane of
// P, when a CTA per head took 343).  T = (I + A)^-1 by 16x16 blocks:
// the four diagonal blocks by forward substitution in fp32 (one lane per column); then warp j
// forms block column j downwards, X_ij = -X_ii sum_{j <= k < i} A_ik X_kj, as
// X_ij^T = -(sum_k X_kj^T A_ik^T) X_ii^T, so that every X_kj^T is an accumulator that becomes the next
// product's left operand in place.
constexpr int kLdF = kChunk + 2;       // row stride of the fp32 matrix in shared memory

struct PrepLayout {
  int k, q, a, x, xd, f, bytes;
};
// `several`: heads per CTA.  For one, the planes of A take Q's place once Q is used.
__host__ __device__ constexpr PrepLayout prep_layout(int dk, int np, bool several) {
  PrepLayout l{};
  const int tile = np * kChunk * dk * 2, planes = 2 * kChunk * kChunk * 2;
  l.k = 0;
  l.q = tile;
  l.a = several ? l.q + tile : l.q;
  l.x = several ? l.a + planes : l.q + (tile > planes ? tile : planes);
  l.xd = l.x + kChunk * kLdF * 4;
  l.f = l.xd + 4 * 2 * 16 * 16 * 2;
  l.bytes = l.f + 2 * (kChunk + 2 * kChunk) * 4 + 16 * 4;
  return l;
}

// Rows of K or Q of a chunk.  A thread holds PASS pieces of 8 entries as they came, piece e being row e % 8 of tile
// e / 8 (so that the planes are written in order); all loads are in flight before the first is used.
template <int DK, int NP, int PASS>
__device__ __forceinline__ void load_rows(const ScanParams &p, const void *src, long long stride, long long token0, int qh,
                                          int n, uint4 (&raw)[PASS][NP], int tid) {
  constexpr int PER = DK / 8;
#pragma unroll
  for (int i = 0; i < PASS; ++i) {
    const int e = tid + i * kPrepThreads, r = (e >> 3) / PER * 8 + (e & 7), c = (e >> 3) % PER * 8;
#pragma unroll
    for (int h = 0; h < NP; ++h) raw[i][h] = make_uint4(0, 0, 0, 0);
    if (r < n) {
      const long long at = (token0 + r) * stride + (long long)qh * DK + c;
      if (NP == 2) {
        const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const float *>(src) + at);
#pragma unroll
        for (int h = 0; h < NP; ++h) raw[i][h] = __ldg(s + h);
      } else if (p.qk16) {
        raw[i][0] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(src) + at));
      } else {
        const uint2 *s = reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(src) + at);
        const uint2 a = __ldg(s), b = __ldg(s + 1);
        raw[i][0] = make_uint4(a.x, a.y, b.x, b.y);
      }
    }
  }
}
template <int NP>
__device__ __forceinline__ void unpack_row(const uint4 (&raw)[NP], int dtype, float (&x)[8]) {
  const uint32_t u[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w,
                         raw[NP - 1].x, raw[NP - 1].y, raw[NP - 1].z, raw[NP - 1].w};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (NP == 2) {
      x[e] = __uint_as_float(u[e]);
    } else if (!(e & 1)) {
      const float2 f = pair_of(u[e >> 1], dtype);
      x[e] = f.x;
      x[e + 1] = f.y;
    }
  }
}
// Bits (of fp32) of the warp's largest finite magnitude; 16-bit types are compared as integers, two at a time.  (What is
// not finite says nothing about a scale: under the scale of an infinity everything else would vanish.)
template <int NP, int PASS>
__device__ __forceinline__ unsigned max_rows(const uint4 (&raw)[PASS][NP], int dtype) {
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < PASS; ++i)
#pragma unroll
    for (int h = 0; h < NP; ++h) {
      const uint32_t u[4] = {raw[i][h].x, raw[i][h].y, raw[i][h].z, raw[i][h].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) m = NP == 2 ? max(m, u[e] & 0x7FFFFFFFu) : __vmaxu2(m, u[e] & 0x7FFF7FFFu);
    }
  if (NP == 1) {
    const uint32_t w = max(m & 0xFFFFu, m >> 16);
    m = dtype == 1 ? w << 16 : __float_as_uint(__half2float(__ushort_as_half((unsigned short)w)));
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if (m >= kInf) {
    float f = 0.0f;
#pragma unroll
    for (int i = 0; i < PASS; ++i) {
      float x[8];
      unpack_row<NP>(raw[i], dtype, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) f = fmaxf(f, finite_abs(x[e]));
    }
    m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(f));
  }
  return m;
}
// The rows over their scale as planes, in shared memory and, where `out` is given, in the workspace.
template <int DK, int NP, int PASS>
__device__ __forceinline__ void put_rows(const uint4 (&raw)[PASS][NP], int dtype, float inv, __half *dst, __half *out, int tid) {
#pragma unroll
  for (int i = 0; i < PASS; ++i) {
    const int e = tid + i * kPrepThreads, at = e * 8;
    if (at >= kChunk * DK) continue;
    float x[8];
    unpack_row<NP>(raw[i], dtype, x);
    uint4 hi, lo;
    split2(x[0] * inv, x[1] * inv, hi.x, lo.x);
    split2(x[2] * inv, x[3] * inv, hi.y, lo.y);
    split2(x[4] * inv, x[5] * inv, hi.z, lo.z);
    split2(x[6] * inv, x[7] * inv, hi.w, lo.w);
    *reinterpret_cast<uint4 *>(dst + at) = hi;
    if (NP == 2) *reinterpret_cast<uint4 *>(dst + kChunk * DK + at) = lo;
    if (out) {
      *reinterpret_cast<uint4 *>(out + at) = hi;
      if (NP == 2) *reinterpret_cast<uint4 *>(out + kChunk * DK + at) = lo;
    }
  }
}

// Two neighbouring entries into a plane and their rest into the plane behind it.
__device__ __forceinline__ void put_at(__half *dst, long long plane, int at, float x, float y) {
  uint32_t hi, lo;
  split2(x, y, hi, lo);
  *reinterpret_cast<uint32_t *>(dst + at) = hi;
  *reinterpret_cast<uint32_t *>(dst + plane + at) = lo;
}
// One accumulator register pair (rows r0 + lane/4, columns c0 + 2 (lane % 4), +1 of an 8x8 tile) into tiled planes.
template <int COLS>
__device__ __forceinline__ void put_pair(__half *dst, long long plane, int r0, int c0, float x, float y, int lane) {
  put_at(dst, plane, tiled<COLS>(r0, c0) + 2 * lane, x, y);
}

template <int DK, int NP, bool DELTA, bool BWD>
__global__ void __launch_bounds__(kPrepThreads, NP == 1 ? 4 : 2) scan_prep_kernel(const ScanParams p) {
  constexpr int PASS = (kChunk * DK / 8 + kPrepThreads - 1) / kPrepThreads;
  const bool several = p.hpc > 1;
  const PrepLayout l = prep_layout(DK, NP, several);
  extern __shared__ __align__(16) uint8_t smem[];
  __half *K = reinterpret_cast<__half *>(smem + l.k), *Q = reinterpret_cast<__half *>(smem + l.q);
  __half *A16 = reinterpret_cast<__half *>(smem + l.a);             // [2][64][64]
  float *X = reinterpret_cast<float *>(smem + l.x);                 // diagonal blocks of A, then T
  __half *XD = reinterpret_cast<__half *>(smem + l.xd);             // [4][2][16][16]: X_ii
  // of this head and of the next: G / ln 2, b over its scale (which is in red[8], red[9])
  auto gate_at = [&](int which) { return reinterpret_cast<float2 *>(smem + l.f + which * (3 * kChunk * 4)); };
  unsigned *red = reinterpret_cast<unsigned *>(smem + l.f + 2 * (3 * kChunk * 4));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t2 = (lane & 3) * 2;
  const int slot = blockIdx.x, head0 = blockIdx.y * p.hpc;
  launch_next();
  long long token0 = 0;
  bool bad;
  const int n = slot_tokens(p, slot, token0, bad, red + 12);
  if (p.n_seq <= kFewSeqs && slot == 0 && head0 == 0) keep_sequences(p, bad);
  if (BWD && head0 == 0 && tid == 0) p.slot_tokens[slot] = make_longlong2(token0, n);
  if (n == 0) return;
  const int qh = head0 / p.share, hq = p.H / p.share;
  const long long qrec = (long long)slot * hq + qh;
  const bool mine = head0 % p.share == 0;          // the first of the heads that share K and Q keeps them
  // log_alpha and beta of tokens 2 lane, 2 lane + 1 of a head, in flight one head ahead
  float la[2], b[2];
  auto load_gates = [&](int head) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      const long long at = (token0 + t) * p.H + head;
      la[i] = t < n ? __ldg(p.log_alpha + at) : 0.0f;
      b[i] = t < n ? __ldg(p.beta + at) : 0.0f;
    }
  };
  if (warp == 0) load_gates(head0);
  float sk, sq;
  {
    __half *ko = mine ? p.khat + qrec * (NP * kChunk * DK) : nullptr, *qo = mine ? p.qhat + qrec * (NP * kChunk * DK) : nullptr;
    uint4 xk[PASS][NP];
    float inv;
    load_rows<DK, NP, PASS>(p, p.k, p.k_stride, token0, qh, n, xk, tid);
    if (NP == 1) {
      uint4 xq[PASS][NP];
      load_rows<DK, NP, PASS>(p, p.q, p.q_stride, token0, qh, n, xq, tid);
      const unsigned mk = max_rows<NP, PASS>(xk, p.dtype), mq = max_rows<NP, PASS>(xq, p.dtype);
      if (lane == 0) {
        red[warp] = mk;
        red[4 + warp] = mq;
      }
      __syncthreads();
      sk = scale_of(max(max(red[0], red[1]), max(red[2], red[3])), kUpK, inv);
      put_rows<DK, NP, PASS>(xk, p.dtype, inv, K, ko, tid);
      sq = scale_of(max(max(red[4], red[5]), max(red[6], red[7])), kUp, inv);
      put_rows<DK, NP, PASS>(xq, p.dtype, inv, Q, qo, tid);
    } else {
      const unsigned mk = max_rows<NP, PASS>(xk, p.dtype);
      if (lane == 0) red[warp] = mk;
      __syncthreads();
      sk = scale_of(max(max(red[0], red[1]), max(red[2], red[3])), kUpK, inv);
      put_rows<DK, NP, PASS>(xk, p.dtype, inv, K, ko, tid);
      load_rows<DK, NP, PASS>(p, p.q, p.q_stride, token0, qh, n, xk, tid);
      const unsigned mq = max_rows<NP, PASS>(xk, p.dtype);
      if (lane == 0) red[4 + warp] = mq;
      __syncthreads();
      sq = scale_of(max(max(red[4], red[5]), max(red[6], red[7])), kUp, inv);
      put_rows<DK, NP, PASS>(xk, p.dtype, inv, Q, qo, tid);
    }
  }
  const Lane<DK> ld(lane);
  const uint32_t sK = smem_addr(K), sQ = smem_addr(Q);
  constexpr uint32_t LO = kChunk * DK * 2;         // bytes from a plane to the next
  const int m0 = warp * 16;
  // one warp, a head's gates
  auto form_gates = [&](int head) {
    // Sums of log_alpha in 64 bits, so that their differences keep their digits behind a
    // strong decay.  Below -1000 exp() is 0 in fp32 whatever follows, so -inf (a = 0) is
    // held there and G stays finite.
    float *gates = p.gates + ((long long)slot * p.H + head) * kGateFloats;
    float2 *G = gate_at((head - head0) & 1);
    float *bn = reinterpret_cast<float *>(G + kChunk);
    const float kn = sk * pow2(kUpK);
    float inv;
    const float sb = scale_of(__reduce_max_sync(0xFFFFFFFFu, abs_bits(fmaxf(0.0f, fmaxf(finite_abs(b[0]), finite_abs(b[1]))))), 0, inv);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (la[i] < -1000.0f) la[i] = -1000.0f;
    double run = (double)la[0] + (double)la[1];
    for (int d = 1; d < 32; d <<= 1) {
      const double up = __shfl_up_sync(0xFFFFFFFFu, run, d);
      if (lane >= d) run += up;
    }
    const double end = __shfl_sync(0xFFFFFFFFu, run, 31);
    const double Gt[2] = {run - (double)la[1], run};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      const float e = expf((float)Gt[i]), c = expf((float)(end - Gt[i])), w = b[i] * c;
      const double l2 = Gt[i] * 1.4426950408889634;
      const float hi = (float)l2;
      const float2 pair = make_float2(hi, (float)(l2 - (double)hi));
      G[t] = pair;
      bn[t] = b[i] * inv;
      gates[kGateE * kChunk + t] = e;
      gates[kGateWk * kChunk + t] = w * kn;
      gates[kGateEk * kChunk + t] = e * kn;
      gates[kGateW * kChunk + t] = w;
      gates[kGateB * kChunk + t] = b[i];
      gates[kGateC * kChunk + t] = c;
      reinterpret_cast<float2 *>(gates + kGateG * kChunk)[t] = pair;
    }
    if (lane == 0) {
      gates[kGateScales] = sk;
      gates[kGateScales + 1] = sq;
      gates[kGateScales + 2] = sb;
      red[8 + ((head - head0) & 1)] = __float_as_uint(sb);
    }
  };
  if (warp == 0) {
    form_gates(head0);
    if (p.hpc > 1) load_gates(head0 + 1);
  }
  // Q K^T and K K^T, the warp's rows
  auto products = [&](float (&P)[8][4], float (&A)[8][4]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) P[i][j] = A[i][j] = 0.0f;
#pragma unroll 2
    for (int ks = 0; ks < DK / 16; ++ks) {
      uint32_t ak[NP][4], aq[NP][4];
#pragma unroll
      for (int c = 0; c < NP; ++c) {
        if (DELTA) ld.a_rows(ak[c], sK + c * LO, m0, ks * 16);
        ld.a_rows(aq[c], sQ + c * LO, m0, ks * 16);
      }
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        if (np <= warp) {
          uint32_t r[4];
          ld.b_rows(r, sK, np * 16, ks * 16);
#pragma unroll
          for (int c = 0; c < NP; ++c) {
            if (DELTA) mma2(A[2 * np], A[2 * np + 1], ak[c], r);
            mma2(P[2 * np], P[2 * np + 1], aq[c], r);
          }
          if (NP == 2) {
            ld.b_rows(r, sK + LO, np * 16, ks * 16);
            if (DELTA) mma2(A[2 * np], A[2 * np + 1], ak[0], r);
            mma2(P[2 * np], P[2 * np + 1], aq[0], r);
          }
        }
      }
    }
  };
  float QK[8][4];                      // without the delta rule one product serves all heads of the group
  if (!DELTA) {
    __syncthreads();
    float none[8][4];
    products(QK, none);
  }
#pragma unroll 1
  for (int head = head0; head < head0 + p.hpc; ++head) {
    const long long rec = (long long)slot * p.H + head;
    __syncthreads();                   // this head's gates are formed, the last head's matrices are used
    const float2 *G = gate_at((head - head0) & 1);
    const float *bn = reinterpret_cast<const float *>(G + kChunk);
    const float sb = __uint_as_float(red[8 + ((head - head0) & 1)]), sbk = sb * sk;
    // the next head's gates, by the warp that has the fewest blocks
    auto next_gates = [&]() {
      if (warp == 0 && head + 1 < head0 + p.hpc) {
        form_gates(head + 1);
        if (head + 2 < head0 + p.hpc) load_gates(head + 2);
      }
    };

    float P[8][4];
    {
      float A[8][4];
      if (DELTA) products(P, A);
      else
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) P[i][j] = QK[i][j];
      if (DELTA && !several) __syncthreads();      // Q's tile becomes A's planes
      // P over the scales of Q, K and b (for Z without its decays) and, strictly below the diagonal, A
      constexpr bool KEEP = !BWD || !DELTA;        // P itself is wanted
      const float2 gt[2] = {G[m0 + g], G[m0 + g + 8]};
      __half *pp = p.pp + rec * (2 * kTri);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i / 2 <= warp) {
          const float4 gs = *reinterpret_cast<const float4 *>(G + 8 * i + t2);
          const float2 bs = *reinterpret_cast<const float2 *>(bn + 8 * i + t2);
          const bool diagonal = i / 2 == warp;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float p0 = P[i][2 * h] * (BWD ? bs.x * pow2(kDownZ) : bs.x), p1 = P[i][2 * h + 1] * (BWD ? bs.y * pow2(kDownZ) : bs.y);
            if (KEEP) {
              p0 *= decay(gt[h], make_float2(gs.x, gs.y));
              p1 *= decay(gt[h], make_float2(gs.z, gs.w));
            }
            const float a0 = A[i][2 * h] * (bs.x * sbk) * sk, a1 = A[i][2 * h + 1] * (bs.y * sbk) * sk;
            if (diagonal) {
              const int t = m0 + g + 8 * h, s = 8 * i + t2;
              p0 = s <= t ? p0 : 0.0f;
              p1 = s + 1 <= t ? p1 : 0.0f;
              if (DELTA) {
                X[t * kLdF + s] = s < t ? a0 : 0.0f;
                X[t * kLdF + s + 1] = s + 1 < t ? a1 : 0.0f;
              }
            } else if (DELTA) {
              put_pair<kChunk>(A16, kChunk * kChunk, m0 + 8 * h, 8 * i, a0, a1, lane);
            }
            P[i][2 * h] = p0;
            P[i][2 * h + 1] = p1;
          }
        }
      }
      if (KEEP) {
        // forward: each row over a scale of its own, since an output takes one row (and is linear in q)
        float to[2] = {1.0f, 1.0f};
        if (!BWD)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i / 2 <= warp) m = fmaxf(m, fmaxf(fabsf(P[i][2 * h]), fabsf(P[i][2 * h + 1])));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
            const float row = scale_of(__float_as_uint(m), kUp, to[h]);
            if ((lane & 3) == 0) p.gates[rec * kGateFloats + kGateP * kChunk + m0 + g + 8 * h] = row * sbk * sq;
          }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i / 2 <= warp)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              put_at(pp, kTri, tri(warp, i / 2) + (2 * h + (i & 1)) * 64 + 2 * lane, P[i][2 * h] * to[h],
                     P[i][2 * h + 1] * to[h]);
      }
    }
    if (!DELTA) {
      next_gates();
      continue;
    }
    __syncwarp();
    {
      // this warp's diagonal block: lanes c and c + 16 hold column c of its inverse
      const int c = lane & 15;
      float x[16];
      float *B = X + m0 * kLdF + m0;
#pragma unroll
      for (int r = 0; r < 16; ++r) x[r] = r == c ? 1.0f : 0.0f;
#pragma unroll
      for (int r = 0; r < 15; ++r)
#pragma unroll
        for (int i = r + 1; i < 16; ++i) x[i] = fmaf(-B[i * kLdF + r], x[r], x[i]);
      __syncwarp();
      if (lane < 16) {
        __half *d = XD + warp * 512;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          B[r * kLdF + c] = x[r];
          const __half hi = __float2half_rn(x[r]);
          d[tiled<16>(r, c)] = hi;
          d[256 + tiled<16>(r, c)] = __float2half_rn(x[r] - __half2float(hi));
        }
      }
    }
    __syncthreads();
    {
      // block column `warp`: yh, yl[k] = planes of X_kj^T
      const Lane<16> l16(lane);
      const Lane<kChunk> l64(lane);
      const uint32_t sA = smem_addr(A16), sD = smem_addr(XD);
      uint32_t yh[4][4], yl[4][4];
      l16.a_cols(yh[0], sD + warp * 1024, 0, 0);     // X_jj^T: element (m, k) = X_jj[k][m]
      l16.a_cols(yl[0], sD + warp * 1024 + 512, 0, 0);
#pragma unroll
      for (int di = 1; di < 4; ++di) {
        const int i = warp + di;
        if (i < 4) {
          float z0[4] = {0, 0, 0, 0}, z1[4] = {0, 0, 0, 0};
#pragma unroll
          for (int dk = 0; dk < di; ++dk) {
            uint32_t r[4];
            l64.b_rows(r, sA, 16 * i, 16 * (warp + dk));
            mma2(z0, z1, yh[dk], r);
            mma2(z0, z1, yl[dk], r);
            l64.b_rows(r, sA + 2 * kChunk * kChunk, 16 * i, 16 * (warp + dk));
            mma2(z0, z1, yh[dk], r);
          }
          uint32_t zh[4], zl[4], r[4];
          split_tiles(z0, z1, -1.0f, zh, zl);
          float y0[4] = {0, 0, 0, 0}, y1[4] = {0, 0, 0, 0};
          l16.b_rows(r, sD + i * 1024, 0, 0);
          mma2(y0, y1, zh, r);
          mma2(y0, y1, zl, r);
          l16.b_rows(r, sD + i * 1024 + 512, 0, 0);
          mma2(y0, y1, zh, r);
          split_tiles(y0, y1, yh[di], yl[di]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {   // y[c][r] -> X[16 i + r][16 warp + c]
            const int c = g + 8 * (j >> 1), r2 = t2 + (j & 1);
            X[(16 * i + r2) * kLdF + m0 + c] = y0[j];
            X[(16 * i + 8 + r2) * kLdF + m0 + c] = y1[j];
          }
        }
      }
    }
    __syncthreads();

    {
      // planes of Tm (blocks on and below the diagonal)
      __half *tm = p.tm + rec * (2 * kTri);
#pragma unroll 1
      for (int j = 0; j < kChunk * 8 / kPrepThreads; ++j) {
        const int i = tid + j * kPrepThreads, r = (i >> 6) * 8 + (i & 7), c = ((i >> 3) & 7) * 8;
        if ((c >> 4) <= (r >> 4)) {
          uint4 hi, lo;
          float x[8];
          const float2 gr = G[r];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = c + e <= r ? X[r * kLdF + c + e] * decay(gr, G[c + e]) : 0.0f;
          split2(x[0], x[1], hi.x, lo.x);
          split2(x[2], x[3], hi.y, lo.y);
          split2(x[4], x[5], hi.z, lo.z);
          split2(x[6], x[7], hi.w, lo.w);
          const int at = tri(r >> 4, c >> 4) + ((r >> 2 & 2) + (c >> 3 & 1)) * 64 + (r & 7) * 8;
          *reinterpret_cast<uint4 *>(tm + at) = hi;
          *reinterpret_cast<uint4 *>(tm + kTri + at) = lo;
        }
      }
    }
    if (BWD) {
      // Z = P Tm (over P's scales), that is dec times the product without decays: rows t of this warp; block (r, s)
      // of T is zero for s > r
      float acc[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        if (ks <= warp) {
          uint32_t ah[4], al[4];
          split_tiles(P[2 * ks], P[2 * ks + 1], ah, al);
#pragma unroll
          for (int i = 0; i < 2 * ks + 2; ++i) {
            const float *c = X + (ks * 16 + t2) * kLdF + 8 * i + g;
            uint32_t h0, l0, h1, l1;
            split2(c[0], c[kLdF], h0, l0);
            split2(c[8 * kLdF], c[9 * kLdF], h1, l1);
            mma(acc[i], ah, h0, h1);
            mma(acc[i], ah, l0, l1);
            mma(acc[i], al, h0, h1);
          }
        }
      }
      __half *z = p.z + rec * (2 * kTri);
      const float2 gt[2] = {G[m0 + g], G[m0 + g + 8]};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i / 2 <= warp) {
          const float4 gs = *reinterpret_cast<const float4 *>(G + 8 * i + t2);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int t = m0 + g + 8 * h, s = 8 * i + t2;
            const float z0 = s <= t ? acc[i][2 * h] * decay(gt[h], make_float2(gs.x, gs.y)) : 0.0f;
            const float z1 = s + 1 <= t ? acc[i][2 * h + 1] * decay(gt[h], make_float2(gs.z, gs.w)) : 0.0f;
            put_at(z, kTri, tri(warp, i / 2) + (2 * h + (i & 1)) * 64 + 2 * lane, z0, z1);
          }
        }
    }
    // Kt = -T K over the scale of K: rows t of this warp, s blocks up to its own; then Kb = T^T diag(b) K over those of
    // K and b: rows s of this warp, t
    // blocks from its own on.  Two halves of the columns, so that the accumulators leave room for
    // four CTAs per SM.
    constexpr int HALVES = DK >= 64 ? 2 : 1, HT = DK / 8 / HALVES;
#pragma unroll
    for (int which = 0; which < (BWD ? 2 : 1); ++which) {
      __half *dst = (which ? p.kb : p.kt) + rec * (2 * kChunk * DK);
      uint32_t ah[4][4], al[4][4];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        if (which ? ks >= warp : ks <= warp)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int m = m0 + g + 8 * (q & 1), k = ks * 16 + t2 + 8 * (q >> 1);
            if (which) split2(X[k * kLdF + m] * bn[k], X[(k + 1) * kLdF + m] * bn[k + 1], ah[ks][q], al[ks][q]);
            else split2(-X[m * kLdF + k], -X[m * kLdF + k + 1], ah[ks][q], al[ks][q]);
          }
#pragma unroll 1
      for (int half = 0; half < HALVES; ++half) {
        float acc[HT][4];
#pragma unroll
        for (int i = 0; i < HT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          if (which ? ks >= warp : ks <= warp) {
            uint32_t r[HT / 2][4];
#pragma unroll
            for (int np = 0; np < HT / 2; ++np) ld.b_cols(r[np], sK, ks * 16, half * (DK / HALVES) + np * 16);
#pragma unroll
            for (int np = 0; np < HT / 2; ++np) mma2(acc[2 * np], acc[2 * np + 1], ah[ks], r[np]);
#pragma unroll
            for (int np = 0; np < HT / 2; ++np) mma2(acc[2 * np], acc[2 * np + 1], al[ks], r[np]);
            if (NP == 2) {
#pragma unroll
              for (int np = 0; np < HT / 2; ++np) ld.b_cols(r[np], sK + LO, ks * 16, half * (DK / HALVES) + np * 16);
#pragma unroll
              for (int np = 0; np < HT / 2; ++np) mma2(acc[2 * np], acc[2 * np + 1], ah[ks], r[np]);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < HT; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            put_pair<DK>(dst, kChunk * DK, m0 + 8 * h, half * (DK / HALVES) + 8 * i, acc[i][2 * h], acc[i][2 * h + 1], lane);
      }
    }
    next_gates();
  }
}

// -------------------------------------------------------------------------------------
// scan_walk
// -------------------------------------------------------------------------------------
// Grid (sequence * H + head, group of p.rb blocks of 16 value rows).  Per block:
//   NH state warps: warp h holds the state's columns [h d_k/NH, (h+1) d_k/NH) in its accumulators and
//     forms, over its columns, a part of S0 Kt^T for all 64 tokens; the parts are added
//     through shared memory (barrier X), E follows, then S for the own columns.  The state of
//     chunk c + 1 waits for this alone, and NH = 2 halves it.
//   2 side warps, 32 tokens each: Tm V before X; Q S0^T beside the state warps' second half, then
//     (barrier Y, which the state warps only arrive at) P E and the output rows.
// Without the delta rule E = V and the state warps have no products before X; a CTA then takes four blocks.
// A loader warp per block fetches the next chunk's tiles meanwhile (two stages where they fit; one
// took 465 us where two took 300): bulk copies, since 16-byte cp.async of the same 96 KB took longer
// than the chunk's arithmetic (665 against 500 us); and it turns the block's rows of V into fp16 over
// their scale.  In the backward pass's recomputation (kRecompute) the planes of S0 and E are kept
// instead of o.
// Bound by the latency of a chunk's chain, close behind it by the side warps' products for o (two planes of S0, P and
// E) and by shared memory (fragments, exchanged parts, copies).  One sequence of 8192 tokens, 32 heads of 128 x 128, bf16:
// 128 chunks in 335 us, 2.6 us a chunk; the same recomputed for 2 x 4096 tokens and 16 heads: 144 us;
// reverse: 186 us (before scales were taken from what E and R hold 172, and 200 to 220 with 67 KB of code in place of 60:
// the instruction cache).
// The reverse walk has the same roles: D for S, R for E, dO^T Z for Tm V; its side warps also
// form D's sum over dO^T Q, which the state warps take last (barrier Z).
constexpr int kSideWarps = 2;
constexpr int kReverseBlocks = 2;        // at most, where E or R has a barrier of the side warps'

enum WalkKind { kForward, kRecompute, kReverse, kWalkKinds };
// Blocks of value rows per CTA, at most: what registers and shared memory leave room for.
__host__ __device__ constexpr int max_blocks(int np, bool delta, int kind) {
  return !delta && kind != kReverse && np == 1 ? 4 : 2;
}
__host__ __device__ constexpr int walk_threads(int blocks) { return 32 * blocks * (2 + kSideWarps + 1); }

struct WalkLayout {
  int kt, k, q, tm, pp, v, gates, bytes;         // byte offsets inside one stage
  int part, side, plus, last, planes, tops, tail;   // behind the stages, one record per block of rows
};
constexpr int kWalkEnd = 48;             // behind the blocks' records: two barriers, `stop`, the sequence
// A block's 64 token rows of V (or dO): as they come, then as fp16 planes in tiles, then (output) again as
// they go.
__host__ __device__ constexpr int tile_bytes(int np) { return kChunk * 16 * 2 * np; }

__host__ __device__ inline WalkLayout walk_layout(int dk, int np, int rb, int nh, bool delta, int kind) {
  const int tile = kChunk * dk * 2, sq = kTri * 2;
  WalkLayout l{};
  int at = 0;
  l.kt = at; at += delta ? 2 * tile : 0;                       // Kt or Kb
  l.k = at; at += np * tile;
  l.q = at; at += kind != kRecompute ? np * tile : 0;
  l.tm = at; at += kind == kReverse || delta ? 2 * sq : 0;     // Tm or Z
  l.pp = at; at += kind == kForward ? 2 * sq : 0;
  l.v = at; at += rb * tile_bytes(np);
  l.gates = at; at += kGateStage * 4;
  l.bytes = (at + 15) / 16 * 16;
  at = 0;
  l.part = at; at += nh > 1 && (delta || kind == kReverse) ? nh * 4096 : 0;   // the state warps' parts of E or R
  l.side = at; at += delta || kind == kReverse ? 4096 : 0;     // Tm V or dO^T Z
  l.last = at; at += delta || kind == kReverse ? 4096 : 0;     // E or R, for the side warps
  l.plus = at; at += kind == kReverse ? 16 * dk * 4 : 0;       // dO^T Q
  l.planes = at; at += kind == kForward ? 2 * 16 * dk * 2 : 0;   // S0 as left operands
  l.tops = at; at += 32;                                       // largest entries: see below
  l.tail = at;
  return l;
}

// The state rows a thread holds: rows r0 and r0 + 8, columns c0 + 8 i, +1.
template <int NTH>
__device__ __forceinline__ void load_state(float (&S)[NTH][4], const float *src, long long tile, int d_v, int dk, int r0,
                                           int c0) {
#pragma unroll
  for (int i = 0; i < NTH; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float2 x = make_float2(0.0f, 0.0f);
      if (src && r0 + 8 * h < d_v)
        x = *reinterpret_cast<const float2 *>(src + (tile * d_v + r0 + 8 * h) * dk + c0 + 8 * i);
      S[i][2 * h] = x.x;
      S[i][2 * h + 1] = x.y;
    }
}
template <int NTH>
__device__ __forceinline__ void save_state(const float (&S)[NTH][4], float *dst, long long tile, int d_v, int dk, int r0,
                                           int c0) {
#pragma unroll
  for (int i = 0; i < NTH; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (r0 + 8 * h < d_v)
        *reinterpret_cast<float2 *>(dst + (tile * d_v + r0 + 8 * h) * dk + c0 + 8 * i) =
            make_float2(S[i][2 * h], S[i][2 * h + 1]);
}
// Bits of the warp's largest finite magnitude.
template <int N, int M>
__device__ __forceinline__ unsigned max_bits(const float (&x)[N][M]) {
  float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};       // (a NaN is passed over: it is in the data all the same)
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < M; ++j) m[j & 3] = fmaxf(m[j & 3], fabsf(x[i][j]));
  unsigned top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]))));
  if (top >= kInf) {                           // (an infinity would make zeros of the rest)
    float f = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < M; ++j) f = fmaxf(f, finite_abs(x[i][j]));
    top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(f));
  }
  return top;
}

// A warp's 64 rows of 16 columns of the caller's tensor (columns >= have, a multiple of 4, and rows >= n are zeros).
template <int NP>
__device__ __forceinline__ void fetch_rows(uint8_t *dst, const void *src, long long stride, long long token0, int col, int n,
                                           int have, bool by16, int lane) {
  constexpr int SIZE = NP == 2 ? 4 : 2;
  const uint8_t *s = static_cast<const uint8_t *>(src) + (token0 * stride + col) * SIZE;
  if (by16) {
    constexpr int PER = SIZE;              // 16-byte pieces of a row
#pragma unroll
    for (int i = 0; i < kChunk * PER / 32; ++i) {
      const int e = i * 32 + lane, r = e / PER, c = e % PER * (16 / SIZE);
      const bool in = r < n && c < have;
      cp16(dst + e * 16, in ? s + (r * stride + c) * SIZE : s, in);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kChunk * 4 / 32; ++i) {
      const int e = i * 32 + lane, r = e / 4, c = e % 4 * 4;
      const bool in = r < n && c < have;
      cp8(dst + e * 8, in ? s + (r * stride + c) * SIZE : s, in);
    }
  }
}
// ... turned in place into fp16 planes [64][16] (in tiles) over their scale; returns the bits of the largest magnitude.
template <int NP, bool LEAST>
__device__ __forceinline__ unsigned convert_rows(uint8_t *tile, int dtype, int lane) {
  float x[2][16];                          // rows lane and lane + 32
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint8_t *row = tile + (lane + 32 * h) * (16 * 2 * NP);
    if (NP == 1) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint4 w = *reinterpret_cast<const uint4 *>(row + 16 * c);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = pair_of(u[e], dtype);
          x[h][8 * c + 2 * e] = f.x;
          x[h][8 * c + 2 * e + 1] = f.y;
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 f = *reinterpret_cast<const float4 *>(row + 16 * c);
        x[h][4 * c] = f.x; x[h][4 * c + 1] = f.y; x[h][4 * c + 2] = f.z; x[h][4 * c + 3] = f.w;
      }
    }
  }
  const unsigned m = max_bits(x);          // (also: every lane has read its rows)
  float inv;
  scale_of<LEAST>(m, kUp, inv);
  __syncwarp();
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float *y = x[h] + 8 * c;
      uint4 hi, lo;
      split2(y[0] * inv, y[1] * inv, hi.x, lo.x);
      split2(y[2] * inv, y[3] * inv, hi.y, lo.y);
      split2(y[4] * inv, y[5] * inv, hi.z, lo.z);
      split2(y[6] * inv, y[7] * inv, hi.w, lo.w);
      const int at = 2 * tiled<16>(lane + 32 * h, 8 * c);
      *reinterpret_cast<uint4 *>(tile + at) = hi;
      if (NP == 2) *reinterpret_cast<uint4 *>(tile + kChunk * 16 * 2 + at) = lo;
    }
  return m;
}

// Writes 4 tiles (tokens 8 (tile0 + i) .., 16 value rows) times `by` to token rows of the
// caller's tensor, through the block's tile so that rows leave in 16-byte pieces.
template <int NP>
__device__ __forceinline__ void store_tokens(const float (&O)[4][4], float by, uint8_t *tile, int tile0, void *dst, int dtype,
                                             long long stride, long long token0, int n, int col, int have, bool by16,
                                             int lane) {
  const int g = lane >> 2, t2 = (lane & 3) * 2;
  if (NP == 1) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t r[4];
      r[0] = pack_as(dtype, O[2 * i][0] * by, O[2 * i][1] * by);
      r[1] = pack_as(dtype, O[2 * i][2] * by, O[2 * i][3] * by);
      r[2] = pack_as(dtype, O[2 * i + 1][0] * by, O[2 * i + 1][1] * by);
      r[3] = pack_as(dtype, O[2 * i + 1][2] * by, O[2 * i + 1][3] * by);
      const int tok = 8 * (tile0 + 2 * i + (lane >> 4)) + (lane & 7);
      stsm4t(smem_addr(tile + tok * 32 + 16 * ((lane >> 3) & 1)), r);
    }
    __syncwarp();
    uint16_t *out = static_cast<uint16_t *>(dst);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = i * 32 + lane, tok = 8 * tile0 + (e >> 1), c = (e & 1) * 8;
      const uint4 x = *reinterpret_cast<const uint4 *>(tile + tok * 32 + 2 * c);
      if (tok < n) {
        uint16_t *to = out + (token0 + tok) * stride + col + c;
        if (by16) {
          if (c < have) *reinterpret_cast<uint4 *>(to) = x;
        } else {
          if (c < have) *reinterpret_cast<uint2 *>(to) = make_uint2(x.x, x.y);
          if (c + 4 < have) *reinterpret_cast<uint2 *>(to + 4) = make_uint2(x.z, x.w);
        }
      }
    }
  } else {
    float *sm = reinterpret_cast<float *>(tile);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sm[(8 * (tile0 + i) + t2 + (j & 1)) * 16 + g + 8 * (j >> 1)] = O[i][j] * by;
    __syncwarp();
    float *out = static_cast<float *>(dst);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = i * 32 + lane, tok = 8 * tile0 + (e >> 2), c = (e & 3) * 4;
      const float4 x = *reinterpret_cast<const float4 *>(sm + tok * 16 + c);
      if (tok < n && c < have) *reinterpret_cast<float4 *>(out + (token0 + tok) * stride + col + c) = x;
    }
  }
}

__device__ __forceinline__ void barrier_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void barrier_arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
template <int V>
struct Const {
  static constexpr int value = V;
};
__device__ __forceinline__ float4 f4(const float (&x)[4]) { return make_float4(x[0], x[1], x[2], x[3]); }
// Tiles of 16 value rows x 64 tokens as planes in the workspace.
__device__ __forceinline__ void keep_tiles(__half *dst, long long plane, int row0, int tile0, const float (&x)[4][4],
                                           float by, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      put_pair<kChunk>(dst, plane, row0 + 8 * h, 8 * (tile0 + i), x[i][2 * h] * by, x[i][2 * h + 1] * by, lane);
}

// Bytes of a chunk's bulk copies.
__host__ __device__ constexpr unsigned walk_bulk_bytes(int dk, int np, bool delta, int kind) {
  const int tile = kChunk * dk * 2, sq = kTri * 2;
  return kGateStage * 4 + (delta ? 2 * tile : 0) + (delta || kind == kReverse ? 2 * sq : 0) + np * tile +
         (kind != kRecompute ? np * tile : 0) + (kind == kForward ? 2 * sq : 0);
}
// The chunk's matrices: one thread issues them, they complete on `bar`.
template <int DK, int NP, bool DELTA, int KIND>
__device__ __forceinline__ void fetch_matrices(const ScanParams &p, uint8_t *st, uint64_t *bar, const WalkLayout &l, int slot,
                                               int head) {
  constexpr unsigned TILE = kChunk * DK * 2, SQ = kTri * 2;
  const long long rec = (long long)slot * p.H + head;
  const long long qrec = (long long)slot * (p.H / p.share) + head / p.share;
  const float *gates = p.gates + rec * kGateFloats;
  mbar_expect_tx(bar, walk_bulk_bytes(DK, NP, DELTA, KIND));
  bulk_g2s(st + l.gates, gates + (KIND == kForward ? kGateE : kGateC) * kChunk, 4 * kChunk * 4, bar);
  bulk_g2s(st + l.gates + 4 * kChunk * 4, gates + kGateScales, 32, bar);
  if (DELTA) bulk_g2s(st + l.kt, (KIND == kReverse ? p.kb : p.kt) + rec * (2 * kChunk * DK), 2 * TILE, bar);
  if (DELTA || KIND == kReverse)
    bulk_g2s(st + l.tm, (KIND != kReverse ? p.tm : DELTA ? p.z : p.pp) + rec * (2 * kTri), 2 * SQ, bar);
  bulk_g2s(st + l.k, p.khat + qrec * (NP * kChunk * DK), NP * TILE, bar);
  if (KIND != kRecompute) bulk_g2s(st + l.q, p.qhat + qrec * (NP * kChunk * DK), NP * TILE, bar);
  if (KIND == kForward) bulk_g2s(st + l.pp, p.pp + rec * (2 * kTri), 2 * SQ, bar);
}

template <int DK, int NP, bool DELTA, int KIND, int NH>
__global__ void __launch_bounds__(walk_threads(max_blocks(NP, DELTA, KIND)), 1) scan_walk_kernel(const ScanParams p) {
  constexpr bool REV = KIND == kReverse, FWD = KIND == kForward;
  constexpr bool JOIN = DELTA || REV;                        // E (or R) has parts in several warps
  constexpr int DKH = DK / NH, NTH = DKH / 8;
  constexpr uint32_t TILE = kChunk * DK * 2, SQ = kTri * 2, VP = kChunk * 16 * 2;
  constexpr int PER = 32 * (NH + kSideWarps);                // threads of a block of rows
  static_assert(NH == 1 || NH == 2, "parts are exchanged between two warps at most");
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t2 = (lane & 3) * 2;
  const int seq = blockIdx.x / p.H, head = blockIdx.x % p.H, row0 = blockIdx.y * 16 * p.rb;
  // state warps first, then side warps, then loaders
  const int first_side = p.rb * NH, first_load = first_side + p.rb * kSideWarps;
  const bool loader = warp >= first_load, side = !loader && warp >= first_side;
  const int blk = loader ? warp - first_load : side ? (warp - first_side) / kSideWarps : warp / NH;
  const int h = loader ? 0 : side ? (warp - first_side) % kSideWarps : NH == 1 ? 0 : warp % NH;
  const WalkLayout l = walk_layout(DK, NP, p.rb, NH, DELTA, KIND);
  // (a kernel that may start beside scan_prep, which writes it, waits first; without the delta rule all do, since the
  // registers of 20 warps do not hold it over the loads of the state: 64 sequences of 32 tokens, 128 heads 488 us against 513)
  const bool late = !DELTA || (!REV && p.early);
  longlong2 range;
  if (!late) range = __ldcg(p.seqs + seq);
  const int brow = row0 + blk * 16, r0 = brow + g, c0 = h * DKH;
  const bool live = brow < p.dvp;
  uint8_t *tail = smem + p.stages * l.bytes + blk * l.tail;
  float4 *part = reinterpret_cast<float4 *>(tail + l.part), *sided = reinterpret_cast<float4 *>(tail + l.side);
  float4 *last = reinterpret_cast<float4 *>(tail + l.last), *plus = reinterpret_cast<float4 *>(tail + l.plus);
  uint4 *planes = reinterpret_cast<uint4 *>(tail + l.planes);
  // bits of the largest magnitudes: [2 (i & 1) + h] of the state warps' columns at the start of the i-th chunk,
  // [4 + stage] of the rows of V or dO, [6 + h] of E or R (forward: by the state warps, else of the side warps' tokens)
  unsigned *tops = reinterpret_cast<unsigned *>(tail + l.tops);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + p.stages * l.bytes + p.rb * l.tail);   // one per stage, `stop`, the sequence
  int *stop = reinterpret_cast<int *>(bars + 2);
  volatile longlong2 *placed = reinterpret_cast<volatile longlong2 *>(bars + 4);
  const Lane<DK> ld(lane);
  const Lane<16> lv(lane);
  const int X = 1 + 3 * blk, Y = X + 1, Z = X + 2, sides = Z + 3 * kReverseBlocks;
  if (tid == 0) {
    mbar_init(bars, 1);
    mbar_init(bars + 1, 1);
    *stop = 0;
    fence_mbar_init();
  }
  __syncthreads();

  float S[NTH][4];
  if (live && !side && !loader) {
    load_state<NTH>(S, REV ? p.d_state_out : p.state_in, blockIdx.x, p.d_v, DK, r0, c0 + t2);
    const unsigned top = max_bits(S);
    if (lane == 0) {
      tops[h] = top;
      if (NH == 1) tops[1] = tops[3] = 0;
    }
  }
  const int by = p.stages == 2 ? 1 : 0;
  auto stage_of = [&](int c) { return smem + (c & by) * l.bytes; };
  // The reverse walk reads nothing of the recomputation, which has waited for scan_prep: it may run beside it, on the
  // SMs that it leaves free, and waits for it at its own end.
  if (!REV) wait_before();
  launch_next();
  if (late) range = __ldcg(p.seqs + seq);
  const int chunks = ((int)range.y + kChunk - 1) / kChunk;
  if (tid == 0) {                        // (kept there and not in registers, of which there are few)
    placed->x = range.x;
    placed->y = range.y;
  }
  auto fetch = [&](int c, longlong2 of) {
    const long long token0 = of.x + (long long)c * kChunk;
    if (blk == 0 && lane == 0)
      fetch_matrices<DK, NP, DELTA, KIND>(p, stage_of(c), bars + (c & by), l, slot_base(of.x, seq) + c, head);
    if (live)
      fetch_rows<NP>(stage_of(c) + l.v + blk * tile_bytes(NP), REV ? p.o : p.v, REV ? p.o_stride : p.v_stride, token0,
                     head * p.d_v + brow, min(kChunk, (int)of.y - c * kChunk), p.d_v - brow, REV ? p.o16 : p.v16, lane);
    cp_commit();
  };
  if (loader && chunks > 0) fetch(REV ? chunks - 1 : 0, range);
  for (int i0 = 0; i0 < chunks; ++i0) {
    const int c = REV ? chunks - 1 - i0 : i0, next = REV ? c - 1 : c + 1;
    uint8_t *st = stage_of(c);
    uint8_t *tile = st + l.v + blk * tile_bytes(NP);
    if (loader) {
      cp_wait<0>();
      __syncwarp();
      if (live) {
        const unsigned m = convert_rows<NP, !FWD>(tile, p.dtype, lane);
        if (lane == 0) tops[4 + (c & by)] = m;
      }
      // the stage's copies; a wait that runs out ends the walk for the whole CTA (after another wait: they write to its
      // shared memory)
      if (blk == 0 && lane == 0 && !mbar_wait_bounded(bars + (c & by), (i0 >> by) & 1, kWaitNs)) {
        *stop = 1;
        atomicOr(p.flag, kFlagWait);
        mbar_wait_bounded(bars + (c & by), (i0 >> by) & 1, kWaitNs);
      }
    }
    __syncthreads();
    if (*stop) break;
    if (by && loader && i0 + 1 < chunks) fetch(next, make_longlong2(placed->x, placed->y));
    const uint32_t kt = smem_addr(st + l.kt), sk = smem_addr(st + l.k), sq = smem_addr(st + l.q),
                   tm = smem_addr(st + l.tm), pp = smem_addr(st + l.pp), sv = smem_addr(tile);
    // (forward: rows kGateE .. kGateP, else kGateC .. kGateEk)
    const float *eC = reinterpret_cast<const float *>(st + l.gates), *eG = FWD ? eC : eC + kChunk, *wk = eG + kChunk,
                *ek = wk + kChunk, *rowP = ek + kChunk, *scalars = eC + 4 * kChunk;
    const float qscale = scalars[1], bkscale = scalars[2] * scalars[0];
    const long long start = placed->x, rec = (long long)(slot_base(start, seq) + c) * p.H + head;
    const int n = min(kChunk, (int)placed->y - c * kChunk);
    if (loader || !live) {
    } else {
      // scales: of the state, of V (or dO, which takes the scale of Q that the planes of Q and Z lack; Z those of K and
      // b too)
      float inv, invV;
      const float scale = scale_of<!FWD>(max(tops[2 * (i0 & 1)], tops[2 * (i0 & 1) + 1]), kUp, inv);
      float scaleV = scale_of<!FWD>(tops[4 + (c & by)], kUp, invV);
      [[maybe_unused]] const float scaleO = scaleV;          // reverse: dO's own
      if (REV) scaleV *= qscale;
      if (!side) {
        // ---- state warp -----------------------------------------------------------------
        float E[8][4];                   // 16 value rows x 64 tokens
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) E[i][j] = 0.0f;
        __half *keep = FWD ? nullptr : (REV ? p.dd : p.s0) + rec * (2ll * p.dvp * DK);
        // (reverse without the delta rule: Kb = diag(w) K.)  Products that share an accumulator are eight
        // instructions apart and the next fragments are under way before the last products are
        // issued, which covers the latencies of the tensor cores and of ldmatrix.
        constexpr bool LO = DELTA || NP == 2;
        const uint32_t right = DELTA ? kt : sk;
        uint32_t rh[4][4], rl[4][4];
        if (JOIN)
#pragma unroll
          for (int np = 0; np < 4; ++np) {
            ld.b_rows(rh[np], right, np * 16, c0);
            if (LO) ld.b_rows(rl[np], right + TILE, np * 16, c0);
          }
#pragma unroll
        for (int ks = 0; ks < DKH / 16; ++ks) {
          uint32_t ah[4], al[4];
          split_tiles(S[2 * ks], S[2 * ks + 1], inv, ah, al);
          if (FWD) {
            planes[(c0 / 16 + ks) * 32 + lane] = make_uint4(ah[0], ah[1], ah[2], ah[3]);
            planes[(DK / 16 + c0 / 16 + ks) * 32 + lane] = make_uint4(al[0], al[1], al[2], al[3]);
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int at = tiled<DK>(brow + 8 * (q & 1), c0 + ks * 16 + 8 * (q >> 1)) + 2 * lane;
              *reinterpret_cast<uint32_t *>(keep + at) = ah[q];
              *reinterpret_cast<uint32_t *>(keep + (long long)p.dvp * DK + at) = al[q];
            }
          }
          if (JOIN) {
            const bool more = ks + 1 < DKH / 16;
#pragma unroll
            for (int np = 0; np < 4; ++np) mma2(E[2 * np], E[2 * np + 1], ah, rh[np]);
#pragma unroll
            for (int np = 0; np < 4; ++np) mma2(E[2 * np], E[2 * np + 1], al, rh[np]);
            if (more)
#pragma unroll
              for (int np = 0; np < 4; ++np) ld.b_rows(rh[np], right, np * 16, c0 + ks * 16 + 16);
            if (LO) {
#pragma unroll
              for (int np = 0; np < 4; ++np) mma2(E[2 * np], E[2 * np + 1], ah, rl[np]);
              if (more)
#pragma unroll
                for (int np = 0; np < 4; ++np) ld.b_rows(rl[np], right + TILE, np * 16, c0 + ks * 16 + 16);
            }
          }
        }
        if (!FWD && lane == 0 && h == 0)
          p.scales[REV ? kScaleD : kScaleS][rec * (p.dvp / 16) + brow / 16] = scale;
        if (JOIN) {
          if (NH > 1)
#pragma unroll
            for (int i = 0; i < 8; ++i) part[(h * 8 + i) * 32 + lane] = f4(E[i]);
          barrier_sync(X, PER);
          const float s = scale * (REV && DELTA ? bkscale : pow2(-kUpK));
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 u = sided[i * 32 + lane];
            if (NH > 1) {
              const float4 y = part[((h ^ 1) * 8 + i) * 32 + lane];
              E[i][0] += y.x; E[i][1] += y.y; E[i][2] += y.z; E[i][3] += y.w;
            }
            const float2 f = *reinterpret_cast<const float2 *>((!DELTA ? wk : REV ? eC : ek) + 8 * i + t2);
            // (not scale times f: that may leave fp32's range below)
            E[i][0] = fmaf(E[i][0] * s, f.x, u.x); E[i][1] = fmaf(E[i][1] * s, f.y, u.y);
            E[i][2] = fmaf(E[i][2] * s, f.x, u.z); E[i][3] = fmaf(E[i][3] * s, f.y, u.w);
          }
        } else {
          if (FWD) barrier_arrive(X, PER);
        }
        if (JOIN) {
          // E (or R) for the side warps: each state warp hands over half of the tokens
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (NH == 1 || (i >> 2) == h) last[i * 32 + lane] = f4(E[i]);
          if (FWD) {                     // (and the largest, for the scale of its planes)
            const unsigned top = max_bits(E);
            if (lane == 0) tops[6 + h] = top;
            if (NH == 1 && lane == 0) tops[7] = top;
          }
          barrier_arrive(Y, PER);
        }
        // S = e^{G_C} S0 + (diag(w) E)^T K, or D = e^{G_C} D + (diag(e^G) dO)^T Q - (diag(e^G) R)^T K: each tile's
        // sum starts from zero and joins the state in one fma, so that the tensor cores'
        // rounding does not pile up in it
        const float eEnd = eG[kChunk - 1];
        // that operand, in fp32, then over its scale
        float scaleW = 1.0f;
        uint32_t wh[4][4], wl[4][4];
        if (!REV || DELTA) {
          if (!JOIN)                     // E = V: the planes of V are over its own scale
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
              uint32_t v[NP][4];
#pragma unroll
              for (int pl = 0; pl < NP; ++pl) lv.a_cols(v[pl], sv + pl * VP, ks * 16, 0);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                float2 x = half2_of(v[0][q]);
                if (NP == 2) {
                  const float2 y = half2_of(v[NP - 1][q]);
                  x.x = __fadd_rn(x.x, y.x);
                  x.y = __fadd_rn(x.y, y.y);
                }
                E[2 * ks + (q >> 1)][2 * (q & 1)] = x.x * scaleV;
                E[2 * ks + (q >> 1)][2 * (q & 1) + 1] = x.y * scaleV;
              }
            }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 f = *reinterpret_cast<const float2 *>((REV ? ek : wk) + 8 * i + t2);
            E[i][0] *= f.x; E[i][1] *= f.y; E[i][2] *= f.x; E[i][3] *= f.y;
          }
          float invW;
          scaleW = scale_of(max_bits(E), kUp, invW) * pow2(-kUpK);
          if (REV) invW = -invW;
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) split_tiles(E[2 * ks], E[2 * ks + 1], invW, wh[ks], wl[ks]);
        }
        if (!JOIN && FWD) barrier_arrive(Y, PER);    // (V is read)
        constexpr int STEP = JOIN && NTH >= 8 ? 4 : NTH >= 4 ? 2 : 1;   // column pairs at a time
#pragma unroll
        for (int n0 = 0; n0 < NTH / 2; n0 += STEP) {
          float a[2 * STEP][4];
#pragma unroll
          for (int i = 0; i < 2 * STEP; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) a[i][j] = 0.0f;
          if (!REV || DELTA) {
            uint32_t r[2][STEP][4];
#pragma unroll
            for (int i = 0; i < STEP; ++i) ld.b_cols(r[0][i], sk, 0, c0 + (n0 + i) * 16);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
              if (ks < 3)
#pragma unroll
                for (int i = 0; i < STEP; ++i) ld.b_cols(r[(ks + 1) & 1][i], sk, ks * 16 + 16, c0 + (n0 + i) * 16);
#pragma unroll
              for (int i = 0; i < STEP; ++i) mma2(a[2 * i], a[2 * i + 1], wh[ks], r[ks & 1][i]);
#pragma unroll
              for (int i = 0; i < STEP; ++i) mma2(a[2 * i], a[2 * i + 1], wl[ks], r[ks & 1][i]);
              if (NP == 2) {
                uint32_t x[STEP][4];
#pragma unroll
                for (int i = 0; i < STEP; ++i) ld.b_cols(x[i], sk + TILE, ks * 16, c0 + (n0 + i) * 16);
#pragma unroll
                for (int i = 0; i < STEP; ++i) mma2(a[2 * i], a[2 * i + 1], wh[ks], x[i]);
              }
            }
          }
          if (REV && n0 == 0) barrier_sync(Z, PER);
#pragma unroll
          for (int i = 0; i < 2 * STEP; ++i) {
            float *x = S[2 * n0 + i];
            if (REV) {
              const float4 y = plus[(c0 / 8 + 2 * n0 + i) * 32 + lane];
              const float z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) x[j] = fmaf(x[j], eEnd, fmaf(a[i][j], scaleW, z[j]));
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) x[j] = fmaf(x[j], eEnd, a[i][j] * scaleW);
            }
          }
        }
        const unsigned top = max_bits(S);
        if (lane == 0) tops[2 * ((i0 + 1) & 1) + h] = top;
      } else {
        // ---- side warp: tokens 32 h .. 32 h + 31 (where a half meets a triangle, a body for each, so that every loop is
        // straight code; nowhere else, since both bodies and the state warps' share the instruction cache)
        auto with_v = [&](auto half) {
          constexpr int H = decltype(half)::value;
          float U[4][4];                   // tokens 32 H + 8 i ..
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) U[i][j] = 0.0f;
          // Tm V: blocks s <= t; dO^T Z: blocks t >= s
          constexpr int K0 = REV ? 2 * H : 0, K1 = REV ? 4 : 2 * H + 2;
          uint32_t v[4][NP][4], b[4][2][2][4];
#pragma unroll
          for (int ks = K0; ks < K1; ++ks) {
#pragma unroll
            for (int pl = 0; pl < NP; ++pl) lv.a_cols(v[ks][pl], sv + pl * VP, ks * 16, 0);
#pragma unroll
            for (int c2 = 0; c2 < 2; ++c2)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                if (REV ? 2 * H + i <= ks : ks <= 2 * H + i) {
                  if (REV) lv.b_cols(b[ks][c2][i], tm + c2 * SQ + 2 * tri(ks, 2 * H + i), 0, 0);
                  else lv.b_rows(b[ks][c2][i], tm + c2 * SQ + 2 * tri(2 * H + i, ks), 0, 0);
                }
          }
#pragma unroll
          for (int ks = K0; ks < K1; ++ks) {
#pragma unroll
            for (int c2 = 0; c2 < 2; ++c2)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                if (REV ? 2 * H + i <= ks : ks <= 2 * H + i) mma2(U[2 * i], U[2 * i + 1], v[ks][0], b[ks][c2][i]);
            if (NP == 2)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                if (REV ? 2 * H + i <= ks : ks <= 2 * H + i) mma2(U[2 * i], U[2 * i + 1], v[ks][NP - 1], b[ks][0][i]);
          }
          const float to = REV ? scaleV * (bkscale * pow2(-kDownZ)) : scaleV;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            sided[(4 * H + i) * 32 + lane] = make_float4(U[i][0] * to, U[i][1] * to, U[i][2] * to, U[i][3] * to);
        };
        if (JOIN) {
          if (h == 0) with_v(Const<0>());
          else with_v(Const<1>());
        }
        // (in reverse the sum over dO^T Q waits too: it then runs beside the state warps' additions and not
        // beside their products, which the chain waits for)
        if (JOIN || FWD) barrier_sync(X, PER);
        if (REV) {
          // (diag(e^G) dO)^T Q, columns [h d_k/2, (h+1) d_k/2)
          constexpr int HALF = DK >= 32 ? DK / 2 : DK, QS = HALF >= 64 ? 4 : HALF / 16;
          if (DK >= 32 || h == 0) {
            // (e^G over a scale of its own: behind a strong decay at the chunk's start all of it is small)
            float invG;
            const float scaleG = scale_of(__float_as_uint(eG[0]), -1, invG), to = scaleV * scaleG;
            uint32_t oh[4][4], ol[4][4];
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
              uint32_t v[NP][4];
#pragma unroll
              for (int pl = 0; pl < NP; ++pl) lv.a_cols(v[pl], sv + pl * VP, ks * 16, 0);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                float2 f = *reinterpret_cast<const float2 *>(eG + ks * 16 + 8 * (q >> 1) + t2);
                f.x *= invG;
                f.y *= invG;
                float2 x = half2_of(v[0][q]);
                if (NP == 2) {
                  const float2 y = half2_of(v[NP - 1][q]);
                  x.x = __fadd_rn(x.x, y.x);
                  x.y = __fadd_rn(x.y, y.y);
                }
                split2(x.x * f.x, x.y * f.y, oh[ks][q], ol[ks][q]);
              }
            }
#pragma unroll
            for (int n0 = 0; n0 < HALF; n0 += 16 * QS) {
              const int col = (DK >= 32 ? h * HALF : 0) + n0;
              float a[2 * QS][4];
#pragma unroll
              for (int i = 0; i < 2 * QS; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) a[i][j] = 0.0f;
              uint32_t r[2][QS][4];
#pragma unroll
              for (int i = 0; i < QS; ++i) ld.b_cols(r[0][i], sq, 0, col + 16 * i);
#pragma unroll
              for (int ks = 0; ks < 4; ++ks) {
                if (ks < 3)
#pragma unroll
                  for (int i = 0; i < QS; ++i) ld.b_cols(r[(ks + 1) & 1][i], sq, ks * 16 + 16, col + 16 * i);
#pragma unroll
                for (int i = 0; i < QS; ++i) mma2(a[2 * i], a[2 * i + 1], oh[ks], r[ks & 1][i]);
#pragma unroll
                for (int i = 0; i < QS; ++i) mma2(a[2 * i], a[2 * i + 1], ol[ks], r[ks & 1][i]);
                if (NP == 2) {
                  uint32_t x[QS][4];
#pragma unroll
                  for (int i = 0; i < QS; ++i) ld.b_cols(x[i], sq + TILE, ks * 16, col + 16 * i);
#pragma unroll
                  for (int i = 0; i < QS; ++i) mma2(a[2 * i], a[2 * i + 1], oh[ks], x[i]);
                }
              }
#pragma unroll
              for (int i = 0; i < 2 * QS; ++i)
                plus[(col / 8 + i) * 32 + lane] =
                    make_float4(a[i][0] * to, a[i][1] * to, a[i][2] * to, a[i][3] * to);
            }
          }
          barrier_arrive(Z, PER);
        }
        float O[4][4];
        if (FWD) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) O[i][j] = 0.0f;
          uint4 y[DK / 16];
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks) y[ks] = planes[ks * 32 + lane];
          uint32_t b[2][2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i) ld.b_rows(b[0][i], sq, (2 * h + i) * 16, 0);
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks) {
            const uint32_t ah[4] = {y[ks].x, y[ks].y, y[ks].z, y[ks].w};
            if (ks + 1 < DK / 16)
#pragma unroll
              for (int i = 0; i < 2; ++i) ld.b_rows(b[(ks + 1) & 1][i], sq, (2 * h + i) * 16, ks * 16 + 16);
#pragma unroll
            for (int i = 0; i < 2; ++i) mma2(O[2 * i], O[2 * i + 1], ah, b[ks & 1][i]);
            const uint4 z = planes[(DK / 16 + ks) * 32 + lane];
            const uint32_t al[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              mma2(O[2 * i], O[2 * i + 1], al, b[ks & 1][i]);
              if (NP == 2) {
                uint32_t x[4];
                ld.b_rows(x, sq + TILE, (2 * h + i) * 16, ks * 16);
                mma2(O[2 * i], O[2 * i + 1], ah, x);
              }
            }
          }
          const float to = scale * qscale;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = *reinterpret_cast<const float2 *>(eG + 32 * h + 8 * i + t2);
            O[i][0] *= f.x * to; O[i][1] *= f.y * to; O[i][2] *= f.x * to; O[i][3] *= f.y * to;
          }
        }
        auto with_p = [&](auto half) {
          constexpr int H = decltype(half)::value;
          uint32_t r[4][2][4];             // P's blocks
#pragma unroll
          for (int ks = 0; ks < 2 * H + 2; ++ks)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (ks <= 2 * H + i) lv.b_rows(r[ks][i], pp + 2 * tri(2 * H + i, ks), 0, 0);
          if (JOIN) barrier_sync(Y, PER);
          // + E^T P^T (E = V of a 16-bit type is exact in one plane)
          constexpr bool EL = JOIN || NP == 2;
          uint32_t eh[4][4], el[4][4];
          float scaleE = scaleV, invE;
          if (JOIN) scaleE = scale_of(max(tops[6], tops[7]), kUp, invE);
#pragma unroll
          for (int ks = 0; ks < 2 * H + 2; ++ks) {
            if (!JOIN) {
              lv.a_cols(eh[ks], sv, ks * 16, 0);
              if (NP == 2) lv.a_cols(el[ks], sv + VP, ks * 16, 0);
              continue;
            }
            const float4 y = last[(2 * ks) * 32 + lane], z = last[(2 * ks + 1) * 32 + lane];
            const float e0[4] = {y.x, y.y, y.z, y.w}, e1[4] = {z.x, z.y, z.z, z.w};
            split_tiles(e0, e1, invE, eh[ks], el[ks]);
          }
          float a[4][4];                   // (a sum of its own: E and S0 may be of very different sizes)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) a[i][j] = 0.0f;
#pragma unroll
          for (int ks = 0; ks < 2 * H + 2; ++ks)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (ks <= 2 * H + i) {
                mma2(a[2 * i], a[2 * i + 1], eh[ks], r[ks][i]);
                if (EL) mma2(a[2 * i], a[2 * i + 1], el[ks], r[ks][i]);
                uint32_t x[4];
                lv.b_rows(x, pp + SQ + 2 * tri(2 * H + i, ks), 0, 0);
                mma2(a[2 * i], a[2 * i + 1], eh[ks], x);
              }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = *reinterpret_cast<const float2 *>(rowP + 32 * h + 8 * i + t2);
#pragma unroll
            for (int j = 0; j < 4; ++j) O[i][j] = fmaf(a[i][j], scaleE * (j & 1 ? f.y : f.x), O[i][j]);
          }
        };
        if (FWD) {
          if (h == 0) with_p(Const<0>());
          else with_p(Const<1>());
          // (without the delta rule the tile holds V until every warp of the block has read it)
          if (!JOIN) barrier_sync(Y, PER);
          store_tokens<NP>(O, 1.0f, tile, 4 * h, p.o, p.dtype, p.o_stride, start + (long long)c * kChunk, n,
                           head * p.d_v + brow, p.d_v - brow, p.o16, lane);
        } else if (!JOIN) {
          // the planes of V, tile by tile (a tile of [64 tokens][16 rows] is kept transposed)
          __half *et = p.et + rec * (2ll * p.dvp * kChunk);
#pragma unroll
          for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
            for (int pl = 0; pl < 2; ++pl) {
              const int ks = 2 * h + k2;
              uint32_t v[4] = {0, 0, 0, 0};
              if (pl < NP) lv.a_cols(v, sv + pl * VP, ks * 16, 0);
#pragma unroll
              for (int q = 0; q < 4; ++q)
                *reinterpret_cast<uint32_t *>(et + pl * (long long)p.dvp * kChunk +
                                              tiled<kChunk>(brow + 8 * (q & 1), ks * 16 + 8 * (q >> 1)) + 2 * lane) = v[q];
            }
          if (lane == 0 && h == 0) p.scales[kScaleE][rec * (p.dvp / 16) + brow / 16] = scaleV;
        } else {
          barrier_sync(Y, PER);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 y = last[(4 * h + i) * 32 + lane];
            O[i][0] = y.x; O[i][1] = y.y; O[i][2] = y.z; O[i][3] = y.w;
          }
          const unsigned top = max_bits(O);
          if (lane == 0) tops[6 + h] = top;
          barrier_sync(sides, 32 * kSideWarps);
          float invE;
          const float scaleE = scale_of<true>(max(tops[6], tops[7]), kUp, invE);
          keep_tiles((REV ? p.rt : p.et) + rec * (2ll * p.dvp * kChunk), (long long)p.dvp * kChunk, brow, 4 * h, O, invE, lane);
          if (lane == 0 && h == 0) {
            p.scales[REV ? kScaleR : kScaleE][rec * (p.dvp / 16) + brow / 16] = scaleE;
            if (REV) p.scales[kScaleO][rec * (p.dvp / 16) + brow / 16] = scaleO;
          }
          if (REV) {
            // (both side warps are done with the rows of dO)
            barrier_sync(sides, 32 * kSideWarps);
            store_tokens<NP>(O, 1.0f, tile, 4 * h, p.dv, p.dtype, p.v_stride, start + (long long)c * kChunk, n,
                             head * p.d_v + brow, p.d_v - brow, p.v16, lane);
          }
        }
      }
    }
    if (!by) {
      __syncthreads();
      if (loader && i0 + 1 < chunks) fetch(next, make_longlong2(placed->x, placed->y));
    }
  }
  if (live && !side && !loader && KIND != kRecompute && !*stop) {
    float *out = REV ? p.d_state_in : p.state_out;
    if (out) save_state<NTH>(S, out, blockIdx.x, p.d_v, DK, r0, c0 + t2);
  }
  if (REV) wait_before();
}

// -------------------------------------------------------------------------------------
// scan_grads
// -------------------------------------------------------------------------------------
// Grid (slot, head), 16 warps in four groups of four; a warp owns 16 of a group's 64 token rows:
//   group 0: dO S0     group 1: R S0     group 2: E D     group 3: dO E^T and R E^T
// with the value rows as the contraction axis, passing through shared memory kGradRows at a time.  Then,
// with dP'_ts = b_s dec_ts dO_t.E_s (s <= t), dL'_ts = -b_s dec_ts R_t.E_s (s < t) from group 3:
//   dQ = diag(e^G) dO S0 + dP' K                                            group 0
//   dK = diag(w) E D + dP'^T Q  - d diag(e^G) R S0 + dL' K  + dL'^T K        groups 2, 1, 3
//   c_s = sum_t dec_ts (q_t.k_s dO_t.E_s - k_t.k_s R_t.E_s)
//   dbeta_s = c_s + e^{G_C - G_s} k_s.(D^T E_s)
//   dG_t = sum_s b_s dec_ts (...) - b_t dbeta_t + e^{G_t} (q_t.(S0^T dO_t) - d k_t.(S0^T R_t))
//   dlog_alpha_r = sum_{t >= r} dG_t + sum_s w_s k_s.(D^T E_s) + e^{G_C} <D, S0>
// (the pair (t, s) enters dG_t and, through dbeta_s, -dG_s with the same value: a token's own pair is left out of both,
// and of the terms of the last state those of the tokens before r are what is left, since behind strong decays the
// others are far larger).
// Scales: the planes of 16 value rows are held over their own powers of two, so a 16-row step
// contributes in units that are the product of two of them; left operands are brought to
// the largest unit F of the group's steps, and the group's sums are held over F.
// Bound by latency and the tensor cores in turn: of an item's 35000 cycles 4300 wait for the first
// copies, 17000 are the sums over value rows (10800 of products), 4200 the matrices dP' and dL', 3200
// their products and 3600 the stores.  2 x 4096 tokens, 16 heads of 128 x 128, bf16 (2048 items): 290
// us (those cycles of 280).  Items of a CTA one behind the other, the next one's copies under way: 357 us (registers).
// The tensor cores cut their sums off instead of rounding them: 768 products in a row (d_v = 4096) leave 1.6e-5, all
// to one side.  So every kGradSum value rows (48 products, below 1.5e-6) the sums are added, rounded, to a copy in the
// thread's local memory; narrower heads (the usual 64 to 256) never touch it.
constexpr int kGradRows = 32, kGradSum = 256;
// Without the delta rule and with one plane of K and Q an item fits half an SM: 8 warps in two groups (dO S0, E D), each
// with every other 16 columns of dO E^T beside it, and two CTAs per SM cover each other's waits (6400
// tokens, 64 heads of 64 x 128, bf16: 366 us; 379 at first, where four groups in one CTA took 487).
__host__ __device__ constexpr bool grad_halves(int np, bool delta) { return np == 1 && !delta; }
__host__ __device__ constexpr int grad_threads(int np, bool delta) { return grad_halves(np, delta) ? 256 : 512; }

struct GradLayout {
  int k, q, x, f, scales, stage, stage_bytes, s0, d, e, r, o;
};
__host__ __device__ inline GradLayout grad_layout(int dk, int np, int dvp, bool delta) {
  GradLayout l{};
  int at = 0;
  l.k = at; at += np * kChunk * dk * 2;
  l.q = at; at += np * kChunk * dk * 2;
  l.x = at; at += (delta ? 4 : 2) * kChunk * kChunk * 2;  // dP' hi, lo, dL' hi, lo
  l.f = at; at += (kGateFloats + 6 * kChunk + 4 * kChunk + 16 + 8) * 4;
  l.scales = at; at += kScales * (dvp / 16) * 4;
  l.stage = (at + 15) / 16 * 16;
  at = 0;
  l.s0 = at; at += 2 * kGradRows * dk * 2;
  l.d = at; at += 2 * kGradRows * dk * 2;
  l.e = at; at += 2 * kGradRows * kChunk * 2;
  l.r = at; at += delta ? 2 * kGradRows * kChunk * 2 : 0;
  l.o = at; at += kChunk * (kGradRows + (np == 2 ? 4 : 8)) * (np == 2 ? 4 : 2);
  l.stage_bytes = at;
  return l;
}
// Behind the fixed part: the stages, and later what groups 1 and 3 hand to group 2.
__host__ __device__ inline int grad_bytes(const GradLayout &l, int dk, int stages, bool delta) {
  const int a = stages * l.stage_bytes, b = delta ? 2 * kChunk * dk * 4 : 0;
  return l.stage + (a > b ? a : b);
}

// A left operand's registers times a power of two <= 1.
__device__ __forceinline__ void scale_frag(uint32_t (&a)[4], __half2 by) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const __half2 y = __hmul2(*reinterpret_cast<__half2 *>(&a[q]), by);
    a[q] = *reinterpret_cast<const uint32_t *>(&y);
  }
}
__device__ __forceinline__ int exponent(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }
// The largest exponent of a[b] c[b] over the blocks of 16 value rows.
__device__ __forceinline__ int top_unit(const float *a, const float *c, int blocks, int lane) {
  int top = -1000;
  for (int b = lane; b < blocks; b += 32) top = max(top, exponent(a[b]) + exponent(c[b]));
  return __reduce_max_sync(0xFFFFFFFFu, top);
}

template <int DK, int NP, bool DELTA>
__global__ void __launch_bounds__(grad_threads(NP, DELTA), grad_halves(NP, DELTA) ? 2 : 1) scan_grads_kernel(const ScanParams p) {
  constexpr bool HALF = grad_halves(NP, DELTA);
  constexpr int kGradThreads = grad_threads(NP, DELTA), KGROUP = HALF ? 1 : 2;     // KGROUP: the group of dK
  constexpr int NT = DK / 8, LDO = kGradRows + (NP == 2 ? 4 : 8), SIZE = NP == 2 ? 4 : 2;
  constexpr uint32_t TILE = kChunk * DK * 2, SQ = kChunk * kChunk * 2, SP = kGradRows * DK * 2, EP = kGradRows * kChunk * 2;
  extern __shared__ __align__(16) uint8_t smem[];
  const GradLayout l = grad_layout(DK, NP, p.dvp, DELTA);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, group = warp >> 2, w4 = warp & 3, g = lane >> 2,
            t2 = (lane & 3) * 2, m0 = w4 * 16;
  const int slot = blockIdx.x / p.H, head = blockIdx.x % p.H;    // (heads that share K and Q run side by side)
  wait_before();
  launch_next();
  const longlong2 tokens = p.slot_tokens[slot];
  const long long token0 = tokens.x;
  const int n = (int)tokens.y;
  if (n == 0) return;
  const long long rec = (long long)slot * p.H + head;
  const long long qrec = (long long)slot * (p.H / p.share) + head / p.share;
  const uint32_t sk = smem_addr(smem + l.k), sq = smem_addr(smem + l.q), sx = smem_addr(smem + l.x);
  float *gates = reinterpret_cast<float *>(smem + l.f);
  const float *eG = gates + kGateE * kChunk, *w = gates + kGateW * kChunk, *be = gates + kGateB * kChunk,
              *eC = gates + kGateC * kChunk;
  const float2 *G = reinterpret_cast<const float2 *>(gates + kGateG * kChunk);
  float *rowv = gates + kGateFloats, *aq = rowv + 2 * kChunk, *ak = aq + kChunk, *kw = ak + kChunk, *diagp = kw + kChunk,
        *colp = diagp + kChunk, *red = colp + 4 * kChunk;
  uint64_t *bars = reinterpret_cast<uint64_t *>(red + 16);                // one per stage
  int *stop = reinterpret_cast<int *>(bars + 2);
  if (tid == 0) {
    mbar_init(bars, 1);
    mbar_init(bars + 1, 1);
    *stop = 0;
    fence_mbar_init();
  }
  const int blocks = (p.dvp + kGradRows - 1) / kGradRows, blocks16 = p.dvp / 16;
  // A block of value rows, with the first one all that belongs to the item: bulk copies of one thread (they complete on
  // the stage's barrier), the rows of dO in 8- or 16-byte pieces.
  auto stage_of = [&](int b) { return smem + l.stage + (p.stages == 2 ? (b & 1) * l.stage_bytes : 0); };
  auto fetch = [&](int b) {
    uint8_t *st = stage_of(b);
    const int v0 = b * kGradRows, rows = min(kGradRows, p.dvp - v0);
    if (tid == 0) {
      uint64_t *bar = bars + (p.stages == 2 ? b & 1 : 0);
      mbar_expect_tx(bar, rows * (DK * 8 + kChunk * (DELTA ? 8 : 4)) + (b == 0 ? 2 * NP * TILE + kGateFloats * 4 : 0));
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const long long at = (rec * 2 + c) * p.dvp + v0;
        bulk_g2s(st + l.s0 + c * SP, p.s0 + at * DK, rows * DK * 2, bar);
        bulk_g2s(st + l.d + c * SP, p.dd + at * DK, rows * DK * 2, bar);
        bulk_g2s(st + l.e + c * EP, p.et + at * kChunk, rows * kChunk * 2, bar);
        if (DELTA) bulk_g2s(st + l.r + c * EP, p.rt + at * kChunk, rows * kChunk * 2, bar);
      }
      if (b == 0) {
        bulk_g2s(smem + l.k, p.khat + qrec * (NP * kChunk * DK), NP * TILE, bar);
        bulk_g2s(smem + l.q, p.qhat + qrec * (NP * kChunk * DK), NP * TILE, bar);
        bulk_g2s(gates, p.gates + rec * kGateFloats, kGateFloats * 4, bar);
      }
    }
    if (b == 0)
      for (int i = tid; i < kScales * blocks16; i += kGradThreads)
        cp4(smem + l.scales + 4 * i, p.scales[i / blocks16] + rec * blocks16 + i % blocks16);
    copy_tokens<SIZE>(st + l.o, LDO,
                      static_cast<const uint8_t *>(p.o) + (token0 * p.o_stride + (long long)head * p.d_v + v0) * SIZE,
                      p.o_stride, kGradRows, n, p.d_v - v0, p.o16, tid, kGradThreads);
    cp_commit();
  };
  fetch(0);
  const float *sS = reinterpret_cast<const float *>(smem + l.scales), *sE = sS + blocks16, *sD = sE + blocks16,
              *sR = sD + blocks16, *sO = sR + blocks16;
  // the group's two scales: of the left operand's planes and of the right one's
  const float *sl = group == KGROUP ? sE : group == 0 || !DELTA ? sO : sR,
              *sr2 = group == KGROUP ? sD : group == 3 ? sE : sS;
  int topDS = 0, topRE = 0, topOE = 0, top = 0;

  // groups 0 to 2: 16 rows x d_k; group 3: tiles 0-7 dO E^T, 8-15 R E^T (in halves: tiles NT .. NT + 3 dO E^T)
  constexpr int NA = HALF ? NT + 4 : NT > 16 ? NT : 16;
  float acc[NA][4], ds = 0.0f;
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
  float kept[NA * 4], *far = kept;
  asm volatile("" : "+l"(far));                          // (memory, not registers)
  const Lane<DK> ld(lane);
  const Lane<kChunk> lc(lane);

  for (int b = 0; b < blocks; ++b) {
    cp_wait<0>();
    if (tid == 0 && !mbar_wait_bounded(bars + (p.stages == 2 ? b & 1 : 0), (p.stages == 2 ? b >> 1 : b) & 1, kWaitNs)) {
      *stop = 1;
      atomicOr(p.flag, kFlagWait);
      mbar_wait_bounded(bars + (p.stages == 2 ? b & 1 : 0), (p.stages == 2 ? b >> 1 : b) & 1, kWaitNs);
    }
    __syncthreads();
    if (*stop) return;
    if (b == 0) {
      topDS = top_unit(sD, sS, blocks16, lane);
      topOE = top_unit(sO, sE, blocks16, lane);
      if (DELTA) topRE = top_unit(sR, sE, blocks16, lane);
      if (DELTA) {
        top = top_unit(sl, sr2, blocks16, lane);
      } else {                           // (both, and no addresses kept: 8 warps an item have no registers for them)
        const int os = top_unit(sO, sS, blocks16, lane), ed = top_unit(sE, sD, blocks16, lane);
        top = group == KGROUP ? ed : group == 0 ? os : topOE;
      }
    }
    if (p.stages == 2 && b + 1 < blocks) fetch(b + 1);
    uint8_t *st = stage_of(b);
    const uint32_t s0 = smem_addr(st + l.s0), dd = smem_addr(st + l.d), se = smem_addr(st + l.e), sr = smem_addr(st + l.r);
#pragma unroll
    for (int kk = 0; kk < kGradRows; kk += 16) {
      const int b16 = b * (kGradRows / 16) + kk / 16;
      if (b16 >= blocks16) break;
      {
        // <D, S0>
        float part = 0.0f;
#pragma unroll
        for (int i = tid; i < 16 * DK / 2; i += kGradThreads) {
          const int at = kk * DK * 2 + i * 4;          // (any order of the block's entries will do)
          auto pair = [&](int off) {
            const float2 hi = half2_of(*reinterpret_cast<const uint32_t *>(st + off + at));
            const float2 lo = half2_of(*reinterpret_cast<const uint32_t *>(st + off + SP + at));
            return make_float2(__fadd_rn(hi.x, lo.x), __fadd_rn(hi.y, lo.y));
          };
          const float2 x = pair(l.s0), y = pair(l.d);
          part = fmaf(x.x, y.x, fmaf(x.y, y.y, part));
        }
        ds = fmaf(part, pow2(exponent(sD[b16]) + exponent(sS[b16]) - topDS), ds);
      }
      const int el = exponent(sl[b16]);
      const float ratio = pow2(el + exponent(sr2[b16]) - top);
      const __half2 by = __float2half2_rn(ratio);
      uint32_t ao[NP][4], ar[2][4], b4[4];
      if (HALF) {
        // dO over its scale, in the unit of dO E^T; of this warp's columns every other 16
        const int eo = exponent(sO[b16]);
        const float to = pow2(-eo) * pow2(eo + exponent(sE[b16]) - topOE);
        uint32_t raw[4], ae[4];
        a_rows_plain(raw, smem_addr(st + l.o), LDO, m0, kk, lane);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 f = pair_of(raw[q], p.dtype);
          ae[q] = pack2(f.x * to, f.y * to);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int np = 2 * j + group;
          if (np <= w4) {
            lc.b_cols(b4, se, kk, np * 16);
            mma2(acc[NT + 2 * j], acc[NT + 2 * j + 1], ae, b4);
            lc.b_cols(b4, se + EP, kk, np * 16);
            mma2(acc[NT + 2 * j], acc[NT + 2 * j + 1], ae, b4);
          }
        }
      }
      if (group == 0 || (!HALF && group == 3)) {
        // dO over its scale, in the unit of the group's product
        const int eo = exponent(sO[b16]);
        const float to = pow2(-eo) * (group == 0 ? ratio : pow2(eo + exponent(sE[b16]) - topOE));
        if (NP == 1) {
          uint32_t raw[4];
          a_rows_plain(raw, smem_addr(st + l.o), LDO, m0, kk, lane);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 f = pair_of(raw[q], p.dtype);
            ao[0][q] = pack2(f.x * to, f.y * to);
          }
        } else {
          const float *so = reinterpret_cast<const float *>(st + l.o);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 f = *reinterpret_cast<const float2 *>(so + (m0 + g + 8 * (q & 1)) * LDO + kk + 8 * (q >> 1) + t2);
            split2(f.x * to, f.y * to, ao[0][q], ao[NP - 1][q]);
          }
        }
      }
      if (group == KGROUP || (DELTA && (group & 1)))
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          lc.a_cols(ar[c], (group == KGROUP ? se : sr) + c * EP, kk, m0);
          scale_frag(ar[c], by);
        }
      if (group == 0) {
#pragma unroll
        for (int np = 0; np < DK / 16; ++np) {
          ld.b_cols(b4, s0, kk, np * 16);
#pragma unroll
          for (int c = 0; c < NP; ++c) mma2(acc[2 * np], acc[2 * np + 1], ao[c], b4);
          ld.b_cols(b4, s0 + SP, kk, np * 16);
          mma2(acc[2 * np], acc[2 * np + 1], ao[0], b4);
        }
      } else if (group == KGROUP || (DELTA && group == 1)) {
        const uint32_t x = group == KGROUP ? dd : s0;
#pragma unroll
        for (int np = 0; np < DK / 16; ++np) {
          ld.b_cols(b4, x, kk, np * 16);
          mma2(acc[2 * np], acc[2 * np + 1], ar[0], b4);
          mma2(acc[2 * np], acc[2 * np + 1], ar[1], b4);
          ld.b_cols(b4, x + SP, kk, np * 16);
          mma2(acc[2 * np], acc[2 * np + 1], ar[0], b4);
        }
      } else if (!HALF && group == 3) {
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          if (np <= w4) {
            lc.b_cols(b4, se, kk, np * 16);
#pragma unroll
            for (int c = 0; c < NP; ++c) mma2(acc[2 * np], acc[2 * np + 1], ao[c], b4);
            if (DELTA) {
              mma2(acc[8 + 2 * np], acc[8 + 2 * np + 1], ar[0], b4);
              mma2(acc[8 + 2 * np], acc[8 + 2 * np + 1], ar[1], b4);
            }
            lc.b_cols(b4, se + EP, kk, np * 16);
            mma2(acc[2 * np], acc[2 * np + 1], ao[0], b4);
            if (DELTA) mma2(acc[8 + 2 * np], acc[8 + 2 * np + 1], ar[0], b4);
          }
        }
      }
    }
    if (p.stages == 1) {
      __syncthreads();
      if (b + 1 < blocks) fetch(b + 1);
    }
    if (blocks > kGradSum / kGradRows && ((b + 1) % (kGradSum / kGradRows) == 0 || b + 1 == blocks)) {
      const bool begun = b >= kGradSum / kGradRows, done = b + 1 == blocks;
#pragma unroll
      for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x = acc[i][j] + (begun ? far[4 * i + j] : 0.0f);
          if (!done) far[4 * i + j] = x;
          acc[i][j] = done ? x : 0.0f;
        }
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) ds += __shfl_xor_sync(0xFFFFFFFFu, ds, d);
  if (lane == 0) red[warp] = ds;
  const float kappa = gates[kGateScales], qscale = gates[kGateScales + 1], sb = gates[kGateScales + 2];
  const float isb = __uint_as_float((254u << 23) - __float_as_uint(sb));
  // The planes of dP' are held over the unit of dO E^T, dvp (rounded up to a power of two) and the scale of b, those of
  // dL' over that of R E^T likewise.  Entries of dO, E and R over their scales are below 2^15, so a sum over d_v of
  // products of two is below 2^30 dvp, and b over its scale below 2: the planes' entries are below
  // 2^15.
  const int lg = 2 + kUp + 32 - __clz(p.dvp - 1);
  // A group's sums over value rows go on in the unit of its planes' products, 2^(topP + lg + eb) times the right operand's
  // scale, or 2^-60 of their own unit where that is larger (the planes' part is then scaled down in turn).  E D is
  // multiplied by w <= b, so its unit takes the scale of b.
  const int topP = DELTA && (group & 1) ? topRE : topOE;
  const int own = top + (group == KGROUP ? exponent(sb) : 0);
  const int unitP = topP + lg + exponent(sb) + exponent(group == KGROUP ? qscale : kappa), unit = max(unitP, own - 60);
  const float F1 = pow2(top / 2), F2 = pow2(top - top / 2);              // unit of the group's sums, as two factors in range
  const float to_unit = pow2(own - unit);
  const float out1 = pow2(unit / 2), out2 = pow2(unit - unit / 2);

  auto finish_rows = [&]() {
    // the row's dot with q or k, then the row in the planes' units
    const uint8_t *x = smem + (group == 0 ? l.q : l.k);
    float *dots = group == 0 ? aq : group == KGROUP ? kw : ak;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = m0 + g + 8 * h;
      float s = 0.0f;
      const float to = (group == KGROUP ? w[t] * isb : group == 1 ? -eG[t] : eG[t]) * to_unit;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int at = 2 * (tiled<DK>(m0 + 8 * h, 8 * i) + 2 * lane);
        float2 v = half2_of(*reinterpret_cast<const uint32_t *>(x + at));
        if (NP == 2) {
          const float2 y = half2_of(*reinterpret_cast<const uint32_t *>(x + TILE + at));
          v.x = __fadd_rn(v.x, y.x);
          v.y = __fadd_rn(v.y, y.y);
        }
        s = fmaf(v.x, acc[i][2 * h], fmaf(v.y, acc[i][2 * h + 1], s));
        acc[i][2 * h] *= to;
        acc[i][2 * h + 1] *= to;
      }
      s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
      s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
      if ((lane & 3) == 0) dots[t] = s * (group == 0 ? qscale : kappa) * F1 * F2;
    }
  };
  auto form_planes = [&]() {
    constexpr int STEPS = HALF ? 2 : 4;
    // the larger of the units of dO E^T and R E^T
    const int topM = DELTA ? max(topOE, topRE) : topOE;
    const float U1 = pow2(topM / 2), U2 = pow2(topM - topM / 2), to_planes = pow2(-lg);
    float rs[2] = {0.0f, 0.0f}, cs[2 * STEPS][2];
#pragma unroll
    for (int i = 0; i < 2 * STEPS; ++i) cs[i][0] = cs[i][1] = 0.0f;
    // q_t.k_s with dO E^T -> dP', k_t.k_s with R E^T -> dL', by 16 columns s, so that few registers hold the products
    const float toq = qscale * kappa * pow2(topOE - topM), tok = -kappa * kappa * pow2(topRE - topM);
    __half *out = reinterpret_cast<__half *>(smem + l.x);
    const float2 gt[2] = {G[m0 + g], G[m0 + g + 8]};
#pragma unroll
    for (int step = 0; step < STEPS; ++step) {
      const int np = HALF ? 2 * step + group : step;
      if (np <= w4) {
        float x[2][2][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[0][0][j] = x[0][1][j] = x[1][0][j] = x[1][1][j] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks) {
          uint32_t a[2][NP][4], b4[4];
#pragma unroll
          for (int c = 0; c < NP; ++c) {
            ld.a_rows(a[0][c], sq + c * TILE, m0, ks * 16);
            if (DELTA) ld.a_rows(a[1][c], sk + c * TILE, m0, ks * 16);
          }
          ld.b_rows(b4, sk, np * 16, ks * 16);
#pragma unroll
          for (int ps = 0; ps < (DELTA ? 2 : 1); ++ps)
#pragma unroll
            for (int c = 0; c < NP; ++c) mma2(x[ps][0], x[ps][1], a[ps][c], b4);
          if (NP == 2) {
            ld.b_rows(b4, sk + TILE, np * 16, ks * 16);
#pragma unroll
            for (int ps = 0; ps < (DELTA ? 2 : 1); ++ps) mma2(x[ps][0], x[ps][1], a[ps][0], b4);
          }
        }
        const bool diagonal = np == w4;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = 2 * np + e, own = (HALF ? NT : 0) + 2 * step + e;
          const float4 gs = *reinterpret_cast<const float4 *>(G + 8 * i + t2);
          const float2 bs = *reinterpret_cast<const float2 *>(be + 8 * i + t2);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int t = m0 + g + 8 * h;
            float y[2], z[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int s = 8 * i + t2 + j;
              const float dec = decay(gt[h], j ? make_float2(gs.z, gs.w) : make_float2(gs.x, gs.y));
              const float b = j ? bs.y : bs.x;
              y[j] = acc[own][2 * h + j] * dec;
              z[j] = DELTA ? acc[(DELTA ? 8 : 0) + own][2 * h + j] * dec : 0.0f;
              if (diagonal) {
                y[j] = s <= t ? y[j] : 0.0f;
                z[j] = s < t ? z[j] : 0.0f;
              }
              float m = y[j] * (x[0][e][2 * h + j] * toq);
              if (DELTA) m = fmaf(z[j], x[1][e][2 * h + j] * tok, m);
              // (a pair that the mask leaves out gives nothing, not 0 times a decay that overflowed)
              if (diagonal && s > t) m = 0.0f;
              // (the pair (t, t) is dbeta's alone: in dG_t it cancels)
              if (diagonal && s == t) {
                diagp[t] = m * U1 * U2;
                m = 0.0f;
              }
              rs[h] = fmaf(b, m, rs[h]);
              cs[2 * step + e][j] += m;
              y[j] *= b * isb * to_planes;
              z[j] *= -b * isb * to_planes;
            }
            put_pair<kChunk>(out, kChunk * kChunk, m0 + 8 * h, 8 * i, y[0], y[1], lane);
            if (DELTA) put_pair<kChunk>(out + 2 * kChunk * kChunk, kChunk * kChunk, m0 + 8 * h, 8 * i, z[0], z[1], lane);
          }
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      rs[h] += __shfl_xor_sync(0xFFFFFFFFu, rs[h], 1);
      rs[h] += __shfl_xor_sync(0xFFFFFFFFu, rs[h], 2);
      if ((lane & 3) == 0) rowv[(HALF ? group * kChunk : 0) + m0 + g + 8 * h] = rs[h] * U1 * U2;
    }
#pragma unroll
    for (int i = 0; i < 2 * STEPS; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int tile = HALF ? 2 * (2 * (i >> 1) + group) + (i & 1) : i;
        float c = cs[i][j];
        c += __shfl_xor_sync(0xFFFFFFFFu, c, 4);
        c += __shfl_xor_sync(0xFFFFFFFFu, c, 8);
        c += __shfl_xor_sync(0xFFFFFFFFu, c, 16);
        if (g == 0) colp[w4 * kChunk + 8 * tile + t2 + j] = c * U1 * U2;
      }
#pragma unroll
    for (int i = 0; i < (HALF ? 0 : NT); ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
  };
  if (HALF || group != 3) finish_rows();
  else form_planes();
  if (HALF) form_planes();
  __syncthreads();
  {
    // dP' K, dL' K: rows t, blocks s <= t; dP'^T Q, dL'^T K: rows s, blocks t >= s
    const bool rows_t = HALF ? group == 0 : group < 2;
    const uint32_t left = sx + (DELTA && (group & 1) ? 2 * SQ : 0), right = group == KGROUP ? sq : sk;
    const __half2 down = __float2half2_rn(pow2(unitP - unit));
    if (DELTA || HALF || !(group & 1))
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        if (rows_t ? ks <= w4 : ks >= w4) {
          uint32_t a[2][4], b4[4];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (rows_t) lc.a_rows(a[c], left + c * SQ, m0, ks * 16);
            else lc.a_cols(a[c], left + c * SQ, ks * 16, m0);
            if (unit != unitP) scale_frag(a[c], down);
          }
#pragma unroll
          for (int np = 0; np < DK / 16; ++np) {
            ld.b_cols(b4, right, ks * 16, np * 16);
            mma2(acc[2 * np], acc[2 * np + 1], a[0], b4);
            mma2(acc[2 * np], acc[2 * np + 1], a[1], b4);
            if (NP == 2) {
              ld.b_cols(b4, right + TILE, ks * 16, np * 16);
              mma2(acc[2 * np], acc[2 * np + 1], a[0], b4);
            }
          }
        }
      }
  }
  float4 *hand = reinterpret_cast<float4 *>(smem + l.stage);             // [2][4 warps][NT][32]
  if (DELTA && (group & 1))
#pragma unroll
    for (int i = 0; i < NT; ++i)
      hand[(((group >> 1) * 4 + w4) * NT + i) * 32 + lane] =
          make_float4(acc[i][0] * out1 * out2, acc[i][1] * out1 * out2, acc[i][2] * out1 * out2, acc[i][3] * out1 * out2);
  if (DELTA) __syncthreads();
  if (group == 0 || group == KGROUP) {
    void *dst = group == 0 ? p.dq : p.dk;
    const long long stride = p.parts ? (long long)p.H * DK : group == 0 ? p.q_stride : p.k_stride;
    const int type = p.parts ? 0 : p.dtype;
    const bool odd = lane & 1;
#pragma unroll
    for (int i = 0; i < NT; i += 2) {
      float x[2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[e][j] = acc[i + e][j] * out1 * out2;
        if (DELTA && group == 2) {
          const float4 y = hand[(w4 * NT + i + e) * 32 + lane], z = hand[((4 + w4) * NT + i + e) * 32 + lane];
          x[e][0] += y.x + z.x; x[e][1] += y.y + z.y; x[e][2] += y.z + z.z; x[e][3] += y.w + z.w;
        }
      }
      // neighbouring lanes trade halves, so that each holds four columns of one of the two tiles
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float rx = __shfl_xor_sync(0xFFFFFFFFu, odd ? x[0][2 * h] : x[1][2 * h], 1);
        const float ry = __shfl_xor_sync(0xFFFFFFFFu, odd ? x[0][2 * h + 1] : x[1][2 * h + 1], 1);
        const float4 y = odd ? make_float4(rx, ry, x[1][2 * h], x[1][2 * h + 1])
                             : make_float4(x[0][2 * h], x[0][2 * h + 1], rx, ry);
        const int t = m0 + g + 8 * h;
        if (t < n) {
          const long long at = (token0 + t) * stride + (long long)head * DK + 8 * (i + odd) + (t2 & 4);
          if (type == 0) *reinterpret_cast<float4 *>(static_cast<float *>(dst) + at) = y;
          else
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(dst) + at) =
                make_uint2(pack_as(type, y.x, y.y), pack_as(type, y.z, y.w));
        }
      }
    }
  }
  if (warp == 4) {
    // gates: two tokens a lane, sums over t >= r from the chunk's end
    float dsum = 0.0f;
    for (int i = 0; i < kGradThreads / 32; ++i) dsum += red[i];
    dsum = dsum * pow2(topDS / 2) * pow2(topDS - topDS / 2);
    double dG[2], x[2];
    float db[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      // (a token's columns are summed by the warps whose rows reach it)
      const float c = (colp[t] + colp[kChunk + t]) + (colp[2 * kChunk + t] + colp[3 * kChunk + t]);
      db[i] = fmaf(eC[t], kw[t], c + diagp[t]);
      // (the last state's part: its sum over all tokens and, in dG, less that of t >= r leave the tokens before r)
      x[i] = (double)be[t] * ((double)eC[t] * (double)kw[t]);
      dG[i] = (double)rowv[t] + (HALF ? (double)rowv[kChunk + t] : 0.0) - (double)be[t] * c +
              (double)eG[t] * (aq[t] - (DELTA ? ak[t] : 0.0f));
    }
    double run = dG[0] + dG[1], past = x[0] + x[1];
    for (int d = 1; d < 32; d <<= 1) {
      const double up = __shfl_down_sync(0xFFFFFFFFu, run, d), down = __shfl_up_sync(0xFFFFFFFFu, past, d);
      if (lane + d < 32) run += up;
      if (lane >= d) past += down;
    }
    past = __shfl_up_sync(0xFFFFFFFFu, past, 1);
    if (lane == 0) past = 0.0;
    const double end = (double)eG[kChunk - 1] * dsum, out[2] = {run + past + end, run - dG[0] + past + x[0] + end};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      if (t < n) {
        const long long at = (token0 + t) * p.H + head;
        // (a state that was dropped has no gradient through its decay: not even the rounding of the sums)
        p.dlog_alpha[at] = __ldg(p.log_alpha + at) < -1000.0f ? 0.0f : (float)out[i];
        p.dbeta[at] = db[i];
      }
    }
  }
}

// Sums the heads' parts of dq and dk where heads share q and k, in head order.  Memory bound: 8192
// tokens, 16 heads on 8, d_k = 128, bf16: 38 us, 4.4 TB/s.  (scan_grads adding its part to the last
// head's instead, heads of a group one behind the other: it took 497 us in place of 320.)
static __global__ void __launch_bounds__(256) scan_shared_kernel(const ScanParams p, const float *parts_q,
                                                                 const float *parts_k, int dk) {
  wait_before();
  const int hq = p.H / p.share, per = hq * (dk / 4);
  const long long n = (long long)p.n_slots * kChunk * per, all = 2 * n;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < all; i += (long long)gridDim.x * 256) {
    const bool second = i >= n;
    const long long j = second ? i - n : i, row = j / per;
    const int r = (int)(j % per), h = r / (dk / 4), c = (r % (dk / 4)) * 4;
    const longlong2 tokens = p.slot_tokens[row / kChunk];
    if (row % kChunk >= tokens.y) continue;
    const long long tok = tokens.x + row % kChunk;
    const float *src = (second ? parts_k : parts_q) + (tok * p.H + (long long)h * p.share) * dk + c;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int m = 0; m < p.share; ++m) {
      const float4 x = *reinterpret_cast<const float4 *>(src + (long long)m * dk);
      s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    const long long at = tok * (second ? p.k_stride : p.q_stride) + (long long)h * dk + c;
    store_pair(second ? p.dk : p.dq, p.dtype, at, s.x, s.y);
    store_pair(second ? p.dk : p.dq, p.dtype, at + 2, s.z, s.w);
  }
}

// -------------------------------------------------------------------------------------
// scan_recurrent: short sequences, token by token in fp32
// -------------------------------------------------------------------------------------
// Grid (sequence * H + head, group of value rows).  d_k/16 lanes share a value row (16 of its columns each, in
// groups of 4 so that the lanes' 16-byte accesses are contiguous) and two rows are in flight per
// lane, their arithmetic as packed pairs.  q, k, v and the gates of kRecTokens tokens at a time pass through
// shared memory as fp32, while the state's loads are under way.  Memory bound for a few tokens (the
// state in and out): 64 sequences of up to 5, 32 heads of 128 x 128: 61 us, 4.6 TB/s; then by issue,
// 8.5 us a token there.  Seven CTAs per SM (72 registers) took 63 us a call where eight
// took 65.
constexpr int kRecThreads = 128, kRecRows = 2, kRecTokens = 8;

template <int DK, bool DELTA>
__global__ void __launch_bounds__(kRecThreads, 7) scan_recurrent_kernel(const ScanParams p) {
  constexpr int LPR = DK / 16, ROWS = kRecThreads / LPR * kRecRows;
  __shared__ float4 sk[kRecTokens][DK / 4], sq[kRecTokens][DK / 4];
  __shared__ float sv[kRecTokens][ROWS];
  __shared__ float2 sg[kRecTokens];                   // a, b
  if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(p);
  const int tid = threadIdx.x, lir = tid % LPR, threads = blockDim.x;
  const int rows = threads / LPR * kRecRows;          // of this block
  const int row0 = blockIdx.y * rows, row = row0 + tid / LPR * kRecRows;
  const long long tile = blockIdx.x;
  const int head = (int)(tile % p.H), seq = (int)(tile / p.H);
  const bool live = row < p.d_v;                      // (d_v is even)
  const long long at = (tile * p.d_v + row) * DK + 4 * lir;
  float2 S[kRecRows][8];
#pragma unroll
  for (int r = 0; r < kRecRows; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (p.state_in && live) x = *reinterpret_cast<const float4 *>(p.state_in + at + r * DK + 4 * LPR * c);
      S[r][2 * c] = make_float2(x.x, x.y);
      S[r][2 * c + 1] = make_float2(x.z, x.w);
    }
  long long start;
  int len;
  seq_range(p, seq, start, len);
  const long long qo = (long long)(head / p.share) * DK;
  for (int t0 = 0; t0 < len; t0 += kRecTokens) {
    const int n = min(kRecTokens, len - t0);
    if (t0) __syncthreads();
    for (int i = tid; i < n * (DK / 4); i += threads) {
      const int t = i / (DK / 4), c = i % (DK / 4);
      float x[4];
      load4(p.k, p.dtype, (start + t0 + t) * p.k_stride + qo + 4 * c, x);
      sk[t][c] = make_float4(x[0], x[1], x[2], x[3]);
      load4(p.q, p.dtype, (start + t0 + t) * p.q_stride + qo + 4 * c, x);
      sq[t][c] = make_float4(x[0], x[1], x[2], x[3]);
    }
    const int vrows = min(rows, p.d_v - row0) / 4;    // (d_v and rows are multiples of 4)
    for (int i = tid; i < n * vrows; i += threads) {
      const int t = i / vrows, c = (i % vrows) * 4;
      float x[4];
      load4(p.v, p.dtype, (start + t0 + t) * p.v_stride + (long long)head * p.d_v + row0 + c, x);
#pragma unroll
      for (int e = 0; e < 4; ++e) sv[t][c + e] = x[e];
    }
    if (tid < n) {
      const long long g = (start + t0 + tid) * p.H + head;
      sg[tid] = make_float2(expf(__ldg(p.log_alpha + g)), __ldg(p.beta + g));
    }
    __syncthreads();
    for (int t = 0; t < n; ++t) {
      const float2 ab = sg[t], aa = make_float2(ab.x, ab.x);
      float2 k[8], q[8];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 x = sk[t][LPR * c + lir], y = sq[t][LPR * c + lir];
        k[2 * c] = make_float2(x.x, x.y); k[2 * c + 1] = make_float2(x.z, x.w);
        q[2 * c] = make_float2(y.x, y.y); q[2 * c + 1] = make_float2(y.z, y.w);
      }
      float u[kRecRows], o[kRecRows];
#pragma unroll
      for (int r = 0; r < kRecRows; ++r) {
        float2 y = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          S[r][e] = __fmul2_rn(S[r][e], aa);
          if (DELTA) y = __ffma2_rn(S[r][e], k[e], y);
        }
        u[r] = y.x + y.y;
      }
      if (DELTA)
#pragma unroll
        for (int d = 1; d < LPR; d <<= 1)
#pragma unroll
          for (int r = 0; r < kRecRows; ++r) u[r] += __shfl_xor_sync(0xFFFFFFFFu, u[r], d);
#pragma unroll
      for (int r = 0; r < kRecRows; ++r) {
        const float w = ab.y * (sv[t][tid / LPR * kRecRows + r] - u[r]);
        const float2 ww = make_float2(w, w);
        float2 y = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          S[r][e] = __ffma2_rn(ww, k[e], S[r][e]);
          y = __ffma2_rn(S[r][e], q[e], y);
        }
        o[r] = y.x + y.y;
      }
#pragma unroll
      for (int d = 1; d < LPR; d <<= 1)
#pragma unroll
        for (int r = 0; r < kRecRows; ++r) o[r] += __shfl_xor_sync(0xFFFFFFFFu, o[r], d);
      if (live && lir == 0)
        store_pair(p.o, p.dtype, (start + t0 + t) * p.o_stride + (long long)head * p.d_v + row, o[0], o[1]);
    }
  }
  if (p.state_out && live)
#pragma unroll
    for (int r = 0; r < kRecRows; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<float4 *>(p.state_out + at + r * DK + 4 * LPR * c) =
            make_float4(S[r][2 * c].x, S[r][2 * c].y, S[r][2 * c + 1].x, S[r][2 * c + 1].y);
}

using ScanFn = void (*)(ScanParams);
// kernels of one key width
struct ScanKernels {
  ScanFn prep[2][2][2];                // [np - 1][delta][backward]
  ScanFn walk[2][2][kWalkKinds];       // [np - 1][delta][WalkKind]
  ScanFn grads[2][2];
};
// Warps that share a block's state: half a 16-column state has no whole k-step.
constexpr int state_warps(int dk) { return dk >= 32 ? 2 : 1; }

}  // namespace scan
}  // namespace lores
