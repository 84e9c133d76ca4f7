// lores_scan.cuh -- device side of the state scan and its backward pass (sm_100a).
//
// The scan runs the decode step's recurrence, without its quantizer, over packed sequences:
//   S'  = a_t S_{t-1},  E_t = v_t - d S' k_t,  S_t = S' + b_t E_t k_t^T,  o_t = S_t q_t
// (General recurrence form; a_t = exp(log_alpha_t), d = delta).  Sequences are cut into
// chunks of kChunk = 64 tokens.  With G_t the sum of log_alpha over the chunk up to t, S0 the
// state at its start, rows t of Q, K, V, E its tokens and dec_ts = exp(G_t - G_s):
//   L_ts = dec_ts k_t.k_s (s < t)      P_ts = dec_ts q_t.k_s b_s (s <= t)
//   Tm   = (I + d L diag(b))^-1        E = Tm (V - d diag(e^G) K S0^T)
//   O    = diag(e^G) Q S0^T + P E      S_C = e^{G_C} S0 + (diag(w) E)^T K,  w = b e^{G_C - G}
// Only S0 -> S_C is sequential, so the work is split in two:
//   scan_prep     all chunks at once: gates, Tm, P, Kt = -d Tm diag(e^G) K (and, for the
//                 backward pass, Z = P Tm and Kb = Tm^T diag(w) K)
//   scan_chain    per (sequence, head, block of value rows): E^T = S0 Kt^T + (Tm V)^T, O^T and
//                 S_C, chunk after chunk.  Value rows are independent (as in the decode
//                 step), so one or two warps own 16 of them, keep S [16][d_k] in their
//                 accumulators and feed it back as the next product's left operand
//                 without leaving registers.
// Backward, D = dL/dS_C:
//   R   = Z^T dO + Kb D^T (= dV)       D0 = e^{G_C} D + (diag(e^G) dO)^T Q - d (diag(e^G) R)^T K
//   scan_reverse  the same walk backwards over R and D;
//   scan_grads    all chunks at once: dQ, dK and the gates' gradients from S0, D, E, R.
//
// Precision.  Sums and states are fp32; the tensor cores multiply fp16.  An fp32 operand x is given
// as two fp16 planes, hi = fp16(x) and lo = fp16(x - hi): 22 bits of significand, or an absolute
// 2^-25 where lo is subnormal.  A product is hi hi + hi lo + lo hi; 16-bit inputs are
// exact as one plane.  fp16's range is met by powers of two that leave the result exactly:
// K and Q are divided by one scale per chunk and head (largest entry in [1, 2)), the walks'
// operands by one scale per 16 value rows and chunk (largest entry of S0 and V, or of D and
// dO, in [2^6, 2^7)).  The error of states and gradients stays near 1e-7; two bf16
// planes would leave 3e-6 to 1e-5, one fp16 plane 2e-4.  Products that only reach a 16-bit
// output (Q S0^T and P E) use one plane.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace lores {
namespace scan {

constexpr int kChunk = 64;
constexpr int kLdC = kChunk + 8;       // row stride of a [64][64] plane in shared memory (rows 16
                                       // bytes apart modulo 128: the 8 rows that ldmatrix
                                       // reads fall into different banks)
constexpr int kPrepThreads = 128;
constexpr int kGradThreads = 256;
constexpr unsigned kFlagOffsets = 1u;  // a sequence's offsets were not 0 <= a <= b <= total

struct ScanParams {
  int n_seq, H, share, d_v, dvp, dtype, n_slots, max_len, stages;
  int rb;                              // walks: blocks of 16 value rows per CTA
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
  // workspace, records of one (slot, head); khat, qhat of one (slot, q/k head)
  float *gates;                        // kGateFloats
  __half *khat, *qhat;                 // [NP][64][d_k], divided by their scales
  __half *kt, *kb;                     // [2][64][d_k]
  __half *tm, *pp, *z;                 // [2][64][64]
  __half *s0, *dd;                     // [2][dvp][d_k]
  __half *et, *rt;                     // [2][dvp][64]
  float *fscale, *bscale;              // [dvp/16]: scales of s0 and et, of dd and rt
  // backward
  const float *d_state_out;
  float *d_state_in;
  void *dv, *dq, *dk;                  // dq, dk: the caller's, or fp32 parts [total][H][d_k]
  int parts;                           // dq, dk are parts
  float *dlog_alpha, *dbeta;
};

// Record of a chunk and head: e^G, w, b, e^(G_C - G) [64] each, G [64] (double), scales of K and Q
constexpr int kGateFloats = 4 * kChunk + 2 * kChunk + 4;
constexpr int kGateScales = 6 * kChunk;

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

// The first token of a slot's chunk and its number of tokens (0: the slot is not used).
__device__ __forceinline__ int slot_tokens(const ScanParams &p, int slot, long long &token0) {
  int lo = 0, hi = p.n_seq - 1;
  if (!p.offsets) {
    const long long each = p.total / p.n_seq;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (slot_base(each * mid, mid) <= slot) lo = mid; else hi = mid - 1;
    }
  } else {
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (slot_base(__ldg(p.offsets + mid), mid) <= slot) lo = mid; else hi = mid - 1;
    }
  }
  long long start;
  int len;
  seq_range(p, lo, start, len);
  const long long first = (long long)(slot - slot_base(start, lo)) * kChunk;
  if (first < 0 || first >= len) return 0;
  token0 = start + first;
  return (int)min((long long)kChunk, len - first);
}

// Whether a token belongs to a sequence (the others' rows are left as they were).
__device__ __forceinline__ bool token_used(const ScanParams &p, long long tok) {
  if (!p.offsets) return true;
  int lo = 0, hi = p.n_seq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(p.offsets + mid) <= tok) lo = mid; else hi = mid - 1;
  }
  long long start;
  int len;
  seq_range(p, lo, start, len);
  return tok >= start && tok < start + len;
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
// fragments
// -------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_addr(const void *x) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(x));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const void *row) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_addr(row)));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], const void *row) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_addr(row)));
}
__device__ __forceinline__ void stsm4t(void *row, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(smem_addr(row)),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
// Fragment loads of 16x16 blocks from row-major shared memory with row stride ld.
//   right operand, two column tiles (r[0], r[1]: columns n0..n0+7; r[2], r[3]: n0+8..):
//     b_rows:  stored [n][k]      b_cols: stored [k][n]
//   left operand:
//     a_rows:  stored [m][k]      a_cols: stored [k][m]
__device__ __forceinline__ void b_rows(uint32_t (&r)[4], const __half *x, int ld, int n0, int k0, int lane) {
  ldsm4(r, x + (n0 + ((lane >> 4) << 3) + (lane & 7)) * ld + k0 + (((lane >> 3) & 1) << 3));
}
__device__ __forceinline__ void b_cols(uint32_t (&r)[4], const __half *x, int ld, int k0, int n0, int lane) {
  ldsm4t(r, x + (k0 + (((lane >> 3) & 1) << 3) + (lane & 7)) * ld + n0 + ((lane >> 4) << 3));
}
__device__ __forceinline__ void a_rows(uint32_t (&r)[4], const __half *x, int ld, int m0, int k0, int lane) {
  ldsm4(r, x + (m0 + (((lane >> 3) & 1) << 3) + (lane & 7)) * ld + k0 + ((lane >> 4) << 3));
}
__device__ __forceinline__ void a_cols(uint32_t (&r)[4], const __half *x, int ld, int k0, int m0, int lane) {
  ldsm4t(r, x + (k0 + ((lane >> 4) << 3) + (lane & 7)) * ld + m0 + (((lane >> 3) & 1) << 3));
}

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
// bits (1 for zero, limits at the ends of the range), and its inverse.
__device__ __forceinline__ float scale_of(unsigned bits, int up, float &inv) {
  int e = (int)(bits >> 23) - up;
  e = bits == 0u ? 127 : max(1, min(253, e));
  inv = __uint_as_float((unsigned)(254 - e) << 23);
  return __uint_as_float((unsigned)e << 23);
}
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
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A [ROWS][COLS] plane of a record (dense rows) into shared rows of LD elements.
template <int ROWS, int COLS, int LD>
__device__ __forceinline__ void copy_plane(__half *dst, const __half *src, int tid, int threads) {
  constexpr int per = COLS / 8;
#pragma unroll 4
  for (int i = tid; i < ROWS * per; i += threads)
    cp16(dst + (i / per) * LD + (i % per) * 8, src + i * 8, true);
}
// The lower triangle of a [64][64] plane, by 16x16 blocks (the others are not read).
__device__ __forceinline__ void copy_lower(__half *dst, const __half *src, int tid, int threads) {
#pragma unroll 4
  for (int i = tid; i < kChunk * 8; i += threads) {
    const int r = i >> 3, c = i & 7;
    if ((c >> 1) <= (r >> 4)) cp16(dst + r * kLdC + c * 8, src + r * kChunk + c * 8, true);
  }
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

__device__ __forceinline__ void store_as(void *base, int dtype, long long i, float x) {
  if (dtype == 0) static_cast<float *>(base)[i] = x;
  else if (dtype == 1) static_cast<__nv_bfloat16 *>(base)[i] = __float2bfloat16_rn(x);
  else static_cast<__half *>(base)[i] = __float2half_rn(x);
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
// 8 entries of a row of the caller's tensor.
__device__ __forceinline__ void load8(const void *src, int dtype, long long i, bool by16, float (&x)[8]) {
  if (dtype != 0 && by16) {
    const uint4 w = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(src) + i));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = pair_of(u[e], dtype);
      x[2 * e] = f.x;
      x[2 * e + 1] = f.y;
    }
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float y[4];
    load4(src, dtype, i + 4 * h, y);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[4 * h + e] = y[e];
  }
}

// -------------------------------------------------------------------------------------
// scan_prep
// -------------------------------------------------------------------------------------
// Grid (slot, head), 4 warps; warp w owns rows 16w .. 16w+15 of every [64][.] result, and only
// blocks on and below the diagonal are formed.  Tm = (I + A)^-1, A = L diag(b), by 16x16 blocks:
// the four diagonal blocks by forward substitution in fp32 (one lane per column); then warp j
// forms block column j downwards, X_ij = -X_ii sum_{j <= k < i} A_ik X_kj, as
// X_ij^T = -(sum_k X_kj^T A_ik^T) X_ii^T, so that every X_kj^T is an accumulator that becomes the next
// product's left operand in place.
constexpr int kLdF = kChunk + 2;       // row stride of the fp32 matrix in shared memory
constexpr int kLdX = 24;               // row stride of a [16][16] plane

struct PrepLayout {
  int k, q, x, xd, f, bytes;           // q: also the planes of A (48 rows) once Q is used
};
__host__ __device__ constexpr PrepLayout prep_layout(int dk, int np) {
  PrepLayout l{};
  const int tile = np * kChunk * (dk + 8) * 2, planes = 2 * 48 * kLdC * 2;
  l.k = 0;
  l.q = tile;
  l.x = l.q + (tile > planes ? tile : planes);
  l.xd = l.x + kChunk * kLdF * 4;
  l.f = l.xd + 4 * 2 * 16 * kLdX * 2;
  l.bytes = l.f + (4 * kChunk + 2 * kChunk + 16) * 4;
  return l;
}

// Rows of K or Q of a chunk: their scale (left in *scale), planes in shared memory, and in the
// workspace where `out` is given.
template <int DK, int NP>
__device__ __forceinline__ float stage_rows(const ScanParams &p, const void *src, long long stride, long long token0,
                                            int qh, int n, __half *dst, __half *out, unsigned *red, int tid) {
  constexpr int LD = DK + 8, PER = DK / 8;
  unsigned m = 0;
  for (int i = tid; i < kChunk * PER; i += kPrepThreads) {
    const int r = i / PER, c = (i % PER) * 8;
    if (r < n) {
      float x[8];
      load8(src, p.dtype, (token0 + r) * stride + (long long)qh * DK + c, p.qk16, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, abs_bits(x[e]));
    }
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((tid & 31) == 0) red[tid >> 5] = m;
  __syncthreads();
  m = max(max(red[0], red[1]), max(red[2], red[3]));
  float inv;
  const float scale = scale_of(m, 0, inv);
  for (int i = tid; i < kChunk * PER; i += kPrepThreads) {
    const int r = i / PER, c = (i % PER) * 8;
    float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (r < n) load8(src, p.dtype, (token0 + r) * stride + (long long)qh * DK + c, p.qk16, x);
    uint4 hi, lo;
    split2(x[0] * inv, x[1] * inv, hi.x, lo.x);
    split2(x[2] * inv, x[3] * inv, hi.y, lo.y);
    split2(x[4] * inv, x[5] * inv, hi.z, lo.z);
    split2(x[6] * inv, x[7] * inv, hi.w, lo.w);
    *reinterpret_cast<uint4 *>(dst + r * LD + c) = hi;
    if (NP == 2) *reinterpret_cast<uint4 *>(dst + kChunk * LD + r * LD + c) = lo;
    if (out) {
      *reinterpret_cast<uint4 *>(out + r * DK + c) = hi;
      if (NP == 2) *reinterpret_cast<uint4 *>(out + kChunk * DK + r * DK + c) = lo;
    }
  }
  return scale;
}

// Accumulators of 16 rows [m0 ..] x COLS as planes of a record with row length COLS.
template <int TILES>
__device__ __forceinline__ void store_planes(__half *dst, long long plane, int cols, int m0, const float (&c)[TILES][4],
                                             int tiles, int lane) {
  const int g = lane >> 2, t2 = (lane & 3) * 2;
#pragma unroll
  for (int i = 0; i < TILES; ++i)
    if (i < tiles)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t hi, lo;
        split2(c[i][2 * h], c[i][2 * h + 1], hi, lo);
        const long long at = (long long)(m0 + g + 8 * h) * cols + 8 * i + t2;
        *reinterpret_cast<uint32_t *>(dst + at) = hi;
        *reinterpret_cast<uint32_t *>(dst + plane + at) = lo;
      }
}

template <int DK, int NP, bool DELTA, bool BWD>
__global__ void __launch_bounds__(kPrepThreads, DK <= 128 && NP == 1 ? 4 : 2) scan_prep_kernel(const ScanParams p) {
  constexpr int LD = DK + 8;
  constexpr PrepLayout l = prep_layout(DK, NP);
  extern __shared__ __align__(16) uint8_t smem[];
  __half *K = reinterpret_cast<__half *>(smem + l.k), *Q = reinterpret_cast<__half *>(smem + l.q);
  __half *A16 = Q;                                                  // [2][48][kLdC]: rows 16..63 of A
  float *X = reinterpret_cast<float *>(smem + l.x);                 // diagonal blocks of A, then Tm
  __half *XD = reinterpret_cast<__half *>(smem + l.xd);             // [4][2][16][kLdX]: X_ii
  double *G = reinterpret_cast<double *>(smem + l.f);
  float *eG = reinterpret_cast<float *>(G + kChunk), *w = eG + kChunk, *be = w + kChunk;
  unsigned *red = reinterpret_cast<unsigned *>(be + 2 * kChunk);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t2 = (lane & 3) * 2;
  const int slot = blockIdx.x, head = blockIdx.y;
  if (slot == 0 && head == 0) check_offsets(p);
  long long token0 = 0;
  const int n = slot_tokens(p, slot, token0);
  if (n == 0) return;
  const int qh = head / p.share, hq = p.H / p.share;
  const long long rec = (long long)slot * p.H + head, qrec = (long long)slot * hq + qh;
  const bool mine = head % p.share == 0;           // the first of the heads that share K and Q keeps them
  float *gates = p.gates + rec * kGateFloats;
  if (warp == 0) {
    // Sums of log_alpha in 64 bits, so that the differences below keep their digits behind a
    // strong decay.  Below -1000 exp() is 0 in fp32 whatever follows, so -inf (a = 0) is
    // held there and G stays finite.
    double a[2], run;
    float b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      const long long at = (token0 + t) * p.H + head;
      float la = t < n ? __ldg(p.log_alpha + at) : 0.0f;
      if (la < -1000.0f) la = -1000.0f;
      a[i] = la;
      b[i] = t < n ? __ldg(p.beta + at) : 0.0f;
    }
    run = a[0] + a[1];
    for (int d = 1; d < 32; d <<= 1) {
      const double up = __shfl_up_sync(0xFFFFFFFFu, run, d);
      if (lane >= d) run += up;
    }
    const double end = __shfl_sync(0xFFFFFFFFu, run, 31);
    const double Gt[2] = {run - a[1], run};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      const float e = expf((float)Gt[i]), c = expf((float)(end - Gt[i]));
      G[t] = Gt[i];
      eG[t] = e; be[t] = b[i]; w[t] = b[i] * c;
      gates[t] = e; gates[kChunk + t] = b[i] * c; gates[2 * kChunk + t] = b[i]; gates[3 * kChunk + t] = c;
      reinterpret_cast<double *>(gates + 4 * kChunk)[t] = Gt[i];
    }
  }
  const float sk = stage_rows<DK, NP>(p, p.k, p.k_stride, token0, qh, n, K,
                                      mine ? p.khat + qrec * (NP * kChunk * DK) : nullptr, red, tid);
  const float sq = stage_rows<DK, NP>(p, p.q, p.q_stride, token0, qh, n, Q,
                                      mine ? p.qhat + qrec * (NP * kChunk * DK) : nullptr, red + 4, tid);
  if (tid == 0) {
    gates[kGateScales] = sk;
    gates[kGateScales + 1] = sq;
  }
  __syncthreads();

  const int m0 = warp * 16;
  float P[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) P[i][j] = 0.0f;
  {
    float A[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) A[i][j] = 0.0f;
#pragma unroll 2
    for (int ks = 0; ks < DK / 16; ++ks) {
      uint32_t ak[NP][4], aq[NP][4];
#pragma unroll
      for (int c = 0; c < NP; ++c) {
        if (DELTA) a_rows(ak[c], K + c * kChunk * LD, LD, m0, ks * 16, lane);
        a_rows(aq[c], Q + c * kChunk * LD, LD, m0, ks * 16, lane);
      }
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        if (np <= warp) {
          uint32_t b[4];
          b_rows(b, K, LD, np * 16, ks * 16, lane);
#pragma unroll
          for (int c = 0; c < NP; ++c) {
            if (DELTA) mma2(A[2 * np], A[2 * np + 1], ak[c], b);
            mma2(P[2 * np], P[2 * np + 1], aq[c], b);
          }
          if (NP == 2) {
            b_rows(b, K + kChunk * LD, LD, np * 16, ks * 16, lane);
            if (DELTA) mma2(A[2 * np], A[2 * np + 1], ak[0], b);
            mma2(P[2 * np], P[2 * np + 1], aq[0], b);
          }
        }
      }
    }
    __syncthreads();                   // Q's tile becomes A's planes
    // P (over the scale of Q) and, strictly below the diagonal, A
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i / 2 <= warp) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int t = m0 + g + 8 * h, s = 8 * i + t2;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float dec = s + j <= t ? expf((float)(G[t] - G[s + j])) * be[s + j] * sk : 0.0f;
            P[i][2 * h + j] = s + j <= t ? P[i][2 * h + j] * dec : 0.0f;
            if (DELTA) A[i][2 * h + j] = s + j < t ? A[i][2 * h + j] * dec * sk : 0.0f;
          }
          if (DELTA) {
            if (i / 2 == warp) {
              X[t * kLdF + s] = A[i][2 * h];
              X[t * kLdF + s + 1] = A[i][2 * h + 1];
            } else {
              uint32_t hi, lo;
              split2(A[i][2 * h], A[i][2 * h + 1], hi, lo);
              *reinterpret_cast<uint32_t *>(A16 + (t - 16) * kLdC + s) = hi;
              *reinterpret_cast<uint32_t *>(A16 + 48 * kLdC + (t - 16) * kLdC + s) = lo;
            }
          }
        }
      }
    }
  }
  if (!BWD || !DELTA) {
    // 16-bit outputs need one plane of P
    __half *pp = p.pp + rec * (2 * kChunk * kChunk);
    if (NP == 2 || BWD) store_planes<8>(pp, kChunk * kChunk, kChunk, m0, P, 2 * warp + 2, lane);
    else
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i / 2 <= warp)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            *reinterpret_cast<uint32_t *>(pp + (m0 + g + 8 * h) * kChunk + 8 * i + t2) = pack2(P[i][2 * h], P[i][2 * h + 1]);
  }
  if (!DELTA) return;
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
      __half *d = XD + warp * (2 * 16 * kLdX);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        B[r * kLdF + c] = x[r];
        const __half hi = __float2half_rn(x[r]);
        d[r * kLdX + c] = hi;
        d[16 * kLdX + r * kLdX + c] = __float2half_rn(x[r] - __half2float(hi));
      }
    }
  }
  __syncthreads();
  {
    // block column `warp`: yh, yl[k] = planes of X_kj^T
    uint32_t yh[4][4], yl[4][4];
    {
      // X_jj^T as a left operand: element (m, k) = X_jj[k][m], read transposed
      const __half *d = XD + warp * (2 * 16 * kLdX);
      a_cols(yh[0], d, kLdX, 0, 0, lane);
      a_cols(yl[0], d + 16 * kLdX, kLdX, 0, 0, lane);
    }
#pragma unroll
    for (int di = 1; di < 4; ++di) {
      const int i = warp + di;
      if (i < 4) {
        float z0[4] = {0, 0, 0, 0}, z1[4] = {0, 0, 0, 0};
#pragma unroll
        for (int dk = 0; dk < di; ++dk) {
          uint32_t b[4];
          b_rows(b, A16, kLdC, 16 * i - 16, 16 * (warp + dk), lane);
          mma2(z0, z1, yh[dk], b);
          mma2(z0, z1, yl[dk], b);
          b_rows(b, A16 + 48 * kLdC, kLdC, 16 * i - 16, 16 * (warp + dk), lane);
          mma2(z0, z1, yh[dk], b);
        }
        uint32_t zh[4], zl[4], b[4];
        split_tiles(z0, z1, -1.0f, zh, zl);
        float y0[4] = {0, 0, 0, 0}, y1[4] = {0, 0, 0, 0};
        const __half *d = XD + i * (2 * 16 * kLdX);
        b_rows(b, d, kLdX, 0, 0, lane);
        mma2(y0, y1, zh, b);
        mma2(y0, y1, zl, b);
        b_rows(b, d + 16 * kLdX, kLdX, 0, 0, lane);
        mma2(y0, y1, zh, b);
        split_tiles(y0, y1, yh[di & 3], yl[di & 3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {   // y[c][r] -> X[16 i + r][16 warp + c]
          const int c = g + 8 * (j >> 1), r = t2 + (j & 1);
          X[(16 * i + r) * kLdF + m0 + c] = y0[j];
          X[(16 * i + 8 + r) * kLdF + m0 + c] = y1[j];
        }
      }
    }
  }
  __syncthreads();

  // planes of Tm (blocks on and below the diagonal)
  __half *tm = p.tm + rec * (2 * kChunk * kChunk);
  for (int i = tid; i < kChunk * 8; i += kPrepThreads) {
    const int r = i >> 3, c = (i & 7) * 8;
    if ((c >> 4) <= (r >> 4)) {
      uint4 hi, lo;
      const float *x = X + r * kLdF + c;
      split2(x[0], x[1], hi.x, lo.x);
      split2(x[2], x[3], hi.y, lo.y);
      split2(x[4], x[5], hi.z, lo.z);
      split2(x[6], x[7], hi.w, lo.w);
      *reinterpret_cast<uint4 *>(tm + r * kChunk + c) = hi;
      *reinterpret_cast<uint4 *>(tm + kChunk * kChunk + r * kChunk + c) = lo;
    }
  }
  // Kt = -Tm diag(e^G) K: rows t of this warp, s blocks up to its own.  Two halves of the columns, so
  // that the accumulators leave room for four CTAs per SM.
  constexpr int HALVES = DK >= 64 ? 2 : 1, HT = DK / 8 / HALVES;
#pragma unroll 1
  for (int half = 0; half < HALVES; ++half) {
    float acc[HT][4];
#pragma unroll
    for (int i = 0; i < HT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      if (ks <= warp) {
        uint32_t ah[4], al[4], b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int t = m0 + g + 8 * (q & 1), s = ks * 16 + t2 + 8 * (q >> 1);
          split2(-X[t * kLdF + s] * eG[s] * sk, -X[t * kLdF + s + 1] * eG[s + 1] * sk, ah[q], al[q]);
        }
#pragma unroll
        for (int np = 0; np < HT / 2; ++np) {
          const int c0 = half * (DK / HALVES) + np * 16;
          b_cols(b, K, LD, ks * 16, c0, lane);
          mma2(acc[2 * np], acc[2 * np + 1], ah, b);
          mma2(acc[2 * np], acc[2 * np + 1], al, b);
          if (NP == 2) {
            b_cols(b, K + kChunk * LD, LD, ks * 16, c0, lane);
            mma2(acc[2 * np], acc[2 * np + 1], ah, b);
          }
        }
      }
    }
    store_planes<HT>(p.kt + rec * (2 * kChunk * DK) + half * (DK / HALVES), kChunk * DK, DK, m0, acc, HT, lane);
  }
  if (!BWD) return;
  // Kb = Tm^T diag(w) K: rows s of this warp, t blocks from its own on
#pragma unroll 1
  for (int half = 0; half < HALVES; ++half) {
    float acc[HT][4];
#pragma unroll
    for (int i = 0; i < HT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      if (ks >= warp) {
        uint32_t ah[4], al[4], b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int s = m0 + g + 8 * (q & 1), t = ks * 16 + t2 + 8 * (q >> 1);
          split2(X[t * kLdF + s] * w[t] * sk, X[(t + 1) * kLdF + s] * w[t + 1] * sk, ah[q], al[q]);
        }
#pragma unroll
        for (int np = 0; np < HT / 2; ++np) {
          const int c0 = half * (DK / HALVES) + np * 16;
          b_cols(b, K, LD, ks * 16, c0, lane);
          mma2(acc[2 * np], acc[2 * np + 1], ah, b);
          mma2(acc[2 * np], acc[2 * np + 1], al, b);
          if (NP == 2) {
            b_cols(b, K + kChunk * LD, LD, ks * 16, c0, lane);
            mma2(acc[2 * np], acc[2 * np + 1], ah, b);
          }
        }
      }
    }
    store_planes<HT>(p.kb + rec * (2 * kChunk * DK) + half * (DK / HALVES), kChunk * DK, DK, m0, acc, HT, lane);
  }
  // Z = P Tm (over the scale of Q): rows t of this warp; block (r, s) of Tm is zero for s > r
  {
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
    store_planes<8>(p.z + rec * (2 * kChunk * kChunk), kChunk * kChunk, kChunk, m0, acc, 2 * warp + 2, lane);
  }
}

// -------------------------------------------------------------------------------------
// scan_chain
// -------------------------------------------------------------------------------------
// Grid (sequence * H + head, group of p.rb blocks of 16 value rows).  NH warps share a block: warp h
// holds the state's columns [h d_k/NH, (h+1) d_k/NH) and forms, over its columns, a part of S0 Kt^T
// and S0 Q^T for all 64 tokens; the parts are added through shared memory, one barrier of the
// NH warps per chunk; then each warp finishes O for its own 64/NH tokens and S for its own
// columns.  (NH = 2 halves the chain from chunk to chunk where there are few blocks.)  Two more
// warps fetch the next chunk's tiles meanwhile (two stages where they fit).
// SAVE: the backward pass's recomputation, which keeps the planes of S0 and E of every chunk;
// otherwise o and the last state are written.
constexpr int kLoadWarps = 2;
constexpr int kWalkWarps = 4;          // compute warps of a CTA, at most

struct WalkLayout {                    // byte offsets inside one stage; `part` after the stages
  int kt, k, q, tm, pp, v, gates, bytes, part;
};
// elements of a token row of the V (or dO) tile
__host__ __device__ constexpr int tile_ld(int np, int rb) { return 16 * rb + (np == 2 ? 4 : 8); }

// what = 0: forward, 1: recomputation, 2: reverse
__host__ __device__ inline WalkLayout walk_layout(int dk, int np, int rb, int nh, bool delta, int what) {
  const int tile = kChunk * (dk + 8) * 2, sq = kChunk * kLdC * 2;
  WalkLayout l{};
  int at = 0;
  l.kt = at; at += delta ? 2 * tile : 0;                       // Kt or Kb
  l.k = at; at += np * tile;
  l.q = at; at += what != 1 ? np * tile : 0;
  l.tm = at; at += what == 2 || delta ? 2 * sq : 0;            // Tm or Z
  l.pp = at; at += what == 0 ? np * sq : 0;
  l.v = at; at += kChunk * tile_ld(np, rb) * (np == 2 ? 4 : 2);
  l.gates = at; at += 2 * kChunk * 4 + 16;
  l.bytes = (at + 15) / 16 * 16;
  // parts of E (32 floats a lane) and, forward, of O for the others' tokens; maxima
  l.part = nh == 1 ? 0 : rb * nh * 32 * (32 + (what == 0 ? 32 - 32 / nh : 0)) * 4;
  return l;
}

// The state rows a thread holds: rows r0 and r0 + 8, columns c0 + 8 i + t2, +1.
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
template <int NTH>
__device__ __forceinline__ unsigned max_bits(const float (&S)[NTH][4]) {
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < NTH; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max(m, abs_bits(S[i][j]));
  return m;
}

// The tile of V (or dO) as left operands V^T: x[ks][2 q], x[ks][2 q + 1] are the two entries of
// register q of k-step ks (tokens 16 ks ..) as fp32 values of the caller's type.
template <int NP>
__device__ __forceinline__ void load_tokens(float (&x)[4][8], const uint8_t *tile, int ld, int col0, int dtype,
                                            int lane) {
  const int g = lane >> 2, t2 = (lane & 3) * 2;
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    if (NP == 1) {
      uint32_t a[4];
      a_cols(a, reinterpret_cast<const __half *>(tile), ld, ks * 16, col0, lane);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 f = pair_of(a[q], dtype);
        x[ks][2 * q] = f.x;
        x[ks][2 * q + 1] = f.y;
      }
    } else {
      const float *f = reinterpret_cast<const float *>(tile);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          x[ks][2 * q + e] = f[(ks * 16 + 8 * (q >> 1) + t2 + e) * ld + col0 + g + 8 * (q & 1)];
    }
  }
}

// Writes OT tiles (tokens 8 (tile0 + i) .., 16 value rows) times `by` to token rows of the
// caller's tensor, through the warp's part of the V tile so that rows leave in 16-byte
// pieces.
template <int NP, int OT>
__device__ __forceinline__ void store_tokens(const float (&O)[OT][4], float by, uint8_t *tile, int ld, int col0, int tile0,
                                             void *dst, int dtype, long long stride, long long token0, int n, int col,
                                             int have, bool by16, int lane) {
  const int g = lane >> 2, t2 = (lane & 3) * 2;
  if (NP == 1) {
    uint16_t *sm = reinterpret_cast<uint16_t *>(tile);
#pragma unroll
    for (int i = 0; i < OT / 2; ++i) {
      uint32_t r[4];
      r[0] = pack_as(dtype, O[2 * i][0] * by, O[2 * i][1] * by);
      r[1] = pack_as(dtype, O[2 * i][2] * by, O[2 * i][3] * by);
      r[2] = pack_as(dtype, O[2 * i + 1][0] * by, O[2 * i + 1][1] * by);
      r[3] = pack_as(dtype, O[2 * i + 1][2] * by, O[2 * i + 1][3] * by);
      const int tok = 8 * (tile0 + 2 * i + (lane >> 4)) + (lane & 7);
      stsm4t(sm + tok * ld + col0 + 8 * ((lane >> 3) & 1), r);
    }
    __syncwarp();
    uint16_t *out = static_cast<uint16_t *>(dst);
#pragma unroll
    for (int i = 0; i < OT / 2; ++i) {
      const int e = i * 32 + lane, tok = 8 * tile0 + (e >> 1), c = (e & 1) * 8;
      const uint4 x = *reinterpret_cast<const uint4 *>(sm + tok * ld + col0 + c);
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
    for (int i = 0; i < OT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        sm[(8 * (tile0 + i) + t2 + (j & 1)) * ld + col0 + g + 8 * (j >> 1)] = O[i][j] * by;
    __syncwarp();
    float *out = static_cast<float *>(dst);
#pragma unroll
    for (int i = 0; i < OT; ++i) {
      const int e = i * 32 + lane, tok = 8 * tile0 + (e >> 2), c = (e & 3) * 4;
      const float4 x = *reinterpret_cast<const float4 *>(sm + tok * ld + col0 + c);
      if (tok < n && c < have) *reinterpret_cast<float4 *>(out + (token0 + tok) * stride + col + c) = x;
    }
  }
}

__device__ __forceinline__ void block_barrier(int block, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + block), "r"(threads) : "memory");
}

template <int DK, int NP, bool DELTA, bool SAVE>
__device__ __forceinline__ void chain_fetch(const ScanParams &p, uint8_t *st, const WalkLayout &l, long long token0, int n,
                                            int slot, int head, int row0, int tid, int threads) {
  constexpr int LD = DK + 8, SIZE = NP == 2 ? 4 : 2;
  const long long rec = (long long)slot * p.H + head;
  const long long qrec = (long long)slot * (p.H / p.share) + head / p.share;
#pragma unroll
  for (int c = 0; c < 2; ++c)
    if (DELTA) {
      copy_plane<kChunk, DK, LD>(reinterpret_cast<__half *>(st + l.kt) + c * kChunk * LD,
                                 p.kt + (rec * 2 + c) * (kChunk * DK), tid, threads);
      copy_lower(reinterpret_cast<__half *>(st + l.tm) + c * kChunk * kLdC, p.tm + (rec * 2 + c) * (kChunk * kChunk),
                 tid, threads);
    }
#pragma unroll
  for (int c = 0; c < NP; ++c) {
    copy_plane<kChunk, DK, LD>(reinterpret_cast<__half *>(st + l.k) + c * kChunk * LD,
                               p.khat + (qrec * NP + c) * (kChunk * DK), tid, threads);
    if (!SAVE) {
      copy_plane<kChunk, DK, LD>(reinterpret_cast<__half *>(st + l.q) + c * kChunk * LD,
                                 p.qhat + (qrec * NP + c) * (kChunk * DK), tid, threads);
      copy_lower(reinterpret_cast<__half *>(st + l.pp) + c * kChunk * kLdC, p.pp + (rec * 2 + c) * (kChunk * kChunk),
                 tid, threads);
    }
  }
  copy_tokens<SIZE>(st + l.v, tile_ld(NP, p.rb),
                    static_cast<const uint8_t *>(p.v) + (token0 * p.v_stride + (long long)head * p.d_v + row0) * SIZE,
                    p.v_stride, min(16 * p.rb, p.dvp - row0), n, p.d_v - row0, p.v16, tid, threads);
  const float *gates = p.gates + rec * kGateFloats;
  for (int i = tid; i < 2 * kChunk / 4 + 1; i += threads)
    cp16(st + l.gates + 16 * i, i < 2 * kChunk / 4 ? gates + 4 * i : gates + kGateScales, true);
}

template <int DK, int NP, bool DELTA, bool SAVE, int NH>
__global__ void __launch_bounds__(32 * (kWalkWarps + kLoadWarps), 1) scan_chain_kernel(const ScanParams p) {
  constexpr int LD = DK + 8, DKH = DK / NH, NTH = DKH / 8, OT = 8 / NH;
  static_assert(NH == 1 || NH == 2, "E without the delta rule is laid out for these");
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t2 = (lane & 3) * 2;
  const int blk = warp / NH, h = NH == 1 ? 0 : warp % NH;
  const int seq = blockIdx.x / p.H, head = blockIdx.x % p.H, row0 = blockIdx.y * 16 * p.rb;
  const WalkLayout l = walk_layout(DK, NP, p.rb, NH, DELTA, SAVE ? 1 : 0);
  const int ldv = tile_ld(NP, p.rb);
  long long start;
  int len;
  seq_range(p, seq, start, len);
  const int chunks = (len + kChunk - 1) / kChunk, base = slot_base(start, seq);
  const bool loader = blk >= p.rb;
  const int r0 = row0 + blk * 16 + g, c0 = h * DKH;    // this thread's value rows: r0, r0 + 8
  const bool live = !loader && row0 + blk * 16 < p.dvp;
  float4 *part = reinterpret_cast<float4 *>(smem + p.stages * l.bytes);
  unsigned *tops = reinterpret_cast<unsigned *>(smem + p.stages * l.bytes + l.part);

  float S[NTH][4];
  load_state<NTH>(S, live ? p.state_in : nullptr, blockIdx.x, p.d_v, DK, r0, c0 + t2);
  unsigned top = __reduce_max_sync(0xFFFFFFFFu, max_bits<NTH>(S));
  if (NH > 1 && live && lane == 0) tops[warp] = top;

  const int ltid = tid - 32 * NH * p.rb, lthreads = 32 * kLoadWarps;
  auto fetch = [&](int c) {
    chain_fetch<DK, NP, DELTA, SAVE>(p, smem + (p.stages == 2 ? (c & 1) * l.bytes : 0), l,
                                     start + (long long)c * kChunk, min(kChunk, len - c * kChunk), base + c, head, row0,
                                     ltid, lthreads);
    cp_commit();
  };
  if (loader && chunks > 0) fetch(0);
  for (int c = 0; c < chunks; ++c) {
    uint8_t *st = smem + (p.stages == 2 ? (c & 1) * l.bytes : 0);
    if (loader) cp_wait<0>();
    __syncthreads();
    if (p.stages == 2 && loader && c + 1 < chunks) fetch(c + 1);
    if (live) {
      const __half *kt = reinterpret_cast<const __half *>(st + l.kt), *sk = reinterpret_cast<const __half *>(st + l.k);
      const __half *sq = reinterpret_cast<const __half *>(st + l.q), *tm = reinterpret_cast<const __half *>(st + l.tm);
      const __half *pp = reinterpret_cast<const __half *>(st + l.pp);
      const float *eG = reinterpret_cast<const float *>(st + l.gates), *w = eG + kChunk;
      const float kappa = w[kChunk], qscale = w[kChunk + 1], eC = eG[kChunk - 1];
      const long long rec = (long long)(base + c) * p.H + head;
      const int n = min(kChunk, len - c * kChunk);
      // V^T and the scale of this chunk
      float x[4][8];
      load_tokens<NP>(x, st + l.v, ldv, blk * 16, p.dtype, lane);
      unsigned m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, abs_bits(x[i][j]));
      m = max(__reduce_max_sync(0xFFFFFFFFu, m), top);
#pragma unroll
      for (int o = 1; o < NH; ++o) m = max(m, tops[blk * NH + ((h + o) & (NH - 1))]);
      float inv;
      const float scale = scale_of(m, 6, inv);

      // Tile i of E and O holds tokens 8 ((i + OT h) % 8) ..: the warp's own come first.
      float E[8][4], O[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) E[i][j] = O[i][j] = 0.0f;
      __half *s0 = SAVE ? p.s0 + rec * (2ll * p.dvp * DK) : nullptr;
#pragma unroll
      for (int ks = 0; ks < DKH / 16; ++ks) {
        uint32_t ah[4], al[4], b[4];
        split_tiles(S[2 * ks], S[2 * ks + 1], inv, ah, al);
        if (SAVE) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const long long at = (long long)(r0 + 8 * (q & 1)) * DK + c0 + ks * 16 + 8 * (q >> 1) + t2;
            *reinterpret_cast<uint32_t *>(s0 + at) = ah[q];
            *reinterpret_cast<uint32_t *>(s0 + (long long)p.dvp * DK + at) = al[q];
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int np = NH == 1 ? i : (i + OT / 2 * h) & 3;
          if (DELTA) {
            b_rows(b, kt, LD, np * 16, c0 + ks * 16, lane);
            mma2(E[2 * i], E[2 * i + 1], ah, b);
            mma2(E[2 * i], E[2 * i + 1], al, b);
            b_rows(b, kt + kChunk * LD, LD, np * 16, c0 + ks * 16, lane);
            mma2(E[2 * i], E[2 * i + 1], ah, b);
          }
          if (!SAVE) {
            b_rows(b, sq, LD, np * 16, c0 + ks * 16, lane);
            mma2(O[2 * i], O[2 * i + 1], ah, b);
            if (NP == 2) {
              mma2(O[2 * i], O[2 * i + 1], al, b);
              b_rows(b, sq + kChunk * LD, LD, np * 16, c0 + ks * 16, lane);
              mma2(O[2 * i], O[2 * i + 1], ah, b);
            }
          }
        }
      }
      if (SAVE && lane == 0 && h == 0) p.fscale[rec * (p.dvp / 16) + (row0 >> 4) + blk] = scale;
      // + V^T Tm^T for the warp's own tokens (without the delta rule Tm = I and E = V for all)
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        uint32_t vh[4], vl[4];
        if (DELTA) {
#pragma unroll
          for (int q = 0; q < 4; ++q) split2(x[ks][2 * q] * inv, x[ks][2 * q + 1] * inv, vh[q], vl[q]);
#pragma unroll
          for (int i = 0; i < OT / 2; ++i) {
            const int np = NH == 1 ? i : (i + OT / 2 * h) & 3;
            if (ks <= np) {
              uint32_t b[4];
              b_rows(b, tm, kLdC, np * 16, ks * 16, lane);
              mma2(E[2 * i], E[2 * i + 1], vh, b);
              if (NP == 2) mma2(E[2 * i], E[2 * i + 1], vl, b);
              b_rows(b, tm + kChunk * kLdC, kLdC, np * 16, ks * 16, lane);
              mma2(E[2 * i], E[2 * i + 1], vh, b);
            }
          }
        }
      }
      // the other warps' parts
      if (NH > 1) {                    // (also what keeps a warp's next maximum behind the others' reading)
        float4 *own = part + warp * (32 * (8 + (SAVE ? 0 : 8 - OT)));
        if (DELTA)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            own[((i + OT * h) & 7) * 32 + lane] = make_float4(E[i][0], E[i][1], E[i][2], E[i][3]);
        if (!SAVE)
#pragma unroll
          for (int i = OT; i < 8; ++i) own[(8 + i - OT) * 32 + lane] = make_float4(O[i][0], O[i][1], O[i][2], O[i][3]);
        block_barrier(blk, 32 * NH);
#pragma unroll
        for (int o = 1; o < NH; ++o) {
          const int other = (h + o) & (NH - 1);
          const float4 *their = part + (blk * NH + other) * (32 * (8 + (SAVE ? 0 : 8 - OT)));
          if (DELTA)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 y = their[((i + OT * h) & 7) * 32 + lane];
              E[i][0] += y.x; E[i][1] += y.y; E[i][2] += y.z; E[i][3] += y.w;
            }
          if (!SAVE)
#pragma unroll
            for (int i = 0; i < OT; ++i) {
              // this warp's tokens are tile i + OT (NH - o) of the other
              const float4 y = their[(8 + i + OT * (NH - o) - OT) * 32 + lane];
              O[i][0] += y.x; O[i][1] += y.y; O[i][2] += y.z; O[i][3] += y.w;
            }
        }
      }
      if (!DELTA)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // (x is indexed by the token; with NH = 2 the halves trade places for h = 1)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int q = (j >> 1) + 2 * (i & 1), e = 2 * q + (j & 1);
            E[i][j] = (NH == 2 && h == 1 ? x[(i / 2 + 2) & 3][e] : x[i / 2][e]) * inv;
          }
        }
      if (SAVE) {
        __half *et = p.et + rec * (2ll * p.dvp * kChunk);
#pragma unroll
        for (int i = 0; i < OT; ++i)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            uint32_t hi, lo;
            split2(E[i][2 * r], E[i][2 * r + 1], hi, lo);
            const long long at = (long long)(r0 + 8 * r) * kChunk + 8 * ((i + OT * h) & 7) + t2;
            *reinterpret_cast<uint32_t *>(et + at) = hi;
            *reinterpret_cast<uint32_t *>(et + (long long)p.dvp * kChunk + at) = lo;
          }
      }
      // S = e^{G_C} S0 + (diag(w) E)^T K: each tile's sum starts from zero and joins the
      // state in one fma, so that the tensor cores' rounding does not pile up in it
      {
        uint32_t wh[4][4], wl[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int ks = NH == 1 ? i : (i + OT / 2 * h) & 3;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 f = *reinterpret_cast<const float2 *>(w + ks * 16 + 8 * (q >> 1) + t2);
            const float *e = &E[2 * i + (q >> 1)][2 * (q & 1)];
            split2(e[0] * f.x * kappa, e[1] * f.y * kappa, wh[i][q], wl[i][q]);
          }
        }
#pragma unroll
        for (int np = 0; np < NTH / 2; ++np) {
          float a0[4] = {0, 0, 0, 0}, a1[4] = {0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int ks = NH == 1 ? i : (i + OT / 2 * h) & 3;
            uint32_t b[4];
            b_cols(b, sk, LD, ks * 16, c0 + np * 16, lane);
            mma2(a0, a1, wh[i], b);
            mma2(a0, a1, wl[i], b);
            if (NP == 2) {
              b_cols(b, sk + kChunk * LD, LD, ks * 16, c0 + np * 16, lane);
              mma2(a0, a1, wh[i], b);
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            S[2 * np][j] = fmaf(S[2 * np][j], eC, a0[j] * scale);
            S[2 * np + 1][j] = fmaf(S[2 * np + 1][j], eC, a1[j] * scale);
          }
        }
        top = __reduce_max_sync(0xFFFFFFFFu, max_bits<NTH>(S));
        if (NH > 1 && lane == 0) tops[warp] = top;
      }
      if (!SAVE) {
        // O^T = diag(e^G) (S0 Q^T) + E^T P^T for the own tokens
#pragma unroll
        for (int i = 0; i < OT; ++i) {
          const float2 f = *reinterpret_cast<const float2 *>(eG + 8 * ((i + OT * h) & 7) + t2);
          O[i][0] *= f.x; O[i][1] *= f.y; O[i][2] *= f.x; O[i][3] *= f.y;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int ks = NH == 1 ? j : (j + OT / 2 * h) & 3;
          uint32_t eh[4], el[4], b[4];
          split_tiles(E[2 * j], E[2 * j + 1], eh, el);
#pragma unroll
          for (int i = 0; i < OT / 2; ++i) {
            const int np = NH == 1 ? i : (i + OT / 2 * h) & 3;
            if (ks <= np) {
              b_rows(b, pp, kLdC, np * 16, ks * 16, lane);
              mma2(O[2 * i], O[2 * i + 1], eh, b);
              if (NP == 2) {
                mma2(O[2 * i], O[2 * i + 1], el, b);
                b_rows(b, pp + kChunk * kLdC, kLdC, np * 16, ks * 16, lane);
                mma2(O[2 * i], O[2 * i + 1], eh, b);
              }
            }
          }
        }
        float own[OT][4];
#pragma unroll
        for (int i = 0; i < OT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) own[i][j] = O[i][j];
        store_tokens<NP, OT>(own, scale * qscale, st + l.v, ldv, blk * 16, OT * h, p.o, p.dtype, p.o_stride,
                             start + (long long)c * kChunk, n, head * p.d_v + row0 + blk * 16,
                             p.d_v - row0 - blk * 16, p.o16, lane);
      }
    }
    if (p.stages == 1) {
      __syncthreads();
      if (loader && c + 1 < chunks) fetch(c + 1);
    }
  }
  if (live && p.state_out && !SAVE) save_state<NTH>(S, p.state_out, blockIdx.x, p.d_v, DK, r0, c0 + t2);
}

// -------------------------------------------------------------------------------------
// scan_reverse
// -------------------------------------------------------------------------------------
// The same grid and roles over the chunks backwards: the planes of D (at every chunk's end) and R
// are kept for scan_grads, dV = R and d_state_in are written.
template <int DK, int NP, bool DELTA>
__device__ __forceinline__ void reverse_fetch(const ScanParams &p, uint8_t *st, const WalkLayout &l, long long token0,
                                              int n, int slot, int head, int row0, int tid, int threads) {
  constexpr int LD = DK + 8, SIZE = NP == 2 ? 4 : 2;
  const long long rec = (long long)slot * p.H + head;
  const long long qrec = (long long)slot * (p.H / p.share) + head / p.share;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    if (DELTA)
      copy_plane<kChunk, DK, LD>(reinterpret_cast<__half *>(st + l.kt) + c * kChunk * LD,
                                 p.kb + (rec * 2 + c) * (kChunk * DK), tid, threads);
    copy_lower(reinterpret_cast<__half *>(st + l.tm) + c * kChunk * kLdC,
               (DELTA ? p.z : p.pp) + (rec * 2 + c) * (kChunk * kChunk), tid, threads);
  }
#pragma unroll
  for (int c = 0; c < NP; ++c) {
    copy_plane<kChunk, DK, LD>(reinterpret_cast<__half *>(st + l.k) + c * kChunk * LD,
                               p.khat + (qrec * NP + c) * (kChunk * DK), tid, threads);
    copy_plane<kChunk, DK, LD>(reinterpret_cast<__half *>(st + l.q) + c * kChunk * LD,
                               p.qhat + (qrec * NP + c) * (kChunk * DK), tid, threads);
  }
  copy_tokens<SIZE>(st + l.v, tile_ld(NP, p.rb),
                    static_cast<const uint8_t *>(p.o) + (token0 * p.o_stride + (long long)head * p.d_v + row0) * SIZE,
                    p.o_stride, min(16 * p.rb, p.dvp - row0), n, p.d_v - row0, p.o16, tid, threads);
  const float *gates = p.gates + rec * kGateFloats;
  for (int i = tid; i < 2 * kChunk / 4 + 1; i += threads)
    cp16(st + l.gates + 16 * i, i < 2 * kChunk / 4 ? gates + 4 * i : gates + kGateScales, true);
}

template <int DK, int NP, bool DELTA, int NH>
__global__ void __launch_bounds__(32 * (kWalkWarps + kLoadWarps), 1) scan_reverse_kernel(const ScanParams p) {
  constexpr int LD = DK + 8, DKH = DK / NH, NTH = DKH / 8, OT = 8 / NH;
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t2 = (lane & 3) * 2;
  const int blk = warp / NH, h = NH == 1 ? 0 : warp % NH;
  const int seq = blockIdx.x / p.H, head = blockIdx.x % p.H, row0 = blockIdx.y * 16 * p.rb;
  const WalkLayout l = walk_layout(DK, NP, p.rb, NH, DELTA, 2);
  const int ldv = tile_ld(NP, p.rb);
  long long start;
  int len;
  seq_range(p, seq, start, len);
  const int chunks = (len + kChunk - 1) / kChunk, base = slot_base(start, seq);
  const bool loader = blk >= p.rb;
  const int r0 = row0 + blk * 16 + g, c0 = h * DKH;
  const bool live = !loader && row0 + blk * 16 < p.dvp;
  float4 *part = reinterpret_cast<float4 *>(smem + p.stages * l.bytes);
  unsigned *tops = reinterpret_cast<unsigned *>(smem + p.stages * l.bytes + l.part);

  float D[NTH][4];
  load_state<NTH>(D, live ? p.d_state_out : nullptr, blockIdx.x, p.d_v, DK, r0, c0 + t2);
  unsigned top = __reduce_max_sync(0xFFFFFFFFu, max_bits<NTH>(D));
  if (NH > 1 && live && lane == 0) tops[warp] = top;

  const int ltid = tid - 32 * NH * p.rb, lthreads = 32 * kLoadWarps;
  auto fetch = [&](int c) {
    reverse_fetch<DK, NP, DELTA>(p, smem + (p.stages == 2 ? (c & 1) * l.bytes : 0), l, start + (long long)c * kChunk,
                                 min(kChunk, len - c * kChunk), base + c, head, row0, ltid, lthreads);
    cp_commit();
  };
  if (loader && chunks > 0) fetch(chunks - 1);
  for (int c = chunks - 1; c >= 0; --c) {
    uint8_t *st = smem + (p.stages == 2 ? (c & 1) * l.bytes : 0);
    if (loader) cp_wait<0>();
    __syncthreads();
    if (p.stages == 2 && loader && c > 0) fetch(c - 1);
    if (live) {
      const __half *kb = reinterpret_cast<const __half *>(st + l.kt), *sk = reinterpret_cast<const __half *>(st + l.k);
      const __half *sq = reinterpret_cast<const __half *>(st + l.q), *z = reinterpret_cast<const __half *>(st + l.tm);
      const float *eG = reinterpret_cast<const float *>(st + l.gates), *w = eG + kChunk;
      const float kappa = w[kChunk], qscale = w[kChunk + 1], eC = eG[kChunk - 1];
      const long long rec = (long long)(base + c) * p.H + head;
      const int n = min(kChunk, len - c * kChunk);
      // dO^T (times the scale of Q, which Z and the planes of Q lack) and the chunk's scale
      float x[4][8];
      load_tokens<NP>(x, st + l.v, ldv, blk * 16, p.dtype, lane);
      unsigned m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[i][j] *= qscale;
          m = max(m, abs_bits(x[i][j]));
        }
      m = max(__reduce_max_sync(0xFFFFFFFFu, m), top);
#pragma unroll
      for (int o = 1; o < NH; ++o) m = max(m, tops[blk * NH + ((h + o) & (NH - 1))]);
      float inv;
      const float scale = scale_of(m, 6, inv);

      float R[8][4];                   // tile i: tokens 8 ((i + OT h) % 8) ..
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) R[i][j] = 0.0f;
      __half *dd = p.dd + rec * (2ll * p.dvp * DK);
      // D Kb^T; without the delta rule Kb = diag(w) K, applied below
#pragma unroll
      for (int ks = 0; ks < DKH / 16; ++ks) {
        uint32_t ah[4], al[4], b[4];
        split_tiles(D[2 * ks], D[2 * ks + 1], inv, ah, al);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const long long at = (long long)(r0 + 8 * (q & 1)) * DK + c0 + ks * 16 + 8 * (q >> 1) + t2;
          *reinterpret_cast<uint32_t *>(dd + at) = ah[q];
          *reinterpret_cast<uint32_t *>(dd + (long long)p.dvp * DK + at) = al[q];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int np = NH == 1 ? i : (i + OT / 2 * h) & 3;
          b_rows(b, DELTA ? kb : sk, LD, np * 16, c0 + ks * 16, lane);
          mma2(R[2 * i], R[2 * i + 1], ah, b);
          mma2(R[2 * i], R[2 * i + 1], al, b);
          if (DELTA || NP == 2) {
            b_rows(b, (DELTA ? kb : sk) + kChunk * LD, LD, np * 16, c0 + ks * 16, lane);
            mma2(R[2 * i], R[2 * i + 1], ah, b);
          }
        }
      }
      if (lane == 0 && h == 0) p.bscale[rec * (p.dvp / 16) + (row0 >> 4) + blk] = scale;
      if (!DELTA)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = *reinterpret_cast<const float2 *>(w + 8 * ((i + OT * h) & 7) + t2);
          R[i][0] *= f.x * kappa; R[i][1] *= f.y * kappa; R[i][2] *= f.x * kappa; R[i][3] *= f.y * kappa;
        }
      // + dO^T Z for the warp's own tokens s, from blocks t >= s
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        uint32_t oh[4], ol[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) split2(x[ks][2 * q] * inv, x[ks][2 * q + 1] * inv, oh[q], ol[q]);
#pragma unroll
        for (int i = 0; i < OT / 2; ++i) {
          const int np = NH == 1 ? i : (i + OT / 2 * h) & 3;
          if (np <= ks) {
            uint32_t b[4];
            b_cols(b, z, kLdC, ks * 16, np * 16, lane);
            mma2(R[2 * i], R[2 * i + 1], oh, b);
            if (NP == 2) mma2(R[2 * i], R[2 * i + 1], ol, b);
            b_cols(b, z + kChunk * kLdC, kLdC, ks * 16, np * 16, lane);
            mma2(R[2 * i], R[2 * i + 1], oh, b);
          }
        }
      }
      if (NH > 1) {
        float4 *own = part + warp * (32 * 8);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          own[((i + OT * h) & 7) * 32 + lane] = make_float4(R[i][0], R[i][1], R[i][2], R[i][3]);
        block_barrier(blk, 32 * NH);
#pragma unroll
        for (int o = 1; o < NH; ++o) {
          const float4 *their = part + (blk * NH + ((h + o) & (NH - 1))) * (32 * 8);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 y = their[((i + OT * h) & 7) * 32 + lane];
            R[i][0] += y.x; R[i][1] += y.y; R[i][2] += y.z; R[i][3] += y.w;
          }
        }
      }
      {
        __half *rt = p.rt + rec * (2ll * p.dvp * kChunk);
        float own[OT][4];
#pragma unroll
        for (int i = 0; i < OT; ++i) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            uint32_t hi, lo;
            split2(R[i][2 * r], R[i][2 * r + 1], hi, lo);
            const long long at = (long long)(r0 + 8 * r) * kChunk + 8 * ((i + OT * h) & 7) + t2;
            *reinterpret_cast<uint32_t *>(rt + at) = hi;
            *reinterpret_cast<uint32_t *>(rt + (long long)p.dvp * kChunk + at) = lo;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) own[i][j] = R[i][j];
        }
        store_tokens<NP, OT>(own, scale, st + l.v, ldv, blk * 16, OT * h, p.dv, p.dtype, p.v_stride,
                             start + (long long)c * kChunk, n, head * p.d_v + row0 + blk * 16,
                             p.d_v - row0 - blk * 16, p.v16, lane);
      }
      // D = e^{G_C} D + (diag(e^G) dO)^T Q - (diag(e^G) R)^T K
      uint32_t oh[4][4], ol[4][4], rh[4][4], rl[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 f = *reinterpret_cast<const float2 *>(eG + i * 16 + 8 * (q >> 1) + t2);
          split2(x[i][2 * q] * inv * f.x, x[i][2 * q + 1] * inv * f.y, oh[i][q], ol[i][q]);
          if (DELTA) {
            const int ks = NH == 1 ? i : (i + OT / 2 * h) & 3;
            const float2 e = *reinterpret_cast<const float2 *>(eG + ks * 16 + 8 * (q >> 1) + t2);
            const float *y = &R[2 * i + (q >> 1)][2 * (q & 1)];
            split2(y[0] * e.x * -kappa, y[1] * e.y * -kappa, rh[i][q], rl[i][q]);
          }
        }
#pragma unroll
      for (int np = 0; np < NTH / 2; ++np) {
        float a0[4] = {0, 0, 0, 0}, a1[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t b[4];
          b_cols(b, sq, LD, i * 16, c0 + np * 16, lane);
          mma2(a0, a1, oh[i], b);
          mma2(a0, a1, ol[i], b);
          if (NP == 2) {
            b_cols(b, sq + kChunk * LD, LD, i * 16, c0 + np * 16, lane);
            mma2(a0, a1, oh[i], b);
          }
          if (DELTA) {
            const int ks = NH == 1 ? i : (i + OT / 2 * h) & 3;
            b_cols(b, sk, LD, ks * 16, c0 + np * 16, lane);
            mma2(a0, a1, rh[i], b);
            mma2(a0, a1, rl[i], b);
            if (NP == 2) {
              b_cols(b, sk + kChunk * LD, LD, ks * 16, c0 + np * 16, lane);
              mma2(a0, a1, rh[i], b);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          D[2 * np][j] = fmaf(D[2 * np][j], eC, a0[j] * scale);
          D[2 * np + 1][j] = fmaf(D[2 * np + 1][j], eC, a1[j] * scale);
        }
      }
      top = __reduce_max_sync(0xFFFFFFFFu, max_bits<NTH>(D));
      if (NH > 1 && lane == 0) tops[warp] = top;
    }
    if (p.stages == 1) {
      __syncthreads();
      if (loader && c > 0) fetch(c - 1);
    }
  }
  if (live && p.d_state_in) save_state<NTH>(D, p.d_state_in, blockIdx.x, p.d_v, DK, r0, c0 + t2);
}

// -------------------------------------------------------------------------------------
// scan_grads
// -------------------------------------------------------------------------------------
// Grid (slot, head), 8 warps.  Warps 0-3 (group A) own 16 rows each of dO S0 and R S0, warps
// 4-7 (group B) of E D, dO E^T and R E^T; the value rows are the contraction
// axis and pass through shared memory kGradRows at a time.  With dP'_ts = b_s dec_ts dO_t.E_s
// (s <= t), dL'_ts = -b_s dec_ts R_t.E_s (s < t):
//   dQ = diag(e^G) dO S0 + dP' K
//   dK = diag(w) E D - d diag(e^G) R S0 + dP'^T Q + dL' K + dL'^T K
//   c_s = sum_t dec_ts (q_t.k_s dO_t.E_s - k_t.k_s R_t.E_s)
//   dbeta_s = c_s + e^{G_C - G_s} k_s.(D^T E_s)
//   dG_t = sum_s b_s dec_ts (...) - b_t dbeta_t + e^{G_t} (q_t.(S0^T dO_t) - d k_t.(S0^T R_t))
//   dlog_alpha_r = sum_{t >= r} dG_t + sum_s w_s k_s.(D^T E_s) + e^{G_C} <D, S0>
// (the pair (t, s) enters dG_t and, through dbeta_s, -dG_s with the same value, so the sums
// over t >= r cancel exactly where they should).
// Scales: every product pairs a plane of the forward walk (16 value rows over c_b) with one
// of the reverse walk (over d_b), so a 16-row step contributes in units of c_b d_b; left operands
// are brought to the largest such unit F, and sums are held over F.
constexpr int kGradRows = 32;

struct GradLayout {
  int k, q, x, f, stage, stage_bytes, s0, d, e, r, o;
};
__host__ __device__ inline GradLayout grad_layout(int dk, int np) {
  const int ld = dk + 8;
  GradLayout l{};
  int at = 0;
  l.k = at; at += np * kChunk * ld * 2;
  l.q = at; at += np * kChunk * ld * 2;
  l.x = at; at += 4 * kChunk * kLdC * 2;                 // dP' hi, lo, dL' hi, lo
  l.f = at; at += (kGateFloats + 3 * kChunk + 4 * kChunk + 16) * 4;
  l.stage = (at + 15) / 16 * 16;
  at = 0;
  l.s0 = at; at += 2 * kGradRows * ld * 2;
  l.d = at; at += 2 * kGradRows * ld * 2;
  l.e = at; at += 2 * kGradRows * kLdC * 2;
  l.r = at; at += 2 * kGradRows * kLdC * 2;
  l.o = at; at += kChunk * tile_ld(np, kGradRows / 16) * (np == 2 ? 4 : 2);
  l.stage_bytes = at;                                    // holds the [64][dk + 4] fp32 exchange too
  return l;
}

// Rows [0, there) of kGradRows rows of a plane; the others are zeros.
template <int COLS, int LD>
__device__ __forceinline__ void copy_rows(__half *dst, const __half *src, int there, int tid, int threads) {
  constexpr int per = COLS / 8;
#pragma unroll 2
  for (int i = tid; i < kGradRows * per; i += threads) {
    const bool in = i / per < there;
    cp16(dst + (i / per) * LD + (i % per) * 8, in ? src + i * 8 : src, in);
  }
}
// A left operand's registers times a power of two <= 1.
__device__ __forceinline__ void scale_frag(uint32_t (&a)[4], __half2 by) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const __half2 y = __hmul2(*reinterpret_cast<__half2 *>(&a[q]), by);
    a[q] = *reinterpret_cast<const uint32_t *>(&y);
  }
}

template <int DK, int NP, bool DELTA>
__global__ void __launch_bounds__(kGradThreads) scan_grads_kernel(const ScanParams p) {
  constexpr int LD = DK + 8, NT = DK / 8, LDX = DK + 4, LDO = tile_ld(NP, kGradRows / 16), SIZE = NP == 2 ? 4 : 2;
  extern __shared__ __align__(16) uint8_t smem[];
  const GradLayout l = grad_layout(DK, NP);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, w4 = warp & 3, g = lane >> 2,
            t2 = (lane & 3) * 2, m0 = w4 * 16;
  const bool groupA = warp < 4;
  const int slot = blockIdx.x, head = blockIdx.y;
  long long token0 = 0;
  const int n = slot_tokens(p, slot, token0);
  if (n == 0) return;
  const long long rec = (long long)slot * p.H + head;
  const long long qrec = (long long)slot * (p.H / p.share) + head / p.share;
  __half *sk = reinterpret_cast<__half *>(smem + l.k), *sq = reinterpret_cast<__half *>(smem + l.q);
  __half *sx = reinterpret_cast<__half *>(smem + l.x);
  float *eG = reinterpret_cast<float *>(smem + l.f), *w = eG + kChunk, *be = w + kChunk, *eC = be + kChunk;
  const double *G = reinterpret_cast<const double *>(eC + kChunk);
  float *rowv = eG + kGateFloats, *aq = rowv + kChunk, *kw = aq + kChunk, *colp = kw + kChunk,
        *red = colp + 4 * kChunk;
#pragma unroll
  for (int c = 0; c < NP; ++c) {
    copy_plane<kChunk, DK, LD>(sk + c * kChunk * LD, p.khat + (qrec * NP + c) * (kChunk * DK), tid, kGradThreads);
    copy_plane<kChunk, DK, LD>(sq + c * kChunk * LD, p.qhat + (qrec * NP + c) * (kChunk * DK), tid, kGradThreads);
  }
  for (int i = tid; i < kGateFloats / 4; i += kGradThreads)
    cp16(eG + 4 * i, p.gates + rec * kGateFloats + 4 * i, true);
  const int blocks = (p.dvp + kGradRows - 1) / kGradRows, blocks16 = p.dvp / 16;
  auto fetch = [&](int b) {
    uint8_t *st = smem + l.stage + (p.stages == 2 ? (b & 1) * l.stage_bytes : 0);
    const int v0 = b * kGradRows, rows = min(kGradRows, p.dvp - v0);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const long long at = (rec * 2 + c) * p.dvp + v0;
      copy_rows<DK, LD>(reinterpret_cast<__half *>(st + l.s0) + c * kGradRows * LD, p.s0 + at * DK, rows, tid, kGradThreads);
      copy_rows<DK, LD>(reinterpret_cast<__half *>(st + l.d) + c * kGradRows * LD, p.dd + at * DK, rows, tid, kGradThreads);
      copy_rows<kChunk, kLdC>(reinterpret_cast<__half *>(st + l.e) + c * kGradRows * kLdC, p.et + at * kChunk, rows, tid, kGradThreads);
      copy_rows<kChunk, kLdC>(reinterpret_cast<__half *>(st + l.r) + c * kGradRows * kLdC, p.rt + at * kChunk, rows, tid, kGradThreads);
    }
    copy_tokens<SIZE>(st + l.o, LDO,
                      static_cast<const uint8_t *>(p.o) + (token0 * p.o_stride + (long long)head * p.d_v + v0) * SIZE,
                      p.o_stride, kGradRows, n, p.d_v - v0, p.o16, tid, kGradThreads);
    cp_commit();
  };
  fetch(0);
  // exponents of the steps' units, the largest one
  const unsigned *cb = reinterpret_cast<const unsigned *>(p.fscale + rec * blocks16);
  const unsigned *db = reinterpret_cast<const unsigned *>(p.bscale + rec * blocks16);
  int top = 0;
  for (int b = lane; b < blocks16; b += 32) top = max(top, (int)(__ldg(cb + b) >> 23) + (int)(__ldg(db + b) >> 23));
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  // F = 2^(top - 254) as two factors, each in range
  const int f1 = (top - 254) / 2, f2 = top - 254 - f1;
  const float F1 = __uint_as_float((unsigned)(127 + max(-126, f1)) << 23), F2 = __uint_as_float((unsigned)(127 + max(-126, f2)) << 23);

  // group A: acc = dO S0, acc2 = R S0; group B: acc = E D, acc2 tiles 0-7 dO E^T, 8-15 R E^T
  constexpr int N2 = NT > 16 ? NT : 16;
  float acc[NT][4], acc2[N2][4], ds = 0.0f;
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
#pragma unroll
  for (int i = 0; i < N2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc2[i][j] = 0.0f;

  for (int b = 0; b < blocks; ++b) {
    cp_wait<0>();
    __syncthreads();
    if (p.stages == 2 && b + 1 < blocks) fetch(b + 1);
    uint8_t *st = smem + l.stage + (p.stages == 2 ? (b & 1) * l.stage_bytes : 0);
    const __half *s0 = reinterpret_cast<const __half *>(st + l.s0), *dd = reinterpret_cast<const __half *>(st + l.d);
    const __half *se = reinterpret_cast<const __half *>(st + l.e), *sr = reinterpret_cast<const __half *>(st + l.r);
#pragma unroll
    for (int kk = 0; kk < kGradRows; kk += 16) {
      const int b16 = b * (kGradRows / 16) + kk / 16;
      if (b16 >= blocks16) break;
      const unsigned ed = __ldg(db + b16) >> 23;
      const int gap = (int)(__ldg(cb + b16) >> 23) + (int)ed - top;       // <= 0
      const float ratio = gap > -126 ? __uint_as_float((unsigned)(127 + gap) << 23) : 0.0f;
      const float dinv = __uint_as_float((254u - ed) << 23);
      const __half2 by = __float2half2_rn(ratio);
      uint32_t ao[NP][4], ar[2][4], b4[4];
      if (NP == 1) {
        uint32_t raw[4];
        a_rows(raw, reinterpret_cast<const __half *>(st + l.o), LDO, m0, kk, lane);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 f = pair_of(raw[q], p.dtype);
          ao[0][q] = pack2(f.x * dinv * ratio, f.y * dinv * ratio);
        }
      } else {
        const float *so = reinterpret_cast<const float *>(st + l.o);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 f = *reinterpret_cast<const float2 *>(so + (m0 + g + 8 * (q & 1)) * LDO + kk + 8 * (q >> 1) + t2);
          split2(f.x * dinv * ratio, f.y * dinv * ratio, ao[0][q], ao[NP - 1][q]);
        }
      }
      if (DELTA)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          a_cols(ar[c], sr + c * kGradRows * kLdC, kLdC, kk, m0, lane);
          scale_frag(ar[c], by);
        }
      // <D, S0>
      {
        float part = 0.0f;
#pragma unroll
        for (int i = tid; i < 16 * DK / 2; i += kGradThreads) {
          const int at = (kk + i / (DK / 2)) * LD + (i % (DK / 2)) * 2;
          auto pair = [&](const __half *x) {
            const float2 hi = half2_of(*reinterpret_cast<const uint32_t *>(x + at));
            const float2 lo = half2_of(*reinterpret_cast<const uint32_t *>(x + kGradRows * LD + at));
            return make_float2(__fadd_rn(hi.x, lo.x), __fadd_rn(hi.y, lo.y));
          };
          const float2 x = pair(s0), y = pair(dd);
          part = fmaf(x.x, y.x, fmaf(x.y, y.y, part));
        }
        ds = fmaf(part, ratio, ds);
      }
      if (groupA) {
#pragma unroll
        for (int np = 0; np < DK / 16; ++np) {
          b_cols(b4, s0, LD, kk, np * 16, lane);
#pragma unroll
          for (int c = 0; c < NP; ++c) mma2(acc[2 * np], acc[2 * np + 1], ao[c], b4);
          if (DELTA) {
            mma2(acc2[2 * np], acc2[2 * np + 1], ar[0], b4);
            mma2(acc2[2 * np], acc2[2 * np + 1], ar[1], b4);
          }
          b_cols(b4, s0 + kGradRows * LD, LD, kk, np * 16, lane);
          mma2(acc[2 * np], acc[2 * np + 1], ao[0], b4);
          if (DELTA) mma2(acc2[2 * np], acc2[2 * np + 1], ar[0], b4);
        }
      } else {
        uint32_t ae[2][4];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          a_cols(ae[c], se + c * kGradRows * kLdC, kLdC, kk, m0, lane);
          scale_frag(ae[c], by);
        }
#pragma unroll
        for (int np = 0; np < DK / 16; ++np) {
          b_cols(b4, dd, LD, kk, np * 16, lane);
          mma2(acc[2 * np], acc[2 * np + 1], ae[0], b4);
          mma2(acc[2 * np], acc[2 * np + 1], ae[1], b4);
          b_cols(b4, dd + kGradRows * LD, LD, kk, np * 16, lane);
          mma2(acc[2 * np], acc[2 * np + 1], ae[0], b4);
        }
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          if (np <= w4) {
            b_cols(b4, se, kLdC, kk, np * 16, lane);
#pragma unroll
            for (int c = 0; c < NP; ++c) mma2(acc2[2 * np], acc2[2 * np + 1], ao[c], b4);
            if (DELTA) {
              mma2(acc2[8 + 2 * np], acc2[8 + 2 * np + 1], ar[0], b4);
              mma2(acc2[8 + 2 * np], acc2[8 + 2 * np + 1], ar[1], b4);
            }
            b_cols(b4, se + kGradRows * kLdC, kLdC, kk, np * 16, lane);
            mma2(acc2[2 * np], acc2[2 * np + 1], ao[0], b4);
            if (DELTA) mma2(acc2[8 + 2 * np], acc2[8 + 2 * np + 1], ar[0], b4);
          }
        }
      }
    }
    if (p.stages == 1) {
      __syncthreads();
      if (b + 1 < blocks) fetch(b + 1);
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) ds += __shfl_xor_sync(0xFFFFFFFFu, ds, d);
  if (lane == 0) red[warp] = ds;
  const float kappa = eG[kGateScales], qscale = eG[kGateScales + 1];
  const float ikappa = __uint_as_float((254u << 23) - __float_as_uint(kappa));
  const float iqscale = __uint_as_float((254u << 23) - __float_as_uint(qscale));
  // planes of dP', dL' are held over F and 4 dvp (rounded up to a power of two): the entries of
  // E, R and dO over their scales stay below 2^7 (E and R somewhat above), so a sum over d_v of their
  // products stays below 2^14 dvp
  const int lg = 32 - __clz(p.dvp - 1);
  const float unit = __uint_as_float((unsigned)(127 - 2 - lg) << 23), iunit = __uint_as_float((unsigned)(127 + 2 + lg) << 23);

  auto row_pair = [&](const __half *x, int row, int col) {
    float2 v = half2_of(*reinterpret_cast<const uint32_t *>(x + row * LD + col));
    if (NP == 2) {
      const float2 y = half2_of(*reinterpret_cast<const uint32_t *>(x + kChunk * LD + row * LD + col));
      v.x = __fadd_rn(v.x, y.x);
      v.y = __fadd_rn(v.y, y.y);
    }
    return v;
  };
  if (groupA) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = m0 + g + 8 * h;
      float s = 0.0f, r = 0.0f;
      const float e = eG[t], to = e * unit * ikappa;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const float2 q = row_pair(sq, t, 8 * i + t2);
        s = fmaf(q.x, acc[i][2 * h], fmaf(q.y, acc[i][2 * h + 1], s));
        acc[i][2 * h] *= to;
        acc[i][2 * h + 1] *= to;
        if (DELTA) {
          const float2 k = row_pair(sk, t, 8 * i + t2);
          r = fmaf(k.x, acc2[i][2 * h], fmaf(k.y, acc2[i][2 * h + 1], r));
          acc2[i][2 * h] *= -to;
          acc2[i][2 * h + 1] *= -to;
        }
      }
      s = fmaf(s, qscale, -r * kappa) * e;
      s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
      s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
      if ((lane & 3) == 0) aq[t] = s * F1 * F2;
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = m0 + g + 8 * h;
      float s = 0.0f;
      const float to = w[t] * unit * iqscale;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const float2 k = row_pair(sk, t, 8 * i + t2);
        s = fmaf(k.x, acc[i][2 * h], fmaf(k.y, acc[i][2 * h + 1], s));
        acc[i][2 * h] *= to;
        acc[i][2 * h + 1] *= to;
      }
      s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
      s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
      if ((lane & 3) == 0) kw[t] = s * kappa * F1 * F2;
    }
    float rs[2] = {0.0f, 0.0f}, cs[8][2];
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i][0] = cs[i][1] = 0.0f;
    // pass 0: q_t.k_s with dO E^T -> dP'; pass 1: k_t.k_s with R E^T -> dL'
#pragma unroll
    for (int ps = 0; ps < (DELTA ? 2 : 1); ++ps) {
      float x[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = 0.0f;
      const __half *left = ps ? sk : sq;
#pragma unroll
      for (int ks = 0; ks < DK / 16; ++ks) {
        uint32_t a[NP][4], b4[4];
#pragma unroll
        for (int c = 0; c < NP; ++c) a_rows(a[c], left + c * kChunk * LD, LD, m0, ks * 16, lane);
#pragma unroll
        for (int np = 0; np < 4; ++np)
          if (np <= w4) {
            b_rows(b4, sk, LD, np * 16, ks * 16, lane);
#pragma unroll
            for (int c = 0; c < NP; ++c) mma2(x[2 * np], x[2 * np + 1], a[c], b4);
            if (NP == 2) {
              b_rows(b4, sk + kChunk * LD, LD, np * 16, ks * 16, lane);
              mma2(x[2 * np], x[2 * np + 1], a[0], b4);
            }
          }
      }
      const float by = (ps ? kappa : qscale) * kappa;
      __half *out = sx + ps * 2 * kChunk * kLdC;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i / 2 <= w4) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int t = m0 + g + 8 * h;
            float y[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int s = 8 * i + t2 + j;
              const bool in = ps ? s < t : s <= t;
              const float dec = in ? expf((float)(G[t] - G[s])) : 0.0f;
              const float z = in ? (ps ? -acc2[8 + i][2 * h + j] : acc2[i][2 * h + j]) * dec : 0.0f;
              const float m = z * (x[i][2 * h + j] * by);
              y[j] = z * be[s] * unit;
              if (in) {
                rs[h] = fmaf(be[s], m, rs[h]);
                cs[i][j] += m;
              }
            }
            uint32_t hi, lo;
            split2(y[0], y[1], hi, lo);
            *reinterpret_cast<uint32_t *>(out + t * kLdC + 8 * i + t2) = hi;
            *reinterpret_cast<uint32_t *>(out + kChunk * kLdC + t * kLdC + 8 * i + t2) = lo;
          }
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      rs[h] += __shfl_xor_sync(0xFFFFFFFFu, rs[h], 1);
      rs[h] += __shfl_xor_sync(0xFFFFFFFFu, rs[h], 2);
      if ((lane & 3) == 0) rowv[m0 + g + 8 * h] = rs[h] * F1 * F2;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float c = cs[i][j];
        c += __shfl_xor_sync(0xFFFFFFFFu, c, 4);
        c += __shfl_xor_sync(0xFFFFFFFFu, c, 8);
        c += __shfl_xor_sync(0xFFFFFFFFu, c, 16);
        if (g == 0) colp[w4 * kChunk + 8 * i + t2 + j] = c * F1 * F2;
      }
  }
  __syncthreads();
  const float out1 = F1 * kappa, out2 = F2 * iunit;      // what the sums of dQ and dK are held over
  if (groupA) {
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      if (ks <= w4) {
        uint32_t a[4][4], b4[4];
#pragma unroll
        for (int c = 0; c < (DELTA ? 4 : 2); ++c) a_rows(a[c], sx + c * kChunk * kLdC, kLdC, m0, ks * 16, lane);
#pragma unroll
        for (int np = 0; np < DK / 16; ++np) {
          b_cols(b4, sk, LD, ks * 16, np * 16, lane);
          mma2(acc[2 * np], acc[2 * np + 1], a[0], b4);
          mma2(acc[2 * np], acc[2 * np + 1], a[1], b4);
          if (DELTA) {
            mma2(acc2[2 * np], acc2[2 * np + 1], a[2], b4);
            mma2(acc2[2 * np], acc2[2 * np + 1], a[3], b4);
          }
          if (NP == 2) {
            b_cols(b4, sk + kChunk * LD, LD, ks * 16, np * 16, lane);
            mma2(acc[2 * np], acc[2 * np + 1], a[0], b4);
            if (DELTA) mma2(acc2[2 * np], acc2[2 * np + 1], a[2], b4);
          }
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = m0 + g + 8 * h;
      const long long tok = token0 + t;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if (t < n) {
          const float x = acc[i][2 * h] * out1 * out2, y = acc[i][2 * h + 1] * out1 * out2;
          if (p.parts) store_pair(p.dq, 0, (tok * p.H + head) * DK + 8 * i + t2, x, y);
          else store_pair(p.dq, p.dtype, tok * p.q_stride + (long long)head * DK + 8 * i + t2, x, y);
        }
        if (DELTA)
          *reinterpret_cast<float2 *>(reinterpret_cast<float *>(smem + l.stage) + t * LDX + 8 * i + t2) =
              make_float2(acc2[i][2 * h], acc2[i][2 * h + 1]);
      }
    }
  } else {
    const float turn = qscale * ikappa;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      if (ks >= w4) {
        uint32_t a[2][4], b4[4];
#pragma unroll
        for (int c = 0; c < 2; ++c) a_cols(a[c], sx + c * kChunk * kLdC, kLdC, ks * 16, m0, lane);
#pragma unroll
        for (int np = 0; np < DK / 16; ++np) {
          b_cols(b4, sq, LD, ks * 16, np * 16, lane);
          mma2(acc[2 * np], acc[2 * np + 1], a[0], b4);
          mma2(acc[2 * np], acc[2 * np + 1], a[1], b4);
          if (NP == 2) {
            b_cols(b4, sq + kChunk * LD, LD, ks * 16, np * 16, lane);
            mma2(acc[2 * np], acc[2 * np + 1], a[0], b4);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] *= turn;
    if (DELTA)
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        if (ks >= w4) {
          uint32_t a[2][4], b4[4];
#pragma unroll
          for (int c = 0; c < 2; ++c) a_cols(a[c], sx + (2 + c) * kChunk * kLdC, kLdC, ks * 16, m0, lane);
#pragma unroll
          for (int np = 0; np < DK / 16; ++np) {
            b_cols(b4, sk, LD, ks * 16, np * 16, lane);
            mma2(acc[2 * np], acc[2 * np + 1], a[0], b4);
            mma2(acc[2 * np], acc[2 * np + 1], a[1], b4);
            if (NP == 2) {
              b_cols(b4, sk + kChunk * LD, LD, ks * 16, np * 16, lane);
              mma2(acc[2 * np], acc[2 * np + 1], a[0], b4);
            }
          }
        }
      }
  }
  __syncthreads();
  if (!groupA) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = m0 + g + 8 * h;
      const long long tok = token0 + t;
      if (t < n)
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          float2 x = make_float2(acc[i][2 * h], acc[i][2 * h + 1]);
          if (DELTA) {
            const float2 y = *reinterpret_cast<const float2 *>(
                reinterpret_cast<const float *>(smem + l.stage) + t * LDX + 8 * i + t2);
            x.x = __fadd_rn(x.x, y.x);
            x.y = __fadd_rn(x.y, y.y);
          }
          x.x = x.x * out1 * out2;
          x.y = x.y * out1 * out2;
          if (p.parts) store_pair(p.dk, 0, (tok * p.H + head) * DK + 8 * i + t2, x.x, x.y);
          else store_pair(p.dk, p.dtype, tok * p.k_stride + (long long)head * DK + 8 * i + t2, x.x, x.y);
        }
    }
  } else if (warp == 0) {
    // gates: two tokens a lane, sums over t >= r from the chunk's end
    float dsum = 0.0f;
    for (int i = 0; i < kGradThreads / 32; ++i) dsum += red[i];
    dsum = dsum * F1 * F2;
    double dG[2], tot = 0.0;
    float db2[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      const float c = (colp[t] + colp[kChunk + t]) + (colp[2 * kChunk + t] + colp[3 * kChunk + t]);
      db2[i] = fmaf(eC[t], kw[t], c);
      dG[i] = (double)rowv[t] - (double)be[t] * db2[i] + aq[t];
      tot += (double)w[t] * kw[t];
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) tot += __shfl_xor_sync(0xFFFFFFFFu, tot, d);
    tot += (double)eG[kChunk - 1] * dsum;
    double run = dG[0] + dG[1];
    for (int d = 1; d < 32; d <<= 1) {
      const double up = __shfl_down_sync(0xFFFFFFFFu, run, d);
      if (lane + d < 32) run += up;
    }
    const double out[2] = {run + tot, run - dG[0] + tot};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      if (t < n) {
        const long long at = (token0 + t) * p.H + head;
        p.dlog_alpha[at] = (float)out[i];
        p.dbeta[at] = db2[i];
      }
    }
  }
}

// Sums the heads' parts of dq and dk where heads share q and k, in head order.
static __global__ void __launch_bounds__(256) scan_shared_kernel(const ScanParams p, const float *parts_q,
                                                                 const float *parts_k, int dk) {
  const int hq = p.H / p.share, per = hq * (dk / 4);
  const long long n = p.total * per, all = 2 * n;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < all; i += (long long)gridDim.x * 256) {
    const bool second = i >= n;
    const long long j = second ? i - n : i, tok = j / per;
    const int r = (int)(j % per), h = r / (dk / 4), c = (r % (dk / 4)) * 4;
    if (!token_used(p, tok)) continue;
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
// d_k/16 lanes share a value row (16 of its columns each, in groups of 4 so that the lanes'
// 16-byte accesses are contiguous) and two rows are in flight per lane.
constexpr int kRecThreads = 128, kRecRows = 2;

template <int DK, bool DELTA>
__global__ void __launch_bounds__(kRecThreads) scan_recurrent_kernel(const ScanParams p) {
  constexpr int LPR = DK / 16;
  if (blockIdx.x == 0) check_offsets(p);
  const int lane = threadIdx.x & 31, lir = lane % LPR;
  const int per = p.d_v / kRecRows;                               // row pairs of one head
  const long long pairs = (long long)p.n_seq * p.H * per;
  const long long id = (blockIdx.x * (long long)kRecThreads + threadIdx.x) / LPR;
  const bool live = id < pairs;
  const long long gr = live ? id : pairs - 1;
  const long long tile = gr / per;
  const int row = (int)(gr % per) * kRecRows, head = (int)(tile % p.H), seq = (int)(tile / p.H);
  long long start;
  int len;
  seq_range(p, seq, start, len);
  if (!live) len = 0;
  const int most = __reduce_max_sync(0xFFFFFFFFu, len);
  float S[kRecRows][16];
  const long long at = (tile * p.d_v + row) * DK + 4 * lir;
#pragma unroll
  for (int r = 0; r < kRecRows; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (p.state_in && live) x = *reinterpret_cast<const float4 *>(p.state_in + at + r * DK + 4 * LPR * c);
      S[r][4 * c] = x.x; S[r][4 * c + 1] = x.y; S[r][4 * c + 2] = x.z; S[r][4 * c + 3] = x.w;
    }
  const long long qo = (long long)(head / p.share) * DK + 4 * lir;
  for (int t = 0; t < most; ++t) {
    const bool on = t < len;
    const long long tok = start + (on ? t : 0);
    float k[16], q[16], v[kRecRows], a = 1.0f, b = 0.0f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float x[4] = {0, 0, 0, 0}, y[4] = {0, 0, 0, 0};
      if (on) {
        load4(p.k, p.dtype, tok * p.k_stride + qo + 4 * LPR * c, x);
        load4(p.q, p.dtype, tok * p.q_stride + qo + 4 * LPR * c, y);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) { k[4 * c + e] = x[e]; q[4 * c + e] = y[e]; }
    }
#pragma unroll
    for (int r = 0; r < kRecRows; ++r) v[r] = 0.0f;
    if (on) {
      a = expf(__ldg(p.log_alpha + tok * p.H + head));
      b = __ldg(p.beta + tok * p.H + head);
      const long long vo = tok * p.v_stride + (long long)head * p.d_v + row;
#pragma unroll
      for (int r = 0; r < kRecRows; ++r)
        v[r] = p.dtype == 0 ? __ldg(static_cast<const float *>(p.v) + vo + r)
               : p.dtype == 1 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p.v)[vo + r])
                              : __half2float(static_cast<const __half *>(p.v)[vo + r]);
    }
    float u[kRecRows], o[kRecRows];
#pragma unroll
    for (int r = 0; r < kRecRows; ++r) {
      u[r] = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        S[r][e] *= a;
        if (DELTA) u[r] = fmaf(S[r][e], k[e], u[r]);
      }
    }
    if (DELTA)
#pragma unroll
      for (int d = 1; d < LPR; d <<= 1)
#pragma unroll
        for (int r = 0; r < kRecRows; ++r) u[r] += __shfl_xor_sync(0xFFFFFFFFu, u[r], d);
#pragma unroll
    for (int r = 0; r < kRecRows; ++r) {
      const float wr = b * (v[r] - u[r]);
      o[r] = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        S[r][e] = fmaf(wr, k[e], S[r][e]);
        o[r] = fmaf(S[r][e], q[e], o[r]);
      }
    }
#pragma unroll
    for (int d = 1; d < LPR; d <<= 1)
#pragma unroll
      for (int r = 0; r < kRecRows; ++r) o[r] += __shfl_xor_sync(0xFFFFFFFFu, o[r], d);
    if (on && lir == 0)
#pragma unroll
      for (int r = 0; r < kRecRows; ++r)
        store_as(p.o, p.dtype, tok * p.o_stride + (long long)head * p.d_v + row + r, o[r]);
  }
  if (p.state_out && live)
#pragma unroll
    for (int r = 0; r < kRecRows; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<float4 *>(p.state_out + at + r * DK + 4 * LPR * c) =
            make_float4(S[r][4 * c], S[r][4 * c + 1], S[r][4 * c + 2], S[r][4 * c + 3]);
}

using ScanFn = void (*)(ScanParams);
// kernels of one key width
struct ScanKernels {
  ScanFn prep[2][2][2];                // [np - 1][delta][backward]
  ScanFn chain[2][2][2][2];            // [np - 1][delta][save][nh - 1]
  ScanFn reverse[2][2][2];             // [np - 1][delta][nh - 1]
  ScanFn grads[2][2];
};

}  // namespace scan
}  // namespace lores
