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
// Only S0 -> S_C is sequential, so the work is split in three:
//   scan_planes   inputs that are not aligned bf16 rows -> one or two bf16 planes (below)
//   scan_prep     all chunks at once: gates, Tm, P, Kt = -d Tm diag(e^G) K (and, for the
//                 backward pass, Z = P Tm and Kb = Tm^T diag(w) K)
//   scan_chain    per (sequence, head, block of value rows): E^T = S0 Kt^T + (Tm V)^T, O^T and
//                 S_C, chunk after chunk.  Value rows are independent (as in the decode
//                 step), so a warp owns 16 of them, keeps S [16][d_k] in its accumulators and
//                 feeds it back as the next product's left operand without leaving registers.
// Backward, D = dL/dS_C:
//   R   = Z^T dO + Kb D^T (= dV)       D0 = e^{G_C} D + (diag(e^G) dO)^T Q - d (diag(e^G) R)^T K
//   scan_reverse  the same walk backwards over R and D;
//   scan_grads    all chunks at once: dQ, dK and the gates' gradients from S0, D, E, R.
//
// Precision.  The tensor cores multiply bf16 and add fp32.  Every fp32 operand x is given as two
// bf16 planes, hi = bf16(x) and lo = bf16(x - hi) (16 bits of significand, 2^-18 at worst), and a product is
// hi hi + hi lo + lo hi; a bf16 input is exact as one plane.  So states, gates' gradients and
// everything between two products keep an error near 1e-6, which one bf16 product (2^-9)
// could not.  The state itself and every sum stay in fp32.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace lores {
namespace scan {

constexpr int kChunk = 64;
constexpr int kLdC = kChunk + 8;       // row stride of a [64][64] plane (16-byte rows apart: no
                                       // bank conflict of the 8 rows that ldmatrix reads)
constexpr int kPrepThreads = 128;
constexpr int kGradThreads = 256;
constexpr unsigned kFlagOffsets = 1u;  // a sequence's offsets were not 0 <= a <= b <= total

// bf16 planes of a token-major tensor: element (token, head, i) at token * stride +
// head * hstride + i.  lo is null for one plane.
struct Planes {
  const __nv_bfloat16 *hi, *lo;
  long long stride;
  int hstride;
};

// A user's tensor that scan_planes turns into planes.
struct Raw {
  const void *src;
  long long stride;                    // elements between tokens
  int heads, dim, dimp;                // dimp: dim rounded up to 16 (zeros behind dim)
  __nv_bfloat16 *hi, *lo;              // [total][heads][dimp]
};

struct ScanParams {
  int n_seq, H, share, d_v, dvp, dtype, n_slots, max_len, stages;
  long long total;
  const int *offsets;
  Planes q, k, v, dO;
  Raw raw[4];
  const float *log_alpha, *beta;       // [total][H]
  const float *state_in;               // [n_seq][H][d_v][d_k] or null
  float *state_out;                    // likewise or null
  void *o;                             // forward: o; backward: dv
  long long o_stride;
  unsigned *flag;
  // workspace, records of one (slot, head)
  float *gates;                        // [64] e^G, w, b, e^(G_C - G); [64] G (double)
  __nv_bfloat16 *kt, *kb;              // [2][64][d_k]
  __nv_bfloat16 *tm, *pp, *z;          // [2][64][64]
  __nv_bfloat16 *s0, *dd;              // [2][dvp][d_k]
  __nv_bfloat16 *et, *rt;              // [2][dvp][64]
  // backward
  const float *d_state_out;
  float *d_state_in;
  void *dq, *dk;                       // user's gradients, or fp32 parts [total][H][d_k]
  long long dq_stride, dk_stride;
  int parts;                           // dq, dk are fp32 parts of each head
  float *dlog_alpha, *dbeta;
  // recurrent form: the user's tensors as they are
  const void *uq, *uk, *uv;
  long long uq_stride, uk_stride, uv_stride;
};

constexpr int kGateFloats = 4 * kChunk + 2 * kChunk;

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

// The sequence and first token of a slot's chunk and its tokens (0: the slot is not used).
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
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const __nv_bfloat16 *row) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_addr(row)));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], const __nv_bfloat16 *row) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_addr(row)));
}
// Fragment loads of 16x16 blocks from row-major shared memory with row stride ld.
//   right operand, two column tiles (r[0], r[1]: columns n0..n0+7; r[2], r[3]: n0+8..):
//     b_rows:  stored [n][k]      b_cols: stored [k][n]
//   left operand:
//     a_rows:  stored [m][k]      a_cols: stored [k][m]
__device__ __forceinline__ void b_rows(uint32_t (&r)[4], const __nv_bfloat16 *x, int ld, int n0,
                                       int k0, int lane) {
  ldsm4(r, x + (n0 + ((lane >> 4) << 3) + (lane & 7)) * ld + k0 + (((lane >> 3) & 1) << 3));
}
__device__ __forceinline__ void b_cols(uint32_t (&r)[4], const __nv_bfloat16 *x, int ld, int k0,
                                       int n0, int lane) {
  ldsm4t(r, x + (k0 + (((lane >> 3) & 1) << 3) + (lane & 7)) * ld + n0 + ((lane >> 4) << 3));
}
__device__ __forceinline__ void a_rows(uint32_t (&r)[4], const __nv_bfloat16 *x, int ld, int m0,
                                       int k0, int lane) {
  ldsm4(r, x + (m0 + (((lane >> 3) & 1) << 3) + (lane & 7)) * ld + k0 + ((lane >> 4) << 3));
}
__device__ __forceinline__ void a_cols(uint32_t (&r)[4], const __nv_bfloat16 *x, int ld, int k0,
                                       int m0, int lane) {
  ldsm4t(r, x + (k0 + ((lane >> 4) << 3) + (lane & 7)) * ld + m0 + (((lane >> 3) & 1) << 3));
}

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
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

// x, y -> packed bf16 (x low) and the packed rest.
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(y), "f"(x));
  const float rx = __fsub_rn(x, __uint_as_float(hi << 16));
  const float ry = __fsub_rn(y, __uint_as_float(hi & 0xFFFF0000u));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(ry), "f"(rx));
}
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// Accumulator tiles 2j, 2j+1 (16 columns) as a left operand's planes: the layouts agree.
__device__ __forceinline__ void split_tiles(const float (&c0)[4], const float (&c1)[4],
                                            uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  split2(c0[0], c0[1], hi[0], lo[0]);
  split2(c0[2], c0[3], hi[1], lo[1]);
  split2(c1[0], c1[1], hi[2], lo[2]);
  split2(c1[2], c1[3], hi[3], lo[3]);
}

// -------------------------------------------------------------------------------------
// asynchronous copies
// -------------------------------------------------------------------------------------
__device__ __forceinline__ void cp16(void *dst, const void *src, bool there) {
  const int n = there ? 16 : 0;        // 0: sixteen zero bytes
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// rows x cols elements of bf16 -> shared rows of ld elements; rows >= there and columns >=
// have are zeros.  cols and have are multiples of 8.
__device__ __forceinline__ void copy_tile(__nv_bfloat16 *dst, int ld, const __nv_bfloat16 *src,
                                          long long stride, int rows, int cols, int there, int have,
                                          int tid, int threads) {
  const int per = cols >> 3;
  for (int i = tid; i < rows * per; i += threads) {
    const int r = i / per, c = (i % per) << 3;
    const bool in = r < there && c < have;
    cp16(dst + r * ld + c, in ? src + r * stride + c : src, in);
  }
}

__device__ __forceinline__ void store_as(void *base, int dtype, long long i, float x) {
  if (dtype == 0) static_cast<float *>(base)[i] = x;
  else if (dtype == 1) static_cast<__nv_bfloat16 *>(base)[i] = __float2bfloat16_rn(x);
  else static_cast<__half *>(base)[i] = __float2half_rn(x);
}
__device__ __forceinline__ void store_pair(void *base, int dtype, long long i, float x, float y) {
  if (dtype == 0) *reinterpret_cast<float2 *>(static_cast<float *>(base) + i) = make_float2(x, y);
  else if (dtype == 1)
    *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(base) + i) = __floats2bfloat162_rn(x, y);
  else *reinterpret_cast<__half2 *>(static_cast<__half *>(base) + i) = __floats2half2_rn(x, y);
}

// -------------------------------------------------------------------------------------
// scan_planes: inputs -> bf16 planes
// -------------------------------------------------------------------------------------
// Grid (blocks over 4-element groups, tensor).  fp32 and fp16 give two planes (fp16's 11 bits
// fit in them exactly), bf16 rows that are not 16-byte aligned one.
__device__ __forceinline__ void load4(const void *src, int dtype, long long i, float (&x)[4]) {
  if (dtype == 0) {
    const float4 f = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(src) + i));
    x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
    return;
  }
  const uint2 w = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(src) + i));
  if (dtype == 1) {
    const float2 a = unpack2(w.x), b = unpack2(w.y);
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  } else {
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&w.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&w.y));
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  }
}

static __global__ void __launch_bounds__(256) scan_planes_kernel(const ScanParams p) {
  const Raw r = p.raw[blockIdx.y];
  if (!r.src) return;
  const int per = r.dimp >> 2;
  const long long n = p.total * r.heads * per;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const int c = (int)(i % per) << 2;
    const long long th = i / per;
    const int h = (int)(th % r.heads);
    const long long t = th / r.heads;
    float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < r.dim) load4(r.src, p.dtype, t * r.stride + (long long)h * r.dim + c, x);
    uint2 hi, lo;
    split2(x[0], x[1], hi.x, lo.x);
    split2(x[2], x[3], hi.y, lo.y);
    const long long at = th * r.dimp + c;
    *reinterpret_cast<uint2 *>(r.hi + at) = hi;
    if (r.lo) *reinterpret_cast<uint2 *>(r.lo + at) = lo;
  }
}

// -------------------------------------------------------------------------------------
// scan_prep
// -------------------------------------------------------------------------------------
// Grid (slot, head), 4 warps; warp w owns rows 16w .. 16w+15 of every [64][.] result, and only
// blocks on and below the diagonal are formed.  Tm is inverted in fp32: the four diagonal
// 16x16 blocks by forward substitution (one lane per column), then pairs of blocks joined as
// [[A,0],[B,C]]^-1 = [[A',0],[-C'BA',C']], twice.
constexpr int kLdF = kChunk + 2;       // row stride of the fp32 matrix in shared memory

template <int DK, int NP>
constexpr int prep_smem() {
  return (2 * NP * kChunk * (DK + 8)) * 2 + kChunk * kLdF * 4 * 2 + kChunk * 8 + kChunk * 4 * 4;
}

__device__ __forceinline__ void inverse_join(float *X, float *Y, int n, int tid, int threads) {
  // X holds, on the diagonal, inverted n x n blocks and below every second one the block B.
  // Y is scratch of the same layout.
  const int pairs = kChunk / (2 * n), per = n * n;
  for (int i = tid; i < pairs * per; i += threads) {         // Y = C' B
    const int b = i / per, r = (i % per) / n, c = i % n, o = b * 2 * n;
    float s = 0.0f;
    for (int m = 0; m <= r; ++m) s = fmaf(X[(o + n + r) * kLdF + o + n + m], X[(o + n + m) * kLdF + o + c], s);
    Y[(o + n + r) * kLdF + o + c] = s;
  }
  __syncthreads();
  for (int i = tid; i < pairs * per; i += threads) {         // X = -Y A'
    const int b = i / per, r = (i % per) / n, c = i % n, o = b * 2 * n;
    float s = 0.0f;
    for (int m = c; m < n; ++m) s = fmaf(Y[(o + n + r) * kLdF + o + m], X[(o + m) * kLdF + o + c], s);
    X[(o + n + r) * kLdF + o + c] = -s;
  }
  __syncthreads();
}

template <int DK, int NP, bool DELTA, bool BWD>
__global__ void __launch_bounds__(kPrepThreads) scan_prep_kernel(const ScanParams p) {
  constexpr int LD = DK + 8;
  extern __shared__ __align__(16) uint8_t smem[];
  __nv_bfloat16 *K = reinterpret_cast<__nv_bfloat16 *>(smem);       // NP planes
  __nv_bfloat16 *Q = K + NP * kChunk * LD;
  float *X = reinterpret_cast<float *>(Q + NP * kChunk * LD);       // Tm
  float *Y = X + kChunk * kLdF;
  double *G = reinterpret_cast<double *>(Y + kChunk * kLdF);
  float *eG = reinterpret_cast<float *>(G + kChunk), *w = eG + kChunk, *be = w + kChunk,
        *eC = be + kChunk;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t2 = (lane & 3) * 2;
  const int slot = blockIdx.x, head = blockIdx.y;
  if (slot == 0 && head == 0) check_offsets(p);
  long long token0 = 0;
  const int n = slot_tokens(p, slot, token0);
  if (n == 0) return;
  const int qh = head / p.share;
#pragma unroll
  for (int c = 0; c < NP; ++c) {
    copy_tile(K + c * kChunk * LD, LD, (c ? p.k.lo : p.k.hi) + token0 * p.k.stride + qh * p.k.hstride,
              p.k.stride, kChunk, DK, n, DK, tid, kPrepThreads);
    copy_tile(Q + c * kChunk * LD, LD, (c ? p.q.lo : p.q.hi) + token0 * p.q.stride + qh * p.q.hstride,
              p.q.stride, kChunk, DK, n, DK, tid, kPrepThreads);
  }
  cp_commit();
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
    float *rec = p.gates + ((long long)slot * p.H + head) * kGateFloats;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      const float e = expf((float)Gt[i]), c = expf((float)(end - Gt[i]));
      G[t] = Gt[i];
      eG[t] = e; be[t] = b[i]; eC[t] = c; w[t] = b[i] * c;
      rec[t] = e; rec[kChunk + t] = b[i] * c; rec[2 * kChunk + t] = b[i]; rec[3 * kChunk + t] = c;
      reinterpret_cast<double *>(rec + 4 * kChunk)[t] = Gt[i];
    }
  }
  cp_wait<0>();
  __syncthreads();

  const long long rec = (long long)slot * p.H + head;
  const int m0 = warp * 16;
  float P[8][4], A[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) P[i][j] = A[i][j] = 0.0f;
#pragma unroll
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
  // decays; A below the diagonal to shared memory, P to its planes
  __nv_bfloat16 *pp = p.pp + rec * (2 * kChunk * kChunk);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i / 2 <= warp) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = m0 + g + 8 * h, s = 8 * i + t2;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float dec = s + j <= t ? expf((float)(G[t] - G[s + j])) * be[s + j] : 0.0f;
          P[i][2 * h + j] = s + j <= t ? P[i][2 * h + j] * dec : 0.0f;
          if (DELTA) X[t * kLdF + s + j] = s + j < t ? A[i][2 * h + j] * dec : 0.0f;
        }
        uint32_t hi, lo;
        split2(P[i][2 * h], P[i][2 * h + 1], hi, lo);
        *reinterpret_cast<uint32_t *>(pp + t * kChunk + s) = hi;
        *reinterpret_cast<uint32_t *>(pp + kChunk * kChunk + t * kChunk + s) = lo;
      }
    }
  }
  if (!DELTA) return;
  __syncthreads();
  if (lane < 16) {                     // this warp's diagonal block, column `lane`
    float x[16];
    float *B = X + m0 * kLdF + m0;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float s0 = r == lane ? 1.0f : 0.0f, s1 = 0.0f;
#pragma unroll
      for (int m = 0; m < r; ++m) {
        if (m & 1) s1 = fmaf(-B[r * kLdF + m], x[m], s1);
        else s0 = fmaf(-B[r * kLdF + m], x[m], s0);
      }
      x[r] = s0 + s1;
    }
    __syncwarp(0x0000FFFFu);
#pragma unroll
    for (int r = 0; r < 16; ++r) B[r * kLdF + lane] = x[r];
  }
  __syncthreads();
  inverse_join(X, Y, 16, tid, kPrepThreads);
  inverse_join(X, Y, 32, tid, kPrepThreads);

  // planes of Tm
  __nv_bfloat16 *tm = p.tm + rec * (2 * kChunk * kChunk);
  for (int i = tid; i < kChunk * kChunk / 2; i += kPrepThreads) {
    const int r = i / (kChunk / 2), c = (i % (kChunk / 2)) * 2;
    uint32_t hi = 0, lo = 0;
    if ((c >> 4) <= (r >> 4)) split2(X[r * kLdF + c], X[r * kLdF + c + 1], hi, lo);
    *reinterpret_cast<uint32_t *>(tm + r * kChunk + c) = hi;
    *reinterpret_cast<uint32_t *>(tm + kChunk * kChunk + r * kChunk + c) = lo;
  }
  // Kt = -Tm diag(e^G) K: rows t of this warp, s blocks up to its own
  {
    float acc[DK / 8][4];
#pragma unroll
    for (int i = 0; i < DK / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      if (ks <= warp) {
        uint32_t ah[4], al[4], b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int t = m0 + g + 8 * (q & 1), s = ks * 16 + t2 + 8 * (q >> 1);
          split2(-X[t * kLdF + s] * eG[s], -X[t * kLdF + s + 1] * eG[s + 1], ah[q], al[q]);
        }
#pragma unroll
        for (int np = 0; np < DK / 16; ++np) {
          b_cols(b, K, LD, ks * 16, np * 16, lane);
          mma2(acc[2 * np], acc[2 * np + 1], ah, b);
          mma2(acc[2 * np], acc[2 * np + 1], al, b);
          if (NP == 2) {
            b_cols(b, K + kChunk * LD, LD, ks * 16, np * 16, lane);
            mma2(acc[2 * np], acc[2 * np + 1], ah, b);
          }
        }
      }
    }
    __nv_bfloat16 *kt = p.kt + rec * (2 * kChunk * DK);
#pragma unroll
    for (int i = 0; i < DK / 8; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t hi, lo;
        split2(acc[i][2 * h], acc[i][2 * h + 1], hi, lo);
        const int at = (m0 + g + 8 * h) * DK + 8 * i + t2;
        *reinterpret_cast<uint32_t *>(kt + at) = hi;
        *reinterpret_cast<uint32_t *>(kt + kChunk * DK + at) = lo;
      }
  }
  if (!BWD) return;
  // Kb = Tm^T diag(w) K: rows s of this warp, t blocks from its own on
  {
    float acc[DK / 8][4];
#pragma unroll
    for (int i = 0; i < DK / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      if (ks >= warp) {
        uint32_t ah[4], al[4], b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int s = m0 + g + 8 * (q & 1), t = ks * 16 + t2 + 8 * (q >> 1);
          split2(X[t * kLdF + s] * w[t], X[(t + 1) * kLdF + s] * w[t + 1], ah[q], al[q]);
        }
#pragma unroll
        for (int np = 0; np < DK / 16; ++np) {
          b_cols(b, K, LD, ks * 16, np * 16, lane);
          mma2(acc[2 * np], acc[2 * np + 1], ah, b);
          mma2(acc[2 * np], acc[2 * np + 1], al, b);
          if (NP == 2) {
            b_cols(b, K + kChunk * LD, LD, ks * 16, np * 16, lane);
            mma2(acc[2 * np], acc[2 * np + 1], ah, b);
          }
        }
      }
    }
    __nv_bfloat16 *kb = p.kb + rec * (2 * kChunk * DK);
#pragma unroll
    for (int i = 0; i < DK / 8; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t hi, lo;
        split2(acc[i][2 * h], acc[i][2 * h + 1], hi, lo);
        const int at = (m0 + g + 8 * h) * DK + 8 * i + t2;
        *reinterpret_cast<uint32_t *>(kb + at) = hi;
        *reinterpret_cast<uint32_t *>(kb + kChunk * DK + at) = lo;
      }
  }
  // Z = P Tm: rows t of this warp; block (r, s) of Tm is zero for s > r
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
    __nv_bfloat16 *z = p.z + rec * (2 * kChunk * kChunk);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i / 2 <= warp)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t hi, lo;
          split2(acc[i][2 * h], acc[i][2 * h + 1], hi, lo);
          const int at = (m0 + g + 8 * h) * kChunk + 8 * i + t2;
          *reinterpret_cast<uint32_t *>(z + at) = hi;
          *reinterpret_cast<uint32_t *>(z + kChunk * kChunk + at) = lo;
        }
  }
}

// -------------------------------------------------------------------------------------
// scan_chain
// -------------------------------------------------------------------------------------
// Grid (sequence * H + head, block of 16 W value rows); W compute warps of 16 rows each and
// two warps that fetch the next chunk's tiles meanwhile (two stages where they fit).
// SAVE: the backward pass's recomputation, which keeps S0 and E of every chunk; otherwise
// o and the last state are written.
constexpr int kLoadWarps = 2;

struct ChainLayout {                   // byte offsets inside one stage
  int kt, k, q, tm, pp, v, gates, bytes;
};
__host__ __device__ inline ChainLayout chain_layout(int dk, int np, int w, bool delta, bool out) {
  const int ld = dk + 8, tile = kChunk * ld * 2, sq = kChunk * kLdC * 2;
  ChainLayout l{};
  int at = 0;
  l.kt = at; at += delta ? 2 * tile : 0;
  l.k = at; at += np * tile;
  l.q = at; at += out ? np * tile : 0;
  l.tm = at; at += delta ? 2 * sq : 0;
  l.pp = at; at += out ? 2 * sq : 0;
  l.v = at; at += np * kChunk * (16 * w + 8) * 2;
  l.gates = at; at += 2 * kChunk * 4;
  l.bytes = at;
  return l;
}

template <int DK, int NP, bool DELTA, bool SAVE>
__device__ __forceinline__ void chain_fetch(const ScanParams &p, uint8_t *st, const ChainLayout &l,
                                            int w, long long token0, int n, long long rec, int head,
                                            int row0, int tid, int threads) {
  constexpr int LD = DK + 8;
  const int qh = head / p.share, ldv = 16 * w + 8;
  const int cols = min(16 * w, p.dvp - row0);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    if (DELTA) {
      copy_tile(reinterpret_cast<__nv_bfloat16 *>(st + l.kt) + c * kChunk * LD, LD,
                p.kt + rec * (2 * kChunk * DK) + c * kChunk * DK, DK, kChunk, DK, kChunk, DK, tid, threads);
      copy_tile(reinterpret_cast<__nv_bfloat16 *>(st + l.tm) + c * kChunk * kLdC, kLdC,
                p.tm + rec * (2 * kChunk * kChunk) + c * kChunk * kChunk, kChunk, kChunk, kChunk,
                kChunk, kChunk, tid, threads);
    }
    if (!SAVE)
      copy_tile(reinterpret_cast<__nv_bfloat16 *>(st + l.pp) + c * kChunk * kLdC, kLdC,
                p.pp + rec * (2 * kChunk * kChunk) + c * kChunk * kChunk, kChunk, kChunk, kChunk,
                kChunk, kChunk, tid, threads);
  }
#pragma unroll
  for (int c = 0; c < NP; ++c) {
    copy_tile(reinterpret_cast<__nv_bfloat16 *>(st + l.k) + c * kChunk * LD, LD,
              (c ? p.k.lo : p.k.hi) + token0 * p.k.stride + qh * p.k.hstride, p.k.stride, kChunk, DK,
              n, DK, tid, threads);
    if (!SAVE)
      copy_tile(reinterpret_cast<__nv_bfloat16 *>(st + l.q) + c * kChunk * LD, LD,
                (c ? p.q.lo : p.q.hi) + token0 * p.q.stride + qh * p.q.hstride, p.q.stride, kChunk,
                DK, n, DK, tid, threads);
    copy_tile(reinterpret_cast<__nv_bfloat16 *>(st + l.v) + c * kChunk * ldv, ldv,
              (c ? p.v.lo : p.v.hi) + token0 * p.v.stride + (long long)head * p.v.hstride + row0,
              p.v.stride, kChunk, cols, n, p.v.hstride - row0, tid, threads);
  }
  const float *gates = p.gates + rec * kGateFloats;
  for (int i = tid; i < 2 * kChunk / 4; i += threads)
    cp16(st + l.gates + 16 * i, gates + 4 * i, true);
}

template <int DK, int NP, bool DELTA, bool SAVE>
__global__ void __launch_bounds__(32 * (4 + kLoadWarps)) scan_chain_kernel(const ScanParams p) {
  constexpr int LD = DK + 8, NT = DK / 8;
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t2 = (lane & 3) * 2;
  const int W = blockDim.x / 32 - kLoadWarps;
  const int seq = blockIdx.x / p.H, head = blockIdx.x % p.H, row0 = blockIdx.y * 16 * W;
  const ChainLayout l = chain_layout(DK, NP, W, DELTA, !SAVE);
  const int ldv = 16 * W + 8;
  long long start;
  int len;
  seq_range(p, seq, start, len);
  const int chunks = (len + kChunk - 1) / kChunk, base = slot_base(start, seq);
  const bool loader = warp >= W;
  const int r0 = row0 + warp * 16 + g;             // this thread's value rows: r0, r0 + 8
  const bool live = !loader && row0 + warp * 16 < p.dvp;

  float S[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float2 x = make_float2(0.0f, 0.0f);
      if (live && p.state_in && r0 + 8 * h < p.d_v)
        x = *reinterpret_cast<const float2 *>(
            p.state_in + ((long long)blockIdx.x * p.d_v + r0 + 8 * h) * DK + 8 * i + t2);
      S[i][2 * h] = x.x;
      S[i][2 * h + 1] = x.y;
    }

  const int ltid = tid - 32 * W, lthreads = 32 * kLoadWarps;
  if (loader && chunks > 0) {
    chain_fetch<DK, NP, DELTA, SAVE>(p, smem, l, W, start, min(kChunk, len), (long long)base * p.H + head,
                                     head, row0, ltid, lthreads);
    cp_commit();
  }
  for (int c = 0; c < chunks; ++c) {
    uint8_t *st = smem + (p.stages == 2 ? (c & 1) * l.bytes : 0);
    if (loader) cp_wait<0>();
    __syncthreads();
    const long long rec = (long long)(base + c) * p.H + head;
    auto fetch_next = [&]() {
      if (loader && c + 1 < chunks) {
        chain_fetch<DK, NP, DELTA, SAVE>(
            p, smem + (p.stages == 2 ? ((c + 1) & 1) * l.bytes : 0), l, W,
            start + (long long)(c + 1) * kChunk, min(kChunk, len - (c + 1) * kChunk), rec + p.H, head,
            row0, ltid, lthreads);
        cp_commit();
      }
    };
    if (p.stages == 2) fetch_next();
    if (live) {
      const __nv_bfloat16 *kt = reinterpret_cast<const __nv_bfloat16 *>(st + l.kt);
      const __nv_bfloat16 *sk = reinterpret_cast<const __nv_bfloat16 *>(st + l.k);
      const __nv_bfloat16 *sq = reinterpret_cast<const __nv_bfloat16 *>(st + l.q);
      const __nv_bfloat16 *tm = reinterpret_cast<const __nv_bfloat16 *>(st + l.tm);
      const __nv_bfloat16 *pp = reinterpret_cast<const __nv_bfloat16 *>(st + l.pp);
      const __nv_bfloat16 *sv = reinterpret_cast<const __nv_bfloat16 *>(st + l.v);
      const float *eG = reinterpret_cast<const float *>(st + l.gates), *w = eG + kChunk;
      float E[8][4], O[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) E[i][j] = O[i][j] = 0.0f;
      // S0 Kt^T and S0 Q^T (and the planes of S0 kept for the backward pass)
      __nv_bfloat16 *s0 = SAVE ? p.s0 + rec * (2ll * p.dvp * DK) : nullptr;
      {
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks) {
          uint32_t ah[4], al[4], b[4];
          split_tiles(S[2 * ks], S[2 * ks + 1], ah, al);
          if (SAVE) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const long long at = (long long)(r0 + 8 * (q & 1)) * DK + ks * 16 + 8 * (q >> 1) + t2;
              *reinterpret_cast<uint32_t *>(s0 + at) = ah[q];
              *reinterpret_cast<uint32_t *>(s0 + (long long)p.dvp * DK + at) = al[q];
            }
          }
#pragma unroll
          for (int np = 0; np < 4; ++np) {
            if (DELTA) {
              b_rows(b, kt, LD, np * 16, ks * 16, lane);
              mma2(E[2 * np], E[2 * np + 1], ah, b);
              mma2(E[2 * np], E[2 * np + 1], al, b);
              b_rows(b, kt + kChunk * LD, LD, np * 16, ks * 16, lane);
              mma2(E[2 * np], E[2 * np + 1], ah, b);
            }
            if (!SAVE) {
              b_rows(b, sq, LD, np * 16, ks * 16, lane);
              mma2(O[2 * np], O[2 * np + 1], ah, b);
              mma2(O[2 * np], O[2 * np + 1], al, b);
              if (NP == 2) {
                b_rows(b, sq + kChunk * LD, LD, np * 16, ks * 16, lane);
                mma2(O[2 * np], O[2 * np + 1], ah, b);
              }
            }
          }
        }
      }
      // E^T += V^T Tm^T (without the delta rule Tm = I)
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        uint32_t av[NP][4];
#pragma unroll
        for (int c2 = 0; c2 < NP; ++c2) a_cols(av[c2], sv + c2 * kChunk * ldv, ldv, ks * 16, warp * 16, lane);
        if (DELTA) {
#pragma unroll
          for (int np = ks; np < 4; ++np) {
            uint32_t b[4];
            b_rows(b, tm, kLdC, np * 16, ks * 16, lane);
#pragma unroll
            for (int c2 = 0; c2 < NP; ++c2) mma2(E[2 * np], E[2 * np + 1], av[c2], b);
            b_rows(b, tm + kChunk * kLdC, kLdC, np * 16, ks * 16, lane);
            mma2(E[2 * np], E[2 * np + 1], av[0], b);
          }
        } else {
#pragma unroll
          for (int c2 = 0; c2 < NP; ++c2)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 x = unpack2(av[c2][q]);
              float *e = &E[2 * ks + (q >> 1)][2 * (q & 1)];
              e[0] = __fadd_rn(e[0], x.x);
              e[1] = __fadd_rn(e[1], x.y);
            }
        }
      }
      if (!SAVE) {
        // O^T = diag(e^G) (S0 Q^T) + E^T P^T
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 e = *reinterpret_cast<const float2 *>(eG + 8 * i + t2);
          O[i][0] *= e.x; O[i][1] *= e.y; O[i][2] *= e.x; O[i][3] *= e.y;
        }
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          uint32_t ah[4], al[4], b[4];
          split_tiles(E[2 * ks], E[2 * ks + 1], ah, al);
#pragma unroll
          for (int np = ks; np < 4; ++np) {
            b_rows(b, pp, kLdC, np * 16, ks * 16, lane);
            mma2(O[2 * np], O[2 * np + 1], ah, b);
            if (DELTA || NP == 2) mma2(O[2 * np], O[2 * np + 1], al, b);
            b_rows(b, pp + kChunk * kLdC, kLdC, np * 16, ks * 16, lane);
            mma2(O[2 * np], O[2 * np + 1], ah, b);
          }
        }
        const int n = min(kChunk, len - c * kChunk);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int t = 8 * i + t2 + (j & 1), r = r0 + 8 * (j >> 1);
            if (t < n && r < p.d_v)
              store_as(p.o, p.dtype, (start + (long long)c * kChunk + t) * p.o_stride +
                                         (long long)head * p.d_v + r, O[i][j]);
          }
      } else {
        __nv_bfloat16 *et = p.et + rec * (2ll * p.dvp * kChunk);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t hi, lo;
            split2(E[i][2 * h], E[i][2 * h + 1], hi, lo);
            const long long at = (long long)(r0 + 8 * h) * kChunk + 8 * i + t2;
            *reinterpret_cast<uint32_t *>(et + at) = hi;
            *reinterpret_cast<uint32_t *>(et + (long long)p.dvp * kChunk + at) = lo;
          }
      }
      // S = e^{G_C} S0 + (diag(w) E)^T K: each tile's sum starts from zero and joins the
      // state in one fma, so that the tensor cores' rounding does not pile up in it
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 x = *reinterpret_cast<const float2 *>(w + 8 * i + t2);
        E[i][0] *= x.x; E[i][1] *= x.y; E[i][2] *= x.x; E[i][3] *= x.y;
      }
      uint32_t wh[4][4], wl[4][4];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) split_tiles(E[2 * ks], E[2 * ks + 1], wh[ks], wl[ks]);
      const float eC = eG[kChunk - 1];
#pragma unroll
      for (int np = 0; np < DK / 16; ++np) {
        float a0[4] = {0, 0, 0, 0}, a1[4] = {0, 0, 0, 0};
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          uint32_t b[4];
          b_cols(b, sk, LD, ks * 16, np * 16, lane);
          mma2(a0, a1, wh[ks], b);
          mma2(a0, a1, wl[ks], b);
          if (NP == 2) {
            b_cols(b, sk + kChunk * LD, LD, ks * 16, np * 16, lane);
            mma2(a0, a1, wh[ks], b);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          S[2 * np][j] = fmaf(S[2 * np][j], eC, a0[j]);
          S[2 * np + 1][j] = fmaf(S[2 * np + 1][j], eC, a1[j]);
        }
      }
    }
    if (p.stages == 1) {
      __syncthreads();
      fetch_next();
    }
  }
  if (live && p.state_out && !SAVE)
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (r0 + 8 * h < p.d_v)
          *reinterpret_cast<float2 *>(p.state_out + ((long long)blockIdx.x * p.d_v + r0 + 8 * h) * DK +
                                      8 * i + t2) = make_float2(S[i][2 * h], S[i][2 * h + 1]);
}

// -------------------------------------------------------------------------------------
// scan_reverse
// -------------------------------------------------------------------------------------
// The same grid and roles over the chunks backwards: D (at every chunk's end) and R of every
// chunk are kept for scan_grads, dV = R and d_state_in are written.
struct ReverseLayout {
  int kb, k, q, z, d, gates, bytes;
};
__host__ __device__ inline ReverseLayout reverse_layout(int dk, int np, int w, bool delta) {
  const int ld = dk + 8, tile = kChunk * ld * 2, sq = kChunk * kLdC * 2;
  ReverseLayout l{};
  int at = 0;
  l.kb = at; at += delta ? 2 * tile : 0;
  l.k = at; at += np * tile;
  l.q = at; at += np * tile;
  l.z = at; at += 2 * sq;
  l.d = at; at += np * kChunk * (16 * w + 8) * 2;
  l.gates = at; at += 2 * kChunk * 4;
  l.bytes = at;
  return l;
}

template <int DK, int NP, bool DELTA>
__device__ __forceinline__ void reverse_fetch(const ScanParams &p, uint8_t *st, const ReverseLayout &l,
                                              int w, long long token0, int n, long long rec, int head,
                                              int row0, int tid, int threads) {
  constexpr int LD = DK + 8;
  const int qh = head / p.share, ldv = 16 * w + 8;
  const int cols = min(16 * w, p.dvp - row0);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    if (DELTA)
      copy_tile(reinterpret_cast<__nv_bfloat16 *>(st + l.kb) + c * kChunk * LD, LD,
                p.kb + rec * (2 * kChunk * DK) + c * kChunk * DK, DK, kChunk, DK, kChunk, DK, tid, threads);
    copy_tile(reinterpret_cast<__nv_bfloat16 *>(st + l.z) + c * kChunk * kLdC, kLdC,
              (DELTA ? p.z : p.pp) + rec * (2 * kChunk * kChunk) + c * kChunk * kChunk, kChunk, kChunk,
              kChunk, kChunk, kChunk, tid, threads);
  }
#pragma unroll
  for (int c = 0; c < NP; ++c) {
    copy_tile(reinterpret_cast<__nv_bfloat16 *>(st + l.k) + c * kChunk * LD, LD,
              (c ? p.k.lo : p.k.hi) + token0 * p.k.stride + qh * p.k.hstride, p.k.stride, kChunk, DK,
              n, DK, tid, threads);
    copy_tile(reinterpret_cast<__nv_bfloat16 *>(st + l.q) + c * kChunk * LD, LD,
              (c ? p.q.lo : p.q.hi) + token0 * p.q.stride + qh * p.q.hstride, p.q.stride, kChunk, DK,
              n, DK, tid, threads);
    copy_tile(reinterpret_cast<__nv_bfloat16 *>(st + l.d) + c * kChunk * ldv, ldv,
              (c ? p.dO.lo : p.dO.hi) + token0 * p.dO.stride + (long long)head * p.dO.hstride + row0,
              p.dO.stride, kChunk, cols, n, p.dO.hstride - row0, tid, threads);
  }
  const float *gates = p.gates + rec * kGateFloats;
  for (int i = tid; i < 2 * kChunk / 4; i += threads)
    cp16(st + l.gates + 16 * i, gates + 4 * i, true);
}

template <int DK, int NP, bool DELTA>
__global__ void __launch_bounds__(32 * (4 + kLoadWarps)) scan_reverse_kernel(const ScanParams p) {
  constexpr int LD = DK + 8, NT = DK / 8;
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t2 = (lane & 3) * 2;
  const int W = blockDim.x / 32 - kLoadWarps;
  const int seq = blockIdx.x / p.H, head = blockIdx.x % p.H, row0 = blockIdx.y * 16 * W;
  const ReverseLayout l = reverse_layout(DK, NP, W, DELTA);
  const int ldv = 16 * W + 8;
  long long start;
  int len;
  seq_range(p, seq, start, len);
  const int chunks = (len + kChunk - 1) / kChunk, base = slot_base(start, seq);
  const bool loader = warp >= W;
  const int r0 = row0 + warp * 16 + g;
  const bool live = !loader && row0 + warp * 16 < p.dvp;

  float D[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float2 x = make_float2(0.0f, 0.0f);
      if (live && p.d_state_out && r0 + 8 * h < p.d_v)
        x = *reinterpret_cast<const float2 *>(
            p.d_state_out + ((long long)blockIdx.x * p.d_v + r0 + 8 * h) * DK + 8 * i + t2);
      D[i][2 * h] = x.x;
      D[i][2 * h + 1] = x.y;
    }
  const int ltid = tid - 32 * W, lthreads = 32 * kLoadWarps;
  if (loader && chunks > 0) {
    const int c = chunks - 1;
    reverse_fetch<DK, NP, DELTA>(p, smem + (p.stages == 2 ? (c & 1) * l.bytes : 0), l, W,
                                 start + (long long)c * kChunk, len - c * kChunk,
                                 (long long)(base + c) * p.H + head, head, row0, ltid, lthreads);
    cp_commit();
  }
  for (int c = chunks - 1; c >= 0; --c) {
    uint8_t *st = smem + (p.stages == 2 ? (c & 1) * l.bytes : 0);
    if (loader) cp_wait<0>();
    __syncthreads();
    const long long rec = (long long)(base + c) * p.H + head;
    auto fetch_next = [&]() {
      if (loader && c > 0) {
        reverse_fetch<DK, NP, DELTA>(p, smem + (p.stages == 2 ? ((c - 1) & 1) * l.bytes : 0), l, W,
                                     start + (long long)(c - 1) * kChunk, kChunk, rec - p.H, head, row0,
                                     ltid, lthreads);
        cp_commit();
      }
    };
    if (p.stages == 2) fetch_next();
    if (live) {
      const __nv_bfloat16 *kb = reinterpret_cast<const __nv_bfloat16 *>(st + l.kb);
      const __nv_bfloat16 *sk = reinterpret_cast<const __nv_bfloat16 *>(st + l.k);
      const __nv_bfloat16 *sq = reinterpret_cast<const __nv_bfloat16 *>(st + l.q);
      const __nv_bfloat16 *z = reinterpret_cast<const __nv_bfloat16 *>(st + l.z);
      const __nv_bfloat16 *sd = reinterpret_cast<const __nv_bfloat16 *>(st + l.d);
      const float *eG = reinterpret_cast<const float *>(st + l.gates), *w = eG + kChunk;
      const int n = min(kChunk, len - c * kChunk);
      float R[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) R[i][j] = 0.0f;
      __nv_bfloat16 *dd = p.dd + rec * (2ll * p.dvp * DK);
      // D Kb^T; without the delta rule Kb = diag(w) K, applied below
#pragma unroll
      for (int ks = 0; ks < DK / 16; ++ks) {
        uint32_t ah[4], al[4], b[4];
        split_tiles(D[2 * ks], D[2 * ks + 1], ah, al);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const long long at = (long long)(r0 + 8 * (q & 1)) * DK + ks * 16 + 8 * (q >> 1) + t2;
          *reinterpret_cast<uint32_t *>(dd + at) = ah[q];
          *reinterpret_cast<uint32_t *>(dd + (long long)p.dvp * DK + at) = al[q];
        }
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          b_rows(b, DELTA ? kb : sk, LD, np * 16, ks * 16, lane);
          mma2(R[2 * np], R[2 * np + 1], ah, b);
          mma2(R[2 * np], R[2 * np + 1], al, b);
          if (DELTA || NP == 2) {
            b_rows(b, (DELTA ? kb : sk) + kChunk * LD, LD, np * 16, ks * 16, lane);
            mma2(R[2 * np], R[2 * np + 1], ah, b);
          }
        }
      }
      if (!DELTA)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 x = *reinterpret_cast<const float2 *>(w + 8 * i + t2);
          R[i][0] *= x.x; R[i][1] *= x.y; R[i][2] *= x.x; R[i][3] *= x.y;
        }
      // + dO^T Z; the same rows of dO times e^G are the left operand of D's sum
      uint32_t oh[4][4], ol[4][4];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        uint32_t a[NP][4], b[4];
#pragma unroll
        for (int c2 = 0; c2 < NP; ++c2) a_cols(a[c2], sd + c2 * kChunk * ldv, ldv, ks * 16, warp * 16, lane);
#pragma unroll
        for (int np = 0; np <= ks; ++np) {
          b_cols(b, z, kLdC, ks * 16, np * 16, lane);
#pragma unroll
          for (int c2 = 0; c2 < NP; ++c2) mma2(R[2 * np], R[2 * np + 1], a[c2], b);
          b_cols(b, z + kChunk * kLdC, kLdC, ks * 16, np * 16, lane);
          mma2(R[2 * np], R[2 * np + 1], a[0], b);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 e = *reinterpret_cast<const float2 *>(eG + ks * 16 + 8 * (q >> 1) + t2);
          float2 x = unpack2(a[0][q]);
          if (NP == 2) {
            const float2 y = unpack2(a[NP - 1][q]);
            x.x = __fadd_rn(x.x, y.x);
            x.y = __fadd_rn(x.y, y.y);
          }
          split2(x.x * e.x, x.y * e.y, oh[ks][q], ol[ks][q]);
        }
      }
      __nv_bfloat16 *rt = p.rt + rec * (2ll * p.dvp * kChunk);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t hi, lo;
          split2(R[i][2 * h], R[i][2 * h + 1], hi, lo);
          const long long at = (long long)(r0 + 8 * h) * kChunk + 8 * i + t2;
          *reinterpret_cast<uint32_t *>(rt + at) = hi;
          *reinterpret_cast<uint32_t *>(rt + (long long)p.dvp * kChunk + at) = lo;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = 8 * i + t2 + (j & 1), r = r0 + 8 * (j >> 1);
          if (t < n && r < p.d_v)
            store_as(p.o, p.dtype, (start + (long long)c * kChunk + t) * p.o_stride +
                                       (long long)head * p.d_v + r, R[i][j]);
        }
      }
      // D = e^{G_C} D + (diag(e^G) dO)^T Q - (diag(e^G) R)^T K
      uint32_t xh[4][4], xl[4][4];
      if (DELTA) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 e = *reinterpret_cast<const float2 *>(eG + 8 * i + t2);
          R[i][0] *= -e.x; R[i][1] *= -e.y; R[i][2] *= -e.x; R[i][3] *= -e.y;
        }
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) split_tiles(R[2 * ks], R[2 * ks + 1], xh[ks], xl[ks]);
      }
      const float eC = eG[kChunk - 1];
#pragma unroll
      for (int np = 0; np < DK / 16; ++np) {
        float a0[4] = {0, 0, 0, 0}, a1[4] = {0, 0, 0, 0};
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          uint32_t b[4];
          b_cols(b, sq, LD, ks * 16, np * 16, lane);
          mma2(a0, a1, oh[ks], b);
          mma2(a0, a1, ol[ks], b);
          if (NP == 2) {
            b_cols(b, sq + kChunk * LD, LD, ks * 16, np * 16, lane);
            mma2(a0, a1, oh[ks], b);
          }
          if (DELTA) {
            b_cols(b, sk, LD, ks * 16, np * 16, lane);
            mma2(a0, a1, xh[ks], b);
            mma2(a0, a1, xl[ks], b);
            if (NP == 2) {
              b_cols(b, sk + kChunk * LD, LD, ks * 16, np * 16, lane);
              mma2(a0, a1, xh[ks], b);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          D[2 * np][j] = fmaf(D[2 * np][j], eC, a0[j]);
          D[2 * np + 1][j] = fmaf(D[2 * np + 1][j], eC, a1[j]);
        }
      }
    }
    if (p.stages == 1) {
      __syncthreads();
      fetch_next();
    }
  }
  if (live && p.d_state_in)
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (r0 + 8 * h < p.d_v)
          *reinterpret_cast<float2 *>(p.d_state_in + ((long long)blockIdx.x * p.d_v + r0 + 8 * h) * DK +
                                      8 * i + t2) = make_float2(D[i][2 * h], D[i][2 * h + 1]);
}

// -------------------------------------------------------------------------------------
// scan_grads
// -------------------------------------------------------------------------------------
// Grid (slot, head), 8 warps.  Warps 0-3 (group A) own 16 rows each of diag(e^G) dO S0 and
// R S0, warps 4-7 (group B) of E D, dO E^T and R E^T; the value rows are the contraction
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
  l.f = at; at += (4 * kChunk + 2 * kChunk + 3 * kChunk + 4 * kChunk + 16) * 4;
  l.stage = at;
  at = 0;
  l.s0 = at; at += 2 * kGradRows * ld * 2;
  l.d = at; at += 2 * kGradRows * ld * 2;
  l.e = at; at += 2 * kGradRows * kLdC * 2;
  l.r = at; at += 2 * kGradRows * kLdC * 2;
  l.o = at; at += np * kChunk * (kGradRows + 8) * 2;
  l.stage_bytes = at;                                    // holds the [64][dk + 4] fp32 exchange too
  return l;
}

template <int DK, int NP, bool DELTA>
__global__ void __launch_bounds__(kGradThreads) scan_grads_kernel(const ScanParams p) {
  constexpr int LD = DK + 8, NT = DK / 8, LDO = kGradRows + 8, LDX = DK + 4;
  extern __shared__ __align__(16) uint8_t smem[];
  const GradLayout l = grad_layout(DK, NP);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, w4 = warp & 3, g = lane >> 2,
            t2 = (lane & 3) * 2, m0 = w4 * 16;
  const bool groupA = warp < 4;
  const int slot = blockIdx.x, head = blockIdx.y;
  long long token0 = 0;
  const int n = slot_tokens(p, slot, token0);
  if (n == 0) return;
  const int qh = head / p.share;
  const long long rec = (long long)slot * p.H + head;
  __nv_bfloat16 *sk = reinterpret_cast<__nv_bfloat16 *>(smem + l.k);
  __nv_bfloat16 *sq = reinterpret_cast<__nv_bfloat16 *>(smem + l.q);
  __nv_bfloat16 *sx = reinterpret_cast<__nv_bfloat16 *>(smem + l.x);
  float *eG = reinterpret_cast<float *>(smem + l.f), *w = eG + kChunk, *be = w + kChunk,
        *eC = be + kChunk;
  double *G = reinterpret_cast<double *>(eC + kChunk);
  float *rowv = reinterpret_cast<float *>(G + kChunk), *aq = rowv + kChunk, *kw = aq + kChunk,
        *colp = kw + kChunk, *red = colp + 4 * kChunk;
#pragma unroll
  for (int c = 0; c < NP; ++c) {
    copy_tile(sk + c * kChunk * LD, LD, (c ? p.k.lo : p.k.hi) + token0 * p.k.stride + qh * p.k.hstride,
              p.k.stride, kChunk, DK, n, DK, tid, kGradThreads);
    copy_tile(sq + c * kChunk * LD, LD, (c ? p.q.lo : p.q.hi) + token0 * p.q.stride + qh * p.q.hstride,
              p.q.stride, kChunk, DK, n, DK, tid, kGradThreads);
  }
  for (int i = tid; i < kGateFloats / 4; i += kGradThreads)
    cp16(eG + 4 * i, p.gates + rec * kGateFloats + 4 * i, true);
  const int blocks = (p.dvp + kGradRows - 1) / kGradRows;
  auto fetch = [&](int b) {
    uint8_t *st = smem + l.stage + (p.stages == 2 ? (b & 1) * l.stage_bytes : 0);
    const int v0 = b * kGradRows, rows = min(kGradRows, p.dvp - v0);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      copy_tile(reinterpret_cast<__nv_bfloat16 *>(st + l.s0) + c * kGradRows * LD, LD,
                p.s0 + (rec * 2 + c) * p.dvp * DK + (long long)v0 * DK, DK, kGradRows, DK, rows, DK, tid,
                kGradThreads);
      copy_tile(reinterpret_cast<__nv_bfloat16 *>(st + l.d) + c * kGradRows * LD, LD,
                p.dd + (rec * 2 + c) * p.dvp * DK + (long long)v0 * DK, DK, kGradRows, DK, rows, DK, tid,
                kGradThreads);
      copy_tile(reinterpret_cast<__nv_bfloat16 *>(st + l.e) + c * kGradRows * kLdC, kLdC,
                p.et + (rec * 2 + c) * p.dvp * kChunk + (long long)v0 * kChunk, kChunk, kGradRows, kChunk,
                rows, kChunk, tid, kGradThreads);
      copy_tile(reinterpret_cast<__nv_bfloat16 *>(st + l.r) + c * kGradRows * kLdC, kLdC,
                p.rt + (rec * 2 + c) * p.dvp * kChunk + (long long)v0 * kChunk, kChunk, kGradRows, kChunk,
                rows, kChunk, tid, kGradThreads);
    }
#pragma unroll
    for (int c = 0; c < NP; ++c)
      copy_tile(reinterpret_cast<__nv_bfloat16 *>(st + l.o) + c * kChunk * LDO, LDO,
                (c ? p.dO.lo : p.dO.hi) + token0 * p.dO.stride + (long long)head * p.dO.hstride + v0,
                p.dO.stride, kChunk, kGradRows, n, p.dO.hstride - v0, tid, kGradThreads);
    cp_commit();
  };
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

  fetch(0);
  for (int b = 0; b < blocks; ++b) {
    cp_wait<0>();
    __syncthreads();
    if (p.stages == 2 && b + 1 < blocks) fetch(b + 1);
    uint8_t *st = smem + l.stage + (p.stages == 2 ? (b & 1) * l.stage_bytes : 0);
    const __nv_bfloat16 *s0 = reinterpret_cast<const __nv_bfloat16 *>(st + l.s0);
    const __nv_bfloat16 *dd = reinterpret_cast<const __nv_bfloat16 *>(st + l.d);
    const __nv_bfloat16 *se = reinterpret_cast<const __nv_bfloat16 *>(st + l.e);
    const __nv_bfloat16 *sr = reinterpret_cast<const __nv_bfloat16 *>(st + l.r);
    const __nv_bfloat16 *so = reinterpret_cast<const __nv_bfloat16 *>(st + l.o);
    for (int i = tid; i < kGradRows * DK / 2; i += kGradThreads) {        // <D, S0>
      const int at = (i / (DK / 2)) * LD + (i % (DK / 2)) * 2;
      auto pair = [&](const __nv_bfloat16 *x) {
        const float2 hi = unpack2(*reinterpret_cast<const uint32_t *>(x + at));
        const float2 lo = unpack2(*reinterpret_cast<const uint32_t *>(x + kGradRows * LD + at));
        return make_float2(__fadd_rn(hi.x, lo.x), __fadd_rn(hi.y, lo.y));
      };
      const float2 x = pair(s0), y = pair(dd);
      ds = fmaf(x.x, y.x, fmaf(x.y, y.y, ds));
    }
#pragma unroll
    for (int kk = 0; kk < kGradRows; kk += 16) {
      uint32_t ao[NP][4], ar[2][4], b4[4];
#pragma unroll
      for (int c = 0; c < NP; ++c) a_rows(ao[c], so + c * kChunk * LDO, LDO, m0, kk, lane);
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (DELTA) a_cols(ar[c], sr + c * kGradRows * kLdC, kLdC, kk, m0, lane);
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
        for (int c = 0; c < 2; ++c) a_cols(ae[c], se + c * kGradRows * kLdC, kLdC, kk, m0, lane);
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

  // row i of a planed tile, columns 8c + t2, +1
  auto row_pair = [&](const __nv_bfloat16 *x, int row, int col) {
    float2 v = unpack2(*reinterpret_cast<const uint32_t *>(x + row * LD + col));
    if (NP == 2) {
      const float2 y = unpack2(*reinterpret_cast<const uint32_t *>(x + kChunk * LD + row * LD + col));
      v.x = __fadd_rn(v.x, y.x);
      v.y = __fadd_rn(v.y, y.y);
    }
    return v;
  };
  if (groupA) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = m0 + g + 8 * h;
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const float2 q = row_pair(sq, t, 8 * i + t2);
        acc[i][2 * h] *= eG[t];
        acc[i][2 * h + 1] *= eG[t];
        s = fmaf(q.x, acc[i][2 * h], fmaf(q.y, acc[i][2 * h + 1], s));
        if (DELTA) {
          const float2 k = row_pair(sk, t, 8 * i + t2);
          acc2[i][2 * h] *= -eG[t];
          acc2[i][2 * h + 1] *= -eG[t];
          s = fmaf(k.x, acc2[i][2 * h], fmaf(k.y, acc2[i][2 * h + 1], s));
        }
      }
      s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
      s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
      if ((lane & 3) == 0) aq[t] = s;
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = m0 + g + 8 * h;
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const float2 k = row_pair(sk, t, 8 * i + t2);
        s = fmaf(k.x, acc[i][2 * h], fmaf(k.y, acc[i][2 * h + 1], s));
        acc[i][2 * h] *= w[t];
        acc[i][2 * h + 1] *= w[t];
      }
      s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
      s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
      if ((lane & 3) == 0) kw[t] = s;
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
      const __nv_bfloat16 *left = ps ? sk : sq;
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
      __nv_bfloat16 *out = sx + ps * 2 * kChunk * kLdC;
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
              const float m = z * x[i][2 * h + j];
              y[j] = z * be[s];
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
      if ((lane & 3) == 0) rowv[m0 + g + 8 * h] = rs[h];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float c = cs[i][j];
        c += __shfl_xor_sync(0xFFFFFFFFu, c, 4);
        c += __shfl_xor_sync(0xFFFFFFFFu, c, 8);
        c += __shfl_xor_sync(0xFFFFFFFFu, c, 16);
        if (g == 0) colp[w4 * kChunk + 8 * i + t2 + j] = c;
      }
  }
  __syncthreads();
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
          if (p.parts) store_pair(p.dq, 0, (tok * p.H + head) * DK + 8 * i + t2, acc[i][2 * h], acc[i][2 * h + 1]);
          else store_pair(p.dq, p.dtype, tok * p.dq_stride + (long long)head * DK + 8 * i + t2, acc[i][2 * h], acc[i][2 * h + 1]);
        }
        if (DELTA)
          *reinterpret_cast<float2 *>(reinterpret_cast<float *>(smem + l.stage) + t * LDX + 8 * i + t2) =
              make_float2(acc2[i][2 * h], acc2[i][2 * h + 1]);
      }
    }
  } else {
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      if (ks >= w4) {
        uint32_t a[4][4], b4[4];
#pragma unroll
        for (int c = 0; c < (DELTA ? 4 : 2); ++c) a_cols(a[c], sx + c * kChunk * kLdC, kLdC, ks * 16, m0, lane);
#pragma unroll
        for (int np = 0; np < DK / 16; ++np) {
          b_cols(b4, sq, LD, ks * 16, np * 16, lane);
          mma2(acc[2 * np], acc[2 * np + 1], a[0], b4);
          mma2(acc[2 * np], acc[2 * np + 1], a[1], b4);
          if (NP == 2) {
            b_cols(b4, sq + kChunk * LD, LD, ks * 16, np * 16, lane);
            mma2(acc[2 * np], acc[2 * np + 1], a[0], b4);
          }
          if (DELTA) {
            b_cols(b4, sk, LD, ks * 16, np * 16, lane);
            mma2(acc[2 * np], acc[2 * np + 1], a[2], b4);
            mma2(acc[2 * np], acc[2 * np + 1], a[3], b4);
            if (NP == 2) {
              b_cols(b4, sk + kChunk * LD, LD, ks * 16, np * 16, lane);
              mma2(acc[2 * np], acc[2 * np + 1], a[2], b4);
            }
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
          if (p.parts) store_pair(p.dk, 0, (tok * p.H + head) * DK + 8 * i + t2, x.x, x.y);
          else store_pair(p.dk, p.dtype, tok * p.dk_stride + (long long)head * DK + 8 * i + t2, x.x, x.y);
        }
    }
  } else if (warp == 0) {
    // gates: two tokens a lane, sums over t >= r from the chunk's end
    float dsum = 0.0f;
    for (int i = 0; i < kGradThreads / 32; ++i) dsum += red[i];
    double dG[2], tot = 0.0;
    float db[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      const float c = (colp[t] + colp[kChunk + t]) + (colp[2 * kChunk + t] + colp[3 * kChunk + t]);
      db[i] = fmaf(eC[t], kw[t], c);
      dG[i] = (double)rowv[t] - (double)be[t] * db[i] + aq[t];
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
        p.dbeta[at] = db[i];
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
    const long long at = tok * (second ? p.dk_stride : p.dq_stride) + (long long)h * dk + c;
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
        load4(p.uk, p.dtype, tok * p.uk_stride + qo + 4 * LPR * c, x);
        load4(p.uq, p.dtype, tok * p.uq_stride + qo + 4 * LPR * c, y);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) { k[4 * c + e] = x[e]; q[4 * c + e] = y[e]; }
    }
#pragma unroll
    for (int r = 0; r < kRecRows; ++r) v[r] = 0.0f;
    if (on) {
      a = expf(__ldg(p.log_alpha + tok * p.H + head));
      b = __ldg(p.beta + tok * p.H + head);
      const long long vo = tok * p.uv_stride + (long long)head * p.d_v + row;
#pragma unroll
      for (int r = 0; r < kRecRows; ++r)
        v[r] = p.dtype == 0 ? __ldg(static_cast<const float *>(p.uv) + vo + r)
               : p.dtype == 1 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p.uv)[vo + r])
                              : __half2float(static_cast<const __half *>(p.uv)[vo + r]);
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
// kernels of one key width: [np - 1][delta]
struct ScanKernels {
  ScanFn prep[2][2][2];                // [np - 1][delta][backward]
  ScanFn chain[2][2][2];               // [np - 1][delta][save]
  ScanFn reverse[2][2];
  ScanFn grads[2][2];
};

}  // namespace scan
}  // namespace lores
