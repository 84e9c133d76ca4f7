// lores_scan.cu -- C entry points of the state scan and its backward pass: checks, workspace
// layout, launches.  The kernels and the mathematics are in lores_scan.cuh.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "lores.h"
#include "lores_host.h"
#include "lores_scan.cuh"

namespace lores {
namespace scan {

void scan_kernels_16_1(ScanKernels &t);
void scan_kernels_16_2(ScanKernels &t);
void scan_kernels_32_1(ScanKernels &t);
void scan_kernels_32_2(ScanKernels &t);
void scan_kernels_64_1(ScanKernels &t);
void scan_kernels_64_2(ScanKernels &t);
void scan_kernels_128_1(ScanKernels &t);
void scan_kernels_128_2(ScanKernels &t);

}  // namespace scan
}  // namespace lores

using namespace lores;
using namespace lores::scan;

namespace {

// Sequences up to this many tokens go token by token: the chunk kernels always pay for 64.  Measured, bf16, heads of
// 128 x 128 with the delta rule, chunks / token by token: 64 sequences of 32 heads 350 / 287 us for 32 tokens and
// 360 / 425 us for 48, one sequence 20.5 / 18.9 and 20.7 / 27.0 us; without it, 64 sequences of 128 heads of 64 x 128 on 8
// pairs of q and k, 414 / 364 us for 24 tokens and 420 / 467 us for 32.  (Narrower heads and fp32 would bear more: 32 heads
// of 64 x 64, 48 tokens 176 / 111, fp32 heads of 128 x 128 446 / 402.)
int recurrent_most(int delta) { return delta ? 32 : 24; }
constexpr int kMaxDevices = 64;

struct Kernels {
  ScanKernels by_width[4];             // 16, 32, 64, 128
  ScanFn recurrent[5][2];              // 16 .. 256, delta
  Kernels() {
    scan_kernels_16_1(by_width[0]); scan_kernels_16_2(by_width[0]);
    scan_kernels_32_1(by_width[1]); scan_kernels_32_2(by_width[1]);
    scan_kernels_64_1(by_width[2]); scan_kernels_64_2(by_width[2]);
    scan_kernels_128_1(by_width[3]); scan_kernels_128_2(by_width[3]);
    recurrent[0][0] = scan_recurrent_kernel<16, false>;  recurrent[0][1] = scan_recurrent_kernel<16, true>;
    recurrent[1][0] = scan_recurrent_kernel<32, false>;  recurrent[1][1] = scan_recurrent_kernel<32, true>;
    recurrent[2][0] = scan_recurrent_kernel<64, false>;  recurrent[2][1] = scan_recurrent_kernel<64, true>;
    recurrent[3][0] = scan_recurrent_kernel<128, false>; recurrent[3][1] = scan_recurrent_kernel<128, true>;
    recurrent[4][0] = scan_recurrent_kernel<256, false>; recurrent[4][1] = scan_recurrent_kernel<256, true>;
  }
};
const Kernels &kernels() {
  static const Kernels k;
  return k;
}

int width_index(int dk) {
  return dk == 16 ? 0 : dk == 32 ? 1 : dk == 64 ? 2 : dk == 128 ? 3 : dk == 256 ? 4 : -1;
}

// A configuration with its defaults filled in.
struct Shape {
  lores_scan_config c;
  int np, dvp, n_slots;
  bool recurrent;
};

lores_status shape_of(const lores_scan_config *cfg, bool backward, Shape &s) {
  if (!cfg) return LORES_ERR_INVALID_ARG;
  lores_scan_config &c = s.c;
  c = *cfg;
  if (c.n_seq < 1 || c.total < 0 || c.total > 0x7FFFFFFFll || c.max_len < 0 || c.heads < 1 ||
      c.heads > 65535 || c.heads_qk < 0 || c.d_v < 4 || c.d_v > 4096 || c.d_v % 4 || width_index(c.d_k) < 0 ||
      c.delta < 0 || c.delta > 1 || c.dtype < LORES_F32 || c.dtype > LORES_F16 || c.device < 0)
    return LORES_ERR_INVALID_ARG;
  if (c.heads_qk == 0) c.heads_qk = c.heads;
  if (c.heads % c.heads_qk) return LORES_ERR_INVALID_ARG;
  if (c.max_len == 0 || c.max_len > c.total) c.max_len = c.total;
  // (grids count sequences and chunks times heads in 31 bits)
  if ((c.total / kChunk + c.n_seq) * c.heads > 0x7FFFFFFFll) return LORES_ERR_INVALID_ARG;
  const long long wq = (long long)c.heads_qk * c.d_k, wv = (long long)c.heads * c.d_v;
  int64_t *st[4] = {&c.q_stride, &c.k_stride, &c.v_stride, &c.o_stride};
  for (int i = 0; i < 4; ++i) {
    const long long width = i < 2 ? wq : wv;
    if (*st[i] == 0) *st[i] = width;
    if (*st[i] < width || *st[i] % 4 || *st[i] > (1ll << 40)) return LORES_ERR_INVALID_ARG;
  }
  if (backward && c.d_k == 256) return LORES_ERR_UNSUPPORTED;
  s.np = c.dtype == LORES_F32 ? 2 : 1;           // fp16 planes that hold the inputs
  s.dvp = (c.d_v + 15) / 16 * 16;
  s.n_slots = (int)(c.total / kChunk + c.n_seq);
  s.recurrent = !backward && (c.max_len <= recurrent_most(c.delta) || c.d_k == 256);
  return LORES_OK;
}

// Hands out the workspace's parts in one order, for sizing and for use.
struct Carver {
  uint8_t *base;
  unsigned long long at = 256;         // the first 256 bytes hold the error word
  template <class T>
  T *take(unsigned long long count) {
    T *r = base ? reinterpret_cast<T *>(base + at) : nullptr;
    at += (count * sizeof(T) + 255) / 256 * 256;
    return r;
  }
};

// Lays the workspace out for the call and returns its bytes.
unsigned long long layout(const Shape &s, bool backward, uint8_t *ws, ScanParams &p) {
  const lores_scan_config &c = s.c;
  Carver w{ws};
  p.flag = reinterpret_cast<unsigned *>(ws);
  if (s.recurrent) return w.at;
  const unsigned long long recs = (unsigned long long)s.n_slots * c.heads, sq = 2 * kTri,
                           tile = 2ull * kChunk * c.d_k, rows = (unsigned long long)s.dvp;
  p.khat = w.take<__half>((unsigned long long)s.n_slots * c.heads_qk * s.np * kChunk * c.d_k);
  p.qhat = w.take<__half>((unsigned long long)s.n_slots * c.heads_qk * s.np * kChunk * c.d_k);
  p.gates = w.take<float>(recs * kGateFloats);
  p.seqs = w.take<longlong2>(s.c.n_seq);
  if (!backward || !c.delta) p.pp = w.take<__half>(recs * sq);
  if (c.delta) {
    p.tm = w.take<__half>(recs * sq);
    p.kt = w.take<__half>(recs * tile);
  }
  if (!backward) return w.at;
  if (c.delta) {
    p.z = w.take<__half>(recs * sq);
    p.kb = w.take<__half>(recs * tile);
  }
  p.s0 = w.take<__half>(recs * 2 * rows * c.d_k);
  p.dd = w.take<__half>(recs * 2 * rows * c.d_k);
  p.et = w.take<__half>(recs * 2 * rows * kChunk);
  p.rt = w.take<__half>(recs * 2 * rows * kChunk);
  for (float *&x : p.scales) x = w.take<float>(recs * (rows / 16));
  p.slot_tokens = w.take<longlong2>(s.n_slots);
  if (c.heads != c.heads_qk) {
    const unsigned long long n = (unsigned long long)c.total * c.heads * c.d_k;
    p.dq = w.take<float>(n);
    p.dk = w.take<float>(n);
  }
  return w.at;
}

ScanParams params_of(const Shape &s) {
  const lores_scan_config &c = s.c;
  ScanParams p{};
  p.n_seq = c.n_seq;
  p.H = c.heads;
  p.share = c.heads / c.heads_qk;
  p.d_v = c.d_v;
  p.dvp = s.dvp;
  p.dtype = c.dtype;
  p.n_slots = s.n_slots;
  p.max_len = (int)c.max_len;
  p.total = c.total;
  p.q_stride = c.q_stride;
  p.k_stride = c.k_stride;
  p.v_stride = c.v_stride;
  p.o_stride = c.o_stride;
  // rows of a 16-bit type are 16-byte aligned where strides and widths are multiples of 8
  p.qk16 = c.dtype == LORES_F32 || (c.q_stride % 8 == 0 && c.k_stride % 8 == 0);
  p.v16 = c.dtype == LORES_F32 || (c.v_stride % 8 == 0 && c.d_v % 8 == 0);
  p.o16 = c.dtype == LORES_F32 || (c.o_stride % 8 == 0 && c.d_v % 8 == 0);
  p.stages = 2;
  return p;
}

constexpr int kMaxShared = 232448;     // dynamic shared memory of one CTA

template <class... Args>
cudaError_t launch_early(const void *fn, dim3 grid, int threads, int smem, cudaStream_t s, bool early,
                         const Args *...args) {
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t l{};
  l.gridDim = grid;
  l.blockDim = dim3(threads);
  l.dynamicSmemBytes = smem;
  l.stream = s;
  l.attrs = &a;
  l.numAttrs = early ? 1 : 0;
  void *list[] = {const_cast<Args *>(args)...};
  return cudaLaunchKernelExC(&l, fn, list);
}

// A kernel's dynamic shared memory differs from call to call; its limit is raised once per device.
// early: it may start beside the kernel before it (see wait_before).
cudaError_t launch(ScanFn fn, dim3 grid, int threads, int smem, cudaStream_t s, int device, const ScanParams &p,
                   bool early, std::atomic<unsigned long long> &raised) {
  if (smem > 48 * 1024) {
    const unsigned long long bit = device < kMaxDevices ? 1ull << device : 0;
    if (!bit || !(raised.load(std::memory_order_acquire) & bit)) {
      const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(fn),
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared);
      if (e != cudaSuccess) return e;
      raised.fetch_or(bit, std::memory_order_release);
    }
  }
  return launch_early(reinterpret_cast<const void *>(fn), grid, threads, smem, s, early, &p);
}

int sm_count(int device) {
  static std::atomic<int> known[kMaxDevices];
  if (device < kMaxDevices) {
    const int n = known[device].load(std::memory_order_relaxed);
    if (n) return n;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || n < 1) n = 148;
  if (device < kMaxDevices) known[device].store(n, std::memory_order_relaxed);
  return n;
}

lores_status device_ok(int device) {
  static std::atomic<int> known[kMaxDevices];
  if (device < kMaxDevices && known[device].load(std::memory_order_relaxed) == 1) return LORES_OK;
  int major = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device) != cudaSuccess) {
    (void)cudaGetLastError();
    return LORES_ERR_CUDA;
  }
  if (major != 10) return LORES_ERR_UNSUPPORTED;
  if (device < kMaxDevices) known[device].store(1, std::memory_order_relaxed);
  return LORES_OK;
}

// Blocks of 16 value rows per CTA of a walk: a CTA's blocks share one fetch of a chunk's tiles, but the CTAs
// should fill the SMs.  Two blocks even where that leaves a quarter of the SMs idle (one sequence of 8192 tokens and 32
// heads of 128 x 128, when 16-bit outputs took one plane: one block per CTA 516 us, two 300), four, without the delta
// rule, only for several rounds of CTAs (heads of 64 x 128: backward 6400 tokens, 64 heads 901 us a call against 933 with
// two blocks; 64 sequences of 32 tokens, 128 heads 488 against 572, of 4 x 2000 tokens 491 against 483; 159 against 146 us
// with 192 CTAs of four).
int walk_blocks(const Shape &s, WalkKind kind) {
  const long long walks = (long long)s.c.n_seq * s.c.heads;
  const int blocks = s.dvp / 16, sms = sm_count(s.c.device);
  const auto ctas = [&](int rb) { return walks * ((blocks + rb - 1) / rb); };
  // the two walks of a backward call side by side, where one of these numbers lets them
  if (kind != kForward)
    for (int rb = 1; rb <= std::min(2, blocks); ++rb)
      if (2 * ctas(rb) <= sms) return rb;
  if (max_blocks(s.np, s.c.delta, kind) == 4 && blocks >= 4 && ctas(4) >= 3ll * sms) return 4;
  return blocks >= 2 && ctas(2) >= sms / 2 ? 2 : 1;
}

bool aligned4(const void *x) { return (reinterpret_cast<uintptr_t>(x) & 3u) == 0; }
bool given16(const void *x, bool needed) { return aligned16(x) && (x || !needed); }

cudaError_t run_prep(const Shape &s, bool backward, ScanParams p, cudaStream_t st) {
  const lores_scan_config &c = s.c;
  static std::atomic<unsigned long long> raised[4][2][2][2];
  const int wi = width_index(c.d_k);
  if (c.n_seq > kFewSeqs) {
    scan_sequences_kernel<<<1, kSeqThreads, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  // as many of the heads that share q and k per CTA as leave every SM its four CTAs
  p.hpc = 1;
  for (int d = 2; d <= p.share; ++d)
    if (p.share % d == 0 && (long long)s.n_slots * (c.heads / d) >= 4ll * sm_count(c.device)) p.hpc = d;
  return launch(kernels().by_width[wi].prep[s.np - 1][c.delta][backward], dim3(s.n_slots, c.heads / p.hpc), kPrepThreads,
                prep_layout(c.d_k, s.np, p.hpc > 1).bytes, st, c.device, p, false,
                raised[wi][s.np - 1][c.delta][backward]);
}

long long walk_ctas(const Shape &s, WalkKind kind) {
  const int rb = walk_blocks(s, kind);
  return (long long)s.c.n_seq * s.c.heads * ((s.dvp / 16 + rb - 1) / rb);
}

// Kernels that fill the GPU more than once start after the one before them: started early, their CTAs hold places on
// SMs in an order that cost 2 to 9 % (backward 2 x 4096 tokens, 16 heads 777 -> 815 us; forward without the delta rule,
// 7897 tokens, 128 heads 395 -> 431 us; 2 x 2048 tokens, 8 heads 56 -> 64 us).  Where each has an SM per CTA, early
// starts hide the launches (forward 1024 tokens, 4 heads of 64 x 64 in fp32 46 -> 42 us, backward 94 -> 64 us), and the
// two walks of a backward call run side by side where both fit (4096 tokens, 16 heads of 128 x 128 546 -> 398 us, 2048
// tokens, 8 heads 224 -> 174 us).
bool early_walk(const Shape &s, WalkKind kind) {
  const int sms = sm_count(s.c.device);
  if (kind == kReverse) return walk_ctas(s, kRecompute) + walk_ctas(s, kReverse) <= sms;
  return (long long)s.n_slots * s.c.heads <= sms && walk_ctas(s, kind) <= sms;
}
bool early_grads(const Shape &s) { return (long long)s.n_slots * s.c.heads <= sm_count(s.c.device); }

cudaError_t run_walk(const Shape &s, WalkKind kind, ScanParams p, cudaStream_t st) {
  const lores_scan_config &c = s.c;
  static std::atomic<unsigned long long> raised[4][2][2][kWalkKinds];
  const int wi = width_index(c.d_k), nh = state_warps(c.d_k);
  p.rb = walk_blocks(s, kind);
  p.early = early_walk(s, kind);
  const WalkLayout l = walk_layout(c.d_k, s.np, p.rb, nh, c.delta, kind);
  p.stages = 2 * l.bytes + p.rb * l.tail + kWalkEnd <= kMaxShared ? 2 : 1;
  return launch(kernels().by_width[wi].walk[s.np - 1][c.delta][kind],
                dim3(c.n_seq * c.heads, (s.dvp / 16 + p.rb - 1) / p.rb), 32 * p.rb * (nh + kSideWarps + 1),
                p.stages * l.bytes + p.rb * l.tail + kWalkEnd, st, c.device, p, p.early != 0,
                raised[wi][s.np - 1][c.delta][kind]);
}

cudaError_t run_grads(const Shape &s, ScanParams p, cudaStream_t st) {
  const lores_scan_config &c = s.c;
  static std::atomic<unsigned long long> raised[4][2][2];
  const int wi = width_index(c.d_k);
  const GradLayout l = grad_layout(c.d_k, s.np, s.dvp, c.delta);
  const int most = grad_halves(s.np, c.delta) ? (kMaxShared + 1024) / 2 - 1024 : kMaxShared;
  p.stages = grad_bytes(l, c.d_k, 2, c.delta) <= most ? 2 : 1;
  return launch(kernels().by_width[wi].grads[s.np - 1][c.delta], dim3((unsigned)s.n_slots * c.heads),
                grad_threads(s.np, c.delta), grad_bytes(l, c.d_k, p.stages, c.delta), st, c.device, p, early_grads(s),
                raised[wi][s.np - 1][c.delta]);
}

lores_status check_inputs(const Shape &s, const void *q, const void *k, const void *v, const float *log_alpha,
                          const float *beta, const int32_t *offsets, const float *state_in, const void *workspace) {
  const bool any = s.c.total > 0;
  if (!given16(q, any) || !given16(k, any) || !given16(v, any) || !aligned4(log_alpha) || !aligned4(beta) ||
      (any && (!log_alpha || !beta)) || !aligned4(offsets) || !given16(state_in, false) ||
      !given16(workspace, true))
    return LORES_ERR_INVALID_ARG;
  if (!offsets && s.c.total % s.c.n_seq) return LORES_ERR_INVALID_ARG;
  return LORES_OK;
}

}  // namespace

extern "C" {

lores_status lores_scan_workspace(const lores_scan_config *cfg, int32_t backward, uint64_t *bytes) {
  if (!bytes || backward < 0 || backward > 1) return LORES_ERR_INVALID_ARG;
  Shape s;
  const lores_status st = shape_of(cfg, backward != 0, s);
  if (st != LORES_OK) return st;
  ScanParams p = params_of(s);
  *bytes = layout(s, backward != 0, nullptr, p);
  return LORES_OK;
}

lores_status lores_scan_forward(const lores_scan_config *cfg, const void *q, const void *k, const void *v,
                                const float *log_alpha, const float *beta, const int32_t *offsets,
                                const float *state_in, void *o, float *state_out, void *workspace,
                                uint64_t workspace_bytes, void *stream) {
  Shape s;
  lores_status st = shape_of(cfg, false, s);
  if (st == LORES_OK) st = check_inputs(s, q, k, v, log_alpha, beta, offsets, state_in, workspace);
  if (st != LORES_OK) return st;
  if (!given16(o, s.c.total > 0) || !given16(state_out, false)) return LORES_ERR_INVALID_ARG;
  ScanParams p = params_of(s);
  if (layout(s, false, static_cast<uint8_t *>(workspace), p) > workspace_bytes)
    return LORES_ERR_INVALID_ARG;
  const lores_scan_config &c = s.c;
  if ((st = device_ok(c.device)) != LORES_OK) return st;
  DeviceGuard guard(c.device);
  if (!guard.ok) return LORES_ERR_CUDA;
  p.q = q;
  p.k = k;
  p.v = v;
  p.offsets = offsets;
  p.log_alpha = log_alpha;
  p.beta = beta;
  p.state_in = state_in;
  p.state_out = state_out;
  p.o = o;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (s.recurrent) {
    const int lpr = c.d_k / 16, groups = c.d_v / kRecRows;
    const int threads = std::min(kRecThreads, (groups * lpr + 31) / 32 * 32), rows = threads / lpr * kRecRows;
    kernels().recurrent[width_index(c.d_k)][c.delta]<<<dim3(c.n_seq * c.heads, (c.d_v + rows - 1) / rows), threads, 0,
                                                       cs>>>(p);
    return cuda_status(cudaGetLastError());
  }
  cudaError_t e = run_prep(s, false, p, cs);
  if (e == cudaSuccess) e = run_walk(s, kForward, p, cs);
  return cuda_status(e);
}

lores_status lores_scan_backward(const lores_scan_config *cfg, const void *q, const void *k, const void *v,
                                 const float *log_alpha, const float *beta, const int32_t *offsets,
                                 const float *state_in, const void *d_o, const float *d_state_out, void *dq,
                                 void *dk, void *dv, float *dlog_alpha, float *dbeta, float *d_state_in,
                                 void *workspace, uint64_t workspace_bytes, void *stream) {
  Shape s;
  lores_status st = shape_of(cfg, true, s);
  if (st == LORES_OK) st = check_inputs(s, q, k, v, log_alpha, beta, offsets, state_in, workspace);
  if (st != LORES_OK) return st;
  const bool any = s.c.total > 0;
  if (!given16(d_o, any) || !given16(d_state_out, false) || !given16(dq, any) || !given16(dk, any) ||
      !given16(dv, any) || !aligned4(dlog_alpha) || !aligned4(dbeta) || (any && (!dlog_alpha || !dbeta)) ||
      !given16(d_state_in, false))
    return LORES_ERR_INVALID_ARG;
  ScanParams p = params_of(s);
  if (layout(s, true, static_cast<uint8_t *>(workspace), p) > workspace_bytes)
    return LORES_ERR_INVALID_ARG;
  const lores_scan_config &c = s.c;
  if ((st = device_ok(c.device)) != LORES_OK) return st;
  DeviceGuard guard(c.device);
  if (!guard.ok) return LORES_ERR_CUDA;
  p.q = q;
  p.k = k;
  p.v = v;
  p.offsets = offsets;
  p.log_alpha = log_alpha;
  p.beta = beta;
  p.state_in = state_in;
  p.d_state_out = d_state_out;
  p.d_state_in = d_state_in;
  p.o = const_cast<void *>(d_o);
  p.dv = dv;
  p.dlog_alpha = dlog_alpha;
  p.dbeta = dbeta;
  p.parts = c.heads != c.heads_qk;
  const float *parts_q = static_cast<const float *>(p.dq), *parts_k = static_cast<const float *>(p.dk);
  if (!p.parts) {
    p.dq = dq;
    p.dk = dk;
  }
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e = run_prep(s, true, p, cs);
  if (e == cudaSuccess) e = run_walk(s, kRecompute, p, cs);
  if (e == cudaSuccess) e = run_walk(s, kReverse, p, cs);
  if (e == cudaSuccess) e = run_grads(s, p, cs);
  if (e == cudaSuccess && p.parts && any) {
    p.dq = dq;
    p.dk = dk;
    const long long n = (long long)s.n_slots * kChunk * c.heads_qk * (c.d_k / 4) * 2;
    const unsigned blocks = (unsigned)std::min<long long>((n + 255) / 256, 32ll * sm_count(c.device));
    const int dk = c.d_k;
    e = launch_early(reinterpret_cast<const void *>(&scan_shared_kernel), dim3(blocks), 256, 0, cs, early_grads(s), &p,
                     &parts_q, &parts_k, &dk);
  }
  return cuda_status(e);
}

lores_status lores_scan_check_errors(const lores_scan_config *cfg, const void *workspace, void *stream) {
  if (!cfg || !workspace || cfg->device < 0) return LORES_ERR_INVALID_ARG;
  DeviceGuard guard(cfg->device);
  if (!guard.ok) return LORES_ERR_CUDA;
  unsigned f = 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyAsync(&f, workspace, sizeof f, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_status(e);
  if (f & kFlagWait) return LORES_ERR_TIMEOUT;
  return f ? LORES_ERR_INVALID_ARG : LORES_OK;
}

}  // extern "C"
