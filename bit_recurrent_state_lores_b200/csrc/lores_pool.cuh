// lores_pool.cuh -- states written into and read out of chosen slots of a handle (sm_100a).
//
// The state of sequence (slot) b is what lores_load_state would quantize and
// lores_dequant_state would dequantize for it; here a list of slots says which ones, so that a
// serving engine moves single sequences in and out of a running batch.  Entry i of the list is one
// [H][d_v][d_k] block of the caller's buffer.
//
// Memory bound: d_k/16 lanes share a row and a lane owns 16 consecutive columns (the code
// format's unit), i.e. 64 bytes of fp32, moved as two 32-byte accesses so that every sector
// is touched by one instruction.  Grid (entry, head, group of rows): no division per row.  64 states
// of 32 heads of 128 x 128 in fp32 into and out of int8 (169 MB each way): written in 33 us, 5.1
// TB/s, read in 27 us, 6.3 TB/s; 96 of them read as bf16 (152 MB): 27 us, 5.6 TB/s.
#pragma once
#include "lores_device.cuh"

namespace lores {

constexpr int kPoolThreads = 256;
constexpr int kPoolRows = 2;    // rows per lane, whose loads are in flight together

struct PoolParams {
  uint8_t *codes;
  float *scales;
  const LaneFmt *fmt;
  const int64_t *head_off;
  long long seq_bytes;
  int H, d_v, ng, G, axis, batch;
  int n;                        // entries
  const int *slots;             // device [n], or null: entry i is slot i
  const void *src;              // write: the caller's states
  void *dst;                    // read
  int dtype;                    // 0 fp32, 1 bf16, 2 fp16
  int wide;                     // the caller's buffer is 32-byte aligned
  uint32_t step_key;
  int stochastic;
  unsigned *flag;
  LORES_RANGES
};

// 32 bytes at once (a 32-byte aligned address).
__device__ __forceinline__ void ld32(const void *src, uint32_t (&w)[8]) {
  asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(src));
}
__device__ __forceinline__ void st32(void *dst, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void get32(const void *src, uint32_t (&w)[8], bool wide) {
  if (wide) {
    ld32(src, w);
    return;
  }
  const uint4 a = __ldg(static_cast<const uint4 *>(src)), b = __ldg(static_cast<const uint4 *>(src) + 1);
  w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
  w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}
__device__ __forceinline__ void put32(void *dst, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    st32(dst, w);
    return;
  }
  static_cast<uint4 *>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  static_cast<uint4 *>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// 16 entries of a state row in the caller's type (element index i, a multiple of 16).
__device__ __forceinline__ void load_row16(const PoolParams &p, long long i, float (&x)[16]) {
  uint32_t w[8];
  if (p.dtype == 0) {
    const float *src = static_cast<const float *>(p.src) + i;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      get32(src + 8 * c, w, p.wide);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[8 * c + e] = __uint_as_float(w[e]);
    }
    return;
  }
  get32(static_cast<const uint16_t *>(p.src) + i, w, p.wide);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (p.dtype == 1) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[e]));
      x[2 * e] = f.x;
      x[2 * e + 1] = f.y;
    }
  }
}
__device__ __forceinline__ void store_row16(const PoolParams &p, long long i, const float (&x)[16]) {
  uint32_t w[8];
  if (p.dtype == 0) {
    float *dst = static_cast<float *>(p.dst) + i;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(x[8 * c + e]);
      put32(dst + 8 * c, w, p.wide);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (p.dtype == 1) {
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[e]) : "f"(x[2 * e + 1]), "f"(x[2 * e]));
    } else {
      const __half2 h = __floats2half2_rn(x[2 * e], x[2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t *>(&h);
    }
  }
  put32(static_cast<uint16_t *>(p.dst) + i, w, p.wide);
}

// The slot of an entry, or -1.
__device__ __forceinline__ int pool_slot(const PoolParams &p, int entry) {
  const int s = p.slots ? __ldg(p.slots + entry) : entry;
  return s >= 0 && s < p.batch ? s : -1;
}

template <int DK>
__global__ void __launch_bounds__(kPoolThreads) write_states_kernel(const PoolParams p) {
  constexpr int LPR = DK / 16, STEP = kPoolThreads / LPR;
  const int entry = blockIdx.x, head = blockIdx.y;
  const int slot = pool_slot(p, entry);
  if (slot < 0) return;
  const int lane = threadIdx.x & 31, lir = threadIdx.x % LPR, col0 = lir * 16;
  const int row0 = blockIdx.z * (STEP * kPoolRows) + threadIdx.x / LPR;
  const long long src_tile = ((long long)entry * p.H + head) * p.d_v;
  float x[kPoolRows][16];
#pragma unroll
  for (int r = 0; r < kPoolRows; ++r) {
    const int row = row0 + r * STEP;
    const long long at = (src_tile + row) * DK + col0;
    [[maybe_unused]] const void *src = static_cast<const uint8_t *>(p.src) + at * (p.dtype == 0 ? 4 : 2);
    if (row < p.d_v && LORES_IN(p, kRgS, src, p.dtype == 0 ? 64 : 32)) load_row16(p, at, x[r]);
    else
#pragma unroll
      for (int e = 0; e < 16; ++e) x[r][e] = 0.0f;
  }
  // the last of several entries with one slot is the one that counts
  int later = 0;
  if (p.slots)
    for (int j = entry + 1 + threadIdx.x; j < p.n; j += kPoolThreads) later |= __ldg(p.slots + j) == slot;
  if (__syncthreads_or(later)) return;
  const LaneFmt f = p.fmt[head * (DK / 16) + lir];
  const int bits = f.bits;
  const long long tile = (long long)slot * p.H + head;
  const int g = col0 / p.G, lpg = p.G / 16;
  uint8_t *codes = p.codes + slot * p.seq_bytes + __ldg(p.head_off + head);
  float *scales = p.scales + tile * p.d_v * p.ng + g;
  const uint32_t tkey = tile_key(p.step_key, (uint32_t)tile);
#pragma unroll
  for (int r = 0; r < kPoolRows; ++r) {
    const int row = row0 + r * STEP;
    const uint32_t n0 = (uint32_t)row * (uint32_t)(DK / 4) + (uint32_t)lir * 4u;
    uint32_t words[4];
    float s_new;
    const bool bad = requantize16<LPR>(x[r], bits == 32 ? 8 : bits, lpg, lane, tkey, n0, p.stochastic, words, s_new,
                                       f.store);
    if (row >= p.d_v) continue;
    // fp32 heads copy a row whatever its size: only what is not finite is reported (0 times it is NaN)
    float zero = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) zero = __fmaf_rn(x[r][e], 0.0f, zero);
    if (bits == 32 ? zero != 0.0f : bad && lir == 0) atomicOr(p.flag, kFlagNonFinite);
    uint8_t *rowp = codes + (size_t)row * f.rowb;
    if (!LORES_IN(p, kRgCodes, rowp, f.rowb)) continue;
    if (bits == 32) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        reinterpret_cast<float4 *>(rowp + f.off)[c] =
            make_float4(x[r][4 * c], x[r][4 * c + 1], x[r][4 * c + 2], x[r][4 * c + 3]);
      continue;
    }
    if (f.store >= 5 && f.store <= 7) {
      const DenseLane dl{words[0], words[1], words[2], words[3]};
      if (f.store == 5) st_dense<5>(rowp, DK, lir, dl);
      else if (f.store == 6) st_dense<6>(rowp, DK, lir, dl);
      else st_dense<7>(rowp, DK, lir, dl);
    } else if (bits != 4) {
      st16_a8(rowp + f.off, make_uint4(words[0], words[1], words[2], words[3]));
    } else {
      *reinterpret_cast<uint2 *>(rowp + f.off) = make_uint2(words[0], words[1]);
    }
    float *sc = scales + (long long)row * p.ng;
    if (lir % lpg == 0 && LORES_IN(p, kRgScales, sc, 4)) *sc = s_new;
  }
}

template <int DK>
__global__ void __launch_bounds__(kPoolThreads) read_states_kernel(const PoolParams p) {
  constexpr int LPR = DK / 16, STEP = kPoolThreads / LPR;
  const int entry = blockIdx.x, head = blockIdx.y;
  const int slot = pool_slot(p, entry);
  if (slot < 0) return;
  const int lir = threadIdx.x % LPR, col0 = lir * 16;
  const int row0 = blockIdx.z * (STEP * kPoolRows) + threadIdx.x / LPR;
  const LaneFmt f = p.fmt[head * (DK / 16) + lir];
  const int bits = f.bits;
  const long long tile = (long long)slot * p.H + head;
  const uint8_t *codes = p.codes + slot * p.seq_bytes + __ldg(p.head_off + head);
  const float *scales = p.axis ? p.scales + tile * DK + col0 : p.scales + tile * p.d_v * p.ng + col0 / p.G;
  const long long dst_tile = ((long long)entry * p.H + head) * p.d_v;
  // 16 codes as they lie (fp32 heads: two rows' worth of registers hold them) and the row's scale
  uint4 raw[kPoolRows];
  float s[kPoolRows];
  bool in[kPoolRows];
#pragma unroll
  for (int r = 0; r < kPoolRows; ++r) {
    const int row = row0 + r * STEP;
    const uint8_t *rowp = codes + (size_t)row * f.rowb;
    const float *sc = p.axis ? scales : scales + (long long)row * p.ng;
    in[r] = row < p.d_v && LORES_IN(p, kRgCodes, rowp, f.rowb) &&
            (bits == 32 || LORES_IN(p, kRgScales, sc, p.axis ? 64 : 4));
    raw[r] = make_uint4(0, 0, 0, 0);
    s[r] = 0.0f;
    if (in[r] && bits != 32) {
      if (f.store >= 5 && f.store <= 7) {
        const DenseLane d = f.store == 5   ? ld_dense<5>(rowp, DK, lir)
                            : f.store == 6 ? ld_dense<6>(rowp, DK, lir)
                                           : ld_dense<7>(rowp, DK, lir);
        raw[r] = make_uint4(d.nib0, d.nib1, d.p2, d.p1);
      } else if (bits != 4) {
        raw[r] = ld16_a8(rowp + f.off);
      } else {
        const uint2 w = *reinterpret_cast<const uint2 *>(rowp + f.off);
        raw[r] = make_uint4(w.x, w.y, 0, 0);
      }
      if (!p.axis) s[r] = *sc;
    }
  }
#pragma unroll
  for (int r = 0; r < kPoolRows; ++r) {
    const int row = row0 + r * STEP;
    if (!in[r]) continue;
    float y[16];
    if (bits == 32) {
      const float4 *src = reinterpret_cast<const float4 *>(codes + (size_t)row * f.rowb + f.off);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 v = src[c];
        y[4 * c] = v.x; y[4 * c + 1] = v.y; y[4 * c + 2] = v.z; y[4 * c + 3] = v.w;
      }
    } else {
      if (f.store >= 5 && f.store <= 7) {
        const DenseLane d{raw[r].x, raw[r].y, raw[r].z, raw[r].w};
        float2 c2[8];
        if (f.store == 5) unpack_dense<5>(d, c2);
        else if (f.store == 6) unpack_dense<6>(d, c2);
        else unpack_dense<7>(d, c2);
#pragma unroll
        for (int e = 0; e < 8; ++e) { y[2 * e] = c2[e].x; y[2 * e + 1] = c2[e].y; }
      } else if (bits != 4) {
        unpack_i8(raw[r], y);
      } else {
        unpack_i4(make_uint2(raw[r].x, raw[r].y), y);
      }
      if (p.axis) {
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = __fmul_rn(y[e], scales[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = __fmul_rn(y[e], s[r]);
      }
    }
    const long long at = (dst_tile + row) * DK + col0;
    [[maybe_unused]] const void *dst = static_cast<const uint8_t *>(p.dst) + at * (p.dtype == 0 ? 4 : 2);
    if (LORES_IN(p, kRgS, dst, p.dtype == 0 ? 64 : 32)) store_row16(p, at, y);
  }
}

using PoolFn = void (*)(PoolParams);

}  // namespace lores
