// KV cache held in 8 bits: written with vg_kv8_append, read back with
// vg_kv8_read, attended to in kv8_attn.cuh.
//
// A code c (int8, or e4m3) of a block of `block` positions and one head stands
// for c * a / Q, a = the block's largest magnitude, Q = 127 (int8) or 448
// (e4m3). `a` is kept, not a / Q: it is always a bf16 value, so every quotient
// that a code is rounded from has few significant bits and ties are exact.
//
// Layout, per (sequence, kv head): groups of 16 positions, 16 * dim bytes each,
// in the order in which the attention's tensor-core fragments take them, so
// that a warp's 16-byte loads are 512 contiguous bytes and no transpose is
// needed (dim = 64 or 128):
//   key   (p, d): [p / 16][d / 64][p % 16][d % 64]
//   value (p, d): [p / 16][d / 4][p % 16 / 4][d % 4][p % 4]
// A "unit" below is 16 bytes of that layout: of a key 16 dimensions of one
// position, of a value 4 dimensions of 4 positions.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace vg {

enum : int32_t { kKv8Int8 = 0, kKv8E4m3 = 1 };
constexpr int kKv8Group = 16;
constexpr float kKv8Tiny = 7.888609e-31f;  // 2^-100: below it quotients by a leave the fp32 range
constexpr float kKv8Lift = 18446744073709551616.0f;  // 2^64

template <int FMT>
__host__ __device__ constexpr float kv8_q() {
  return FMT == kKv8Int8 ? 127.0f : 448.0f;
}

struct Kv8View {
  int32_t B, L_max, n_kv, block, log2;  // block = 2^log2
  uint8_t* k;
  uint8_t* v;
  float* k_amax;  // [B, n_kv, L_max / block]
  float* v_amax;
};

// Where unit u of a 16-position group lies in (position, dimension).
template <bool IS_V>
__device__ __forceinline__ void kv8_unit(int u, int* p, int* d) {
  if (IS_V) {
    *p = (u & 3) * 4;
    *d = (u >> 2) * 4;
  } else {
    *p = (u >> 2) & 15;
    *d = (u >> 6) * 64 + (u & 3) * 16;
  }
}

// Rounds r = numerator / a, computed with up to three fp32 roundings, to the
// code grid as the exact quotient would be, ties to even. The numerator has at
// most 15 significant bits (x * Q, or an earlier code * its old magnitude) and a
// has 8, so a quotient that is not a tie is at least 1.5e-5 (int8: 1 / (2 * 127
// * 255)) or 1.2e-4 (e4m3) of itself away from one; the rounding error is below
// 2e-7 of it. Rounding r to 17 significant bits (3.8e-6) thus restores exact
// ties and moves nothing across one.
__device__ __forceinline__ float kv8_snap(float r) {
  return __uint_as_float((__float_as_uint(r) + 0x40u) & 0xFFFFFF80u);
}

// Codes of four quotients (|r| <= Q but for rounding), packed.
template <int FMT>
__device__ __forceinline__ uint32_t kv8_pack4(float r0, float r1, float r2, float r3) {
  r0 = kv8_snap(r0), r1 = kv8_snap(r1), r2 = kv8_snap(r2), r3 = kv8_snap(r3);
  if constexpr (FMT == kKv8Int8) {
    // 1.5 * 2^23 + r holds the rounded integer in its low byte
    const float magic = 12582912.0f;
    const uint32_t a = __float_as_uint(r0 + magic), b = __float_as_uint(r1 + magic);
    const uint32_t c = __float_as_uint(r2 + magic), d = __float_as_uint(r3 + magic);
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
  } else {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(r0, r1), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(r2, r3), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  }
}

// Four codes as two f16 pairs, exactly.
template <int FMT>
__device__ __forceinline__ void kv8_to_half(uint32_t x, uint32_t* lo, uint32_t* hi) {
  if constexpr (FMT == kKv8Int8) {
    x ^= 0x80808080u;  // code + 128, put behind the exponent of 1024
    const uint32_t l = __byte_perm(x, 0x64646464u, 0x4140), h = __byte_perm(x, 0x64646464u, 0x4342);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&l), off);
    const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&h), off);
    *lo = *reinterpret_cast<const uint32_t*>(&a);
    *hi = *reinterpret_cast<const uint32_t*>(&b);
  } else {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}\n"
        : "=r"(*lo), "=r"(*hi)
        : "r"(x));
  }
}

// Four int8 codes + 128 as two pairs of f16 subnormals, (code + 128) * 2^-24.
__device__ __forceinline__ void kv8_to_tiny(uint32_t x, uint32_t* lo, uint32_t* hi) {
  x ^= 0x80808080u;
  *lo = __byte_perm(x, 0u, 0x4140);
  *hi = __byte_perm(x, 0u, 0x4342);
}

template <int FMT>
__device__ __forceinline__ float4 kv8_to_float4(uint32_t x) {
  uint32_t lo, hi;
  kv8_to_half<FMT>(x, &lo, &hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return make_float4(a.x, a.y, b.x, b.y);
}

struct Kv8AppendArgs {
  Kv8View c;
  int32_t rows, nb;  // rows per sequence; blocks that `rows` consecutive positions can touch
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t k_stride, v_stride;  // elements between rows
  const int32_t* pos;     // [B]
  const int32_t* n_new;   // [B] or null: all rows
};

// Running magnitudes of packed bf16 pairs (NaN stays), and the larger one over a
// warp as a bit pattern: those order as the magnitudes do; 0x7F80 is infinity and
// above it NaN.
__device__ __forceinline__ uint32_t kv8_top2(uint32_t top, uint32_t x) {
  const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&top), __habs2(*reinterpret_cast<const __nv_bfloat162*>(&x)));
  return *reinterpret_cast<const uint32_t*>(&m);
}
__device__ __forceinline__ uint32_t kv8_warp_top(uint32_t top) {
  return __reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16));
}
// The same without infinities and NaN.
__device__ __forceinline__ uint32_t kv8_finite(uint32_t x) {
  const uint32_t lo = x & 0x7FFFu, hi = (x >> 16) & 0x7FFFu;
  return (lo < 0x7F80u ? lo : 0u) | (hi < 0x7F80u ? hi << 16 : 0u);
}

// How a block's values become codes.
struct Kv8Rule {
  float inv, lift;  // Q / (a lift)
  float turn;       // a_old / a_new for the earlier codes
  bool odd;         // lift is not 1, or the block has infinities or NaN
  bool grown;       // there are earlier codes, and a became larger
};
template <int FMT>
__device__ __forceinline__ Kv8Rule kv8_rule(float was, float now, bool holds, bool bad) {
  Kv8Rule c;
  c.lift = now < kKv8Tiny ? kKv8Lift : 1.0f;
  c.inv = now > 0.0f ? kv8_q<FMT>() / (now * c.lift) : 0.0f;
  c.odd = bad || now < kKv8Tiny;
  c.grown = holds && now > was;
  c.turn = c.grown ? was / now : 1.0f;
  return c;
}

// A unit's sixteen bf16 values, x[2 i], x[2 i + 1] of row i of a value's four (or
// in order, of a key's sixteen), to its codes.
template <int FMT, bool IS_V>
__device__ __forceinline__ void kv8_encode(const uint32_t (&x)[8], const Kv8Rule& c, uint32_t (&w)[4]) {
  float r[16];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    r[2 * e] = bf16_lo(x[e]);
    r[2 * e + 1] = bf16_hi(x[e]);
  }
  if (c.odd) {  // infinities take the largest code, NaN takes 0
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float y = r[e] * c.lift * c.inv;
      r[e] = y == y ? fminf(fmaxf(y, -kv8_q<FMT>()), kv8_q<FMT>()) : 0.0f;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) r[e] *= c.inv;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    w[e] = IS_V ? kv8_pack4<FMT>(r[e], r[4 + e], r[8 + e], r[12 + e])
                : kv8_pack4<FMT>(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
}

template <int FMT>
__device__ __forceinline__ uint32_t kv8_turn4(uint32_t x, float turn) {
  const float4 f = kv8_to_float4<FMT>(x);
  return kv8_pack4<FMT>(f.x * turn, f.y * turn, f.z * turn, f.w * turn);
}

// Stores a unit of which the bytes in `keep` stay as they are and those in
// `again` are earlier codes rounded again (the rest are w's).
template <int FMT>
__device__ __forceinline__ void kv8_put(uint4* dst, const uint32_t (&w)[4], uint32_t keep, uint32_t again, float turn) {
  if (keep == 0xFFFFFFFFu) return;
  if ((keep | again) == 0) {
    *dst = make_uint4(w[0], w[1], w[2], w[3]);
    return;
  }
  const uint4 old = *dst;
  const uint32_t o[4] = {old.x, old.y, old.z, old.w};
  uint32_t v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    v[e] = (w[e] & ~(keep | again)) | (o[e] & keep) | (again ? kv8_turn4<FMT>(o[e], turn) & again : 0u);
  *dst = make_uint4(v[0], v[1], v[2], v[3]);
}

// A unit at (position p of the block, dimension d): its bf16 values (0 where the
// position is not new), and which of its bytes are not new.
template <int DIM, bool IS_V, bool FULL = false>
__device__ __forceinline__ void kv8_fetch(const __nv_bfloat16* src, int64_t row0, int64_t stride, int p, int d, int p_lo,
                                          int p_hi, uint32_t (&x)[8]) {
  const __nv_bfloat16* row = src + (row0 + p) * stride + d;
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = 0u;
  if constexpr (IS_V) {
#pragma unroll
    for (int j = 0; j < 4; ++j, row += stride)
      if (FULL || (p + j >= p_lo && p + j < p_hi)) {
        const uint2 w = *reinterpret_cast<const uint2*>(row);
        x[2 * j] = w.x, x[2 * j + 1] = w.y;
      }
  } else if (FULL || (p >= p_lo && p < p_hi)) {
    const uint4* w = reinterpret_cast<const uint4*>(row);
    const uint4 w0 = w[0], w1 = w[1];
    x[0] = w0.x, x[1] = w0.y, x[2] = w0.z, x[3] = w0.w, x[4] = w1.x, x[5] = w1.y, x[6] = w1.z, x[7] = w1.w;
  }
}
template <bool IS_V>
__device__ __forceinline__ void kv8_masks(int p, int p_lo, int p_hi, bool grown, uint32_t* keep, uint32_t* again) {
  *keep = *again = 0u;
  if constexpr (IS_V) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (p + j < p_lo || p + j >= p_hi) (p + j < p_lo && grown ? *again : *keep) |= 0xFFu << (8 * j);
  } else if (p < p_lo || p >= p_hi) {
    (p < p_lo && grown ? *again : *keep) = 0xFFFFFFFFu;
  }
}

// What a block of one head's keys or values is written from and to.
template <int DIM, bool IS_V>
struct Kv8Block {
  const __nv_bfloat16* src;
  int64_t row0, stride;  // row of the block's first position, elements between rows
  uint4* codes;
  float* amax;
  __device__ __forceinline__ Kv8Block(const Kv8AppendArgs& a, int b, int h, int blk, int pos) {
    const size_t head = (size_t)b * a.c.n_kv + h;
    src = (IS_V ? a.v : a.k) + (size_t)h * DIM;
    stride = IS_V ? a.v_stride : a.k_stride;
    row0 = (int64_t)b * a.rows - pos + (int64_t)blk * a.c.block;
    codes = reinterpret_cast<uint4*>((IS_V ? a.c.v : a.c.k) + (head * a.c.L_max + (size_t)blk * a.c.block) * DIM);
    amax = (IS_V ? a.c.v_amax : a.c.k_amax) + head * (a.c.L_max >> a.c.log2) + blk;
  }
};

// One block by one CTA, every unit in registers between the pass that finds the
// magnitude and the pass that encodes: one read of the rows. FULL: the whole block
// is new.
template <int FMT, int DIM, int UPT, bool IS_V, bool FULL>
__device__ __forceinline__ void kv8_append_block(const Kv8AppendArgs& a, int b, int h, int blk, int pos, int p_lo, int p_hi,
                                                 uint32_t* red) {
  const int tid = threadIdx.x, nthreads = blockDim.x;
  const Kv8Block<DIM, IS_V> k(a, b, h, blk, pos);
  uint32_t x[UPT][8], top = 0u;
#pragma unroll
  for (int i = 0; i < UPT; ++i) {
    const int u = tid + i * nthreads;
    int p, d;
    kv8_unit<IS_V>(u % DIM, &p, &d);
    kv8_fetch<DIM, IS_V, FULL>(k.src, k.row0, k.stride, p + u / DIM * kKv8Group, d, p_lo, p_hi, x[i]);
  }
#pragma unroll
  for (int i = 0; i < UPT; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) top = kv8_top2(top, x[i][e]);
  auto join = [&](uint32_t t) {  // over the CTA
    t = kv8_warp_top(t);
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = t;
    __syncthreads();
    for (int w = 0; w < nthreads / 32; ++w) t = max(t, red[w]);
    return t;
  };
  const bool holds = !FULL && p_lo > 0;
  const float was = holds ? *k.amax : 0.0f;
  top = join(top);
  const bool bad = top >= 0x7F80u;
  if (bad) {
    top = 0u;
#pragma unroll
    for (int i = 0; i < UPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = kv8_top2(top, kv8_finite(x[i][e]));
    top = join(top);
  }
  const float now = fmaxf(was, __uint_as_float(top << 16));
  const Kv8Rule c = kv8_rule<FMT>(was, now, holds, bad);
  if (tid == 0) {  // (every thread has read the old magnitude: join() has barriers)
    *k.amax = now;
    if (bad) record_error(kErrBounds, 341);
  }
#pragma unroll
  for (int i = 0; i < UPT; ++i) {
    const int u = tid + i * nthreads;
    int p, d;
    kv8_unit<IS_V>(u % DIM, &p, &d);
    uint32_t w[4], keep = 0u, again = 0u;
    if (!FULL) kv8_masks<IS_V>(p + u / DIM * kKv8Group, p_lo, p_hi, c.grown, &keep, &again);
    kv8_encode<FMT, IS_V>(x[i], c, w);
    kv8_put<FMT>(k.codes + u, w, keep, again, c.turn);
  }
}

// Sequence b's positions of this call, or false (and an error recorded) where they are bad.
__device__ __forceinline__ bool kv8_append_span(const Kv8AppendArgs& a, int b, bool report, int* pos, int* n) {
  *pos = a.pos[b];
  *n = a.n_new ? a.n_new[b] : a.rows;
  if (*n >= 0 && *n <= a.rows && *pos >= 0 && *pos <= a.c.L_max - *n) return true;
  if (report) record_error(kErrBounds, 340);
  return false;
}

// grid: B * n_kv * nb * 2 CTAs (keys and values apart), block * dim / 16 / UPT
// threads: UPT = 4 units of 16 values a thread, 2 where that would leave less than
// a warp. (29,086 rows x 10 heads x 128: 45 us with 4, 53 with 2, 60 with 8.)
template <int FMT, int DIM, int UPT>
__global__ void __launch_bounds__(256) kv8_append(const Kv8AppendArgs a) {
  __shared__ uint32_t red[8];
  griddep_launch_dependents();
  griddep_wait();
  int id = blockIdx.x;
  const int is_v = id & 1;
  id >>= 1;
  const int j = id % a.nb;
  id /= a.nb;
  const int h = id % a.c.n_kv, b = id / a.c.n_kv;
  int pos, n;
  if (!kv8_append_span(a, b, threadIdx.x == 0 && h == 0 && j == 0, &pos, &n)) return;
  const int blk = (pos >> a.c.log2) + j, p0 = blk << a.c.log2;
  const int lo = max(pos - p0, 0), hi = min(pos + n - p0, a.c.block);
  if (hi <= lo) return;
  if (lo == 0 && hi == a.c.block) {
    if (is_v)
      kv8_append_block<FMT, DIM, UPT, true, true>(a, b, h, blk, pos, lo, hi, red);
    else
      kv8_append_block<FMT, DIM, UPT, false, true>(a, b, h, blk, pos, lo, hi, red);
  } else if (is_v) {
    kv8_append_block<FMT, DIM, UPT, true, false>(a, b, h, blk, pos, lo, hi, red);
  } else {
    kv8_append_block<FMT, DIM, UPT, false, false>(a, b, h, blk, pos, lo, hi, red);
  }
}

// Up to kKv8Few new rows a sequence (a verify step): one warp per block, the
// units with new positions alone in registers; the earlier ones are visited only
// where the magnitude grew. A step is latency: launch, positions, rows, codes.
constexpr int kKv8Few = 8;

template <int FMT, int DIM, bool IS_V>
__device__ __forceinline__ void kv8_append_few_block(const Kv8AppendArgs& a, int b, int h, int blk, int pos, int p_lo,
                                                     int p_hi) {
  // units across the dimensions, positions per unit; units with new positions: a key's one position each, of a
  // value's quads of positions at most three
  constexpr int kAcross = IS_V ? DIM / 4 : DIM / 16, kPer = IS_V ? 4 : 1, kMost = cdiv((IS_V ? 3 : kKv8Few) * kAcross, 32);
  const int lane = threadIdx.x & 31;
  const Kv8Block<DIM, IS_V> k(a, b, h, blk, pos);
  const int first = p_lo / kPer, n_units = (cdiv(p_hi, kPer) - first) * kAcross;
  auto unit = [&](int q, int s) {  // the unit of positions q * kPer .. and the s-th share of the dimensions
    const int p = q * kPer, in = p % kKv8Group;
    return p / kKv8Group * DIM + (IS_V ? s * 4 + in / 4 : (s / 4) * 64 + in * 4 + s % 4);
  };
  uint32_t x[kMost][8], top = 0u;
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int e = lane + 32 * i;
    const int q = first + e / kAcross, s = e % kAcross;
    kv8_fetch<DIM, IS_V>(k.src, k.row0, k.stride, q * kPer, s * (DIM / kAcross), p_lo, e < n_units ? p_hi : 0, x[i]);
  }
  const bool holds = p_lo > 0;
  const float was = holds ? *k.amax : 0.0f;
#pragma unroll
  for (int i = 0; i < kMost; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) top = kv8_top2(top, x[i][e]);
  top = kv8_warp_top(top);
  const bool bad = top >= 0x7F80u;
  if (bad) {
    top = 0u;
#pragma unroll
    for (int i = 0; i < kMost; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = kv8_top2(top, kv8_finite(x[i][e]));
    top = kv8_warp_top(top);
  }
  const float now = fmaxf(was, __uint_as_float(top << 16));
  const Kv8Rule c = kv8_rule<FMT>(was, now, holds, bad);
  __syncwarp();
  if (lane == 0) {
    *k.amax = now;
    if (bad) record_error(kErrBounds, 341);
  }
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int e = lane + 32 * i;
    const int q = first + e / kAcross;
    if (e >= n_units) continue;
    uint32_t w[4], keep, again;
    kv8_masks<IS_V>(q * kPer, p_lo, p_hi, c.grown, &keep, &again);
    kv8_encode<FMT, IS_V>(x[i], c, w);
    kv8_put<FMT>(k.codes + unit(q, e % kAcross), w, keep, again, c.turn);
  }
  if (c.grown)  // the units of earlier positions alone
    for (int e = lane; e < first * kAcross; e += 32) {
      uint4* at = k.codes + unit(e / kAcross, e % kAcross);
      const uint4 o = *at;
      *at = make_uint4(kv8_turn4<FMT>(o.x, c.turn), kv8_turn4<FMT>(o.y, c.turn), kv8_turn4<FMT>(o.z, c.turn),
                       kv8_turn4<FMT>(o.w, c.turn));
    }
}

// One warp per (sequence, head, block of the two that the rows can touch, keys or values).
template <int FMT, int DIM>
__global__ void __launch_bounds__(128) kv8_append_few(const Kv8AppendArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  int id = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int is_v = id & 1, j = (id >> 1) & 1;
  id >>= 2;
  const int h = id % a.c.n_kv, b = id / a.c.n_kv;
  if (b >= a.c.B) return;
  int pos, n;
  if (!kv8_append_span(a, b, (threadIdx.x & 31) == 0 && h == 0 && j == 0, &pos, &n)) return;
  const int blk = (pos >> a.c.log2) + j, p0 = blk << a.c.log2;
  const int lo = max(pos - p0, 0), hi = min(pos + n - p0, a.c.block);
  if (hi <= lo) return;
  if (is_v)
    kv8_append_few_block<FMT, DIM, true>(a, b, h, blk, pos, lo, hi);
  else
    kv8_append_few_block<FMT, DIM, false>(a, b, h, blk, pos, lo, hi);
}

struct Kv8ReadArgs {
  Kv8View c;
  int32_t rows, ng, sides;  // rows per sequence; CTAs per (sequence, head, side); 2: keys and values, 1: one of them
  const int32_t* pos;
  const int32_t* n_rows;  // [B] or null
  void* k_out;
  void* v_out;
  int64_t k_stride, v_stride;
};

template <typename T>
__device__ __forceinline__ void kv8_store4(T* dst, float4 v) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(dst) = v;
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}

// The values of four codes: c * (a / Q), two roundings; magnitudes so small that
// a / Q would leave the normal range take the product first.
template <int FMT>
struct Kv8Back {
  float s, drop;
  bool tiny;
  __device__ __forceinline__ explicit Kv8Back(float a) {
    tiny = a < kKv8Tiny;
    s = a * (tiny ? kKv8Lift : 1.0f) / kv8_q<FMT>();
    drop = 1.0f / kKv8Lift;
  }
  __device__ __forceinline__ float4 operator()(uint32_t x) const {
    const float4 f = kv8_to_float4<FMT>(x);
    float4 y = make_float4(f.x * s, f.y * s, f.z * s, f.w * s);
    if (tiny) y.x *= drop, y.y *= drop, y.z *= drop, y.w *= drop;
    return y;
  }
};

constexpr int kKv8ReadThreads = 256;
constexpr int kKv8ReadGroups = kKv8ReadThreads / 32;  // 16-position groups a CTA of vg_kv8_read takes: one a warp

// A warp reads a group's keys word by word (4 dimensions of a position), of its
// values 4 dimensions of 8 or 16 positions a lane, so that its stores are whole
// rows: 128 or 256 contiguous bytes of bf16, twice that of fp32. (16-byte units a
// lane, as the attention takes them, gave stores of 8 bytes 32 apart: 87 us for
// 8 sequences of 6,800 positions, 427 MB, against the 65 of a copy.)
template <int FMT, int DIM, typename T, bool IS_V>
__device__ __forceinline__ void kv8_read_group(const Kv8ReadArgs& a, int bh, int b, int h, int pos, int n, int grp) {
  const Kv8View& c = a.c;
  const int lane = threadIdx.x & 31;
  const size_t head = (size_t)bh;
  const uint8_t* codes = (IS_V ? c.v : c.k) + (head * c.L_max + (size_t)grp * kKv8Group) * DIM;
  const float am = (IS_V ? c.v_amax : c.k_amax)[head * (c.L_max >> c.log2) + (grp * kKv8Group >> c.log2)];
  const int64_t stride = IS_V ? a.v_stride : a.k_stride;
  const int p0 = grp * kKv8Group - pos;  // row of the group's first position
  const bool all = p0 >= 0 && p0 + kKv8Group <= n;
  T* rows = static_cast<T*>(IS_V ? a.v_out : a.k_out) + ((int64_t)b * a.rows + p0) * stride + h * DIM;
  if constexpr (IS_V) {
    constexpr int kQuads = DIM / 32;  // quads of positions a lane: DIM / 4 lanes across the dimensions
    const int d = lane % (DIM / 4) * 4, q0 = lane / (DIM / 4) * kQuads;
    uint4 x[kQuads];
#pragma unroll
    for (int i = 0; i < kQuads; ++i) x[i] = *reinterpret_cast<const uint4*>(codes + d * 16 + (q0 + i) * 16);
    const Kv8Back<FMT> back(am);
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      const float4 f[4] = {back(x[i].x), back(x[i].y), back(x[i].z), back(x[i].w)};
      const float4 row[4] = {make_float4(f[0].x, f[1].x, f[2].x, f[3].x), make_float4(f[0].y, f[1].y, f[2].y, f[3].y),
                             make_float4(f[0].z, f[1].z, f[2].z, f[3].z), make_float4(f[0].w, f[1].w, f[2].w, f[3].w)};
      const int p = (q0 + i) * 4;
      T* to = rows + p * stride + d;
#pragma unroll
      for (int e = 0; e < 4; ++e, to += stride)
        if (all || (p0 + p + e >= 0 && p0 + p + e < n)) kv8_store4<T>(to, row[e]);
    }
  } else {
    constexpr int kWords = kKv8Group * DIM / 128;  // words a lane: two positions' 64 dimensions at a time
    const int p_in = lane / 16, d_in = lane % 16 * 4;
    uint32_t x[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) x[i] = *reinterpret_cast<const uint32_t*>(codes + i * 128 + lane * 4);
    const Kv8Back<FMT> back(am);
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int p = i % 8 * 2 + p_in, d = i / 8 * 64 + d_in;
      if (all || (p0 + p >= 0 && p0 + p < n)) kv8_store4<T>(rows + p * stride + d, back(x[i]));
    }
  }
}

// grid: B * n_kv * ng * sides CTAs.
template <int FMT, int DIM, typename T>
__global__ void __launch_bounds__(kKv8ReadThreads) kv8_read(const Kv8ReadArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int side = blockIdx.x % a.sides, id = blockIdx.x / a.sides;
  const int bh = id / a.ng, j = id - bh * a.ng, b = bh / a.c.n_kv, h = bh - b * a.c.n_kv;
  const int pos = a.pos[b], n = a.n_rows ? a.n_rows[b] : a.rows;
  if (n < 0 || n > a.rows || pos < 0 || pos > a.c.L_max - n) {
    if (threadIdx.x == 0 && j == 0 && h == 0) record_error(kErrBounds, 342);
    return;
  }
  const int grp = pos / kKv8Group + j * kKv8ReadGroups + (int)threadIdx.x / 32;
  if (n == 0 || grp * kKv8Group >= pos + n) return;
  if (side == 0 && a.k_out)
    kv8_read_group<FMT, DIM, T, false>(a, bh, b, h, pos, n, grp);
  else
    kv8_read_group<FMT, DIM, T, true>(a, bh, b, h, pos, n, grp);
}

}  // namespace vg
