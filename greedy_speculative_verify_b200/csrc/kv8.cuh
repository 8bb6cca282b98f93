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
  int32_t B, L_max, n_kv, block;
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

// One block of one head's keys (IS_V false) or values: the largest magnitude of
// the new rows, then their codes; the earlier positions' codes again if the
// block's magnitude grew.
template <int FMT, int DIM, int UPT, bool IS_V>
__device__ __forceinline__ void kv8_append_block(const Kv8AppendArgs& a, int b, int h, int blk, int p_lo, int p_hi,
                                                 bool holds, float* red, int* bad_s) {
  // [p_lo, p_hi): the new positions inside the block; holds: positions below p_lo are earlier ones
  const Kv8View& c = a.c;
  const int tid = threadIdx.x, nthreads = blockDim.x;
  const __nv_bfloat16* src = (IS_V ? a.v : a.k) + (size_t)h * DIM;
  const int64_t stride = IS_V ? a.v_stride : a.k_stride;
  const size_t head = (size_t)b * c.n_kv + h;
  uint4* codes = reinterpret_cast<uint4*>((IS_V ? c.v : c.k) + (head * c.L_max + (size_t)blk * c.block) * DIM);
  float* amax = (IS_V ? c.v_amax : c.k_amax) + head * (c.L_max / c.block) + blk;
  const int p0 = blk * c.block;  // first position of the block
  const int64_t row0 = (int64_t)b * a.rows - (a.pos[b] - p0);  // row of the block's first position

  uint32_t x[UPT][8];  // 16 bf16 of each unit: a key's dimensions, or 4 dimensions of each of 4 positions
  float top = 0.0f;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < UPT; ++i) {
    const int u = tid + i * nthreads;
    int p, d;
    kv8_unit<IS_V>(u % DIM, &p, &d);
    p += u / DIM * kKv8Group;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[i][e] = 0u;
    if constexpr (IS_V) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (p + j >= p_lo && p + j < p_hi) {
          const uint2 w = *reinterpret_cast<const uint2*>(src + (row0 + p + j) * stride + d);
          x[i][2 * j] = w.x, x[i][2 * j + 1] = w.y;
        }
    } else if (p >= p_lo && p < p_hi) {
      const uint4* w = reinterpret_cast<const uint4*>(src + (row0 + p) * stride + d);
      const uint4 w0 = w[0], w1 = w[1];
      x[i][0] = w0.x, x[i][1] = w0.y, x[i][2] = w0.z, x[i][3] = w0.w;
      x[i][4] = w1.x, x[i][5] = w1.y, x[i][6] = w1.z, x[i][7] = w1.w;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float lo = fabsf(bf16_lo(x[i][e])), hi = fabsf(bf16_hi(x[i][e]));
      const bool fl = lo < INFINITY, fh = hi < INFINITY;  // false for NaN too
      bad |= !fl || !fh;
      top = fmaxf(top, fmaxf(fl ? lo : 0.0f, fh ? hi : 0.0f));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((tid & 31) == 0) red[tid >> 5] = top;
  if (bad) *bad_s = 1;
  __syncthreads();
  for (int w = 0; w < nthreads / 32; ++w) top = fmaxf(top, red[w]);
  bad = *bad_s != 0;
  const float was = holds ? *amax : 0.0f;
  const float now = fmaxf(was, top);
  __syncthreads();  // every thread has read the old magnitude (and red)
  if (tid == 0) {
    *amax = now;
    if (bad) record_error(kErrBounds, 341);
  }
  const float lift = now < kKv8Tiny ? kKv8Lift : 1.0f;
  const float inv = now > 0.0f ? kv8_q<FMT>() / (now * lift) : 0.0f;
  const bool grown = holds && now > was;
  const float turn = grown ? was / now : 1.0f;
#pragma unroll
  for (int i = 0; i < UPT; ++i) {
    const int u = tid + i * nthreads;
    int p, d;
    kv8_unit<IS_V>(u % DIM, &p, &d);
    p += u / DIM * kKv8Group;
    float r[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      r[2 * e] = bf16_lo(x[i][e]) * lift * inv;
      r[2 * e + 1] = bf16_hi(x[i][e]) * lift * inv;
    }
    if (bad) {  // infinities take the largest code, NaN takes 0
#pragma unroll
      for (int e = 0; e < 16; ++e)
        r[e] = r[e] == r[e] ? fminf(fmaxf(r[e], -kv8_q<FMT>()), kv8_q<FMT>()) : 0.0f;
    }
    uint32_t w[4], keep = 0, again = 0;  // per byte: new codes; bytes kept as they are; bytes rounded again
    if constexpr (IS_V) {
#pragma unroll
      for (int e = 0; e < 4; ++e)  // dimension d + e, positions p .. p + 3
        w[e] = kv8_pack4<FMT>(r[e], r[4 + e], r[8 + e], r[12 + e]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool fresh = p + j >= p_lo && p + j < p_hi;
        if (!fresh) (p + j < p_lo && grown ? again : keep) |= 0xFFu << (8 * j);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = kv8_pack4<FMT>(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
      if (p < p_lo || p >= p_hi) (p < p_lo && grown ? again : keep) = 0xFFFFFFFFu;
    }
    if (keep == 0xFFFFFFFFu) continue;
    if ((keep | again) != 0) {
      const uint4 old = codes[u];
      const uint32_t o[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 f = kv8_to_float4<FMT>(o[e]);
        const uint32_t t = kv8_pack4<FMT>(f.x * turn, f.y * turn, f.z * turn, f.w * turn);
        w[e] = (w[e] & ~(keep | again)) | (o[e] & keep) | (t & again);
      }
    }
    codes[u] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// grid: B * n_kv * nb * 2 CTAs (keys and values apart), block * dim / 16 / UPT threads.
template <int FMT, int DIM, int UPT>
__global__ void __launch_bounds__(256) kv8_append(const Kv8AppendArgs a) {
  __shared__ float red[8];
  __shared__ int bad_s;
  griddep_launch_dependents();
  griddep_wait();
  int id = blockIdx.x;
  const int is_v = id & 1;
  id >>= 1;
  const int j = id % a.nb;
  id /= a.nb;
  const int h = id % a.c.n_kv, b = id / a.c.n_kv;
  const int pos = a.pos[b], n = a.n_new ? a.n_new[b] : a.rows;
  if (n == 0) return;
  if (n < 0 || n > a.rows || pos < 0 || pos > a.c.L_max - n) {
    if (threadIdx.x == 0 && h == 0 && j == 0) record_error(kErrBounds, 340);
    return;
  }
  const int blk = pos / a.c.block + j, p0 = blk * a.c.block;
  const int lo = max(pos - p0, 0), hi = min(pos + n - p0, a.c.block);
  if (hi <= lo) return;
  if (threadIdx.x == 0) bad_s = 0;
  __syncthreads();
  if (is_v)
    kv8_append_block<FMT, DIM, UPT, true>(a, b, h, blk, lo, hi, lo > 0, red, &bad_s);
  else
    kv8_append_block<FMT, DIM, UPT, false>(a, b, h, blk, lo, hi, lo > 0, red, &bad_s);
}

struct Kv8ReadArgs {
  Kv8View c;
  int32_t rows, ng;  // rows per sequence; 16-position groups that `rows` consecutive positions can touch
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

// One thread per unit of keys and the unit of values at the same place. Values
// are c * (a / Q) in fp32 (two roundings), then rounded to the output type.
template <int FMT, int DIM, typename T>
__global__ void __launch_bounds__(256) kv8_read(const Kv8ReadArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const Kv8View& c = a.c;
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int u = (int)(id % DIM);
  int64_t w = id / DIM;
  const int j = (int)(w % a.ng);
  w /= a.ng;
  const int h = (int)(w % c.n_kv), b = (int)(w / c.n_kv);
  if (b >= c.B) return;
  const int pos = a.pos[b], n = a.n_rows ? a.n_rows[b] : a.rows;
  if (n < 0 || n > a.rows || pos < 0 || pos > c.L_max - n) {
    if (u == 0 && j == 0 && h == 0) record_error(kErrBounds, 342);
    return;
  }
  const int grp = pos / kKv8Group + j, g0 = grp * kKv8Group;
  if (n == 0 || g0 >= pos + n) return;
  const size_t head = (size_t)b * c.n_kv + h;
  const size_t at = (head * c.L_max + g0) * DIM / 16 + u, blk = head * (c.L_max / c.block) + g0 / c.block;
  const int64_t row0 = (int64_t)b * a.rows - pos;  // row of position 0
  const bool want_k = a.k_out != nullptr, want_v = a.v_out != nullptr;
  const uint4 kc = want_k ? reinterpret_cast<const uint4*>(c.k)[at] : make_uint4(0, 0, 0, 0);
  const uint4 vc = want_v ? reinterpret_cast<const uint4*>(c.v)[at] : make_uint4(0, 0, 0, 0);
  auto value = [](uint32_t x, float s, float drop) {
    const float4 f = kv8_to_float4<FMT>(x);
    return make_float4(f.x * s * drop, f.y * s * drop, f.z * s * drop, f.w * s * drop);
  };
  if (want_k) {
    int p, d;
    kv8_unit<false>(u, &p, &d);
    p += g0;
    const float am = c.k_amax[blk], lift = am < kKv8Tiny ? kKv8Lift : 1.0f;
    const float s = am * lift / kv8_q<FMT>(), drop = am < kKv8Tiny ? 1.0f / kKv8Lift : 1.0f;
    if (p >= pos && p < pos + n) {
      T* dst = static_cast<T*>(a.k_out) + (row0 + p) * a.k_stride + h * DIM + d;
      const uint32_t x[4] = {kc.x, kc.y, kc.z, kc.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) kv8_store4<T>(dst + 4 * e, value(x[e], s, drop));
    }
  }
  if (want_v) {
    int p, d;
    kv8_unit<true>(u, &p, &d);
    p += g0;
    const float am = c.v_amax[blk], lift = am < kKv8Tiny ? kKv8Lift : 1.0f;
    const float s = am * lift / kv8_q<FMT>(), drop = am < kKv8Tiny ? 1.0f / kKv8Lift : 1.0f;
    const float4 x0 = value(vc.x, s, drop), x1 = value(vc.y, s, drop), x2 = value(vc.z, s, drop),
                 x3 = value(vc.w, s, drop);
    T* dst = static_cast<T*>(a.v_out) + (row0 + p) * a.v_stride + h * DIM + d;
    const float4 row[4] = {make_float4(x0.x, x1.x, x2.x, x3.x), make_float4(x0.y, x1.y, x2.y, x3.y),
                           make_float4(x0.z, x1.z, x2.z, x3.z), make_float4(x0.w, x1.w, x2.w, x3.w)};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (p + e >= pos && p + e < pos + n) kv8_store4<T>(dst + e * a.v_stride, row[e]);
  }
}

}  // namespace vg
