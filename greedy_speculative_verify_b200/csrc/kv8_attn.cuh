// Attention of the verify rows over an 8-bit KV cache (layout: kv8.cuh):
//   o[r] = sum_p w_p v_p / sum_p w_p,  w_p = exp(scale * q_r . k_p - m_r),
// over the positions first[b] <= p <= lens[b] + i that row i of sequence b
// sees; query head h reads kv head h / (n_heads / n_kv). A row that sees
// nothing gets o = 0.
//
// Both products run on the tensor cores (m16n8k16, f16 operands, fp32 sums)
// with the cache as the 16-row operand and up to 8 * NT query rows of one kv
// head as the columns, so no tile row is empty padding:
//   S^T[position][row] = K Q^T, O^T[dimension][row] += V^T P^T.
// Codes are exact in f16. A query row is brought to [2^14, 2^15) by a power of
// two, which f16 holds exactly down to 2^-29 of the row's largest element.
// Weights are rounded to f16 (2^-12 relative) after scaling by 2^15 times the
// block's share of the largest value scale seen, so that none down to 2^-29 of
// the largest loses precision; the sum of weights is taken in fp32 unrounded.
#pragma once
#include "attention.cuh"
#include "kv8.cuh"

namespace vg {

constexpr int kKaWarps = 4;
constexpr int kKaChunk = 256;      // positions per CTA
constexpr int kKaMaxRows = 8;      // new rows per sequence
constexpr int kKaMaxGroup = 16;    // query heads per kv head
constexpr float kKaLift = 32768.0f;  // 2^15, on the f16 weights

struct Kv8AttnArgs {
  Kv8View c;
  int32_t rows, n_heads, n_tiles;  // rows per sequence; n_tiles: 8 NT-row tiles of a kv head's rows * group query rows
  const __nv_bfloat16* q;
  int64_t q_stride;
  const int32_t* lens;   // [B] positions before the new rows
  const int32_t* first;  // [B] or null: 0
  const int32_t* n_new;  // [B] or null: all rows
  float scale_log2;      // scale * log2(e) / Q
  float* part;           // [unit][chunk][row][2 + dim]
  int32_t n_chunks;
  __nv_bfloat16* o;
  int64_t o_stride;
};

// m16n8k16, f16 operands, fp32 accumulators; fragments as in mma_16816.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Sequence b's visible range for this step: positions [lo, hi) any row may see.
struct Kv8Span {
  int L, lo, hi, n;  // cached positions, range, rows that are real
};
__device__ __forceinline__ bool kv8_span(const Kv8AttnArgs& a, int b, Kv8Span* s) {
  s->L = a.lens[b];
  s->n = a.n_new ? a.n_new[b] : a.rows;
  s->lo = a.first ? a.first[b] : 0;
  if (s->n < 0 || s->n > a.rows || s->L < 0 || s->L > a.c.L_max - s->n || s->lo < 0) {
    s->n = s->lo = s->hi = 0;
    return false;
  }
  s->hi = s->n > 0 ? s->L + s->n : 0;
  if (s->lo > s->hi) s->lo = s->hi;
  return true;
}

// One warp's running softmax over groups of 16 positions, for NT tiles of 8
// query rows. Lane (g, t) = (lane / 4, lane % 4) holds columns (rows) 2t, 2t+1
// of every tile.
template <int FMT, int DIM, int NT>
struct Kv8Warp {
  uint32_t q[NT][DIM / 16][2];   // Q^T fragments
  float mult[NT][2];             // softmax scale * log2(e) / Q * 2^e of rows 2t, 2t+1
  int last[NT][2];               // last position those rows see (-1: none)
  float m[NT][2], l[NT][2];      // running maximum (log2 units) and this lane's share of the sum
  float o[NT][DIM / 32][2][4];   // O^T: dimensions 4 (g + 8 j) + 0..3
  float top_v;                   // largest magnitude of a value block seen: o is in units of it / Q / 2^15

  __device__ __forceinline__ void init(const Kv8AttnArgs& a, int b, int kvh, int tile, const Kv8Span& s, int lane) {
    const int g = lane >> 2, t = lane & 3, group = a.n_heads / a.c.n_kv, n_q = s.n * group;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // column g of the tile: query row r = i * group + head in the group
      const int r = (tile * NT + nt) * 8 + g;
      const bool real = r < n_q;
      const int i = real ? r / group : 0, h = kvh * group + (real ? r - i * group : 0);
      const __nv_bfloat16* src = a.q + ((int64_t)b * a.rows + i) * a.q_stride + h * DIM + 16 * t;
      uint32_t x[DIM / 16][4];
      float big = 0.0f;
#pragma unroll
      for (int s16 = 0; s16 < DIM / 64; ++s16) {
        uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
        if (real) {
          w0 = *reinterpret_cast<const uint4*>(src + 64 * s16);
          w1 = *reinterpret_cast<const uint4*>(src + 64 * s16 + 8);
        }
        const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[s16 * 4 + e / 2][e % 2] = w[e];
          big = fmaxf(big, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
        }
      }
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // 2^(14 - floor(log2 big)), and its inverse (two factors: either may leave the normal range)
      const int ex = big > 0.0f && big < INFINITY ? ilogbf(big) : 0;
      const float up0 = exp2f((float)((14 - ex) / 2)), up1 = exp2f((float)((14 - ex) - (14 - ex) / 2));
#pragma unroll
      for (int k = 0; k < DIM / 16; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          q[nt][k][e] = pack_half2(bf16_lo(x[k][e]) * up0 * up1, bf16_hi(x[k][e]) * up0 * up1);
      const float back = a.scale_log2 / up0 / up1;
      const int seen = real ? s.L + i : -1;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mult[nt][e] = __shfl_sync(0xffffffffu, back, 4 * (2 * t + e));
        last[nt][e] = __shfl_sync(0xffffffffu, seen, 4 * (2 * t + e));
        m[nt][e] = -INFINITY;
        l[nt][e] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < DIM / 32; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][j][0][e] = o[nt][j][1][e] = 0.0f;
    }
    top_v = 0.0f;
  }

  // 16 positions p0 .. p0 + 15, of which [lo, hi) are the sequence's: their keys
  // and values (the group's bytes), and the magnitudes of their blocks.
  __device__ __forceinline__ void group16(const uint8_t* kb, const uint8_t* vb, float ks, float vs, int p0, int lo,
                                          int hi, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const int tok = 4 * (g >> 1) + (g & 1);  // tile row g; row g + 8 is position tok + 2
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = 0.0f;
    uint4 vf[DIM / 32];
#pragma unroll
    for (int j = 0; j < DIM / 32; ++j) vf[j] = *reinterpret_cast<const uint4*>(vb + (g + 8 * j) * 64 + t * 16);
#pragma unroll
    for (int h = 0; h < DIM / 64; ++h) {
      const uint4 ka = *reinterpret_cast<const uint4*>(kb + h * 1024 + tok * 64 + t * 16);
      const uint4 kc = *reinterpret_cast<const uint4*>(kb + h * 1024 + (tok + 2) * 64 + t * 16);
      const uint32_t xa[4] = {ka.x, ka.y, ka.z, ka.w}, xc[4] = {kc.x, kc.y, kc.z, kc.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t a0, a1, a2, a3;
        kv8_to_half<FMT>(xa[w], &a0, &a2);
        kv8_to_half<FMT>(xc[w], &a1, &a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16(s[nt], a0, a1, a2, a3, q[nt][h * 4 + w][0], q[nt][h * 4 + w][1]);
      }
    }
    // ---- weights
    const float grow_v = vs > top_v ? top_v / vs : 1.0f;  // what a larger value scale leaves of o
    top_v = fmaxf(top_v, vs);
    const float share = top_v > 0.0f ? vs / top_v * kKaLift : 0.0f;
    const int pa = p0 + tok, pc = pa + 2;
    uint32_t b0[NT], b1[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float f[2], w[2][2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mu = mult[nt][e] * ks;
        float za = s[nt][e] * mu, zc = s[nt][2 + e] * mu;
        za = pa >= lo && pa <= last[nt][e] ? za : -INFINITY;
        zc = pc >= lo && pc <= last[nt][e] ? zc : -INFINITY;
        float mx = fmaxf(za, zc);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        const float now = fmaxf(m[nt][e], mx), base = now > -INFINITY ? now : 0.0f;
        f[e] = exp2f(m[nt][e] - base);
        m[nt][e] = now;
        w[e][0] = exp2f(za - base);
        w[e][1] = exp2f(zc - base);
        l[nt][e] = l[nt][e] * f[e] + (w[e][0] + w[e][1]);
        f[e] *= grow_v;
      }
      if (__any_sync(0xffffffffu, f[0] != 1.0f || f[1] != 1.0f)) {
#pragma unroll
        for (int j = 0; j < DIM / 32; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            o[nt][j][0][e] *= f[e & 1];
            o[nt][j][1][e] *= f[e & 1];
          }
      }
      // rows 2t, 2t+1 of positions g, g + 8 -> positions 2t, 2t+1 (+ 8) of row g
      b0[nt] = movmatrix_trans(pack_half2(w[0][0] * share, w[1][0] * share));
      b1[nt] = movmatrix_trans(pack_half2(w[0][1] * share, w[1][1] * share));
    }
    // ---- values
    if (FMT == kKv8E4m3 && p0 + kKv8Group > hi) {  // a code never written may be NaN, and 0 * NaN is not 0
      const int real = hi - p0 - 4 * t;            // of this lane's four positions
      const uint32_t keep = real >= 4 ? 0xFFFFFFFFu : real <= 0 ? 0u : (1u << (8 * real)) - 1u;
#pragma unroll
      for (int j = 0; j < DIM / 32; ++j) vf[j].x &= keep, vf[j].y &= keep, vf[j].z &= keep, vf[j].w &= keep;
    }
#pragma unroll
    for (int j = 0; j < DIM / 32; ++j) {
      const uint32_t x[4] = {vf[j].x, vf[j].y, vf[j].z, vf[j].w};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t a0, a1, a2, a3;
        kv8_to_half<FMT>(x[2 * e], &a0, &a2);
        kv8_to_half<FMT>(x[2 * e + 1], &a1, &a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][j][e], a0, a1, a2, a3, b0[nt], b1[nt]);
      }
    }
  }
};

// grid (B * n_kv * n_tiles, n_chunks): the chunk's partial (maximum, sum,
// weighted values) of each of the tile's rows.
template <int FMT, int DIM, int NT>
__global__ void __launch_bounds__(32 * kKaWarps) kv8_attn_chunk(const Kv8AttnArgs a) {
  __shared__ float wm[kKaWarps][8 * NT], wl[kKaWarps][8 * NT];
  __shared__ __align__(16) float wo[kKaWarps][8 * NT][DIM + 4];
  griddep_launch_dependents();
  griddep_wait();
  const int tile = blockIdx.x % a.n_tiles, bh = blockIdx.x / a.n_tiles;
  const int kvh = bh % a.c.n_kv, b = bh / a.c.n_kv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  Kv8Span s;
  if (!kv8_span(a, b, &s) && threadIdx.x == 0 && blockIdx.y == 0 && kvh == 0 && tile == 0) record_error(kErrBounds, 343);
  const int c0 = max(s.lo / kKv8Group * kKv8Group, (int)blockIdx.y * kKaChunk), c1 = min(s.hi, ((int)blockIdx.y + 1) * kKaChunk);
  float* part = a.part + ((size_t)blockIdx.x * a.n_chunks + blockIdx.y) * (8 * NT) * (2 + DIM);
  if (c0 >= c1) {
    for (int r = threadIdx.x; r < 8 * NT; r += blockDim.x) part[(size_t)r * (2 + DIM)] = -INFINITY;
    return;
  }
  Kv8Warp<FMT, DIM, NT> w;
  w.init(a, b, kvh, tile, s, lane);
  const size_t head = (size_t)b * a.c.n_kv + kvh, blocks = a.c.L_max / a.c.block;
  for (int p = c0 + warp * kKv8Group; p < c1; p += kKaWarps * kKv8Group) {
    const size_t at = (head * a.c.L_max + p) * DIM;
    const size_t blk = head * blocks + p / a.c.block;
    w.group16(a.c.k + at, a.c.v + at, a.c.k_amax[blk], a.c.v_amax[blk], p, s.lo, s.hi, lane);
  }
  // ---- merge the warps
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = w.l[nt][e];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      if (g == 0) {
        wm[warp][nt * 8 + 2 * t + e] = w.m[nt][e];
        wl[warp][nt * 8 + 2 * t + e] = l;
      }
      const float back = w.top_v / (kv8_q<FMT>() * kKaLift);
#pragma unroll
      for (int j = 0; j < DIM / 32; ++j)
        *reinterpret_cast<float4*>(&wo[warp][nt * 8 + 2 * t + e][4 * (g + 8 * j)]) =
            make_float4(w.o[nt][j][0][e] * back, w.o[nt][j][0][2 + e] * back, w.o[nt][j][1][e] * back,
                        w.o[nt][j][1][2 + e] * back);
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 8 * NT * DIM; i += blockDim.x) {
    const int r = i / DIM, d = i % DIM;
    float mm = -INFINITY;
#pragma unroll
    for (int k = 0; k < kKaWarps; ++k) mm = fmaxf(mm, wm[k][r]);
    float acc = 0.0f, ls = 0.0f;
    if (mm > -INFINITY) {
#pragma unroll
      for (int k = 0; k < kKaWarps; ++k) {
        const float f = exp2f(wm[k][r] - mm);
        acc += wo[k][r][d] * f;
        ls += wl[k][r] * f;
      }
    }
    float* dst = part + (size_t)r * (2 + DIM);
    dst[2 + d] = acc;
    if (d == 0) dst[0] = mm, dst[1] = ls;
  }
}

// grid B * n_kv * n_tiles * 8 NT, DIM threads.
template <int DIM, int NT>
__global__ void __launch_bounds__(DIM) kv8_attn_merge(const Kv8AttnArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int group = a.n_heads / a.c.n_kv;
  const int unit = blockIdx.x / (8 * NT), rr = blockIdx.x % (8 * NT), d = threadIdx.x;
  const int tile = unit % a.n_tiles, bh = unit / a.n_tiles, kvh = bh % a.c.n_kv, b = bh / a.c.n_kv;
  const int r = tile * 8 * NT + rr;
  if (r >= a.rows * group) return;
  float m = -INFINITY, l = 0.0f, acc = 0.0f;
  const float* part = a.part + ((size_t)unit * a.n_chunks * (8 * NT) + rr) * (2 + DIM);
  for (int c = 0; c < a.n_chunks; ++c) m = fmaxf(m, part[(size_t)c * (8 * NT) * (2 + DIM)]);
  if (m > -INFINITY)
    for (int c = 0; c < a.n_chunks; ++c) {
      const float* p = part + (size_t)c * (8 * NT) * (2 + DIM);
      if (p[0] == -INFINITY) continue;
      const float f = exp2f(p[0] - m);
      l += p[1] * f;
      acc += p[2 + d] * f;
    }
  const int i = r / group, h = kvh * group + r % group;
  a.o[((int64_t)b * a.rows + i) * a.o_stride + h * DIM + d] = __float2bfloat16_rn(l > 0.0f ? acc / l : 0.0f);
}

}  // namespace vg
