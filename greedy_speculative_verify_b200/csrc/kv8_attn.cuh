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
// The running maximum m is only raised when a score exceeds it by 2^kKaSlack, so
// that the common step has one vote instead of a reduction over positions;
// weights are then at most 2^kKaSlack. They are rounded to f16 (2^-11 relative)
// after scaling by 2^kKaLift times the block's share of the largest value
// magnitude seen, so that none down to 2^-(14 + kKaLift) loses precision; the sum
// of weights is taken in fp32 unrounded.
//
// Work: a unit is (sequence, kv head, 8 NT query rows), cut into tiles of 16
// positions a warp. All tiles of the batch form one list, of which every CTA
// takes an equal contiguous share, whatever the lengths are. Warp w runs its own
// softmax over positions 16 w .. 16 w + 15 of every tile. Its codes come by 16-byte
// asynchronous copies into its own place in shared memory: a lane reads what it
// copied itself, so there is no barrier, and requests the next tile's keys as soon
// as this tile's are read, its values likewise. At a unit's end the warps are merged
// in shared memory. A unit that lies in several CTAs' shares leaves partials, which
// the last of them to finish merges in CTA order, so results do not depend on
// timing.
//
// Bound by HBM where caches are long: 16 sequences x 10 heads at 32,760 positions,
// 8 rows each, 200 us for 1.34 GB (6.7 TB/s, what a copy reaches). At 2,048
// positions (32 sequences, 1,650 on average, 135 MB) 32 us against 21: about 5 us
// until every SM has its first tile, the turns from unit to unit, 4 us for the units
// that CTAs share. With 16 rows to a kv head (32 heads on 8, 491 MB) 91 us against
// 75, with 32 rows 154: 12 warps an SM wait for their own chains of products. One
// sequence of 777 positions: 9.7 us, of which the tile itself is 2; 3,000: 14.7, with
// 47 partials a unit to join.
// Loads into registers instead of the copies: 104.6 and 188.5 us where these take
// 91 and 154 (the 32 registers they free are what the loop waits for), 205 where
// these take 200. The copies go by way of L1, and the rest of L1 matters to them: a
// larger part of it given to shared memory, or more tiles a warp under way, took 105
// to 108 us; past L1 (.cg) 108. Bulk copies by a producer warp, or rings that a warp
// shares, took 264 and 350 us at 32,760 positions: their barriers.
#pragma once
#include "attention.cuh"
#include "kv8.cuh"

namespace vg {

constexpr int kKaMaxRows = 8;      // new rows per sequence
constexpr int kKaMaxGroup = 16;    // query heads per kv head
constexpr int kKaTable = 128;      // sequences per launch
constexpr float kKaSlack = 6.0f;   // log2 of the largest weight
constexpr float kKaLift = 512.0f;  // 2^9, on the f16 weights
constexpr float kKaTiny = 5.9604645e-8f;  // 2^-24, the unit of f16 subnormals

struct Kv8AttnArgs {
  Kv8View c;
  int32_t b0, nb;                // the launch's sequences: b0 .. b0 + nb - 1
  int32_t rows, n_heads, n_tiles;  // rows per sequence; n_tiles: 8 NT-row tiles of a kv head's rows * group query rows
  const __nv_bfloat16* q;
  int64_t q_stride;
  const int32_t* lens;   // [B] positions before the new rows
  const int32_t* first;  // [B] or null: 0
  const int32_t* n_new;  // [B] or null: all rows
  float scale_log2;      // scale * log2(e) / Q
  float* part;           // [2 grid][8 NT][DIM + 4]: weighted values, then maximum and sum
  uint32_t* arrived;     // [grid]: partials written of the unit that starts in CTA i and ends in a later one; zero between calls
  __nv_bfloat16* o;
  int64_t o_stride;
};

// Warps per CTA and CTAs per SM: 16 warps of at most 128 registers where a unit
// has up to 8 query rows, 12 of at most 168 where it has 16 (8 of 240: 120 us where
// 12 took 109). Small CTAs: their turns from unit to unit fall apart in time (8
// warps x 2: 33.4 us where 4 x 4 takes 32.2).
constexpr int kKaWarps = 4;
__host__ __device__ constexpr int ka_ctas(int nt) { return nt == 1 ? 4 : 3; }
// Tiles of a warp on their way to shared memory: 4 KB of codes. (Two at 128
// dimensions: 236 us at 32,760 positions where one takes 200.)
__host__ __device__ constexpr int ka_slots(int dim) { return dim == 128 ? 1 : 2; }
__host__ __device__ constexpr int ka_ring_bytes(int dim) { return kKaWarps * ka_slots(dim) * 2 * kKv8Group * dim; }

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

// The query rows of a unit as Q^T fragments, with what belongs to each row: in a
// CTA's shared memory where a unit has several tiles of 8 rows (32 registers a
// lane less: 12 warps an SM without spills), else in every warp's registers.
template <int DIM, int NT>
struct Kv8Rows {
  uint2 frag[NT][DIM / 16][32];  // of lane (g, t): row g, the k-step's two pairs
  float mult[8 * NT], bias[8 * NT];
  int last[8 * NT];
};

// One warp's running softmax over groups of 16 positions, for NT tiles of 8
// query rows. Lane (g, t) = (lane / 4, lane % 4) holds columns (rows) 2t, 2t+1
// of every tile.
template <int FMT, int DIM, int NT>
struct Kv8Warp {
  static constexpr bool kShared = NT > 1;  // the fragments are in shared memory: q holds one tile while it is set up
  uint32_t q[kShared ? 1 : NT][DIM / 16][2];  // Q^T fragments
  float mult[NT][2];             // softmax scale * log2(e) / Q * 2^e of rows 2t, 2t+1
  int last[NT][2];               // last position those rows see (-1: none)
  float bias[NT][2];             // int8: what the 128 in every code adds to a score's sum
  float m[NT][2], l[NT][2];      // running maximum (log2 units) and this lane's share of the sum
  float o[NT][DIM / 32][2][4];   // O^T: dimensions 4 (g + 8 j) + 0..3
  float top_v;                   // largest magnitude of a value block seen: o is in units of it / Q / kKaLift

  // One tile of 8 query rows, 16 dimensions of every 64 a lane; zeros behind the real ones.
  __device__ __forceinline__ void load(const Kv8AttnArgs& a, int b, int kvh, int tile8, int n_q, int lane) {
    const int g = lane >> 2, t = lane & 3, group = a.n_heads / a.c.n_kv;
    // column g of the tile: query row r = i * group + head in the group
    const int r = tile8 * 8 + g;
    const bool real = r < n_q;
    const int i = real ? r / group : 0, h = kvh * group + (real ? r - i * group : 0);
    const __nv_bfloat16* src = a.q + ((int64_t)b * a.rows + i) * a.q_stride + h * DIM + 16 * t;
#pragma unroll
    for (int k = 0; k < DIM / 64; ++k) {
      uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
      if (real) {
        w0 = *reinterpret_cast<const uint4*>(src + 64 * k);
        w1 = *reinterpret_cast<const uint4*>(src + 64 * k + 8);
      }
      q[0][4 * k][0] = w0.x, q[0][4 * k][1] = w0.y, q[0][4 * k + 1][0] = w0.z, q[0][4 * k + 1][1] = w0.w;
      q[0][4 * k + 2][0] = w1.x, q[0][4 * k + 2][1] = w1.y, q[0][4 * k + 3][0] = w1.z, q[0][4 * k + 3][1] = w1.w;
    }
  }

  // Turns the loaded rows into f16 fragments; row g's factor, bias and last position.
  __device__ __forceinline__ void convert(const Kv8AttnArgs& a, int tile8, const Kv8Span& s, int lane, float* row_mult,
                                          float* row_bias, int* row_last) {
    const int group = a.n_heads / a.c.n_kv;
    float big = 0.0f;
#pragma unroll
    for (int k = 0; k < DIM / 16; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e) big = fmaxf(big, fmaxf(fabsf(bf16_lo(q[0][k][e])), fabsf(bf16_hi(q[0][k][e]))));
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
    // 2^(14 - floor(log2 big)), as two factors: the product may leave the normal range
    const int ex = big > 0.0f && big < INFINITY ? ilogbf(big) : 0, lift = 14 - ex;
    const float up0 = __int_as_float((lift / 2 + 127) << 23), up1 = __int_as_float((lift - lift / 2 + 127) << 23);
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < DIM / 16; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const __half2 h2 = __floats2half2_rn(bf16_lo(q[0][k][e]) * up0 * up1, bf16_hi(q[0][k][e]) * up0 * up1);
        q[0][k][e] = *reinterpret_cast<const uint32_t*>(&h2);
        sum += __low2float(h2) + __high2float(h2);
      }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    const float down0 = __int_as_float((127 - lift / 2) << 23), down1 = __int_as_float((127 - (lift - lift / 2)) << 23);
    const int r = tile8 * 8 + (lane >> 2);
    *row_bias = FMT == kKv8Int8 ? sum * (kKaTiny * 128.0f) : 0.0f;
    *row_mult = a.scale_log2 * down0 * down1 * (FMT == kKv8Int8 ? 1.0f / kKaTiny : 1.0f);
    *row_last = r < s.n * group ? s.L + r / group : -1;
  }

  // Sets up the loaded rows and clears the sums. With shared fragments warp nt has
  // loaded tile nt, and the CTA meets here.
  __device__ __forceinline__ void begin(const Kv8AttnArgs& a, int tile, const Kv8Span& s, int warp, int lane,
                                        Kv8Rows<DIM, NT>* rows) {
    const int t = lane & 3;
    float row_mult, row_bias;
    int row_last;
    if constexpr (kShared) {
      if (warp < NT) {
        convert(a, tile * NT + warp, s, lane, &row_mult, &row_bias, &row_last);
#pragma unroll
        for (int k = 0; k < DIM / 16; ++k) rows->frag[warp][k][lane] = make_uint2(q[0][k][0], q[0][k][1]);
        if (t == 0) {
          const int r = warp * 8 + (lane >> 2);
          rows->mult[r] = row_mult;
          rows->bias[r] = row_bias;
          rows->last[r] = row_last;
        }
      }
      __syncthreads();
    } else {
      convert(a, tile, s, lane, &row_mult, &row_bias, &row_last);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 2 * t + e;
        if constexpr (kShared) {
          mult[nt][e] = rows->mult[nt * 8 + r];
          bias[nt][e] = rows->bias[nt * 8 + r];
          last[nt][e] = rows->last[nt * 8 + r];
        } else {
          mult[nt][e] = __shfl_sync(0xffffffffu, row_mult, 4 * r);
          bias[nt][e] = __shfl_sync(0xffffffffu, row_bias, 4 * r);
          last[nt][e] = __shfl_sync(0xffffffffu, row_last, 4 * r);
        }
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

  // A group of 16 positions in three steps: scores of its keys, weights, values.
  // Keys in int8 enter as (code + 128) 2^-24, f16 subnormals that cost no
  // subtraction; 128 times the row's sum is taken off the score. (Values do not:
  // their weights are all positive, so the 128s would not cancel and the sums
  // would lose what they add.)
  __device__ __forceinline__ void scores(const uint4 (&kf)[DIM / 32], float (&s)[NT][4], const Kv8Rows<DIM, NT>* rows,
                                         int lane) const {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = 0.0f;
#pragma unroll
    for (int h = 0; h < DIM / 64; ++h) {
      const uint4 ka = kf[2 * h], kc = kf[2 * h + 1];
      const uint32_t xa[4] = {ka.x, ka.y, ka.z, ka.w}, xc[4] = {kc.x, kc.y, kc.z, kc.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t a0, a1, a2, a3;
        if constexpr (FMT == kKv8Int8) {
          kv8_to_tiny(xa[w], &a0, &a2);
          kv8_to_tiny(xc[w], &a1, &a3);
        } else {
          kv8_to_half<FMT>(xa[w], &a0, &a2);
          kv8_to_half<FMT>(xc[w], &a1, &a3);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (kShared) {
            const uint2 f = rows->frag[nt][h * 4 + w][lane];
            mma_f16(s[nt], a0, a1, a2, a3, f.x, f.y);
          } else {
            mma_f16(s[nt], a0, a1, a2, a3, q[nt][h * 4 + w][0], q[nt][h * 4 + w][1]);
          }
        }
      }
    }
  }

  // ks, vs: the magnitudes of the positions' blocks. plain: every row sees all of
  // p0 .. p0 + 15.
  __device__ __forceinline__ void weights(float (&s)[NT][4], float ks, float vs, int p0, int lo, bool plain, int lane,
                                          uint32_t (&b0)[NT], uint32_t (&b1)[NT]) {
    const int tok = 4 * (lane >> 3) + ((lane >> 2) & 1);  // tile row g = lane / 4; row g + 8 is position tok + 2
    bool above = vs > top_v;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float mu[2] = {mult[nt][0] * ks, mult[nt][1] * ks};
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = (FMT == kKv8Int8 ? s[nt][e] - bias[nt][e & 1] : s[nt][e]) * mu[e & 1];
    }
    if (!plain) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int p = p0 + tok + (e & 2);
          if (p < lo || p > last[nt][e & 1]) s[nt][e] = -INFINITY;
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) above |= fmaxf(s[nt][e], s[nt][2 + e]) > m[nt][e] + kKaSlack;
    if (__any_sync(0xffffffffu, above)) {  // new maxima (or a larger value magnitude)
      const float grow_v = vs > top_v ? top_v / vs : 1.0f;
      top_v = fmaxf(top_v, vs);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(s[nt][e], s[nt][2 + e]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float now = fmaxf(m[nt][e], mx);
          const float f = now > -INFINITY ? ex2(m[nt][e] - now) : 1.0f;
          m[nt][e] = now;
          l[nt][e] *= f;
#pragma unroll
          for (int j = 0; j < DIM / 32; ++j) {
            o[nt][j][0][e] *= f * grow_v;
            o[nt][j][0][2 + e] *= f * grow_v;
            o[nt][j][1][e] *= f * grow_v;
            o[nt][j][1][2 + e] *= f * grow_v;
          }
        }
    }
    float share = kKaLift;
    if (vs != top_v) share = top_v > 0.0f ? vs / top_v * kKaLift : 0.0f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float base = m[nt][e & 1] > -INFINITY ? m[nt][e & 1] : 0.0f;
        w[e] = ex2(s[nt][e] - base);
      }
      l[nt][0] += w[0] + w[2];
      l[nt][1] += w[1] + w[3];
      // rows 2t, 2t+1 of positions g, g + 8 -> positions 2t, 2t+1 (+ 8) of row g
      b0[nt] = movmatrix_trans(pack_half2(w[0] * share, w[1] * share));
      b1[nt] = movmatrix_trans(pack_half2(w[2] * share, w[3] * share));
    }
  }

  // lo, hi: the sequence's positions that any row sees, counted from the group's first
  __device__ __forceinline__ void values(const uint4 (&vf)[DIM / 32], const uint32_t (&b0)[NT], const uint32_t (&b1)[NT],
                                         int lo, int hi, int lane) {
    uint32_t keep = 0xFFFFFFFFu;
    if (FMT == kKv8E4m3 && (lo > 0 || hi < kKv8Group)) {  // a code never written may be NaN, and 0 * NaN is not 0
      const int p = 4 * (lane & 3);
      if (hi < p + 4) keep = hi <= p ? 0u : 0xFFFFFFFFu >> (8 * (p + 4 - hi));
      if (lo > p) keep = lo >= p + 4 ? 0u : keep & (0xFFFFFFFFu << (8 * (lo - p)));
    }
#pragma unroll
    for (int j = 0; j < DIM / 32; ++j) {
      uint32_t x[4] = {vf[j].x, vf[j].y, vf[j].z, vf[j].w};
      if (FMT == kKv8E4m3)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] &= keep;
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

// Where a tile of the launch's list lies.
struct KaPlace {
  int b, kvh, tile;  // sequence of the launch, kv head, row tile
  int j, n;          // tile of the unit, and how many it has
};

// 16 bytes global -> shared, asynchronous; groups of them complete in order. (By way
// of L1: past it, .cg, 32 heads on 8 took 108 us where this takes 91.)
__device__ __forceinline__ void ka_cp16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void ka_cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void ka_cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// A lane's 16 bytes of every 512 from p on.
template <int N>
__device__ __forceinline__ void ka_lds(uint4 (&v)[N], uint32_t p) {
#pragma unroll
  for (int j = 0; j < N; ++j)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[j].x), "=r"(v[j].y), "=r"(v[j].z), "=r"(v[j].w)
                 : "r"(p + j * 512)
                 : "memory");
}

// o of row r of p's tile, dimensions d .. d + 3, from the weighted values and the
// sum of weights; rows from n_q on are not real: 0.
template <int DIM, int NT>
__device__ __forceinline__ void ka_store(const Kv8AttnArgs& a, const KaPlace& p, int n_q, int r, int d, float4 v, float l) {
  const int group = a.n_heads / a.c.n_kv, rr = p.tile * 8 * NT + r;
  if (rr >= a.rows * group) return;
  const int i = rr / group, h = p.kvh * group + rr - i * group;
  const float inv = rr < n_q && l != 0.0f ? 1.0f / l : 0.0f;  // NaN sums stay NaN
  if (inv == 0.0f) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const __nv_bfloat162 x = __floats2bfloat162_rn(v.x * inv, v.y * inv), y = __floats2bfloat162_rn(v.z * inv, v.w * inv);
  *reinterpret_cast<uint2*>(a.o + ((int64_t)(a.b0 + p.b) * a.rows + i) * a.o_stride + h * DIM + d) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

template <int FMT, int DIM, int NT>
__global__ void __launch_bounds__(32 * kKaWarps, ka_ctas(NT)) kv8_attn(const Kv8AttnArgs a) {
  constexpr int W = kKaWarps, kThreads = 32 * W, kTile = kKv8Group * W;
  constexpr int kRowW = DIM + 4, kPartW = DIM + 4;  // floats of a row: of a warp's sums, of a CTA's partials
  constexpr int S = ka_slots(DIM), kHalf = kKv8Group * DIM, kSlot = 2 * kHalf;  // a slot: a group's keys, its values
  extern __shared__ __align__(16) uint8_t ring_smem[];
  __shared__ __align__(16) float wo[W * 8 * kRowW];
  __shared__ float wm[W * 8], wl[W * 8];
  __shared__ Kv8Rows<DIM, NT> rows_s;  // (unused with one tile of rows)
  __shared__ int start[kKaTable + 1];  // first tile of each sequence
  __shared__ int4 span[kKaTable];      // lo, hi, L, n
  __shared__ int sums[kKaTable / 32];
  __shared__ int last_s[2];
  __shared__ KaPlace edge[2];  // the units of this share's first and last tile
  __shared__ int ends[2][2];   // their first and last CTA
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = a.n_heads / a.c.n_kv, units = a.c.n_kv * a.n_tiles;  // units per sequence
  griddep_launch_dependents();
  griddep_wait();
  // ---- the list of tiles: every sequence's range and first tile
  for (int c = warp; c * 32 < a.nb; c += W) {
    const int i = c * 32 + lane;
    int n = 0;
    if (i < a.nb) {
      Kv8Span s;
      if (!kv8_span(a, a.b0 + i, &s) && blockIdx.x == 0) record_error(kErrBounds, 343);
      span[i] = make_int4(s.lo, s.hi, s.L, s.n);
      // an empty sequence has one tile a unit, without positions: its rows become 0
      n = units * max(1, cdiv(s.hi - s.lo / kKv8Group * kKv8Group, kTile));
    }
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (i < a.nb) start[i] = sum - n;
    if (lane == 31) sums[c] = sum;
  }
  __syncthreads();
  for (int i = tid; i <= a.nb; i += kThreads) {
    int before = 0;
    for (int c = 0; c < (i < a.nb ? i / 32 : cdiv(a.nb, 32)); ++c) before += sums[c];
    start[i] = (i < a.nb ? start[i] : 0) + before;
  }
  __syncthreads();
  // G CTAs with a share each, none of it empty (the count of a split unit's CTAs
  // relies on that): CTA i has `each` tiles from i * each + min(i, more) on, and
  // one more if i < more
  const int total = start[a.nb], G = min((int)gridDim.x, total), me = blockIdx.x;
  const int each = total / G, more = total - each * G;
  if (me >= G) return;
  const int t0 = me * each + min(me, more), t1 = t0 + each + (me < more);
  auto owner = [&](int T) {  // the CTA whose share holds tile T
    const int big = more * (each + 1);
    return T < big ? T / (each + 1) : more + (T - big) / each;
  };
  auto place = [&](int T, int b) {  // tile T, in sequence b or a later one
    while (T >= start[b + 1]) ++b;
    KaPlace p;
    p.b = b;
    p.n = (start[b + 1] - start[b]) / units;
    const int rem = T - start[b], u = rem / p.n;
    p.j = rem - u * p.n;
    p.kvh = u / a.n_tiles;
    p.tile = u - p.kvh * a.n_tiles;
    return p;
  };
  auto locate = [&](int T) {
    int lo = 0, hi = a.nb - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (start[mid] <= T) lo = mid;
      else hi = mid - 1;
    }
    return place(T, lo);
  };
  const size_t blocks = (size_t)a.c.L_max >> a.c.log2;
  const int g = lane >> 2, t = lane & 3;
  // this lane's bytes in a group: of the keys positions tok and tok + 2, of the values 4 dimensions of 4 positions
  const int k_at = (4 * (g >> 1) + (g & 1)) * 64 + t * 16, v_at = lane * 16;

  Kv8Warp<FMT, DIM, NT> w;
  uint4 kf[DIM / 32], vf[DIM / 32];
  float ks = 0.0f, vs = 0.0f;
  KaPlace p = locate(t0);
  Kv8Span s;
  const uint32_t ring = smem_u32(ring_smem) + warp * S * kSlot + lane * 16;  // this lane's 16 bytes of every 512
  const uint8_t *kp = nullptr, *vp = nullptr;  // this lane's bytes of the next keys and values to request
  const float *ka = nullptr, *va = nullptr;
  int p0 = 0, mine = 0;  // this warp's first position, and its groups of the share of the unit
  auto load_k = [&](int slot) {
#pragma unroll
    for (int h = 0; h < DIM / 64; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i) ka_cp16(ring + slot * kSlot + (2 * h + i) * 512, kp + h * 1024 + i * 128);
    kp += kTile * DIM;
  };
  auto load_v = [&](int slot) {
#pragma unroll
    for (int j = 0; j < DIM / 32; ++j) ka_cp16(ring + slot * kSlot + kHalf + j * 512, vp + j * 512);
    vp += kTile * DIM;
  };
  auto magnitudes = [&](int p) {
    ks = ka[p >> a.c.log2];
    vs = va[p >> a.c.log2];
  };
  auto enter = [&](int T) {  // a unit's share from tile T on: request its query rows, then its first tiles
    const int4 sp = span[p.b];
    s = Kv8Span{sp.z, sp.x, sp.y, sp.w};
    if (NT == 1 || warp < NT) w.load(a, a.b0 + p.b, p.kvh, p.tile * NT + (NT == 1 ? 0 : warp), s.n * group, lane);
    p0 = s.lo / kKv8Group * kKv8Group + p.j * kTile + warp * kKv8Group;
    mine = p0 < s.hi ? min(min(p.n - p.j, t1 - T), cdiv(s.hi - p0, kTile)) : 0;
    const size_t head = (size_t)(a.b0 + p.b) * a.c.n_kv + p.kvh;
    kp = a.c.k + (head * a.c.L_max + p0) * DIM + k_at;
    vp = a.c.v + (head * a.c.L_max + p0) * DIM + v_at;
    ka = a.c.k_amax + head * blocks, va = a.c.v_amax + head * blocks;
    if (mine > 0) magnitudes(p0);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      if (i < mine) load_k(i);
      ka_cp_commit();
      if (i < mine) load_v(i);
      ka_cp_commit();
    }
  };
  enter(t0);
  for (int T = t0; T < t1;) {
    const int seg0 = T - p.j, seg1 = seg0 + p.n;  // the unit's tiles
    const int n = min(seg1, t1) - T;              // those of this CTA
    w.begin(a, p.tile, s, warp, lane, &rows_s);
    int slot = 0;
    for (int i = 0; i < mine; ++i) {
      const bool more = i + S < mine;  // another tile to request
      float z[NT][4];
      uint32_t b0[NT], b1[NT];
      // a lane reads what it copied itself, and requests the next 16 bytes into the
      // same place: no barrier. Copies complete in the order K0 V0 K1 V1 ..; 2 S are
      // under way (empty ones at the end), the oldest is wanted.
      ka_cp_wait<2 * S - 1>();
      ka_lds(kf, ring + slot * kSlot);
      w.scores(kf, z, &rows_s, lane);
      const float ks_now = ks, vs_now = vs;
      if (more) load_k(slot);
      ka_cp_commit();
      if (i + 1 < mine) magnitudes(p0 + kTile);
      w.weights(z, ks_now, vs_now, p0, s.lo, p0 >= s.lo && p0 + kKv8Group - 1 <= s.L, lane, b0, b1);
      ka_cp_wait<2 * S - 1>();
      ka_lds(vf, ring + slot * kSlot + kHalf);
      w.values(vf, b0, b1, s.lo - p0, s.hi - p0, lane);
      if (more) load_v(slot);
      ka_cp_commit();
      if (++slot == S) slot = 0;
      p0 += kTile;
    }
    T += n;
    const bool whole = seg0 >= t0 && T == seg1;
    const KaPlace done = p;
    if (tid == 0) {
      if (T - n == t0) edge[0] = p;
      if (T == t1) edge[1] = p;
    }
    const int n_q = s.n * group;
    // ---- merge the warps, 8 rows at a time: their sums to shared memory, then a thread per row and 4 dimensions
    const float back = w.top_v / (kv8_q<FMT>() * kKaLift);
    float* slot_out = a.part + (size_t)(2 * me + (seg0 < t0 ? 0 : 1)) * (8 * NT) * kPartW;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (nt > 0) __syncthreads();
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 2 * t + e;
        float l = w.l[nt][e];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (g == 0) {
          wm[warp * 8 + r] = w.m[nt][e];
          wl[warp * 8 + r] = l;
        }
#pragma unroll
        for (int j = 0; j < DIM / 32; ++j)
          *reinterpret_cast<float4*>(wo + (warp * 8 + r) * kRowW + 4 * (g + 8 * j)) =
              make_float4(w.o[nt][j][0][e] * back, w.o[nt][j][0][2 + e] * back, w.o[nt][j][1][e] * back,
                          w.o[nt][j][1][2 + e] * back);
      }
      if (nt == NT - 1 && T < t1) {  // the next unit's data travels while this one's warps are merged
        p = place(T, p.b);
        enter(T);
      }
      __syncthreads();
      for (int i = tid; i < 8 * (DIM / 4); i += kThreads) {
        const int r = i / (DIM / 4), d = i % (DIM / 4) * 4;
        float mm = -INFINITY, ls = 0.0f;
#pragma unroll
        for (int k = 0; k < W; ++k) mm = fmaxf(mm, wm[k * 8 + r]);
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float base = mm > -INFINITY ? mm : 0.0f;  // (a row of NaN has no maximum and keeps its NaN)
#pragma unroll
        for (int k = 0; k < W; ++k) {
          const float f = ex2(wm[k * 8 + r] - base);
          const float4 v = *reinterpret_cast<const float4*>(wo + (k * 8 + r) * kRowW + d);
          ls += wl[k * 8 + r] * f;
          acc.x += v.x * f, acc.y += v.y * f, acc.z += v.z * f, acc.w += v.w * f;
        }
        if (whole) {
          ka_store<DIM, NT>(a, done, n_q, nt * 8 + r, d, acc, ls);
        } else {
          float* x = slot_out + (nt * 8 + r) * kPartW;
          *reinterpret_cast<float4*>(x + d) = acc;
          if (d == 0) *reinterpret_cast<float2*>(x + DIM) = make_float2(mm, ls);
        }
      }
    }
    __syncthreads();  // the merge buffers are free again
  }

  // ---- units that lie in other CTAs' shares too: the one of this share's first
  // tile, and the one of its last. Whoever is the last of a unit's CTAs to get
  // here joins its partials. (At the share's end, both counters at once, so that no
  // unit's turn waits for a round trip.)
  if (warp < 2 && lane == 0) {
    const int seg0 = start[edge[warp].b] + (edge[warp].kvh * a.n_tiles + edge[warp].tile) * edge[warp].n, seg1 = seg0 + edge[warp].n;
    int last = 0;
    if (warp == 0 ? seg0 < t0 : seg0 >= t0 && seg1 > t1) {
      const int c0 = owner(seg0), c1 = owner(seg1 - 1);
      ends[warp][0] = c0, ends[warp][1] = c1;
      // (releases the partials of the whole CTA, written before the barrier above; acquires the others')
      last = atomic_add_acq_rel(a.arrived + c0, 1u) == (uint32_t)(c1 - c0);
    }
    last_s[warp] = last;
  }
  __syncthreads();
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    if (!last_s[side]) continue;
    const KaPlace e = edge[side];
    const int c0 = ends[side][0], c1 = ends[side][1];
    const int n_q = span[e.b].w * group;
    // A row belongs to kLanes lanes, 4 dimensions each. They take as many CTAs'
    // partials at a time: their maxima and sums a lane each, then the values, 8
    // requests of 16 bytes under way. (4: 47 partials take 3.6 us longer; 16: the
    // registers cost the main loop 1.3 us at 32 sequences of 2,048 positions.)
    constexpr int kLanes = DIM / 4, kItems = 8 * NT * kLanes / kThreads, kBatch = 8 / kItems;
    static_assert(kLanes <= 32 && kLanes % kBatch == 0 && kItems * kThreads == 8 * NT * kLanes);
    const int sub = tid % kLanes, r0 = tid / kLanes;  // rows r0 + u * (kThreads / kLanes)
    float mm[kItems], ls[kItems];
    float4 acc[kItems];
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
      mm[u] = -INFINITY, ls[u] = 0.0f;
      acc[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
#pragma unroll 1
    for (int c = c0; c <= c1; c += kLanes) {
      const int nc = min(kLanes, c1 + 1 - c);
      auto row = [&](int j, int u) {  // row u of this thread in the partials of CTA c + j
        const int slot = 2 * (c + j) + (c + j == c0 ? 1 : 0);
        return a.part + ((size_t)slot * (8 * NT) + r0 + u * (kThreads / kLanes)) * kPartW;
      };
      float2 ml[kItems];
      float f[kItems];
#pragma unroll
      for (int u = 0; u < kItems; ++u)
        ml[u] = sub < nc ? __ldcg(reinterpret_cast<const float2*>(row(sub, u) + DIM)) : make_float2(-INFINITY, 0.0f);
#pragma unroll 1
      for (int j0 = 0; j0 < nc; j0 += kBatch) {
        float4 v[kBatch][kItems];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
#pragma unroll
          for (int u = 0; u < kItems; ++u)
            if (j0 + j < nc) v[j][u] = __ldcg(reinterpret_cast<const float4*>(row(j0 + j, u) + 4 * sub));
        if (j0 == 0) {
#pragma unroll
          for (int u = 0; u < kItems; ++u) {
            float now = ml[u].x;
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, o));
            now = fmaxf(now, mm[u]);
            const float base = now > -INFINITY ? now : 0.0f, back = ex2(mm[u] - base);
            f[u] = ex2(ml[u].x - base);
            float l = ml[u].y * f[u];
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            mm[u] = now;
            ls[u] = ls[u] * back + l;
            acc[u].x *= back, acc[u].y *= back, acc[u].z *= back, acc[u].w *= back;
          }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
#pragma unroll
          for (int u = 0; u < kItems; ++u) {
            const float h = __shfl_sync(0xffffffffu, f[u], j0 + j, kLanes);
            if (j0 + j < nc)
              acc[u].x += v[j][u].x * h, acc[u].y += v[j][u].y * h, acc[u].z += v[j][u].z * h, acc[u].w += v[j][u].w * h;
          }
      }
    }
#pragma unroll
    for (int u = 0; u < kItems; ++u) ka_store<DIM, NT>(a, e, n_q, r0 + u * (kThreads / kLanes), 4 * sub, acc[u], ls[u]);
    if (tid == 0) atomicExch(a.arrived + c0, 0u);
  }
}

}  // namespace vg
