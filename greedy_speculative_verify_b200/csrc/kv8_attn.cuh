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
// Work: a unit is (sequence, kv head, 8 NT query rows), cut into tiles of 128
// positions. All tiles of the batch form one list, of which every CTA (one per
// SM) takes an equal contiguous share, whatever the lengths are. One warp feeds
// a ring of tiles (two bulk copies each: a tile's keys, and its values, are
// contiguous; the blocks' magnitudes beside them); warp w of the other eight
// runs its own softmax over positions 16 w .. 16 w + 15 of every tile. At a
// unit's end the warps are merged in shared memory. A unit that lies in several
// CTAs' shares leaves partials, which the last of them to finish merges in CTA
// order, so results do not depend on timing.
#pragma once
#include "attention.cuh"
#include "kv8.cuh"

namespace vg {

constexpr int kKaWarps = 8;        // consumer warps
constexpr int kKaTile = 16 * kKaWarps;  // positions per tile
constexpr int kKaThreads = 32 * (kKaWarps + 1);
constexpr int kKaMaxRows = 8;      // new rows per sequence
constexpr int kKaMaxGroup = 16;    // query heads per kv head
constexpr int kKaTable = 512;      // sequences per launch
constexpr int kKaStages = 8;       // ring slots at most
constexpr float kKaSlack = 6.0f;   // log2 of the largest weight
constexpr float kKaLift = 512.0f;  // 2^9, on the f16 weights

struct Kv8AttnArgs {
  Kv8View c;
  int32_t b0, nb;                // the launch's sequences: b0 .. b0 + nb - 1
  int32_t rows, n_heads, n_tiles;  // rows per sequence; n_tiles: 8 NT-row tiles of a kv head's rows * group query rows
  int32_t stages;
  const __nv_bfloat16* q;
  int64_t q_stride;
  const int32_t* lens;   // [B] positions before the new rows
  const int32_t* first;  // [B] or null: 0
  const int32_t* n_new;  // [B] or null: all rows
  float scale_log2;      // scale * log2(e) / Q
  float* part;           // [2 grid][8 NT][DIM + 2]: weighted values, then maximum and sum
  uint32_t* arrived;     // [grid]: partials written of the unit that starts in CTA i and ends in a later one; zero between calls
  __nv_bfloat16* o;
  int64_t o_stride;
};

__host__ __device__ constexpr int ka_stage_bytes(int dim) { return 2 * kKaTile * dim; }
__host__ __device__ constexpr int ka_merge_bytes(int dim, int nt) { return kKaWarps * 8 * nt * (dim + 4 + 2) * 4; }
__host__ __device__ constexpr int ka_fixed_bytes(int dim, int nt) {
  return 1024 + kKaTable * 24 + 16 + ka_merge_bytes(dim, nt) + kKaStages * 16 * 4;
}

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
  float top_v;                   // largest magnitude of a value block seen: o is in units of it / Q / kKaLift

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
  // and values (the group's bytes), and the magnitudes of their blocks. plain:
  // every row sees all 16.
  __device__ __forceinline__ void group16(const uint8_t* kb, const uint8_t* vb, float ks, float vs, int p0, int lo,
                                          int hi, bool plain, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const int tok = 4 * (g >> 1) + (g & 1);  // tile row g; row g + 8 is position tok + 2
    float s[NT][4], s2[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = s2[nt][e] = 0.0f;
    uint4 vf[DIM / 32];
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
        for (int nt = 0; nt < NT; ++nt)  // two chains of sums
          mma_f16(w & 1 ? s2[nt] : s[nt], a0, a1, a2, a3, q[nt][h * 4 + w][0], q[nt][h * 4 + w][1]);
      }
    }
#pragma unroll
    for (int j = 0; j < DIM / 32; ++j) vf[j] = *reinterpret_cast<const uint4*>(vb + (g + 8 * j) * 64 + t * 16);
    // ---- weights
    float z[NT][2][2];
    bool above = vs > top_v;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mu = mult[nt][e] * ks;
        z[nt][e][0] = (s[nt][e] + s2[nt][e]) * mu;
        z[nt][e][1] = (s[nt][2 + e] + s2[nt][2 + e]) * mu;
        if (!plain) {
          const int pa = p0 + tok, pc = pa + 2;
          if (pa < lo || pa > last[nt][e]) z[nt][e][0] = -INFINITY;
          if (pc < lo || pc > last[nt][e]) z[nt][e][1] = -INFINITY;
        }
        above |= fmaxf(z[nt][e][0], z[nt][e][1]) > m[nt][e] + kKaSlack;
      }
    if (__any_sync(0xffffffffu, above)) {  // new maxima (or a larger value scale)
      const float grow_v = vs > top_v ? top_v / vs : 1.0f;
      top_v = fmaxf(top_v, vs);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(z[nt][e][0], z[nt][e][1]);
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
    const float share = top_v > 0.0f ? vs / top_v * kKaLift : 0.0f;
    uint32_t b0[NT], b1[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float w[2][2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float base = m[nt][e] > -INFINITY ? m[nt][e] : 0.0f;
        w[e][0] = ex2(z[nt][e][0] - base);
        w[e][1] = ex2(z[nt][e][1] - base);
        l[nt][e] += w[e][0] + w[e][1];
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

// Where a tile of the launch's list lies.
struct KaPlace {
  int b, kvh, tile;  // sequence of the launch, kv head, row tile
  int j, n;          // tile of the unit, and how many it has
};

__device__ __forceinline__ void ka_bar() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kKaWarps) : "memory"); }

// Four bytes global -> shared, asynchronous; ka_cp_arrive makes the barrier see
// this lane's copies complete (one arrival, counted at initialisation).
__device__ __forceinline__ void ka_cp4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void ka_cp_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

template <int FMT, int DIM, int NT>
__global__ void __launch_bounds__(kKaThreads, 1) kv8_attn(const Kv8AttnArgs a) {
  constexpr int kTileBytes = kKaTile * DIM, kRowW = DIM + 4;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem;  // [stages][keys | values]
  uint8_t* at = smem + a.stages * ka_stage_bytes(DIM);
  float* wo = reinterpret_cast<float*>(at);                 // [kKaWarps][8 NT][kRowW]
  float* wm = wo + kKaWarps * 8 * NT * kRowW;               // [kKaWarps][8 NT]
  float* wl = wm + kKaWarps * 8 * NT;
  float* mag = wl + kKaWarps * 8 * NT;                      // [stages][keys 8 | values 8]
  int64_t* start = reinterpret_cast<int64_t*>(mag + kKaStages * 16);  // [kKaTable + 1] first tile of each sequence
  int4* span = reinterpret_cast<int4*>(start + kKaTable + 2);         // [kKaTable] lo, hi, L, n
  __shared__ __align__(8) uint64_t full[kKaStages], empty[kKaStages];
  __shared__ int64_t sums[kKaTable / 32];
  __shared__ int last_s;
  __shared__ volatile int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = a.n_heads / a.c.n_kv, units = a.c.n_kv * a.n_tiles;  // units per sequence
  griddep_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&full[i], 1 + 16);
      mbar_init(&empty[i], kKaWarps);
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  griddep_wait();
  // ---- the list of tiles: every sequence's range and first tile
  for (int c = warp; c * 32 < a.nb; c += kKaWarps + 1) {
    const int i = c * 32 + lane;
    int64_t n = 0;
    if (i < a.nb) {
      Kv8Span s;
      if (!kv8_span(a, a.b0 + i, &s) && blockIdx.x == 0) record_error(kErrBounds, 343);
      span[i] = make_int4(s.lo, s.hi, s.L, s.n);
      // an empty sequence has one tile a unit, without positions: its rows become 0
      n = (int64_t)units * max(1, cdiv(s.hi - s.lo / kKv8Group * kKv8Group, kKaTile));
    }
    int64_t sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (i < a.nb) start[i] = sum - n;
    if (lane == 31) sums[c] = sum;
  }
  __syncthreads();
  for (int i = tid; i <= a.nb; i += kKaThreads) {
    int64_t before = 0;
    for (int c = 0; c < (i < a.nb ? i / 32 : cdiv(a.nb, 32)); ++c) before += sums[c];
    start[i] = (i < a.nb ? start[i] : 0) + before;
  }
  __syncthreads();
  // G CTAs with a share each, none of it empty (the count of a split unit's CTAs relies on that)
  const int64_t total = start[a.nb], G = min((int64_t)gridDim.x, total);
  const int64_t t0 = blockIdx.x < G ? total * blockIdx.x / G : 0, t1 = blockIdx.x < G ? total * (blockIdx.x + 1) / G : 0;
  const uint64_t limit = g_wait_timeout_ns;
  auto place = [&](int64_t T, int b) {  // tile T, in sequence b or a later one
    while (T >= start[b + 1]) ++b;
    KaPlace p;
    p.b = b;
    p.n = (int)((start[b + 1] - start[b]) / units);
    const int64_t rem = T - start[b];
    const int u = (int)(rem / p.n);
    p.j = (int)(rem - (int64_t)u * p.n);
    p.kvh = u / a.n_tiles;
    p.tile = u - p.kvh * a.n_tiles;
    return p;
  };
  auto locate = [&](int64_t T) {
    int lo = 0, hi = a.nb - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (start[mid] <= T) lo = mid;
      else hi = mid - 1;
    }
    return place(T, lo);
  };
  auto advance = [&](KaPlace& p) {  // to the next tile
    if (++p.j < p.n) return;
    p.j = 0;
    if (++p.tile < a.n_tiles) return;
    p.tile = 0;
    if (++p.kvh < a.c.n_kv) return;
    p.kvh = 0;
    if (++p.b < a.nb) p.n = (int)((start[p.b + 1] - start[p.b]) / units);
  };
  const size_t blocks = a.c.L_max / a.c.block;

  if (t0 < t1) {
    if (warp == kKaWarps) {
      // ---- producer
      KaPlace p = locate(t0);
      int stage = 0;
      uint32_t phase = 0, issued = 0, last_par = 0;
      for (int64_t T = t0; T < t1; ++T) {
        bool go = true;
        if (lane == 0) go = !abort_flag && mbar_wait(&empty[stage], phase ^ 1, limit);
        go = __shfl_sync(0xffffffffu, go, 0);
        __syncwarp();
        if (!go) {
          if (lane == 0 && !abort_flag) record_error(kErrTimeout, 344);
          abort_flag = 1;
          break;
        }
        const int4 s = span[p.b];
        const int p0 = s.x / kKv8Group * kKv8Group + p.j * kKaTile;
        const int groups = max(0, min(kKaWarps, cdiv(s.y - p0, kKv8Group)));
        const size_t head = (size_t)(a.b0 + p.b) * a.c.n_kv + p.kvh;
        if (lane == 0) {
          const uint32_t bytes = (uint32_t)groups * kKv8Group * DIM;
          mbar_arrive_expect_tx(&full[stage], 2 * bytes);
          if (bytes) {
            uint8_t* dst = ring + stage * ka_stage_bytes(DIM);
            const size_t src = (head * a.c.L_max + p0) * DIM;
            bulk_load(dst, a.c.k + src, bytes, &full[stage]);
            bulk_load(dst + kTileBytes, a.c.v + src, bytes, &full[stage]);
          }
        }
        if (lane < 16) {  // the magnitude of each group's block
          const int gi = lane & 7;
          if (gi < groups)
            ka_cp4(mag + stage * 16 + lane, (lane < 8 ? a.c.k_amax : a.c.v_amax) + head * blocks + (p0 + gi * kKv8Group) / a.c.block);
          ka_cp_arrive(&full[stage]);
        }
        issued |= 1u << stage;
        last_par = (last_par & ~(1u << stage)) | (phase << stage);
        if (++stage == a.stages) {
          stage = 0;
          phase ^= 1;
        }
        advance(p);
      }
      // every copy has landed before the CTA exits (also after a timeout)
      if (lane == 0)
        for (int i = 0; i < a.stages; ++i)
          if (issued & (1u << i)) mbar_wait(&full[i], (last_par >> i) & 1, limit);
    } else {
      // ---- consumers
      KaPlace p = locate(t0);
      int stage = 0;
      uint32_t phase = 0;
      Kv8Warp<FMT, DIM, NT> w;
      bool fresh = true;
      int64_t seg0 = t0 - p.j;  // the unit's first tile
      for (int64_t T = t0; T < t1; ++T) {
        const int4 sp = span[p.b];
        const Kv8Span s{sp.z, sp.x, sp.y, sp.w};
        if (fresh) {
          w.init(a, a.b0 + p.b, p.kvh, p.tile, s, lane);
          seg0 = T - p.j;
          fresh = false;
        }
        const bool go = __all_sync(0xffffffffu, !abort_flag && mbar_wait(&full[stage], phase, limit));
        if (!go) {  // the loop goes on without the data, so that the barriers below stay met
          if (!abort_flag) record_error(kErrTimeout, 345);
          abort_flag = 1;
        } else {
          const int p0 = s.lo / kKv8Group * kKv8Group + p.j * kKaTile + warp * kKv8Group;
          if (p0 < s.hi) {
            const uint8_t* kb = ring + stage * ka_stage_bytes(DIM) + warp * kKv8Group * DIM;
            w.group16(kb, kb + kTileBytes, mag[stage * 16 + warp], mag[stage * 16 + 8 + warp], p0, s.lo, s.hi,
                      p0 >= s.lo && p0 + kKv8Group - 1 <= s.L, lane);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[stage]);
        }
        if (++stage == a.stages) {
          stage = 0;
          phase ^= 1;
        }
        const bool ends = p.j == p.n - 1;
        if (ends || T == t1 - 1) {
          // ---- merge the warps
          const int g = lane >> 2, t = lane & 3;
          const float back = w.top_v / (kv8_q<FMT>() * kKaLift);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = nt * 8 + 2 * t + e;
              float l = w.l[nt][e];
              l += __shfl_xor_sync(0xffffffffu, l, 4);
              l += __shfl_xor_sync(0xffffffffu, l, 8);
              l += __shfl_xor_sync(0xffffffffu, l, 16);
              if (g == 0) {
                wm[warp * 8 * NT + r] = w.m[nt][e];
                wl[warp * 8 * NT + r] = l;
              }
#pragma unroll
              for (int j = 0; j < DIM / 32; ++j)
                *reinterpret_cast<float4*>(wo + (warp * 8 * NT + r) * kRowW + 4 * (g + 8 * j)) =
                    make_float4(w.o[nt][j][0][e] * back, w.o[nt][j][0][2 + e] * back, w.o[nt][j][1][e] * back,
                                w.o[nt][j][1][2 + e] * back);
            }
          ka_bar();
          const int64_t seg1 = seg0 + p.n;
          const bool whole = seg0 >= t0 && ends;
          float* slot = a.part + (size_t)(2 * blockIdx.x + (seg0 < t0 ? 0 : 1)) * (8 * NT) * (DIM + 2);
          const int n_q = s.n * group;
          auto store = [&](int r, int d, float4 v) {  // row r of the tile: o of its query row and head
            const int rr = p.tile * 8 * NT + r;
            if (rr >= a.rows * group) return;
            const int i = rr / group, h = p.kvh * group + rr - i * group;
            if (rr >= n_q) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
            *reinterpret_cast<uint2*>(a.o + ((int64_t)(a.b0 + p.b) * a.rows + i) * a.o_stride + h * DIM + d) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
          };
          for (int i = tid; i < 8 * NT * (DIM / 4); i += 32 * kKaWarps) {
            const int r = i / (DIM / 4), d = i % (DIM / 4) * 4;
            float mm = -INFINITY, ls = 0.0f;
#pragma unroll
            for (int k = 0; k < kKaWarps; ++k) mm = fmaxf(mm, wm[k * 8 * NT + r]);
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (mm > -INFINITY) {
#pragma unroll
              for (int k = 0; k < kKaWarps; ++k) {
                const float f = ex2(wm[k * 8 * NT + r] - mm);
                const float4 v = *reinterpret_cast<const float4*>(wo + (k * 8 * NT + r) * kRowW + d);
                ls += wl[k * 8 * NT + r] * f;
                acc.x += v.x * f, acc.y += v.y * f, acc.z += v.z * f, acc.w += v.w * f;
              }
            }
            if (whole) {
              const float inv = ls > 0.0f ? 1.0f / ls : 0.0f;
              store(r, d, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
            } else {
              *reinterpret_cast<float2*>(slot + r * (DIM + 2) + d) = make_float2(acc.x, acc.y);
              *reinterpret_cast<float2*>(slot + r * (DIM + 2) + d + 2) = make_float2(acc.z, acc.w);
              if (d == 0) *reinterpret_cast<float2*>(slot + r * (DIM + 2) + DIM) = make_float2(mm, ls);
            }
          }
          if (!whole) {
            // the unit's CTAs: those whose shares hold its first and its last tile
            const int64_t c0 = ((seg0 + 1) * G - 1) / total, c1 = (seg1 * G - 1) / total;
            __threadfence();
            ka_bar();
            if (tid == 0) last_s = atomicAdd(a.arrived + c0, 1u) == (uint32_t)(c1 - c0);
            ka_bar();
            if (last_s) {
              __threadfence();
              for (int i = tid; i < 8 * NT * (DIM / 4); i += 32 * kKaWarps) {
                const int r = i / (DIM / 4), d = i % (DIM / 4) * 4;
                float mm = -INFINITY, ls = 0.0f;
                float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (int64_t c = c0; c <= c1; ++c) {
                  const float* x = a.part + ((size_t)(2 * c + (c == c0 ? 1 : 0)) * (8 * NT) + r) * (DIM + 2);
                  const float2 ml = __ldcg(reinterpret_cast<const float2*>(x + DIM));
                  const float2 v0 = __ldcg(reinterpret_cast<const float2*>(x + d)), v1 = __ldcg(reinterpret_cast<const float2*>(x + d + 2));
                  if (ml.x == -INFINITY) continue;
                  const float now = fmaxf(mm, ml.x), f = ex2(mm - now), h = ex2(ml.x - now);
                  mm = now;
                  ls = ls * f + ml.y * h;
                  acc.x = acc.x * f + v0.x * h, acc.y = acc.y * f + v0.y * h;
                  acc.z = acc.z * f + v1.x * h, acc.w = acc.w * f + v1.y * h;
                }
                const float inv = ls > 0.0f ? 1.0f / ls : 0.0f;
                store(r, d, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
              }
              if (tid == 0) atomicExch(a.arrived + c0, 0u);
            }
          }
          ka_bar();  // the merge buffers are free again
          fresh = true;
        }
        advance(p);
      }
    }
  }
  __syncthreads();
}

}  // namespace vg
