// Log probabilities from the LM head, without the logits in memory:
//   z[r,v] = sum_h h[r,h] W[v,h],  lse[r] = log sum_v exp(z[r,v]),
//   logprob[r] = z[r, token[r]] - lse[r],
//   entropy[r] = lse[r] - sum_v p[r,v] z[r,v],  p = exp(z - lse),
//   the n largest z[r,.] - lse[r] with their indices, ties to the lower index.
//
// logprob_tiles: tcgen05 GEMM with 128 rows of h as M and a tile of vocabulary
// rows as N; a unit of work is a group of consecutive vocabulary tiles for one
// 128-row block (PAIR: for 256 rows, by two CTAs that share the vocabulary tile:
// cta_group::2). The epilogue thread that owns a row reads its logits from
// tensor memory and keeps, in one pass, the running maximum m, S = sum e^(z-m),
// T = sum e^(z-m) (z-m), and the candidates: the largest logits, at least
// kLpSpare more than the n asked for.
// logprob_finish: one CTA per row joins the units' partials (S and T rescaled to
// the common maximum), takes the best candidates of all units and recomputes
// their logits and the given token's as sums of exact products in fp64, so that
// the order of close alternatives is that of the exact dot products and does not
// depend on the tensor cores' summation; kLpSpare or more candidates beyond n
// keep one from being lost at the border to what the tensor cores' sums are off by.
//
// Up to 128 rows the LM head's stream bounds it: 60 us for 4 rows (331 MB: 50.4 at
// copy speed), of which 8 are the finishing kernel's round trips, 70 us for 128
// rows with 20 alternatives, 63 with up to 8 (captured in graphs; called without end,
// under the power cap, 65 and 77). 256 rows with 20: 88. 4,096 rows: 0.98
// to 1.01 ms, and 1.16 under the power cap, for 1.36 TFLOP (0.82 at cuBLAS's burst
// rate, 0.99 at its rate under the cap), 56 us of it finishing. Two epilogue threads a row, or tensor memory
// read a chunk ahead, changed nothing at 4,096 rows and cost 3 to 11 us at 128.
#pragma once
#include "common.cuh"
#include "gemm_moe.cuh"
#include "lmhead.cuh"

namespace vg {

constexpr int kLpMaxTop = 20;
constexpr int kLpSpare = 4;
constexpr int kLpM = 128;
constexpr int kLpABytes = kLpM * kBK * 2;
constexpr int kLpAux = 1024;
constexpr int kLpPeaks = 24 * 768;       // words of LpArgs::peaks at most: 768 rows with lists of 24, 1,536 with 12
// Its rows (as a constant: worked out, the NC addresses cost 40 registers and 1.3 us).
__host__ __device__ constexpr int lp_peak_rows(bool pair, int nc) { return pair ? kLpPeaks / nc : kLpM; }
constexpr int kLpChunk = 16;             // columns read from tensor memory at a time
constexpr int kLpPend = 8 + kLpChunk;    // columns a row can have waiting for its candidate list

struct LpArgs {
  int R, V, k_chunks, n_mblk, n_vblk, group_tiles, n_groups, a_box_rows, b_box_rows;
  int tile_n, stages;          // vocabulary rows per tile, pipeline stages
  float* stat;                 // [n_groups][4][R]: m, S, T, what rounding took off S
  unsigned long long* cand;    // [n_groups][R][NC]: order-preserving keys, descending; 0 = none
  uint32_t* floor;             // [R] or null: order-preserving image of a logit that NC others reach (0: none known)
  uint32_t* peaks;             // [NC][lp_peak_rows] or null: images of the largest logits of NC parts of the vocabulary; zero between calls
};

// b_rows: vocabulary rows of a tile that one CTA holds
__host__ __device__ constexpr int lp_stage_bytes(int b_rows) { return kLpABytes + b_rows * kBK * 2; }
__host__ __device__ constexpr int lp_smem_bytes(int b_rows, int stages) {
  return 1024 + stages * lp_stage_bytes(b_rows) + kLpAux + kLpPend * kLpM * 8;
}

// Candidates kept for n alternatives: n + kLpSpare or more, of the two sizes that the
// kernels are built for.
__host__ __device__ constexpr int lp_cands(int n_top) { return n_top + kLpSpare <= 12 ? 12 : 24; }
static_assert(lp_cands(kLpMaxTop) >= kLpMaxTop + kLpSpare);

// A row's best logits so far, descending (equal ones by index), in registers.
template <int NC>
struct LpList {
  float z[NC];
  int v[NC];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < NC; ++k) z[k] = -INFINITY, v[k] = -1;
  }
  // Columns come in increasing order, so an equal logit goes behind.
  __device__ __forceinline__ void insert(float x, int i) {
    bool ahead[NC];
#pragma unroll
    for (int k = 0; k < NC; ++k) ahead[k] = x > z[k];
#pragma unroll
    for (int k = NC - 1; k > 0; --k) {
      z[k] = ahead[k] ? (ahead[k - 1] ? z[k - 1] : x) : z[k];
      v[k] = ahead[k] ? (ahead[k - 1] ? v[k - 1] : i) : v[k];
    }
    z[0] = ahead[0] ? x : z[0];
    v[0] = ahead[0] ? i : v[0];
  }
};

// The largest fp32 value below x (x not NaN; zero: below -0).
__device__ __forceinline__ float lp_below(float x) {
  const int b = __float_as_int(x);
  return x == 0.0f ? __int_as_float(0x80000001) : x == -INFINITY ? x : __int_as_float(b > 0 ? b - 1 : b + 1);
}

// An fp32 logit's image in the order of argmax_key's high word, and back.
__device__ __forceinline__ float lp_unkey(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? u & 0x7FFFFFFFu : ~u);
}

// PAIR: the two CTAs of a cluster take row blocks 2 i and 2 i + 1; each loads its
// own rows of h and its half of the vocabulary tile into its own shared memory and
// epilogues its own rows. All loads of a stage complete on the even CTA's barrier,
// which expects both CTAs' bytes; the even CTA issues the MMAs. (The odd CTA
// watching its own stages and passing them on took 1,920 us for 4,096 rows, against
// 1,080 us: a round trip more than six stages cover.) Shared memory then
// carries 64 + 64 instead of 96 + 96 bytes a cycle at full tensor rate, operands read
// and tiles written, against the 128 it has.
template <int NC, bool PAIR>
__global__ void __launch_bounds__(192, 1)
    logprob_tiles(const __grid_constant__ CUtensorMap mapH, const __grid_constant__ CUtensorMap mapLM, const LpArgs a) {
  constexpr int kMaxStages = 8;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int b_rows = PAIR ? a.tile_n / 2 : a.tile_n;
  const int stages = a.stages, stage_bytes = lp_stage_bytes(b_rows);
  uint8_t* aux = tiles + stages * stage_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(aux);
  uint64_t* empty = full + kMaxStages;
  uint64_t* tfull = empty + kMaxStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* mma_done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float2* pend = reinterpret_cast<float2*>(aux + kLpAux);  // [kLpPend][kLpM]: (logit, column) waiting

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR ? (int)cluster_rank() : 0;
  const int n_rb = PAIR ? cdiv(a.n_mblk, 2) : a.n_mblk;
  const int total = a.n_groups * n_rb;  // unit = (vocabulary group, row block or pair of them), rows fastest
  const int unit0 = PAIR ? blockIdx.x / 2 : blockIdx.x, unit_step = PAIR ? gridDim.x / 2 : gridDim.x;
  const int b_row0 = rank * b_rows;  // this CTA's share of a vocabulary tile
  const uint32_t a_bytes = a.a_box_rows * kBK * 2, b_bytes = a.b_box_rows * kBK * 2;
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], PAIR ? 8 : 4);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&mapH);
    prefetch_tmap(&mapLM);
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(tmem_slot, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();  // the other CTA's barriers are there
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint64_t limit = g_wait_timeout_ns;

  // vocabulary tiles of the first stages before the dependency wait: the LM head is immutable
  int npre = 0;
  const uint64_t pol_w = a.n_mblk == 1 ? policy_evict_first() : policy_evict_normal();
  if (warp == 0 && lane == 0 && unit0 < total) {
    const int g = unit0 / n_rb;
    const int vb1 = min(a.n_vblk, (g + 1) * a.group_tiles);
    for (int vb = g * a.group_tiles; vb < vb1 && npre < stages; ++vb)
      for (int kc = 0; kc < a.k_chunks && npre < stages; ++kc, ++npre) {
        uint8_t* dst = tiles + npre * stage_bytes + kLpABytes;
        if (PAIR) {  // (expected with the stage's arrival: bytes may land before)
          tma_load_2d_pair(dst, &mapLM, &full[npre], kc * kBK, vb * a.tile_n + b_row0, pol_w);
        } else {
          mbar_expect_tx(&full[npre], b_bytes);
          tma_load_2d_hint(dst, &mapLM, &full[npre], kc * kBK, vb * a.tile_n, pol_w);
        }
      }
  }
  griddep_wait();

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol_h = policy_evict_last();
      int stage = 0, it = 0;
      uint32_t phase = 0, issued = 0, last_par = 0;
      for (int u = unit0; u < total && !*abort_flag; u += unit_step) {
        const int g = u / n_rb, mb = PAIR ? 2 * (u - g * n_rb) + rank : u - g * n_rb;
        const int vb1 = min(a.n_vblk, (g + 1) * a.group_tiles);
        for (int vb = g * a.group_tiles; vb < vb1 && !*abort_flag; ++vb) {
          for (int kc = 0; kc < a.k_chunks; ++kc, ++it) {
            if (!mbar_wait(&empty[stage], phase ^ 1, limit)) {
              record_error(kErrTimeout, 351);
              *abort_flag = 1;
              break;
            }
            uint8_t* st = tiles + stage * stage_bytes;
            const bool pre = it < npre;  // its vocabulary tile is already in flight
            if (PAIR) {
              if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * (a_bytes + b_bytes));
              tma_load_2d_pair(st, &mapH, &full[stage], kc * kBK, mb * kLpM, pol_h);
              if (!pre) tma_load_2d_pair(st + kLpABytes, &mapLM, &full[stage], kc * kBK, vb * a.tile_n + b_row0, pol_w);
            } else {
              mbar_arrive_expect_tx(&full[stage], pre ? a_bytes : a_bytes + b_bytes);
              tma_load_2d_hint(st, &mapH, &full[stage], kc * kBK, mb * kLpM, pol_h);
              if (!pre) tma_load_2d_hint(st + kLpABytes, &mapLM, &full[stage], kc * kBK, vb * a.tile_n, pol_w);
            }
            issued |= 1u << stage;
            last_par = (last_par & ~(1u << stage)) | (phase << stage);
            if (++stage == stages) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
      }
      // stages armed before the wait but never reached (an abort): arrive, so
      // their copies complete the phase and can be drained below
      for (; it < npre; ++it) {
        if (PAIR && rank == 0) mbar_arrive_expect_tx(&full[it], 2 * b_bytes);
        if (!PAIR) mbar_arrive(&full[it]);
        issued |= 1u << it;
        last_par &= ~(1u << it);
      }
      // (a pair's copies are all counted in the even CTA)
      for (int s = 0; s < stages; ++s)
        if (rank == 0 && (issued & (1u << s))) mbar_wait(&full[s], (last_par >> s) & 1, limit);
    }
  } else if (warp == 1 && PAIR && rank == 1) {
    // The even CTA issues the pair's MMAs; its commits arrive on this CTA's barriers
    // too, the last of them on mma_done: not to leave before that has come.
    if (lane == 0) mbar_wait(mma_done, 0, limit);
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16_f32(PAIR ? 2 * kLpM : kLpM, a.tile_n);
      int stage = 0;
      uint32_t phase = 0;
      int lt = 0;  // local tile counter: selects the accumulator buffer
      bool ok = true;
      for (int u = unit0; u < total && ok; u += unit_step) {
        const int g = u / n_rb;
        const int vb1 = min(a.n_vblk, (g + 1) * a.group_tiles);
        for (int vb = g * a.group_tiles; vb < vb1 && ok; ++vb, ++lt) {
          const int ab = lt & 1;
          const uint32_t ap = (lt >> 1) & 1;
          if (*abort_flag ||
              !(PAIR ? mbar_wait_cluster(&tempty[ab], ap ^ 1, limit) : mbar_wait(&tempty[ab], ap ^ 1, limit))) {
            record_error(kErrTimeout, 352);
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + ab * 256;
          for (int kc = 0; kc < a.k_chunks; ++kc) {
            if (!mbar_wait(&full[stage], phase, limit)) {
              record_error(kErrTimeout, 353);
              *abort_flag = 1;
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t st = smem_u32(tiles + stage * stage_bytes);
            const uint64_t da = sw128_kmajor_desc(st), db = sw128_kmajor_desc(st + kLpABytes);
#pragma unroll
            for (int k16 = 0; k16 < kBK / 16; ++k16) {
              if (PAIR)
                umma_bf16_pair(d, da + 2 * k16, db + 2 * k16, idesc, (kc | k16) != 0);
              else
                umma_bf16(d, da + 2 * k16, db + 2 * k16, idesc, (kc | k16) != 0);
            }
            if (PAIR)
              umma_commit_pair(&empty[stage]);
            else
              umma_commit(&empty[stage]);
            if (++stage == stages) {
              stage = 0;
              phase ^= 1;
            }
          }
          if (ok) {
            if (PAIR)
              umma_commit_pair(&tfull[ab]);
            else
              umma_commit(&tfull[ab]);
          }
        }
      }
      if (PAIR)
        umma_commit_pair(mma_done);
      else
        umma_commit(mma_done);
      mbar_wait(mma_done, 0, limit);
    }
  } else {
    // Candidates: a logit above the list's last one is first parked in shared
    // memory, and the parked ones of all 32 rows of the warp enter their lists
    // together, so the insertion runs about as often as a row has insertions and
    // not whenever any of 32 rows has one.
    const int q = warp & 3;
    const int row = q * 32 + lane;
    int lt = 0;
    bool ok = true;
    LpList<NC> list;
    for (int u = unit0; u < total && ok; u += unit_step) {
      const int g = u / n_rb, mb = PAIR ? 2 * (u - g * n_rb) + rank : u - g * n_rb;
      const int vb1 = min(a.n_vblk, (g + 1) * a.group_tiles);
      const int r = mb * kLpM + row;
      const bool busy = mb * kLpM + q * 32 < a.R;  // this warp has rows
      float m = -INFINITY, S = 0.0f, T = 0.0f, low = 0.0f;
      float least = -INFINITY;  // only larger logits enter
      int parked = 0;
      list.clear();
      if (r >= a.R) {
        least = INFINITY;  // nothing enters
      } else if (a.floor) {
        const uint32_t f = *reinterpret_cast<volatile uint32_t*>(a.floor + r);
        if (f > 0u) least = lp_below(lp_unkey(f));
      }
      auto settle = [&]() {  // the parked columns into the list
        const int most = __reduce_max_sync(0xffffffffu, parked);
        for (int i = 0; i < most; ++i) {
          const float2 p = pend[i * kLpM + row];
          list.insert(i < parked ? p.x : -INFINITY, __float_as_int(p.y));
        }
        parked = 0;
        least = fmaxf(least, list.z[NC - 1]);
      };
      for (int vb = g * a.group_tiles; vb < vb1; ++vb, ++lt) {
        const int ab = lt & 1;
        const uint32_t ap = (lt >> 1) & 1;
        // one decision for the warp: the votes below need all its lanes
        ok = __all_sync(0xffffffffu, !*abort_flag && mbar_wait(&tfull[ab], ap, limit));
        if (!ok) {
          if (!*abort_flag) record_error(kErrTimeout, 354);
          *abort_flag = 1;
          break;
        }
        tc_fence_after();
        const uint32_t t0 = tmem_base + ((uint32_t)(q * 32) << 16) + ab * 256;
        const int v0 = vb * a.tile_n, cols = busy ? min(a.tile_n, a.V - v0) : 0;
        auto own_bound = [&]() {
          // A bound to start with: NC groups of kLpBound columns have a maximum of
          // at least the NC-th largest of the groups' maxima, so NC logits reach it.
          // Finding it moves values alone (two instructions a place, and groups
          // follow each other through the list), where a column that enters costs
          // five a place: of a first tile of 176 columns 31 enter the list of 24
          // then, and 72 without.
          constexpr int kLpBound = NC == 12 ? 8 : 4;
#pragma unroll 1
          for (int c0 = 0; c0 + kLpChunk <= cols; c0 += kLpChunk) {
            uint32_t zb[kLpChunk];
            tmem_ld16(t0 + c0, zb);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < kLpChunk; j += kLpBound) {
              float x = __uint_as_float(zb[j]);
#pragma unroll
              for (int i = 1; i < kLpBound; ++i) x = fmaxf(x, __uint_as_float(zb[j + i]));
#pragma unroll
              for (int k = 0; k < NC; ++k) {
                const float z = list.z[k];
                list.z[k] = fmaxf(z, x);
                x = fminf(z, x);
              }
            }
          }
          least = fmaxf(least, lp_below(list.z[NC - 1]));
          list.clear();
        };
        // the tile's logits once: into the sums, into the lists
        auto pass = [&](bool sums, bool lists) {
#pragma unroll 1
          for (int c0 = 0; c0 < cols; c0 += kLpChunk) {
            uint32_t zb[kLpChunk];
            tmem_ld16(t0 + c0, zb);
            tmem_ld_wait();
            float z[kLpChunk], top = -INFINITY;
#pragma unroll
            for (int j = 0; j < kLpChunk; ++j) z[j] = __uint_as_float(zb[j]);
            if (c0 + kLpChunk > cols) {  // behind the vocabulary
#pragma unroll
              for (int j = 0; j < kLpChunk; ++j)
                if (c0 + j >= cols) z[j] = -INFINITY;
            }
#pragma unroll
            for (int j = 0; j < kLpChunk; ++j) top = fmaxf(top, z[j]);
            if (sums) {
              const float now = fmaxf(m, top), base = now > -INFINITY ? now : 0.0f;
              if (now > m && m > -INFINITY) {  // to the new maximum
                const float d = fmaxf(m - now, -1000.0f), f = ex2(d * 1.4426950408889634f);
                T = f * (T + S * d);
                S *= f, low *= f;
              }
              m = now;
              float e[kLpChunk], t1 = 0.0f;
#pragma unroll
              for (int j = 0; j < kLpChunk; ++j) {
                const float d = z[j] - base;
                e[j] = ex2(d * 1.4426950408889634f);
                t1 = fmaf(e[j], fmaxf(d, -1000.0f), t1);  // a weight of 0 adds 0, also where z is -inf
              }
              // Where one token has nearly all the mass its log probability is what
              // the others add to its 1: summed in pairs, so that the 1 is rounded
              // with four times a chunk, and with the rounding of S kept.
#pragma unroll
              for (int n = kLpChunk / 2; n > 0; n /= 2)
#pragma unroll
                for (int j = 0; j < n; ++j) e[j] += e[j + n];
              const float sum = S + e[0], back = sum - S;
              low += (S - (sum - back)) + (e[0] - back);
              S = sum;
              T += t1;
            }
            if (lists && __any_sync(0xffffffffu, top > least)) {
#pragma unroll
              for (int j = 0; j < kLpChunk; ++j)
                if (z[j] > least) {
                  pend[parked * kLpM + row] = make_float2(z[j], __int_as_float(v0 + c0 + j));
                  ++parked;
                }
              if (__any_sync(0xffffffffu, parked > kLpPend - kLpChunk)) settle();
            }
          }
        };
        if (vb > g * a.group_tiles) {
          pass(true, true);
        } else if (a.peaks && __any_sync(0xffffffffu, least == -INFINITY && r < a.R)) {
          // The first tile fixes what may enter the lists. NC parts of the
          // vocabulary, each the groups that leave one rest by NC, have a largest
          // logit each, so NC logits reach the smallest of those. Every CTA has its
          // first tile at about the same time: it gives its rows' maxima away, takes
          // the tile into the sums, and by then finds the others'. Of 129,280 tokens
          // some 400 reach the bound then, one or two of a CTA's 880; with what a
          // CTA's own tile shows, 70 of them entered its list of 24 (20 alternatives,
          // 128 rows: 74 us where this took 68; 256 rows 101 and 89).
          float top = -INFINITY;
#pragma unroll 1
          for (int c0 = 0; c0 < cols; c0 += kLpChunk) {
            uint32_t zb[kLpChunk];
            tmem_ld16(t0 + c0, zb);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < kLpChunk; ++j)
              if (c0 + j < cols) top = fmaxf(top, __uint_as_float(zb[j]));
          }
          if (r < a.R && top > -INFINITY)
            atomicMax(a.peaks + g % NC * lp_peak_rows(PAIR, NC) + r, (uint32_t)(argmax_key(top, 0u) >> 32));
          pass(true, false);
          if (r < a.R) {
            uint32_t f = 0xFFFFFFFFu;
#pragma unroll
            for (int k = 0; k < NC; ++k) f = min(f, __ldcg(a.peaks + k * lp_peak_rows(PAIR, NC) + r));
            if (f > 0u) least = fmaxf(least, lp_below(lp_unkey(f)));
          }
          if (__any_sync(0xffffffffu, least == -INFINITY && r < a.R)) own_bound();
          pass(false, true);
        } else {
          if (__any_sync(0xffffffffu, least == -INFINITY && r < a.R)) own_bound();
          pass(true, true);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR)
            mbar_arrive_at(&tempty[ab], 0);
          else
            mbar_arrive(&tempty[ab]);
        }
      }
      if (busy) settle();
      if (ok && r < a.R) {
        float* st = a.stat + (size_t)g * 4 * a.R + r;
        st[0] = m;
        st[a.R] = S;
        st[2 * (size_t)a.R] = T;
        st[3 * (size_t)a.R] = low;
        unsigned long long* dst = a.cand + ((size_t)g * a.R + r) * NC;
#pragma unroll
        for (int k = 0; k < NC; ++k) dst[k] = list.v[k] >= 0 ? argmax_key(list.z[k], (uint32_t)list.v[k]) : 0ull;
        if (a.floor && list.v[NC - 1] >= 0)
          atomicMax(a.floor + r, (uint32_t)(argmax_key(list.z[NC - 1], 0u) >> 32));
      }
    }
  }
  __syncthreads();
  if (PAIR) cluster_sync();  // neither CTA's memory is read or signalled any more
  if (warp == 1) {
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem_base, 512);
    else
      tmem_dealloc(tmem_base, 512);
  }
}

struct LpFinishArgs {
  int R, H, V, n_groups, n_top;
  const float* stat;
  const unsigned long long* cand;
  const __nv_bfloat16* h;
  const __nv_bfloat16* lm;
  const int32_t* tokens;  // [R] or null
  float* logprob;         // [R] or null
  float* entropy;         // [R] or null
  int32_t* top_ids;       // [R, n_top]
  float* top_logprobs;    // [R, n_top]
  uint32_t* peaks;        // as in LpArgs
  int peak_rows;
};

constexpr int kLpMaxGroups = 512;
constexpr int kLpFix = 12;  // candidates whose exact logits enter the sums: the same however many alternatives are asked for
static_assert(kLpFix <= lp_cands(0));

// One CTA per row. The best NC candidates of all units: the NC-th largest of the
// units' first ones bounds them from below, so at most NC lists have any, and a
// rank count orders what is left. Their tensor-core logits are replaced by the
// exact ones in the sums too: the tensor cores cut every partial sum towards
// zero (measured: some 1.5e-8 of a logit for each 16 products, 1.2e-6 at H = 1,280), which
// shifts all logits alike but for their size, so where a few tokens hold the
// mass, correcting those removes most of the error. The kernel is a chain of round
// trips (statistics and heads; the lists; the candidates' rows), each with all its
// loads under way at once.
// NT threads: 512 where every row has an SM to itself and the chain's length is what
// counts, 128 where there are many rows, so that more of them are under way (4,096
// rows: 121 us with 512, 56 with 128).
template <int NC, int NT>
__global__ void __launch_bounds__(NT) logprob_finish(const LpFinishArgs a) {
  constexpr int NW = NT / 32, kOwn = kLpMaxGroups / NT;  // units a thread may own: tid, tid + NT, ..
  __shared__ float red_m[NW];
  __shared__ double red_s[NW], red_t[NW], z_s[NC + 1], s_fix[kLpFix], t_fix[kLpFix], s_raw[kLpFix], t_raw[kLpFix], short_of[kLpFix], square[kLpFix];
  __shared__ unsigned long long head[kLpMaxGroups], pool[NC * NC], best[NC];
  __shared__ unsigned long long floor_s;
  __shared__ int id_s[NC + 1], rank_s[NC], head_rank[kLpMaxGroups], n_pool;
  griddep_launch_dependents();
  griddep_wait();
  const int r = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (a.peaks && tid < NC) a.peaks[tid * a.peak_rows + r] = 0u;
  const int tok = a.tokens ? a.tokens[r] : -1;
  if (tid == 0) n_pool = 0, floor_s = 1ull;  // 0 keys are no candidates
  if (tid < NC) best[tid] = 0ull, rank_s[tid] = 0;
  for (int g = tid; g < a.n_groups; g += NT) head_rank[g] = 0;
  // ---- the units' sums, rescaled to the common maximum
  float mg[kOwn], Sg[kOwn], Tg[kOwn], low[kOwn], m = -INFINITY;
  unsigned long long first[kOwn];
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int g = tid + i * NT;
    mg[i] = -INFINITY, Sg[i] = Tg[i] = low[i] = 0.0f, first[i] = 0ull;
    if (g < a.n_groups) {
      const float* st = a.stat + (size_t)g * 4 * a.R + r;
      mg[i] = st[0], Sg[i] = st[a.R], Tg[i] = st[2 * (size_t)a.R], low[i] = st[3 * (size_t)a.R];
      first[i] = a.cand[((size_t)g * a.R + r) * NC];
      head[g] = first[i];
    }
    m = fmaxf(m, mg[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red_m[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NW; ++w) m = fmaxf(m, red_m[w]);
  // ranks of the units' first candidates, every thread with a part of the comparisons
  {
    const int parts = max(1, NT / a.n_groups), per = cdiv(a.n_groups, parts);
    for (int i = tid; i < parts * a.n_groups; i += NT) {
      const int part = i / a.n_groups, g = i - part * a.n_groups, k1 = min(a.n_groups, (part + 1) * per);
      const unsigned long long key = head[g];
      int above = 0;
#pragma unroll 8
      for (int k = part * per; k < k1; ++k) above += head[k] > key;
      if (above) atomicAdd(&head_rank[g], above);
    }
  }
  double S = 0.0, T = 0.0;
  if (warp * 32 < a.n_groups) {  // whole warps
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      if (i * NT >= a.n_groups) break;
      // a unit's largest term is 1 before rescaling, so the factor needs fp32 accuracy only
      const float d = mg[i] > -INFINITY ? mg[i] - m : 0.0f, f = mg[i] > -INFINITY ? ex2(d * 1.4426950408889634f) : 1.0f;
      S += (double)f * ((double)Sg[i] + (double)low[i]);
      T += (double)f * ((double)Tg[i] + (double)Sg[i] * fmaxf(d, -1000.0f));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      S += __shfl_xor_sync(0xffffffffu, S, o);
      T += __shfl_xor_sync(0xffffffffu, T, o);
    }
    if (lane == 0) red_s[warp] = S, red_t[warp] = T;
  }
  __syncthreads();
  // (the lists of the NC units with the largest first candidates; their smallest is the bound)
#pragma unroll
  for (int i = 0; i < kOwn; ++i)
    if (first[i] && head_rank[tid + i * NT] == NC - 1) floor_s = first[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kOwn; ++i)
    if (first[i] >= floor_s) {
      const uint4* l = reinterpret_cast<const uint4*>(a.cand + ((size_t)(tid + i * NT) * a.R + r) * NC);
      uint4 x[NC / 2];
#pragma unroll
      for (int k = 0; k < NC / 2; ++k) x[k] = l[k];
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        const unsigned long long key = k & 1 ? (unsigned long long)x[k / 2].w << 32 | x[k / 2].z
                                             : (unsigned long long)x[k / 2].y << 32 | x[k / 2].x;
        if (key >= floor_s) pool[atomicAdd(&n_pool, 1)] = key;
      }
    }
  __syncthreads();
  for (int i = tid; i < n_pool; i += NT) {
    const unsigned long long key = pool[i];
    int rank = 0;
#pragma unroll 8
    for (int k = 0; k < n_pool; ++k) rank += pool[k] > key;
    if (rank < NC) best[rank] = key;
  }
  __syncthreads();
  // ---- their logits from exact products (a product of two bf16 is exact in fp32),
  // summed in fp64; a warp takes two candidates at a time (the conversions to fp64,
  // 16 a clock, are the cost: none for a second candidate that is not there)
  for (int k0 = warp; k0 <= NC; k0 += 2 * NW) {
    int v[2];
    double z[2] = {0.0, 0.0};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int k = k0 + c * NW;
      const unsigned long long key = k < NC ? best[k] : 0ull;
      v[c] = key ? (int)(0xFFFFFFFFu - (uint32_t)(key & 0xFFFFFFFFull)) : -1;
      if (k == NC && tok >= 0 && tok < a.V) v[c] = tok;
    }
    if (v[0] >= 0 || v[1] >= 0) {
      const uint4* x = reinterpret_cast<const uint4*>(a.h + (size_t)r * a.H);
      const uint4* w0 = reinterpret_cast<const uint4*>(a.lm + (size_t)(v[0] >= 0 ? v[0] : v[1]) * a.H);
      const uint4* w1 = reinterpret_cast<const uint4*>(a.lm + (size_t)(v[1] >= 0 ? v[1] : v[0]) * a.H);
      double y[2][2] = {{0.0, 0.0}, {0.0, 0.0}};
      auto add = [&](int c, const uint4& xv, const uint4& wv) {
        const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w}, ws[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[c][0] += (double)(bf16_lo(xs[e]) * bf16_lo(ws[e]));
          y[c][1] += (double)(bf16_hi(xs[e]) * bf16_hi(ws[e]));
        }
      };
      if (v[1] >= 0) {
#pragma unroll 5
        for (int i = lane; i < a.H / 8; i += 32) {
          const uint4 xv = x[i], wv[2] = {w0[i], w1[i]};
          add(0, xv, wv[0]);
          add(1, xv, wv[1]);
        }
      } else {
#pragma unroll 5
        for (int i = lane; i < a.H / 8; i += 32) add(0, x[i], w0[i]);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) z[c] = y[c][0] + y[c][1];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        z[0] += __shfl_xor_sync(0xffffffffu, z[0], o);
        z[1] += __shfl_xor_sync(0xffffffffu, z[1], o);
      }
    }
    if (lane < 2 && k0 + lane * NW <= NC) {
      const int id = lane ? v[1] : v[0];
      z_s[k0 + lane * NW] = id >= 0 ? (lane ? z[1] : z[0]) : -INFINITY;
      id_s[k0 + lane * NW] = id;
    }
  }
  if (tid == 0 && tok >= a.V) record_error(kErrBounds, 355);
  __syncthreads();
  if (tid < kLpFix) {  // what the exact logits change in S and T
    double ds = 0.0, dt = 0.0, s0 = 0.0, t0 = 0.0, off = 0.0, sq = 0.0;
    if (id_s[tid] >= 0 && m < INFINITY) {
      const double z0 = (double)lp_unkey((uint32_t)(best[tid] >> 32)), d0 = z0 - (double)m, d1 = z_s[tid] - (double)m;
      // e^d1 - e^d0 = e^d0 (e^(d1 - d0) - 1): d1 - d0 is a rounding's worth, and needs no more than fp32 accuracy
      const double e0 = (double)expf((float)d0), g = d1 - d0, gain = (double)expm1f((float)g);
      ds = e0 * gain;
      dt = e0 * (g + gain * d1);
      s0 = e0, t0 = e0 * d0, off = g * z0, sq = z0 * z0;
    }
    s_fix[tid] = ds, t_fix[tid] = dt, s_raw[tid] = s0, t_raw[tid] = t0, short_of[tid] = off, square[tid] = sq;
  }
  // ---- order: rank of each candidate by (logit, lower index first); those that are
  // missing (fewer logits above -inf than asked for) come last, in list order
  for (int i = tid; i < NC * NC; i += NT) {
    const int c = i / NC, k = i - c * NC, vc = id_s[c], vk = id_s[k];
    const bool ahead = vk < 0 ? (vc < 0 && k < c) : (vc < 0 || z_s[k] > z_s[c] || (z_s[k] == z_s[c] && vk < vc));
    if (ahead && k != c) atomicAdd(&rank_s[c], 1);
  }
  __syncthreads();
  if (warp != 0) return;
  // The other tokens' logits fell short like these, by a share of themselves (the
  // least squares' over the candidates; no more than half a place for each 16
  // products): their mean logit's worth is put back on their S and T. (The entropy
  // misses that share of the logits' variance with it, 1.6e-7 of itself at H = 1,280;
  // for that the epilogue would have to sum e^(z-m) (z-m)^2 too.) What is left of
  // the sums without the candidates is a difference: where these hold all the mass it
  // is rounding alone, a residue of 1e-16 beside one of 1e-8 in T, and their quotient
  // any number. So both are kept within what the other tokens can be: V - kLpFix of
  // them, none above the last candidate, and none below where ex2 gives 0. (Two tokens
  // with all the mass, H = 8,192: the entropy was off by up to 1e-4 without.)
  double sum[6] = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0};  // S, T, then of the candidates: S, T, shortfall times logit, logit squared
  if (lane < NW && lane * 32 < a.n_groups) sum[0] = red_s[lane], sum[1] = red_t[lane];
  if (lane < kLpFix) sum[2] = s_raw[lane], sum[3] = t_raw[lane], sum[4] = short_of[lane], sum[5] = square[lane];
  double ds = lane < kLpFix ? s_fix[lane] : 0.0, dt = lane < kLpFix ? t_fix[lane] : 0.0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    ds += __shfl_xor_sync(0xffffffffu, ds, o);
    dt += __shfl_xor_sync(0xffffffffu, dt, o);
#pragma unroll
    for (int k = 0; k < 6; ++k) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], o);
  }
  S = sum[0] + ds, T = sum[1] + dt;
  const unsigned long long last = best[kLpFix - 1];  // (0: there are no others)
  const double most = last ? (double)lp_unkey((uint32_t)(last >> 32)) - (double)m : -INFINITY;
  const double rest = fmin(sum[0] - sum[2], 1.0001 * (double)(a.V - kLpFix) * (double)expf((float)most));
  if (sum[5] > 0.0 && rest > 0.0) {
    const double share = fmin(fmax(sum[4] / sum[5], 0.0), (double)(a.H / 16) * 5.9604645e-8);
    const double mean = fmin(fmax((sum[1] - sum[3]) / rest, -88.0), most);
    const double move = share * ((double)m + mean) * rest;
    S += move;
    T += move * (1.0 + mean);
  }
  const double log_s = log(S), lse = (double)m + log_s;
  // A token with all the mass may come out a rounding of the sums (1e-10) on the
  // wrong side of 0: what a program takes a logarithm or a root of. NaN stays.
  auto not_above_0 = [](double x) { return x > 0.0 ? 0.0f : (float)x; };
  if (lane == 0) {
    if (a.logprob) a.logprob[r] = not_above_0(z_s[NC] - lse);
    if (a.entropy) a.entropy[r] = fabsf(not_above_0(T / S - log_s));
  }
  if (lane < NC && rank_s[lane] < a.n_top) {
    a.top_ids[(size_t)r * a.n_top + rank_s[lane]] = id_s[lane];
    a.top_logprobs[(size_t)r * a.n_top + rank_s[lane]] = not_above_0(z_s[lane] - lse);
  }
}

}  // namespace vg
