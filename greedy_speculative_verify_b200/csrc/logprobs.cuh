// Log probabilities from the LM head, without the logits in memory:
//   z[r,v] = sum_h h[r,h] W[v,h],  lse[r] = log sum_v exp(z[r,v]),
//   logprob[r] = z[r, token[r]] - lse[r],
//   entropy[r] = lse[r] - sum_v p[r,v] z[r,v],  p = exp(z - lse),
//   the n largest z[r,.] - lse[r] with their indices, ties to the lower index.
//
// logprob_tiles: tcgen05 GEMM with 128 rows of h as M and a tile of vocabulary
// rows as N; a unit of work is a group of consecutive vocabulary tiles for one
// 128-row block. The epilogue thread that owns a row reads its logits from
// tensor memory and keeps, in one pass, the running maximum m, S = sum e^(z-m),
// T = sum e^(z-m) (z-m), and the candidates: the n + kLpSpare largest logits.
// logprob_finish: one CTA per row joins the units' partials (S and T rescaled to
// the common maximum), takes the n + kLpSpare best candidates of all units and
// recomputes their logits and the given token's as sums of exact products in
// fp64, so that the order of close alternatives is that of the exact dot
// products and does not depend on the tensor cores' summation; kLpSpare
// candidates beyond n keep one from being lost to fp32 rounding at the border.
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

struct LpArgs {
  int R, V, k_chunks, n_mblk, n_vblk, group_tiles, n_groups, a_box_rows, b_box_rows;
  int tile_n, stages, n_cand;  // vocabulary rows per tile, pipeline stages, candidates kept per unit (0: none)
  float* stat;                 // [n_groups][3][R]: m, S, T
  unsigned long long* cand;    // [n_groups][R][n_cand]: order-preserving keys, descending; 0 = none
};

__host__ __device__ constexpr int lp_stage_bytes(int tile_n) { return kLpABytes + tile_n * kBK * 2; }
__host__ __device__ constexpr int lp_smem_bytes(int tile_n, int stages, int n_cand) {
  return 1024 + stages * lp_stage_bytes(tile_n) + kLpAux + n_cand * kLpM * 8;
}

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__global__ void __launch_bounds__(192, 1)
    logprob_tiles(const __grid_constant__ CUtensorMap mapH, const __grid_constant__ CUtensorMap mapLM, const LpArgs a) {
  constexpr int kMaxStages = 8;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stages = a.stages, stage_bytes = lp_stage_bytes(a.tile_n);
  uint8_t* aux = tiles + stages * stage_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(aux);
  uint64_t* empty = full + kMaxStages;
  uint64_t* tfull = empty + kMaxStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* mma_done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  unsigned long long* list = reinterpret_cast<unsigned long long*>(aux + kLpAux);  // [n_cand][kLpM]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int total = a.n_groups * a.n_mblk;  // unit = (vocabulary group, row block), row block fastest
  const uint32_t a_bytes = a.a_box_rows * kBK * 2, b_bytes = a.b_box_rows * kBK * 2;
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 4);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&mapH);
    prefetch_tmap(&mapLM);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint64_t limit = g_wait_timeout_ns;

  // vocabulary tiles of the first stages before the dependency wait: the LM head is immutable
  int npre = 0;
  const uint64_t pol_w = a.n_mblk == 1 ? policy_evict_first() : policy_evict_normal();
  if (warp == 0 && lane == 0 && (int)blockIdx.x < total) {
    const int g = blockIdx.x / a.n_mblk;
    const int vb1 = min(a.n_vblk, (g + 1) * a.group_tiles);
    for (int vb = g * a.group_tiles; vb < vb1 && npre < stages; ++vb)
      for (int kc = 0; kc < a.k_chunks && npre < stages; ++kc, ++npre) {
        mbar_expect_tx(&full[npre], b_bytes);
        tma_load_2d_hint(tiles + npre * stage_bytes + kLpABytes, &mapLM, &full[npre], kc * kBK, vb * a.tile_n, pol_w);
      }
  }
  griddep_wait();

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol_h = policy_evict_last();
      int stage = 0, it = 0;
      uint32_t phase = 0, issued = 0, last_par = 0;
      for (int u = blockIdx.x; u < total && !*abort_flag; u += gridDim.x) {
        const int g = u / a.n_mblk, mb = u - g * a.n_mblk;
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
            mbar_arrive_expect_tx(&full[stage], pre ? a_bytes : a_bytes + b_bytes);
            tma_load_2d_hint(st, &mapH, &full[stage], kc * kBK, mb * kLpM, pol_h);
            if (!pre) tma_load_2d_hint(st + kLpABytes, &mapLM, &full[stage], kc * kBK, vb * a.tile_n, pol_w);
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
        mbar_arrive(&full[it]);
        issued |= 1u << it;
        last_par &= ~(1u << it);
      }
      for (int s = 0; s < stages; ++s)
        if (issued & (1u << s)) mbar_wait(&full[s], (last_par >> s) & 1, limit);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16_f32(kLpM, a.tile_n);
      int stage = 0;
      uint32_t phase = 0;
      int lt = 0;  // local tile counter: selects the accumulator buffer
      bool ok = true;
      for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
        const int g = u / a.n_mblk;
        const int vb1 = min(a.n_vblk, (g + 1) * a.group_tiles);
        for (int vb = g * a.group_tiles; vb < vb1 && ok; ++vb, ++lt) {
          const int ab = lt & 1;
          const uint32_t ap = (lt >> 1) & 1;
          if (*abort_flag || !mbar_wait(&tempty[ab], ap ^ 1, limit)) {
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
            for (int k16 = 0; k16 < kBK / 16; ++k16)
              umma_bf16(d, da + 2 * k16, db + 2 * k16, idesc, (kc | k16) != 0);
            umma_commit(&empty[stage]);
            if (++stage == stages) {
              stage = 0;
              phase ^= 1;
            }
          }
          if (ok) umma_commit(&tfull[ab]);
        }
      }
      umma_commit(mma_done);
      mbar_wait(mma_done, 0, limit);
    }
  } else {
    const int q = warp & 3;
    const int row = q * 32 + lane;
    const int nc = a.n_cand;
    int lt = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
      const int g = u / a.n_mblk, mb = u - g * a.n_mblk;
      const int vb1 = min(a.n_vblk, (g + 1) * a.group_tiles);
      const int r = mb * kLpM + row;
      float m = -INFINITY, S = 0.0f, T = 0.0f;
      float worst = -INFINITY;  // the last candidate's logit: only larger ones enter
      for (int k = 0; k < nc; ++k) list[k * kLpM + row] = 0ull;
      for (int vb = g * a.group_tiles; vb < vb1; ++vb, ++lt) {
        if (*abort_flag) {
          ok = false;
          break;
        }
        const int ab = lt & 1;
        const uint32_t ap = (lt >> 1) & 1;
        if (!mbar_wait(&tfull[ab], ap, limit)) {
          record_error(kErrTimeout, 354);
          *abort_flag = 1;
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t t0 = tmem_base + ((uint32_t)(q * 32) << 16) + ab * 256;
        const int v0 = vb * a.tile_n;
#pragma unroll 1
        for (int c0 = 0; c0 < a.tile_n; c0 += 16) {
          if (v0 + c0 >= a.V) break;
          uint32_t zb[16];
          tmem_ld16(t0 + c0, zb);
          tmem_ld_wait();
          float z[16], top = -INFINITY;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            z[j] = v0 + c0 + j < a.V ? __uint_as_float(zb[j]) : -INFINITY;
            top = fmaxf(top, z[j]);
          }
          const float now = fmaxf(m, top), base = now > -INFINITY ? now : 0.0f;
          if (now > m && m > -INFINITY) {  // to the new maximum
            const float d = fmaxf(m - now, -1000.0f), f = ex2_approx(d * 1.4426950408889634f);
            T = f * (T + S * d);
            S *= f;
          }
          m = now;
          float s1 = 0.0f, t1 = 0.0f;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float d = z[j] - base, e = ex2_approx(d * 1.4426950408889634f);
            s1 += e;
            t1 = fmaf(e, fmaxf(d, -1000.0f), t1);  // a weight of 0 adds 0, also where z is -inf
          }
          S += s1;
          T += t1;
          if (nc > 0 && r < a.R && top > worst) {
            for (int j = 0; j < 16; ++j) {
              if (!(z[j] > worst)) continue;
              unsigned long long key = argmax_key(z[j], (uint32_t)(v0 + c0 + j));
              int k = nc - 1;
              while (k > 0 && list[(k - 1) * kLpM + row] < key) {
                list[k * kLpM + row] = list[(k - 1) * kLpM + row];
                --k;
              }
              list[k * kLpM + row] = key;
              const unsigned long long w = list[(nc - 1) * kLpM + row];
              if (w != 0ull) {
                const uint32_t uw = (uint32_t)(w >> 32);
                worst = __uint_as_float((uw & 0x80000000u) ? uw & 0x7FFFFFFFu : ~uw);
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[ab]);
      }
      if (ok && r < a.R) {
        float* st = a.stat + (size_t)g * 3 * a.R + r;
        st[0] = m;
        st[a.R] = S;
        st[2 * (size_t)a.R] = T;
        unsigned long long* dst = a.cand + ((size_t)g * a.R + r) * nc;
        for (int k = 0; k < nc; ++k) dst[k] = list[k * kLpM + row];
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

struct LpFinishArgs {
  int R, H, V, n_groups, n_cand, n_top;
  const float* stat;
  const unsigned long long* cand;
  const __nv_bfloat16* h;
  const __nv_bfloat16* lm;
  const int32_t* tokens;  // [R] or null
  float* logprob;         // [R] or null
  float* entropy;         // [R] or null
  int32_t* top_ids;       // [R, n_top]
  float* top_logprobs;    // [R, n_top]
};

constexpr int kLpFinishThreads = 128;

// One CTA per row.
__global__ void __launch_bounds__(kLpFinishThreads) logprob_finish(const LpFinishArgs a) {
  constexpr int NW = kLpFinishThreads / 32, kMost = kLpMaxTop + kLpSpare;
  __shared__ float red_m[NW];
  __shared__ double red_s[NW], red_t[NW], z_s[kMost + 1];
  __shared__ int id_s[kMost + 1];
  griddep_launch_dependents();
  griddep_wait();
  const int r = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // ---- the units' sums, rescaled to the common maximum
  float m = -INFINITY;
  for (int g = tid; g < a.n_groups; g += kLpFinishThreads) m = fmaxf(m, a.stat[(size_t)g * 3 * a.R + r]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red_m[warp] = m;
  __syncthreads();
  for (int w = 0; w < NW; ++w) m = fmaxf(m, red_m[w]);
  double S = 0.0, T = 0.0;
  for (int g = tid; g < a.n_groups; g += kLpFinishThreads) {
    const float* st = a.stat + (size_t)g * 3 * a.R + r;
    const float mg = st[0], Sg = st[a.R], Tg = st[2 * (size_t)a.R];
    const double d = mg > -INFINITY ? (double)mg - (double)m : 0.0, f = mg > -INFINITY ? exp(d) : 1.0;
    S += f * Sg;
    T += f * (Tg + Sg * d);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    S += __shfl_xor_sync(0xffffffffu, S, o);
    T += __shfl_xor_sync(0xffffffffu, T, o);
  }
  if (lane == 0) red_s[warp] = S, red_t[warp] = T;
  // ---- the best candidates of all units: one warp, each lane walking the lists g = lane, lane + 32, ...
  if (warp == 0 && a.n_cand > 0) {
    for (int k = 0; k < a.n_cand; ++k) {
      // the k-th best key is the largest below the previous one
      const unsigned long long below = k == 0 ? ~0ull : ((unsigned long long)__double_as_longlong(z_s[k - 1]));
      unsigned long long best = 0ull;
      for (int g = lane; g < a.n_groups; g += 32) {
        const unsigned long long* l = a.cand + ((size_t)g * a.R + r) * a.n_cand;
        for (int i = 0; i < a.n_cand; ++i) {
          const unsigned long long key = l[i];
          if (key < below) {
            best = key > best ? key : best;
            break;
          }
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long other = __shfl_xor_sync(0xffffffffu, best, o);
        best = other > best ? other : best;
      }
      if (lane == 0) {
        z_s[k] = __longlong_as_double((long long)best);  // the key itself, until the logits replace it
        id_s[k] = best ? (int)(0xFFFFFFFFu - (uint32_t)(best & 0xFFFFFFFFull)) : -1;
      }
      __syncwarp();
    }
  }
  const int tok = a.tokens ? a.tokens[r] : -1;
  if (tid == 0) {
    id_s[a.n_cand] = tok >= 0 && tok < a.V ? tok : -1;
    if (tok >= a.V) record_error(kErrBounds, 355);
  }
  __syncthreads();
  // ---- their logits from exact products (a product of two bf16 is exact in fp32), summed in fp64
  for (int k = warp; k <= a.n_cand; k += NW) {
    const int v = id_s[k];
    double z = -INFINITY;
    if (v >= 0) {
      z = 0.0;
      const uint4* x = reinterpret_cast<const uint4*>(a.h + (size_t)r * a.H);
      const uint4* w = reinterpret_cast<const uint4*>(a.lm + (size_t)v * a.H);
      for (int i = lane; i < a.H / 8; i += 32) {
        const uint4 xv = x[i], wv = w[i];
        const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w}, ws[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          z += (double)(bf16_lo(xs[e]) * bf16_lo(ws[e]));
          z += (double)(bf16_hi(xs[e]) * bf16_hi(ws[e]));
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    }
    __syncwarp();
    if (lane == 0) z_s[k] = z;
  }
  __syncthreads();
  S = 0.0, T = 0.0;
  for (int w = 0; w < NW; ++w) S += red_s[w], T += red_t[w];
  const double log_s = log(S), lse = (double)m + log_s;
  if (tid == 0) {
    if (a.logprob) a.logprob[r] = (float)(z_s[a.n_cand] - lse);
    if (a.entropy) a.entropy[r] = (float)(log_s - T / S);
  }
  // ---- order: rank of each candidate by (logit, lower index first)
  if (tid < a.n_cand) {
    const double z = z_s[tid];
    const int v = id_s[tid];
    int rank = 0;
    for (int k = 0; k < a.n_cand; ++k) {
      if (k == tid) continue;
      // candidates that are missing (fewer finite logits than asked for) come last, in list order
      const bool ahead = id_s[k] < 0 ? (v < 0 && k < tid) : (v < 0 || z_s[k] > z || (z_s[k] == z && id_s[k] < v));
      rank += ahead;
    }
    if (rank < a.n_top) {
      a.top_ids[(size_t)r * a.n_top + rank] = v;
      a.top_logprobs[(size_t)r * a.n_top + rank] = (float)(z - lse);
    }
  }
}

}  // namespace vg
