// mk_verify.cu -- verification of drafted tokens by the target's probabilities
// (speculative sampling: Leviathan et al. 2023, algorithm 1; Chen et al. 2023),
// the sampled counterpart of the greedy acceptance of mk_verify_steps.
//
// Two launches.  verify_rows finds, for every target and draft row, what
// mk_sample_top_p decides by: the largest logit, the threshold key tau of the
// nucleus, how many tokens tied at tau belong to it, its mass, and the drafted
// token's share of it.  verify_draw walks each sequence's drafts with these
// numbers and draws the block's last token from the residual (or the target's
// own) masses of the row it ends at.
//
// All masses are the fixed-point integers round_half_even(exp((l - max) / T) *
// 2^46), as in mk_sample.cu, so that every sum is exact and no result depends on
// the order in which threads add.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

#include "mk_internal.h"

namespace cg = cooperative_groups;

namespace mk {
namespace {

typedef unsigned long long u64;

constexpr int kVThreads = 512;
constexpr int kVWarps = kVThreads / 32;
constexpr int kMaxCluster = 8;
constexpr double kMassScale = 70368744177664.0;  // 2^46
constexpr int kBins = 1024;   // histogram bins over max - l
constexpr int kCand = 512;    // candidates of the threshold bin that one list holds

// What verify_rows leaves for a row.
struct RowStat {
  u64 mass;      // nucleus mass S
  u64 drafted;   // mass of the draft that the row decides on, 0 outside the nucleus
  u64 ties;      // tokens tied at tau that belong to the nucleus, lowest ids first
  uint32_t max_key, tau;
  int32_t best;  // argmax (lowest id), temperature <= 0 only
  int32_t pad;
};
static_assert(sizeof(RowStat) == 40, "workspace layout");

// Order-preserving key: larger logit <-> larger key; -0 and +0 share one key.
__device__ __forceinline__ uint32_t logit_key(float x) {
  uint32_t b = __float_as_uint(x);
  if (b == 0x80000000u) b = 0u;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

__device__ __forceinline__ u64 mass_of(float l, float m, double inv_t) {
  const double z = ((double)l - (double)m) * inv_t;
  // exp(-33) 2^46 < 0.5: the mass rounds to zero (NaN takes the other branch)
  return z < -33.0 ? 0 : __double2ull_rn(exp(z) * kMassScale);
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

__device__ __forceinline__ u64 nucleus_need(float top_p, u64 total) {
  const double x = ceil((double)top_p * __ull2double_rn(total));
  u64 need;
  if (!(x >= 1.0)) need = 1;
  else if (x >= 18446744073709551616.0) need = total;
  else need = min((u64)x, total);
  return need > 0 ? need : 1;
}

struct RowsArgs {
  const float *logits, *draft;
  const int32_t *tokens;
  int B, T, V, slice, vec4, greedy;
  double inv_t;
  float top_p, bin_scale;
  RowStat *stats;  // [B * T] target rows, then [B * (T - 1)] draft rows
};

struct RowsShared {
  u64 hist[kBins];
  u64 red[kVWarps], red2[kVWarps];
  uint32_t wkey[kVWarps];
  int32_t wid[kVWarps];
  u64 cta_sum, cta_min;   // read by the cluster
  u64 least;
  uint32_t cta_key, n_cand, n_eq;
  int32_t cta_id;
  uint32_t gmax;
  u64 total, above, need;
  int bin;
  uint32_t cand_key[kCand];
  u64 cand_mass[kCand];
  uint32_t tau;
  u64 tau_above;
};

// Sums v over the block; every thread gets the result.
__device__ __forceinline__ u64 block_sum(u64 v, u64 *red, int lane, int warp) {
  v = warp_sum(v);
  if (lane == 0) red[warp] = v;
  __syncthreads();
  u64 s = 0;
#pragma unroll
  for (int w = 0; w < kVWarps; ++w) s += red[w];
  __syncthreads();
  return s;
}

// f(l, id) for this thread's logits of a slice [0, n) of row src (ids from lo).
template <typename F>
__device__ __forceinline__ void each(const float *src, int n, int vec4, int tid, F f) {
  if (vec4) {
    const float4 *s4 = reinterpret_cast<const float4 *>(src);
#pragma unroll 2
    for (int i = tid; i < n / 4; i += kVThreads) {
      const float4 x = s4[i];
      f(x.x, 4 * i);
      f(x.y, 4 * i + 1);
      f(x.z, 4 * i + 2);
      f(x.w, 4 * i + 3);
    }
  } else {
#pragma unroll 4
    for (int i = tid; i < n; i += kVThreads) f(src[i], i);
  }
}

// One cluster per row.  The row is read from memory once (the largest logit) and
// then from L2: for the masses' sum, for the histogram, and for the threshold.
__global__ void __launch_bounds__(kVThreads) verify_rows(const __grid_constant__ RowsArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ RowsShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned rank = cluster.block_rank(), size = cluster.num_blocks();
  const int row = blockIdx.x / size;
  const bool is_draft = row >= a.B * a.T;
  const int r = is_draft ? row - a.B * a.T : row;
  const int per = is_draft ? a.T - 1 : a.T, b = r / per, t = r % per;
  const int lo = (int)rank * a.slice, n = max(0, min(a.slice, a.V - lo));
  const float *base = (is_draft ? a.draft : a.logits) + (size_t)r * a.V;
  const float *src = base + lo;

  // ---- the largest logit ---------------------------------------------------------
  uint32_t kmax = 0;
  each(src, n, a.vec4, tid, [&](float x, int) { kmax = max(kmax, logit_key(x)); });
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  if (lane == 0) sh.wkey[warp] = kmax;
  for (int i = tid; i < kBins; i += kVThreads) sh.hist[i] = 0;
  if (tid == 0) sh.n_cand = 0;
  __syncthreads();
  if (tid == 0) {
    uint32_t k = 0;
    for (int w = 0; w < kVWarps; ++w) k = max(k, sh.wkey[w]);
    sh.cta_key = k;
  }
  cluster.sync();
  if (tid == 0) {
    uint32_t k = 0;
    for (unsigned i = 0; i < size; ++i) k = max(k, *cluster.map_shared_rank(&sh.cta_key, i));
    sh.gmax = k;
  }
  __syncthreads();
  const uint32_t gmax = sh.gmax;

  if (a.greedy) {
    int best = 0x7fffffff;
    each(src, n, a.vec4, tid, [&](float x, int i) {
      if (logit_key(x) == gmax) best = min(best, lo + i);
    });
    best = __reduce_min_sync(0xffffffffu, best);
    if (lane == 0) sh.wid[warp] = best;
    __syncthreads();
    if (tid == 0) {
      int m = 0x7fffffff;
      for (int w = 0; w < kVWarps; ++w) m = min(m, sh.wid[w]);
      sh.cta_id = m;
    }
    cluster.sync();
    if (rank == 0 && tid == 0) {
      int m = 0x7fffffff;
      for (unsigned i = 0; i < size; ++i) m = min(m, *cluster.map_shared_rank(&sh.cta_id, i));
      a.stats[row].best = m;
    }
    cluster.sync();  // no CTA leaves while its shared memory is being read
    return;
  }

  // ---- the masses' sum and the smallest that is not zero -----------------------------
  const float m = key_logit(gmax);
  const bool whole = a.top_p >= 1.0f;  // the histogram is then hardly ever needed
  u64 sum = 0, least = ~0ull;
  each(src, n, a.vec4, tid, [&](float x, int) {
    const u64 q = mass_of(x, m, a.inv_t);
    if (q) {
      sum += q;
      least = min(least, q);
      if (!whole) {
        const int bin = (int)fminf((m - x) * a.bin_scale, (float)(kBins - 1));
        atomicAdd(&sh.hist[max(bin, 0)], q);
      }
    }
  });
#pragma unroll
  for (int o = 16; o; o >>= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
  if (lane == 0) sh.red2[warp] = least;
  sum = block_sum(sum, sh.red, lane, warp);
  if (tid == 0) {
    u64 x = ~0ull;
    for (int w = 0; w < kVWarps; ++w) x = min(x, sh.red2[w]);
    sh.cta_sum = sum;
    sh.cta_min = x;
  }
  cluster.sync();
  if (tid == 0) {
    u64 s = 0, x = ~0ull;
    for (unsigned i = 0; i < size; ++i) {
      s += *cluster.map_shared_rank(&sh.cta_sum, i);
      x = min(x, *cluster.map_shared_rank(&sh.cta_min, i));
    }
    sh.total = s;
    sh.least = x;
    sh.need = nucleus_need(a.top_p, s);
  }
  __syncthreads();
  const u64 total = sh.total, need = sh.need;
  cluster.sync();  // cta_sum is written again
  const u64 smallest = sh.least;

  uint32_t tau = 0;       // every token with a mass
  u64 ties = 0, mass = total;
  if (smallest <= total - need) {  // some token may be left out
    // ---- the bin that holds the threshold ---------------------------------------------
    if (whole) {
      each(src, n, a.vec4, tid, [&](float x, int) {
        const u64 q = mass_of(x, m, a.inv_t);
        if (q) {
          const int bin = (int)fminf((m - x) * a.bin_scale, (float)(kBins - 1));
          atomicAdd(&sh.hist[max(bin, 0)], q);
        }
      });
    }
    __syncthreads();
    cluster.sync();
    u64 v[kBins / kVThreads], s = 0;
#pragma unroll
    for (int k = 0; k < kBins / kVThreads; ++k) {
      v[k] = 0;
      for (unsigned i = 0; i < size; ++i)
        v[k] += *cluster.map_shared_rank(&sh.hist[tid * (kBins / kVThreads) + k], i);
      s += v[k];
    }
    u64 incl = warp_scan(s, lane);
    if (lane == 31) sh.red[warp] = incl;
    if (tid == 0) {  // reached only if no bin is found (non-finite logits)
      sh.bin = kBins - 1;
      sh.above = 0;
    }
    __syncthreads();
    u64 before = incl - s;
    for (int w = 0; w < warp; ++w) before += sh.red[w];
#pragma unroll
    for (int k = 0; k < kBins / kVThreads; ++k) {
      if (before < need && before + v[k] >= need) {
        sh.bin = tid * (kBins / kVThreads) + k;
        sh.above = before;
      }
      before += v[k];
    }
    __syncthreads();
    const int bin = sh.bin;
    const u64 above = sh.above;
    // ---- the tokens of that bin --------------------------------------------------------
    each(src, n, a.vec4, tid, [&](float x, int) {
      const int i = max((int)fminf((m - x) * a.bin_scale, (float)(kBins - 1)), 0);
      if (i == bin) {
        const u64 q = mass_of(x, m, a.inv_t);
        if (q) {
          const uint32_t at = atomicAdd(&sh.n_cand, 1u);
          if (at < kCand) {
            sh.cand_key[at] = logit_key(x);
            sh.cand_mass[at] = q;
          }
        }
      }
    });
    if (tid == 0) {  // before the barrier: another CTA may write them after it
      sh.tau = 0;
      sh.tau_above = above;
    }
    cluster.sync();
    // Every CTA decides from the same lists.  tau is the key of the candidate with
    // mass(bins above) + mass(candidates above it) < need <= that + its ties' mass.
    bool fits = true;
    for (unsigned i = 0; i < size; ++i) fits = fits && *cluster.map_shared_rank(&sh.n_cand, i) <= kCand;
    if (fits) {
      const uint32_t own = sh.n_cand;
      for (uint32_t c = tid; c < own; c += kVThreads) {
        const uint32_t key = sh.cand_key[c];
        u64 more = above, same = 0;
        for (unsigned i = 0; i < size; ++i) {
          const uint32_t cnt = *cluster.map_shared_rank(&sh.n_cand, i);
          const uint32_t *ck = cluster.map_shared_rank(sh.cand_key, i);
          const u64 *cm = cluster.map_shared_rank(sh.cand_mass, i);
          for (uint32_t j = 0; j < cnt; ++j) {
            const uint32_t kj = ck[j];
            if (kj > key) more += cm[j];
            else if (kj == key) same += cm[j];
          }
        }
        if (more < need && need <= more + same)  // tied candidates write the same values, in every CTA
          for (unsigned i = 0; i < size; ++i) {
            *cluster.map_shared_rank(&sh.tau, i) = key;
            *cluster.map_shared_rank(&sh.tau_above, i) = more;
          }
      }
      cluster.sync();
    } else {
      // Too many for the list (a row of equal logits): bisection of the key, bit
      // by bit, for the largest key with mass(keys >= it) >= need.
      uint32_t lo_key = 0;
      for (int bit = 31; bit >= 0; --bit) {
        const uint32_t mid = lo_key | (1u << bit);
        u64 part = 0;
        each(src, n, a.vec4, tid, [&](float x, int) {
          if (logit_key(x) >= mid) part += mass_of(x, m, a.inv_t);
        });
        part = block_sum(part, sh.red, lane, warp);
        if (tid == 0) sh.cta_sum = part;
        cluster.sync();
        u64 all = 0;
        for (unsigned i = 0; i < size; ++i) all += *cluster.map_shared_rank(&sh.cta_sum, i);
        cluster.sync();
        if (all >= need) lo_key = mid;
      }
      u64 part = 0;
      each(src, n, a.vec4, tid, [&](float x, int) {
        if (logit_key(x) > lo_key) part += mass_of(x, m, a.inv_t);
      });
      part = block_sum(part, sh.red, lane, warp);
      if (tid == 0) sh.cta_sum = part;
      cluster.sync();
      u64 all = 0;
      for (unsigned i = 0; i < size; ++i) all += *cluster.map_shared_rank(&sh.cta_sum, i);
      cluster.sync();
      if (tid == 0) {
        sh.tau = lo_key;
        sh.tau_above = all;
      }
      __syncthreads();
    }
    tau = sh.tau;
    const u64 at_tau = sh.tau_above;
    u64 q_tau = mass_of(key_logit(tau), m, a.inv_t);
    if (q_tau == 0) q_tau = 1;  // only on non-finite input
    ties = need > at_tau ? (need - at_tau + q_tau - 1) / q_tau : 1;
    mass = at_tau + ties * q_tau;
  }

  // ---- the draft that this row decides on ---------------------------------------------
  const int x = t < a.T - 1 ? a.tokens[b * a.T + t + 1] : -1;
  u64 drafted = 0;
  if (x >= 0 && x < a.V) {
    const uint32_t key = logit_key(base[x]);
    if (key > tau) {
      drafted = mass_of(base[x], m, a.inv_t);
    } else if (key == tau) {  // in the nucleus if fewer than `ties` of its ties have lower ids
      u64 lower = 0;
      each(src, n, a.vec4, tid, [&](float y, int i) { lower += logit_key(y) == tau && lo + i < x; });
      lower = block_sum(lower, sh.red, lane, warp);
      if (tid == 0) sh.cta_sum = lower;
      cluster.sync();
      u64 all = 0;
      for (unsigned i = 0; i < size; ++i) all += *cluster.map_shared_rank(&sh.cta_sum, i);
      if (all < ties) drafted = mass_of(base[x], m, a.inv_t);
    }
  }
  if (rank == 0 && tid == 0) {
    RowStat &o = a.stats[row];
    o.mass = mass;
    o.drafted = drafted;
    o.ties = ties;
    o.max_key = gmax;
    o.tau = tau;
  }
  cluster.sync();  // no CTA leaves while its shared memory is being read
}

struct DrawArgs {
  const float *logits, *draft;
  const int32_t *tokens;
  const double *uniforms;
  int B, T, V, slice, greedy;
  double inv_t;
  const RowStat *stats;
  int32_t *out_tokens, *out_accepted;
};

// One row's membership: mass of id with logit l, `tied` of its ties before it.
struct RowMass {
  float m;
  uint32_t tau;
  u64 ties;
  double inv_t;
  __device__ u64 of(float l, uint32_t key, u64 tied) const {
    if (key > tau || (key == tau && tied < ties)) return mass_of(l, m, inv_t);
    return 0;
  }
};

// One cluster per sequence; warp w of CTA r holds segment r * kVWarps + w of the
// row's ids.  Ties at the two thresholds are counted per segment first, so that
// a token's rank among its ties is known when its mass is taken.
__global__ void __launch_bounds__(kVThreads) verify_draw(const __grid_constant__ DrawArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ u64 red[kVWarps], seg[kVWarps];
  __shared__ uint32_t tie_a[kVWarps], tie_d[kVWarps];
  __shared__ u64 c_sum;
  __shared__ uint32_t c_tie[2];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned rank = cluster.block_rank(), size = cluster.num_blocks();
  const int b = blockIdx.x / size, T = a.T;
  const RowStat *st = a.stats + (size_t)b * T;
  const RowStat *sd = a.stats + (size_t)a.B * T + (size_t)b * (T - 1);
  const int32_t *tok = a.tokens + (size_t)b * T;
  const bool lead = rank == 0 && tid == 0;

  // ---- how many drafts stand ------------------------------------------------------
  int s = 0;
  for (; s < T - 1; ++s) {
    const int x = tok[s + 1];
    if (x < 0 || x >= a.V) break;
    if (a.greedy) {
      if (x != st[s].best) break;
      continue;
    }
    double u = a.uniforms[(size_t)b * T + s];
    const double am = __ull2double_rn(st[s].mass), ax = __ull2double_rn(st[s].drafted);
    bool ok;
    if (a.draft) {
      const double dm = __ull2double_rn(sd[s].mass), dx = __ull2double_rn(sd[s].drafted);
      ok = __dmul_rn(u, __dmul_rn(dx, am)) < __dmul_rn(ax, dm);
    } else {
      ok = __dmul_rn(u, am) < ax;
    }
    if (!ok) break;
  }
  if (lead) {
    a.out_accepted[b] = s + 1;
    for (int i = 0; i < T; ++i)
      if (i != s) a.out_tokens[(size_t)b * T + i] = i < s ? tok[i + 1] : -1;
  }
  if (a.greedy) {
    if (lead) a.out_tokens[(size_t)b * T + s] = st[s].best;
    return;
  }

  const int x = s < T - 1 ? tok[s + 1] : -1;
  bool residual = x >= 0 && x < a.V;  // a draft that did not stand
  const float *la = a.logits + ((size_t)b * T + s) * a.V;
  const bool with_d = residual && a.draft;
  const float *ld = with_d ? a.draft + ((size_t)b * (T - 1) + s) * a.V : nullptr;
  const RowMass A{key_logit(st[s].max_key), st[s].tau, st[s].ties, a.inv_t};
  const RowMass D = with_d ? RowMass{key_logit(sd[s].max_key), sd[s].tau, sd[s].ties, a.inv_t} : A;
  const double ra = with_d ? kMassScale / __ull2double_rn(st[s].mass) : 0.0;
  const double rd = with_d ? kMassScale / __ull2double_rn(sd[s].mass) : 0.0;

  const int per = (a.slice + kVWarps - 1) / kVWarps;
  const int lo = (int)rank * a.slice, hi = min(a.V, lo + a.slice);
  const int s0 = min(hi, lo + warp * per), s1 = min(hi, s0 + per);

  // ---- ties before each segment ------------------------------------------------------
  uint32_t ca = 0, cd = 0;
  for (int i = s0 + lane; i < s1; i += 32) {
    ca += logit_key(la[i]) == A.tau;
    if (with_d) cd += logit_key(ld[i]) == D.tau;
  }
  ca = __reduce_add_sync(0xffffffffu, ca);
  cd = __reduce_add_sync(0xffffffffu, cd);
  if (lane == 0) {
    tie_a[warp] = ca;
    tie_d[warp] = cd;
  }
  __syncthreads();
  if (tid == 0) {
    c_tie[0] = c_tie[1] = 0;
    for (int w = 0; w < kVWarps; ++w) {
      c_tie[0] += tie_a[w];
      c_tie[1] += tie_d[w];
    }
  }
  cluster.sync();
  u64 before_a = 0, before_d = 0;
  for (unsigned i = 0; i < rank; ++i) {
    const uint32_t *o = cluster.map_shared_rank(c_tie, i);
    before_a += o[0];
    before_d += o[1];
  }
  for (int w = 0; w < warp; ++w) {
    before_a += tie_a[w];
    before_d += tie_d[w];
  }

  // The mass that id i (this lane's of 32 neighbours) is drawn with; ta, td count
  // the ties before these 32.
  auto mass_at = [&](int i, bool in, bool res, u64 &ta, u64 &td) -> u64 {
    const float l = in ? la[i] : 0.f;
    const uint32_t k = in ? logit_key(l) : 0u;
    const unsigned eq = __ballot_sync(0xffffffffu, in && k == A.tau);
    u64 q = in ? A.of(l, k, ta + __popc(eq & ((1u << lane) - 1u))) : 0;
    ta += __popc(eq);
    if (!res) return q;
    if (!with_d) return i == x ? 0 : q;
    const float y = in ? ld[i] : 0.f;
    const uint32_t kd = in ? logit_key(y) : 0u;
    const unsigned ed = __ballot_sync(0xffffffffu, in && kd == D.tau);
    const u64 w = in ? D.of(y, kd, td + __popc(ed & ((1u << lane) - 1u))) : 0;
    td += __popc(ed);
    const u64 p = __double2ull_rn(__dmul_rn(__ull2double_rn(q), ra)), o = __double2ull_rn(__dmul_rn(__ull2double_rn(w), rd));
    return p > o ? p - o : 0;
  };

  // ---- the masses' sums: the residual's, and the target's own where that is zero -------
  u64 total = 0;
  for (int round = residual ? 0 : 1; round < 2; ++round) {
    const bool res = round == 0;
    u64 ta = before_a, td = before_d, mine = 0;
    for (int i0 = s0; i0 < s1; i0 += 32) mine += mass_at(i0 + lane, i0 + lane < s1, res, ta, td);
    mine = warp_sum(mine);
    if (lane == 0) seg[warp] = mine;
    __syncthreads();
    if (tid == 0) {
      u64 c = 0;
      for (int w = 0; w < kVWarps; ++w) c += seg[w];
      c_sum = c;
    }
    cluster.sync();
    total = 0;
    u64 before = 0;
    for (unsigned i = 0; i < size; ++i) {
      const u64 c = *cluster.map_shared_rank(&c_sum, i);
      if (i < rank) before += c;
      total += c;
    }
    for (int w = 0; w < warp; ++w) before += seg[w];
    const u64 own = seg[warp];
    if (res && total == 0) {
      cluster.sync();  // c_sum and seg are written again
      continue;
    }
    // ---- the draw: the segment that holds y, then the id in it -------------------------
    double uu = a.uniforms[(size_t)b * T + T - 1];
    if (!(uu >= 0.0)) uu = 0.0;
    u64 y = (u64)floor(__dmul_rn(fmin(uu, 1.0), __ull2double_rn(total)));
    if (y >= total) y = total > 0 ? total - 1 : 0;
    if (lead && total == 0) a.out_tokens[(size_t)b * T + s] = 0;  // only on rows without a finite logit
    if (before <= y && y < before + own) {
      u64 ra_ = before_a, rd_ = before_d, run = before;
      for (int i0 = s0; i0 < s1; i0 += 32) {
        const u64 q = mass_at(i0 + lane, i0 + lane < s1, res, ra_, rd_);
        const u64 cum = run + warp_scan(q, lane);
        const unsigned hit = __ballot_sync(0xffffffffu, cum > y);
        if (hit) {
          if (lane == __ffs(hit) - 1) a.out_tokens[(size_t)b * T + s] = i0 + lane;
          break;
        }
        run = __shfl_sync(0xffffffffu, cum, 31);
      }
    }
    break;
  }
  cluster.sync();  // no CTA leaves while its shared memory is being read
}

// CTAs per row: the smallest power of two that gives every SM a block.
int cluster_for(int rows, int n_sm) {
  int c = 1;
  while (c < kMaxCluster && static_cast<long long>(rows) * c < n_sm) c *= 2;
  return c;
}

template <typename Args>
cudaError_t launch(void (*kernel)(Args), int grid, int cluster, bool after, cudaStream_t st, const Args &args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid) * cluster);
  cfg.blockDim = dim3(kVThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

}  // namespace

size_t verify_sample_workspace(int B, int T) { return sizeof(RowStat) * static_cast<size_t>(B) * (2 * static_cast<size_t>(T) - 1); }

cudaError_t launch_verify_sample(const VerifySample &v, cudaStream_t st) {
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int greedy = !(v.temperature > 0.0f);
  const double inv_t = greedy ? 0.0 : 1.0 / (double)v.temperature;
  const bool draft = v.draft_logits && !greedy;
  const int rows = v.B * v.T + (draft ? v.B * (v.T - 1) : 0);
  RowStat *stats = static_cast<RowStat *>(v.workspace);

  RowsArgs r{};
  r.logits = v.logits;
  r.draft = draft ? v.draft_logits : nullptr;
  r.tokens = v.tokens;
  r.B = v.B;
  r.T = v.T;
  r.V = v.V;
  const int cr = cluster_for(rows, n_sm);
  r.slice = ((v.V + cr - 1) / cr + 3) & ~3;
  r.vec4 = v.V % 4 == 0 && (reinterpret_cast<uintptr_t>(v.logits) & 15) == 0 &&
           (!draft || (reinterpret_cast<uintptr_t>(v.draft_logits) & 15) == 0);
  r.greedy = greedy;
  r.inv_t = inv_t;
  r.top_p = v.top_p;
  // masses are zero beyond max - l = 33 T; bins of equal width cover that range
  r.bin_scale = greedy ? 0.f : static_cast<float>(kBins * inv_t / 33.0);
  r.stats = stats;
  e = launch(verify_rows, rows, cr, false, st, r);
  if (e != cudaSuccess) return e;

  DrawArgs d{};
  d.logits = v.logits;
  d.draft = r.draft;
  d.tokens = v.tokens;
  d.uniforms = v.uniforms;
  d.B = v.B;
  d.T = v.T;
  d.V = v.V;
  const int cd = greedy ? 1 : cluster_for(v.B, n_sm);
  d.slice = (v.V + cd - 1) / cd;
  d.greedy = greedy;
  d.inv_t = inv_t;
  d.stats = stats;
  d.out_tokens = v.out_tokens;
  d.out_accepted = v.out_accepted;
  return launch(verify_draw, v.B, cd, true, st, d);
}

}  // namespace mk
