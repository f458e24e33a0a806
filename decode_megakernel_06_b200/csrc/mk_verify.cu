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

#include <algorithm>
#include <atomic>
#include <mutex>

#include "mk_internal.h"

namespace cg = cooperative_groups;

namespace mk {
namespace {

typedef unsigned long long u64;

constexpr int kVThreads = 1024;
constexpr int kVWarps = kVThreads / 32;
constexpr int kMaxCluster = 8;
constexpr double kMassScale = 70368744177664.0;  // 2^46
constexpr int kBins = 1024;   // histogram bins over max - l
constexpr int kFine = 10;     // each of 2^kFine fine ones: 2^20 in all, exact in fp32
constexpr int kQueue = 16;    // logits of the nucleus that a thread keeps at hand
constexpr int kCache = 32768; // logits of a slice that are kept in shared memory where a nucleus is looked for
constexpr int kCand = 512;    // tokens of the threshold's fine bin that the list holds
constexpr int kVerifyDevices = 64;
constexpr int kDrawThreads = 512;
constexpr int kDrawWarps = kDrawThreads / 32;

// What verify_rows leaves for a row.
struct RowStat {
  u64 mass;      // nucleus mass S
  u64 drafted;   // mass of the draft that the row decides on, 0 outside the nucleus
  u64 ties;      // tokens tied at tau that belong to the nucleus, lowest ids first
  uint32_t max_key, tau;
  int32_t best;  // argmax (lowest id), temperature <= 0 only
  int32_t cut;   // not all tokens at tau belong to the nucleus
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

constexpr double kRound = 4503599627370496.0;  // 2^52: adding it rounds to a whole number

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A whole number x, 0 <= x < 2^52, from x + 2^52; zero from NaN.
__device__ __forceinline__ u64 whole_bits(double x) {
  return static_cast<unsigned>(__double2hiint(x)) < 0x43400000u ? __double_as_longlong(x) - 0x4330000000000000ll : 0;
}

// round_half_even(exp((l - m) / T) 2^46).  The product is exact, so its sum with 2^52 is
// its rounding.  No test for masses that round to zero: a branch around the
// exponential cost 20 of 65 cycles a warp.
__device__ __forceinline__ u64 mass_of(float l, float m, double inv_t) {
  return whole_bits(fma(exp(((double)l - (double)m) * inv_t), kMassScale, kRound));
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

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

struct RowsArgs {
  const float *logits, *draft;
  const int32_t *tokens;
  int B, T, V, slice, vec4, greedy, cached;
  double inv_t;
  float top_p, bin_scale, inv_t2;  // fine bins per unit of the logits; log2(e) / temperature
  RowStat *stats;  // [B * T] target rows, then [B * (T - 1)] draft rows
};

struct alignas(16) RowsShared {  // the queue and the cache behind it are read 16 bytes at a time
  uint32_t hist[kBins];       // read by the cluster
  u64 fine[1 << kFine];       // read by the cluster
  u64 red[kVWarps], red2[kVWarps];
  uint32_t wkey[kVWarps], wkey2[kVWarps];
  // Read by the cluster, each written again only behind a cluster barrier: the first sum has a
  // word of its own, since no barrier stands between its reading and the search's sums
  // where no histogram is taken (top_p >= 1).
  u64 cta_total, cta_sum, cta_sum2;
  float cta_least;
  uint32_t cta_key, cta_lo, cta_hi, n_cand;
  int32_t cta_id;
  u64 before, at_tau, same;
  uint32_t tau, found;
  int bin, last_bin;
  uint32_t cand_key[kCand], all_key[kCand];
  u64 cand_mass[kCand], all_mass[kCand];
};
static_assert(sizeof(RowsShared) % 16 == 0, "alignment of what follows");

// The block's sum of v, in every thread.
__device__ __forceinline__ u64 block_sum(u64 v, u64 *red, int lane, int warp) {
  v = warp_sum(v);
  __syncthreads();
  if (lane == 0) red[warp] = v;
  __syncthreads();
  u64 s = 0;
#pragma unroll
  for (int w = 0; w < kVWarps; ++w) s += red[w];
  return s;
}

// The cluster's sum of a value that each CTA holds at *mine (written by thread 0 before
// the last cluster barrier), in every thread.
__device__ __forceinline__ u64 cluster_total(cg::cluster_group &cluster, u64 *mine, unsigned size, int lane) {
  u64 v = lane < (int)size ? *cluster.map_shared_rank(mine, lane) : 0;
  return warp_sum(v);
}

// f(l, i) for this thread's logits of the slice [0, n) of a row; padded: the same number
// of calls in every lane of a warp, with i >= n behind the end.
template <int UNROLL, typename F>
__device__ __forceinline__ void each(const float *src, int n, int vec4, int tid, F f) {
  if (vec4) {
    const float4 *s4 = reinterpret_cast<const float4 *>(src);
#pragma unroll 1
    for (int i0 = tid & ~31; i0 < n / 4; i0 += UNROLL * kVThreads) {
      float4 x[UNROLL];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int i = i0 + (tid & 31) + u * kVThreads;
        x[u] = i < n / 4 ? s4[i] : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int i = i0 + (tid & 31) + u * kVThreads, at = i < n / 4 ? 4 * i : n;
        f(x[u].x, at);
        f(x[u].y, at + 1);
        f(x[u].z, at + 2);
        f(x[u].w, at + 3);
      }
    }
  } else {
#pragma unroll 1
    for (int i0 = tid & ~31; i0 < n; i0 += 4 * UNROLL * kVThreads) {
      float x[4 * UNROLL];
#pragma unroll
      for (int u = 0; u < 4 * UNROLL; ++u) {
        const int i = i0 + (tid & 31) + u * kVThreads;
        x[u] = i < n ? src[i] : -INFINITY;
      }
#pragma unroll
      for (int u = 0; u < 4 * UNROLL; ++u) f(x[u], min(i0 + (tid & 31) + u * kVThreads, n));
    }
  }
}

// One cluster per row (of one CTA where there are rows enough).  The row is read from
// memory once and from L2 or shared memory after that: for the largest logit, for the
// masses, and where a nucleus has to be found for its tokens.  What bounds it with a nucleus
// is one phase after another: of some 31 us for 104 rows of 32000 the masses, an fp64
// exponential per logit, and their exact pass take 13, issue slots are 62% used and the
// fp64 pipe 17%.  Of the whole distribution the masses are most.
//
// The nucleus: a token is left out if all tokens whose masses are no larger weigh no
// more than Q - need, so one whose mass is below (Q - need) / V need not be counted.
// The others go into a histogram over max - l, bins of equal width, of fp32 masses in
// 32 bits: a guess of the threshold's bin, which the exact sums of the next pass
// confirm or move.  That bin's tokens are ranked.  Where they are more than a list
// holds, they first go into 1024 finer bins, exactly, whose one that holds the
// threshold is nearly always a single logit of many tokens.
__global__ void __launch_bounds__(kVThreads, 1) verify_rows(const __grid_constant__ RowsArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  extern __shared__ __align__(16) unsigned char dyn[];
  RowsShared &sh = *reinterpret_cast<RowsShared *>(dyn);
  float *queue = reinterpret_cast<float *>(dyn + sizeof(RowsShared));  // [kQueue + 1][kVThreads], then [kCache]
  float *cache = queue + (kQueue + 1) * kVThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned rank = cluster.block_rank(), size = cluster.num_blocks();
  const int row = blockIdx.x / size;
  const bool is_draft = row >= a.B * a.T;
  const int r = is_draft ? row - a.B * a.T : row;
  const int per = is_draft ? a.T - 1 : a.T, b = r / per, t = r % per;
  const int lo = (int)rank * a.slice, n = max(0, min(a.slice, a.V - lo));
  const float *base = (is_draft ? a.draft : a.logits) + (size_t)r * a.V;
  const float *src = base + lo;
  auto sync_all = [&] {
    if (size > 1) cluster.sync();
    else __syncthreads();
  };
  const bool whole = a.top_p >= 1.0f;  // a nucleus is then hardly ever looked for
  pdl_wait();
  pdl_launch();

  // ---- the largest logit ---------------------------------------------------------------
  float mx = -INFINITY;
  if (a.cached && a.vec4) {
    const float4 *s4 = reinterpret_cast<const float4 *>(src);
    float4 *c4 = reinterpret_cast<float4 *>(cache);
#pragma unroll 8
    for (int i = tid; i < n / 4; i += kVThreads) {
      const float4 x = s4[i];
      c4[i] = x;
      mx = fmaxf(mx, fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)));
    }
  } else if (a.cached) {
    each<4>(src, n, 0, tid, [&](float x, int i) {
      if (i < n) cache[i] = x;
      mx = fmaxf(mx, x);
    });
  } else {
    each<4>(src, n, a.vec4, tid, [&](float x, int) { mx = fmaxf(mx, x); });
  }
  uint32_t kmax = __reduce_max_sync(0xffffffffu, logit_key(mx));
  if (lane == 0) sh.wkey[warp] = kmax;
  sh.hist[tid] = 0;
  if (tid == 0) sh.n_cand = 0;
  __syncthreads();
  if (a.cached) src = cache;
  if (warp == 0) {
    kmax = __reduce_max_sync(0xffffffffu, sh.wkey[lane]);
    if (lane == 0) sh.cta_key = kmax;
  }
  sync_all();
  kmax = __reduce_max_sync(0xffffffffu, lane < (int)size ? *cluster.map_shared_rank(&sh.cta_key, lane) : 0u);
  mx = key_logit(kmax);
  const float m = mx;
  const uint32_t gmax = logit_key(m);

  if (a.greedy) {
    int best = 0x7fffffff;
    each<4>(src, n, a.vec4, tid, [&](float x, int i) {
      if (x == m && i < n) best = min(best, lo + i);
    });
    best = __reduce_min_sync(0xffffffffu, best);
    if (lane == 0) sh.wkey[warp] = best;
    __syncthreads();
    if (warp == 0) {
      const int v = __reduce_min_sync(0xffffffffu, static_cast<int>(sh.wkey[lane]));
      if (lane == 0) sh.cta_id = v;
    }
    sync_all();
    if (rank == 0 && warp == 0) {
      const int v = __reduce_min_sync(0xffffffffu, lane < (int)size ? *cluster.map_shared_rank(&sh.cta_id, lane) : 0x7fffffff);
      if (lane == 0) a.stats[row].best = min(v, a.V - 1);
    }
    sync_all();  // no CTA leaves while its shared memory is being read
    return;
  }

  // The fine bin of a logit, rising as it falls (each step is monotone): the sum with 2^23
  // rounds to a whole number, for less than a conversion costs.
  auto fine_of = [&](float v) {
    const float at = fminf(fmaxf((m - v) * a.bin_scale, 0.f), (float)((kBins << kFine) - 1));
    return (int)(__float_as_uint(at + 8388608.f) - 0x4b000000u);
  };
  // ---- the masses' sum and the smallest that is not zero -----------------------------------
  u64 sum = 0;
  float least = INFINITY;  // the smallest logit with a mass
  each<1>(src, n, a.vec4, tid, [&](float x, int) {
    const u64 q = mass_of(x, m, a.inv_t);
    sum += q;
    if (q) least = fminf(least, x);
  });
  sum = warp_sum(sum);
  const uint32_t lk = __reduce_min_sync(0xffffffffu, logit_key(least));
  if (lane == 0) {
    sh.red[warp] = sum;
    sh.wkey[warp] = lk;
  }
  __syncthreads();
  if (warp == 0) {
    sum = warp_sum(sh.red[lane]);
    const uint32_t k = __reduce_min_sync(0xffffffffu, sh.wkey[lane]);
    if (lane == 0) {
      sh.cta_total = sum;
      sh.cta_least = key_logit(k);
    }
  }
  sync_all();
  const u64 total = cluster_total(cluster, &sh.cta_total, size, lane);
  least = lane < (int)size ? *cluster.map_shared_rank(&sh.cta_least, lane) : INFINITY;
  least = key_logit(__reduce_min_sync(0xffffffffu, logit_key(least)));
  const u64 smallest = least < INFINITY ? mass_of(least, m, a.inv_t) : ~0ull;
  const u64 need = nucleus_need(a.top_p, total);

  uint32_t tau = 0;       // every token with a mass
  u64 ties = 0, nucleus = total;
  bool cut = false;
  if (total > 0 && smallest <= total - need) {  // some token may be left out
    // ---- the guess: the bin where fp32 masses, scaled to a sum of 2^22, reach need -----------
    // for top_p = 1 (fp64 rounded need below Q) at most 2^10 units are left out: the last bin with
    // a mass, or one shortly before it
    int bin = min((fine_of(least) >> kFine) + 1, kBins - 1);
    if (!whole) {
      const float up = 4194304.f * (float)kMassScale / __ull2float_rn(total);  // a mass of 2^46
      const float skip = 4194304.f * 0.99f * __ull2float_rn(total - need) / __ull2float_rn(total) / a.V;
      each<2>(src, n, a.vec4, tid, [&](float x, int) {
        const float w = ex2((x - m) * a.inv_t2) * up;
        if (w > skip) atomicAdd(&sh.hist[fine_of(x) >> kFine], __float_as_uint(w + 8388608.f) - 0x4b000000u);
      });
      sync_all();
      uint32_t v = 0;
      for (unsigned i = 0; i < size; ++i) v += cluster.map_shared_rank(&sh.hist[0], i)[tid];
      static_assert(kBins == kVThreads && (1 << kFine) == kVThreads, "a thread per bin");
      uint32_t incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t w = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += w;
      }
      if (lane == 31) sh.wkey[warp] = incl;
      if (tid == 0) {
        sh.bin = kBins;
        sh.last_bin = 0;
      }
      __syncthreads();
      uint32_t w = sh.wkey[lane];
      w = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0u);
      incl += w;
      const float want = 4194304.f * __ull2float_rn(need) / __ull2float_rn(total);
      if (v && (float)incl >= want) atomicMin(&sh.bin, tid);
      if (v) atomicMax(&sh.last_bin, tid);
      __syncthreads();
      bin = min(sh.bin, sh.last_bin);
    }
    // ---- the exact sum above the bin and in it; the bin moves where the guess was off ---------
    u64 above = 0;
    int queued = 0;      // this thread's logits up to the bin, in queue[k][tid]
    bool listed = false;  // all of the CTA's are
#pragma unroll 1
    for (int tries = 0; tries < kBins; ++tries) {
      queued = 0;
      // fine_of(x) >> kFine <= bin, as the sum with 2^23 rounds; behind the end at is infinite
      const float lim = bin < kBins - 1 ? static_cast<float>((bin + 1) << kFine) - 0.5f : 3e38f;
      each<2>(src, n, a.vec4, tid, [&](float x, int) {
        // written at the queue's end in any case, which a branch would cost more than
        queue[min(queued, kQueue) * kVThreads + tid] = x;
        queued += (m - x) * a.bin_scale < lim;
      });
      listed = !__syncthreads_or(queued > kQueue);
      u64 more = 0, in = 0;
      auto add = [&](float x, int i) {
        const int at = fine_of(x) >> kFine;
        if (i >= n || at > bin) return;
        const u64 q = mass_of(x, m, a.inv_t);
        if (at < bin) {
          more += q;
        } else {
          in += q;
          const uint32_t c = atomicAdd(&sh.n_cand, 1u);
          if (c < kCand) {
            sh.cand_key[c] = logit_key(x);
            sh.cand_mass[c] = q;
          }
        }
      };
      if (listed) {
#pragma unroll 1
        for (int k = 0; k < queued; ++k) add(queue[k * kVThreads + tid], 0);
      } else {
        each<1>(src, n, a.vec4, tid, add);
      }
      more = warp_sum(more);
      in = warp_sum(in);
      if (lane == 0) {
        sh.red[warp] = more;
        sh.red2[warp] = in;
      }
      __syncthreads();
      if (warp == 0) {
        more = warp_sum(sh.red[lane]);
        in = warp_sum(sh.red2[lane]);
        if (lane == 0) {
          sh.cta_sum = more;
          sh.cta_sum2 = in;
        }
      }
      sync_all();
      above = cluster_total(cluster, &sh.cta_sum, size, lane);
      const u64 inside = cluster_total(cluster, &sh.cta_sum2, size, lane);
      const bool up = above >= need && bin > 0, down = above + inside < need && bin < kBins - 1;
      if (!up && !down) break;
      bin += up ? -1 : 1;
      sync_all();  // the sums have been read
      if (tid == 0) sh.n_cand = 0;
      __syncthreads();
    }
    // Ranks up to kCand listed tokens: tau is the key with sum(above it) < need <= sum(above
    // it) + its ties' sum.  `before`: what is above all of them.
    u64 at_tau = above, same = 0;
    auto rank_listed = [&](u64 before) {
      const uint32_t cnt = lane < (int)size ? *cluster.map_shared_rank(&sh.n_cand, lane) : 0u;
      const uint32_t all = __reduce_add_sync(0xffffffffu, min(cnt, kCand + 1u));
      if (all > kCand) return false;
      uint32_t first = cnt;
#pragma unroll
      for (int o = 1; o < kMaxCluster; o <<= 1) {
        const uint32_t w = __shfl_up_sync(0xffffffffu, first, o);
        if (lane >= o) first += w;
      }
      first -= cnt;  // entries of the CTAs before CTA `lane`
#pragma unroll 1
      for (unsigned i = 0; i < size; ++i) {
        const uint32_t f = __shfl_sync(0xffffffffu, first, i), c = __shfl_sync(0xffffffffu, cnt, i);
        if (tid < (int)c) {
          sh.all_key[f + tid] = cluster.map_shared_rank(sh.cand_key, i)[tid];
          sh.all_mass[f + tid] = cluster.map_shared_rank(sh.cand_mass, i)[tid];
        }
      }
      if (tid == 0) sh.found = 0;
      __syncthreads();
      if (tid < (int)all) {
        const uint32_t key = sh.all_key[tid];
        u64 over = before, tied = 0;
#pragma unroll 4
        for (uint32_t e = 0; e < all; ++e) {
          const uint32_t ke = sh.all_key[e];
          const u64 qe = sh.all_mass[e];
          if (ke > key) over += qe;
          if (ke == key) tied += qe;
        }
        if (over < need && need <= over + tied) {  // tied tokens write the same values
          sh.tau = key;
          sh.at_tau = over;
          sh.same = tied;
          sh.found = 1;
        }
      }
      __syncthreads();
      if (sh.found) {  // always, on finite input
        tau = sh.tau;
        at_tau = sh.at_tau;
        same = sh.same;
      }
      return true;
    };
    // f(l) for the bin's tokens in this CTA
    auto of_bin = [&](auto f) {
      if (listed) {
#pragma unroll 1
        for (int k = 0; k < queued; ++k) {
          const float x = queue[k * kVThreads + tid];
          if ((fine_of(x) >> kFine) == bin) f(x);
        }
      } else {
        each<1>(src, n, a.vec4, tid, [&](float x, int i) {
          if (i < n && (fine_of(x) >> kFine) == bin) f(x);
        });
      }
    };
    if (!rank_listed(above)) {
      // ---- many tokens in the bin: its fine bins, exactly -----------------------------------
      sh.fine[tid] = 0;
      __syncthreads();
      of_bin([&](float x) {
        const u64 q = mass_of(x, m, a.inv_t);
        if (q) atomicAdd(&sh.fine[fine_of(x) & ((1 << kFine) - 1)], q);
      });
      sync_all();
      u64 v = 0;
      for (unsigned i = 0; i < size; ++i) v += cluster.map_shared_rank(&sh.fine[0], i)[tid];
      u64 incl = warp_scan(v, lane);
      if (lane == 31) sh.red[warp] = incl;
      if (tid == 0) {  // kept only on non-finite input
        sh.bin = 0;
        sh.before = above;
        sh.n_cand = 0;
      }
      __syncthreads();
      incl += above + warp_sum(lane < warp ? sh.red[lane] : 0);
      if (incl - v < need && need <= incl) {
        sh.bin = tid;
        sh.before = incl - v;
      }
      __syncthreads();
      const int fine = sh.bin | bin << kFine;
      const u64 before = sh.before;
      at_tau = before;
      // ---- its tokens: one key, or a list of them to rank --------------------------------------
      uint32_t klo = 0xffffffffu, khi = 0;
      of_bin([&](float x) {
        if (fine_of(x) != fine) return;
        const uint32_t key = logit_key(x);
        klo = min(klo, key);
        khi = max(khi, key);
        const uint32_t at = atomicAdd(&sh.n_cand, 1u);
        if (at < kCand) {
          sh.cand_key[at] = key;
          sh.cand_mass[at] = mass_of(x, m, a.inv_t);
        }
      });
      klo = __reduce_min_sync(0xffffffffu, klo);
      khi = __reduce_max_sync(0xffffffffu, khi);
      if (lane == 0) {
        sh.wkey[warp] = klo;
        sh.wkey2[warp] = khi;
      }
      __syncthreads();
      if (warp == 0) {
        klo = __reduce_min_sync(0xffffffffu, sh.wkey[lane]);
        khi = __reduce_max_sync(0xffffffffu, sh.wkey2[lane]);
        if (lane == 0) {
          sh.cta_lo = klo;
          sh.cta_hi = khi;
        }
      }
      sync_all();
      klo = __reduce_min_sync(0xffffffffu, lane < (int)size ? *cluster.map_shared_rank(&sh.cta_lo, lane) : 0xffffffffu);
      khi = __reduce_max_sync(0xffffffffu, lane < (int)size ? *cluster.map_shared_rank(&sh.cta_hi, lane) : 0u);
      if (klo == khi) {
        tau = klo;
        same = cluster_total(cluster, &sh.fine[fine & ((1 << kFine) - 1)], size, lane);
      } else if (!rank_listed(before)) {
        // More than the list holds, and not one key: the keys between klo and khi are halved
        // until one is left, the largest with sum(keys >= it) >= need.
        auto sum_from = [&](uint32_t key, bool only) {
          u64 part = 0;
          of_bin([&](float x) {
            const uint32_t k = logit_key(x);
            if (fine_of(x) == fine && (only ? k == key : k >= key)) part += mass_of(x, m, a.inv_t);
          });
          part = block_sum(part, sh.red, lane, warp);
          sync_all();  // cta_sum has been read
          if (tid == 0) sh.cta_sum = part;
          sync_all();
          return cluster_total(cluster, &sh.cta_sum, size, lane);
        };
#pragma unroll 1
        while (klo < khi) {
          const uint32_t mid = klo + (khi - klo + 1) / 2;
          if (before + sum_from(mid, false) >= need) klo = mid;
          else khi = mid - 1;
        }
        tau = klo;
        at_tau = before + sum_from(tau, false);
        same = sum_from(tau, true);
        at_tau -= same;
      }
    }
    sync_all();  // lists have been read, cta_sum is written again below
    u64 q_tau = mass_of(key_logit(tau), m, a.inv_t);
    if (q_tau == 0) q_tau = 1;  // only on non-finite input
    ties = need > at_tau ? (need - at_tau + q_tau - 1) / q_tau : 1;
    nucleus = at_tau + ties * q_tau;
    cut = ties * q_tau < same;
  }

  // ---- the draft that this row decides on ---------------------------------------------
  const int d = t < a.T - 1 ? a.tokens[b * a.T + t + 1] : -1;
  u64 drafted = 0;
  if (d >= 0 && d < a.V) {
    const float l = base[d];
    const uint32_t key = logit_key(l);
    if (key > tau || (key == tau && !cut)) {
      drafted = mass_of(l, m, a.inv_t);
    } else if (key == tau) {  // in the nucleus if fewer than `ties` of its ties have lower ids
      u64 lower = 0;
      each<2>(src, n, a.vec4, tid, [&](float y, int i) { lower += logit_key(y) == tau && i < n && lo + i < d; });
      lower = block_sum(lower, sh.red, lane, warp);
      if (tid == 0) sh.cta_sum = lower;
      sync_all();
      if (cluster_total(cluster, &sh.cta_sum, size, lane) < ties) drafted = mass_of(l, m, a.inv_t);
    }
  }
  if (rank == 0 && tid == 0) {
    RowStat &o = a.stats[row];
    o.mass = nucleus;
    o.drafted = drafted;
    o.ties = ties;
    o.max_key = gmax;
    o.tau = tau;
    o.cut = cut;
  }
  sync_all();  // no CTA leaves while its shared memory is being read
}

struct DrawArgs {
  const float *logits, *draft;
  const int32_t *tokens;
  const double *uniforms;
  int B, T, V, slice, per, greedy;  // ids per CTA and per warp (a multiple of 32)
  double inv_t;
  const RowStat *stats;
  int32_t *out_tokens, *out_accepted;
};

// A row's nucleus: the mass of an id with logit l, `tied` of its ties before it.
struct RowMass {
  float m;
  uint32_t tau;
  u64 ties;
  double inv_t;
  bool cut;
  // + 2^52: a whole number, see whole_bits
  __device__ __forceinline__ double of(float l, u64 tied) const {
    const uint32_t key = logit_key(l);
    const bool in = key > tau || (key == tau && (!cut || tied < ties));
    const double q = fma(exp(((double)l - (double)m) * inv_t), kMassScale, kRound);
    return in ? q : kRound;
  }
};

// One cluster per sequence; warp w of CTA r holds ids r * slice + w * per, .. in id
// order, and keeps the masses that they are drawn with in shared memory: the sums
// of the segments give the one that holds the draw's point, and its warp scans it.
// Where a threshold cuts through tied tokens, their ranks are counted first.
__global__ void __launch_bounds__(kDrawThreads) verify_draw(const __grid_constant__ DrawArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  extern __shared__ u64 mass[];  // [kDrawWarps][per]
  __shared__ u64 seg[kDrawWarps];
  __shared__ uint32_t tie_a[kDrawWarps], tie_d[kDrawWarps];
  __shared__ u64 c_sum;
  __shared__ u64 c_tie[2];
  pdl_wait();
  pdl_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned rank = cluster.block_rank(), size = cluster.num_blocks();
  const int b = blockIdx.x / size, T = a.T;
  const RowStat *st = a.stats + (size_t)b * T;
  const RowStat *sd = a.stats + (size_t)a.B * T + (size_t)b * (T - 1);
  const int32_t *tok = a.tokens + (size_t)b * T;
  int32_t *out = a.out_tokens + (size_t)b * T;
  const bool lead = rank == 0 && tid == 0;

  // ---- how many drafts stand: a lane each ---------------------------------------------
  int s = 0;
  for (int s0 = 0; s0 < T; s0 += 32) {
    const int i = s0 + lane;
    bool ok = false;
    const int x = i < T - 1 ? tok[i + 1] : -1;
    if (x >= 0 && x < a.V) {
      if (a.greedy) {
        ok = x == st[i].best;
      } else {
        const double u = a.uniforms[(size_t)b * T + i];
        const double am = __ull2double_rn(st[i].mass), ax = __ull2double_rn(st[i].drafted);
        if (a.draft) {
          const double dm = __ull2double_rn(sd[i].mass), dx = __ull2double_rn(sd[i].drafted);
          ok = __dmul_rn(u, __dmul_rn(dx, am)) < __dmul_rn(ax, dm);
        } else {
          ok = __dmul_rn(u, am) < ax;
        }
      }
    }
    const unsigned bad = ~__ballot_sync(0xffffffffu, ok);
    if (bad) {  // lane T - 1 at the latest
      s = s0 + __ffs(bad) - 1;
      break;
    }
  }
  if (rank == 0) {
    for (int i = tid; i < T; i += kDrawThreads)
      if (i != s) out[i] = i < s ? tok[i + 1] : -1;
    if (tid == 0) a.out_accepted[b] = s + 1;
  }
  if (a.greedy) {
    if (lead) out[s] = st[s].best;
    return;
  }

  const int x = s < T - 1 ? tok[s + 1] : -1;
  const bool residual = x >= 0 && x < a.V;  // a draft that did not stand
  const bool with_d = residual && a.draft;
  const float *la = a.logits + ((size_t)b * T + s) * a.V;
  const float *ld = with_d ? a.draft + ((size_t)b * (T - 1) + s) * a.V : la;
  const RowMass A{key_logit(st[s].max_key), st[s].tau, st[s].ties, a.inv_t, st[s].cut != 0};
  const RowMass D = with_d ? RowMass{key_logit(sd[s].max_key), sd[s].tau, sd[s].ties, a.inv_t, sd[s].cut != 0} : A;
  const double ra = with_d ? kMassScale / __ull2double_rn(st[s].mass) : 0.0;
  const double rd = with_d ? kMassScale / __ull2double_rn(sd[s].mass) : 0.0;
  const int lo = (int)rank * a.slice, hi = min(a.V, lo + a.slice);
  const int s0 = min(hi, lo + warp * a.per), s1 = min(hi, s0 + a.per);
  u64 *mine = mass + warp * a.per;

  // ---- ties before each segment, where they matter ----------------------------------------
  const bool cut = A.cut || (with_d && D.cut);
  u64 before_a = 0, before_d = 0;
  if (cut) {
    uint32_t ca = 0, cd = 0;
#pragma unroll 4
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
      for (int w = 0; w < kDrawWarps; ++w) {
        c_tie[0] += tie_a[w];
        c_tie[1] += tie_d[w];
      }
    }
    cluster.sync();
    for (unsigned i = 0; i < rank; ++i) {
      const u64 *o = cluster.map_shared_rank(c_tie, i);
      before_a += o[0];
      before_d += o[1];
    }
    for (int w = 0; w < warp; ++w) {
      before_a += tie_a[w];
      before_d += tie_d[w];
    }
  }

  // ---- the masses and their sum: the residual's, and the target's own where that is zero ----
  for (int round = residual ? 0 : 1; round < 2; ++round) {
    const bool res = round == 0, two = res && with_d;
    u64 ta = before_a, td = before_d, sum = 0;
    constexpr int kBatch = 8;  // loads in flight per lane and row
#pragma unroll 1
    for (int i0 = s0; i0 < s1; i0 += 32 * kBatch) {
      float va[kBatch], vd[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + 32 * k + lane;
        va[k] = i < s1 ? la[i] : -INFINITY;  // no mass
        vd[k] = two && i < s1 ? ld[i] : -INFINITY;
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + 32 * k + lane;
        if (i0 + 32 * k >= s1) break;
        u64 na = ta, nd = td;
        if (cut) {
          const unsigned ea = __ballot_sync(0xffffffffu, i < s1 && logit_key(va[k]) == A.tau);
          const unsigned ed = __ballot_sync(0xffffffffu, two && i < s1 && logit_key(vd[k]) == D.tau);
          na += __popc(ea & ((1u << lane) - 1u));
          nd += __popc(ed & ((1u << lane) - 1u));
          ta += __popc(ea);
          td += __popc(ed);
        }
        double q = A.of(va[k], na);
        if (two) {
          // each share rounded to a whole number, as its mass times 2^46 / sum
          const double p = __dadd_rn(__dmul_rn(q - kRound, ra), kRound), o = __dadd_rn(__dmul_rn(D.of(vd[k], nd) - kRound, rd), kRound);
          q = p > o ? kRound + (p - o) : kRound;
        } else if (res && i == x) {
          q = kRound;
        }
        const u64 w = whole_bits(q);
        if (i < s1) mine[i - s0] = w;
        sum += w;
      }
    }
    sum = warp_sum(sum);
    if (lane == 0) seg[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      const u64 c = warp_sum(lane < kDrawWarps ? seg[lane] : 0);
      if (lane == 0) c_sum = c;
    }
    cluster.sync();
    const u64 c = lane < (int)size ? *cluster.map_shared_rank(&c_sum, lane) : 0;
    const u64 total = warp_sum(c);
    u64 before = warp_sum(lane < (int)rank ? c : 0);
    if (res && total == 0) {
      cluster.sync();  // c_sum and seg are written again
      continue;
    }
    before += warp_sum(lane < warp ? seg[lane] : 0);
    // ---- the draw: the segment that holds y, then the id in it -------------------------
    double uu = a.uniforms[(size_t)b * T + T - 1];
    if (!(uu >= 0.0)) uu = 0.0;
    u64 y = (u64)floor(__dmul_rn(fmin(uu, 1.0), __ull2double_rn(total)));
    if (y >= total) y = total > 0 ? total - 1 : 0;
    if (lead && total == 0) out[s] = 0;  // only on rows without a finite logit
    if (before <= y && y < before + sum) {
      u64 run = before;
#pragma unroll 1
      for (int i0 = s0; i0 < s1; i0 += 32) {
        const u64 cum = run + warp_scan(i0 + lane < s1 ? mine[i0 - s0 + lane] : 0, lane);
        const unsigned hit = __ballot_sync(0xffffffffu, cum > y);
        if (hit) {
          if (lane == __ffs(hit) - 1) out[s] = i0 + lane;
          break;
        }
        run = __shfl_sync(0xffffffffu, cum, 31);
      }
    }
    break;
  }
  cluster.sync();  // no CTA leaves while its shared memory is being read
}

// Sets a kernel's dynamic shared memory limit where a launch needs more than so far.
template <typename K>
cudaError_t allow_smem(K *kernel, size_t bytes, std::atomic<size_t> (&set)[kVerifyDevices]) {
  if (bytes <= 28 * 1024) return cudaSuccess;  // beside up to 17 KB of static shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kVerifyDevices) return cudaErrorInvalidDevice;
  if (bytes <= set[dev].load(std::memory_order_acquire)) return cudaSuccess;
  static std::mutex mu;
  std::lock_guard<std::mutex> lock(mu);
  if (bytes > set[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    set[dev].store(bytes, std::memory_order_release);
  }
  return cudaSuccess;
}

template <typename Args>
cudaError_t launch(void (*kernel)(Args), int grid, int cluster, int threads, size_t smem, cudaStream_t st,
                   const Args &args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid) * cluster);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

// Shared memory of verify_rows: with a queue per thread, and with a row's cache.
size_t rows_smem(bool queue, bool cache) {
  return sizeof(RowsShared) + (queue ? sizeof(float) * (kQueue + 1) * kVThreads : 0) + (cache ? sizeof(float) * kCache : 0);
}

std::atomic<size_t> g_rows_smem[kVerifyDevices];

// Clusters of verify_rows that the current device holds at once, with the cache's shared
// memory: a CTA takes an SM, and a cluster its SMs from one group of them, so that fewer
// than n_sm / C may fit.  Asked once per device and size.
cudaError_t clusters_at_once(int log2c, int dev, int *n) {
  static std::atomic<int> known[kVerifyDevices][4];
  static_assert((1 << 3) == kMaxCluster);
  if (dev < 0 || dev >= kVerifyDevices) return cudaErrorInvalidDevice;
  *n = known[dev][log2c].load(std::memory_order_relaxed);
  if (*n > 0) return cudaSuccess;
  const size_t smem = rows_smem(true, true);
  cudaError_t e = allow_smem(verify_rows, smem, g_rows_smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 1u << log2c;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(1u << log2c);
  cfg.blockDim = dim3(kVThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(n, verify_rows, &cfg);
  if (e != cudaSuccess) return e;
  if (*n < 1) *n = 1;
  known[dev][log2c].store(*n, std::memory_order_relaxed);
  return cudaSuccess;
}

// CTAs per row.  The rows' clusters run in ceil(rows / clusters at once) turns.  A turn
// takes a fixed time and a time that goes with a CTA's share of the row: 15 us + 0.7 ns
// a logit where a nucleus is searched, 8 us + 0.3 ns a logit where the whole
// distribution stands; a doubling of the cluster costs its barriers 2 us or 1 us.
// Measured with 1 | 2 | 4 | 8 CTAs, nucleus 0.9: 248 rows of 64000 152 | 183 | 253 |
// 464 us, 104 of 32000 44 | 58 | 90 | 167, 28 of 20000 31 | 29 | 28 | 51, 16 of 32000
// 42 | 33 | 29 | 51, 7 of 64000 88 | 64 | 50 | 46, 10 of 5000 19 | 21 | 21 | 26; whole
// distribution: 72 of 32000 24 | 20 | 33 | 49, 8 of 32000 21 | 17 | 15 | 15.
cudaError_t cluster_for(int rows, int V, bool nucleus, int *best) {
  const double fixed = nucleus ? 15.0 : 8.0, logit = nucleus ? 0.7e-3 : 0.3e-3, doubling = nucleus ? 2.0 : 1.0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  double least = 1e30;
  for (int i = 0; e == cudaSuccess && (1 << i) <= kMaxCluster; ++i) {
    int n = 1;
    e = clusters_at_once(i, dev, &n);
    const double us = static_cast<double>((static_cast<long long>(rows) + n - 1) / n) * (fixed + logit * V / (1 << i)) + doubling * i;
    if (us < least) {
      least = us;
      *best = 1 << i;
    }
  }
  return e;
}

}  // namespace

size_t verify_sample_workspace(int B, int T) { return sizeof(RowStat) * static_cast<size_t>(B) * (2 * static_cast<size_t>(T) - 1); }

cudaError_t launch_verify_sample(const VerifySample &v, cudaStream_t st) {
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
  int cr = 1;
  cudaError_t e = cluster_for(rows, v.V, !greedy && v.top_p < 1.0f, &cr);
  if (e != cudaSuccess) return e;
  r.slice = ((v.V + cr - 1) / cr + 3) & ~3;
  r.vec4 = v.V % 4 == 0 && (reinterpret_cast<uintptr_t>(v.logits) & 15) == 0 &&
           (!draft || (reinterpret_cast<uintptr_t>(v.draft_logits) & 15) == 0);
  r.greedy = greedy;
  r.inv_t = inv_t;
  r.top_p = v.top_p;
  // masses are zero beyond max - l = 33 T; bins of equal width cover that range
  const double most = 3e38;  // a temperature near zero: still finite in fp32
  r.bin_scale = greedy ? 0.f : static_cast<float>(std::min((kBins << kFine) * inv_t / 33.0, most));
  r.inv_t2 = static_cast<float>(std::min(inv_t * 1.4426950408889634, most));  // log2(e)
  r.stats = stats;
  r.cached = !greedy && v.top_p < 1.0f && r.slice <= kCache;
  const size_t smem_rows = rows_smem(!greedy, r.cached);
  e = allow_smem(verify_rows, smem_rows, g_rows_smem);
  if (e == cudaSuccess) e = launch(verify_rows, rows, cr, kVThreads, smem_rows, st, r);
  if (e != cudaSuccess) return e;

  DrawArgs d{};
  d.logits = v.logits;
  d.draft = r.draft;
  d.tokens = v.tokens;
  d.uniforms = v.uniforms;
  d.B = v.B;
  d.T = v.T;
  d.V = v.V;
  // two ids a thread or more; clusters of 16 were slower (20 us against 17 for 8 draws of
  // 64000: not all of them resident)
  int cd = 1;
  while (!greedy && cd < kMaxCluster && v.V > cd * 2 * kDrawThreads) cd *= 2;
  d.per = ((v.V + cd * kDrawWarps - 1) / (cd * kDrawWarps) + 31) & ~31;
  d.slice = d.per * kDrawWarps;
  d.greedy = greedy;
  d.inv_t = inv_t;
  d.stats = stats;
  d.out_tokens = v.out_tokens;
  d.out_accepted = v.out_accepted;
  static std::atomic<size_t> set[kVerifyDevices];
  const size_t smem = greedy ? 0 : sizeof(u64) * d.slice;
  e = allow_smem(verify_draw, smem, set);
  return e != cudaSuccess ? e : launch(verify_draw, v.B, cd, kDrawThreads, smem, st, d);
}

}  // namespace mk
