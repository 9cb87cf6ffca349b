// Draws from rows of logits, and their k largest.
//
// The order of a row's tokens is that of common.cuh: falling logits, equal ones by rising id.
// Every filter keeps a prefix of it, so the kept set is known by its border, the last (logit,
// id) kept:
//   top_k   the border is the k-th of the order
//   top_p   the first whose mass, with all before it, reaches p times the mass after top_k
//   min_p   the last whose weight is at least min_p times the largest's
// and the token is the first by id whose mass, with all kept ids below it, exceeds u times the
// kept mass (weights: rows.cuh).
//
// Few rows, or rows that one CTA's shared memory holds: each is held by a cluster of 1 to 8 CTAs
// (76 KB of each for 151936 fp32 logits in 8, two CTAs a SM), read from memory once, and every
// later pass is one over shared memory.  CTAs tell each other by stores into all of their shared
// memories before a barrier of the cluster, and read only their own after it.  Many long rows:
// one CTA each, which reads its row again for every pass (the 128 KB that two CTAs have in flight
// keep the memory busy where barriers of clusters did not: a greedy token of 2048 fp32 rows 503 us
// held by clusters, 198 by single CTAs, 184 the floor).  Where their settings differ, the rows
// that no list serves are begun first.
//
//   top_k, and the k largest: a list of what is not below the least of some groups' maxima; with
//     at least k groups it holds the k largest.  Single CTAs look at a ninth of the row first and
//     list what is not below a bound that some twice k will reach, in the pass that reads the
//     row (the 64 largest of 2048 fp32 rows: 494 us in two passes, 300 in one).  One CTA sorts the
//     list, and does the rest alone.
//   nothing but a draw: single CTAs sum the weights in the pass that reads the row, in units that
//     the look at its ninth gives, and rise by octaves where that was too low.
//   top_p: masses by 2048 classes of weights, 1/64 of an octave wide, off by 2^-13 of themselves
//     (32-bit sums by shared memory atomics); then, in one pass, the exact mass, that of the
//     classes surely kept, and a list of the few classes that the border may lie in, or for bf16
//     the counts of their logits.  The draw takes its sums by warp from that pass.  (2048 fp32 rows,
//     p 0.95: 1.25 ms, 95 instructions for 32 logits, at 2.5 a clock and SM: bound by their issue.)
//   Where a list does not do (more entries than it holds, many equal logits): histograms of the
//     logits' order keys, 2048 bins at a time, with exact masses.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "rows.cuh"
#include "tokens.h"

namespace dspark {

namespace {

// floor(x mass) for 0 <= x < 1, in whole numbers; `rest`: whether that cut anything off.
__device__ __forceinline__ u64 share_of(float x, u64 mass, bool& rest) {
  const u64 f = (u64)(x * 9223372036854775808.f) * 2;            // (x in units of 2^-64)
  rest = f * mass != 0;
  return __umul64hi(f, mass);
}
__device__ __forceinline__ u64 draw_target(float u, u64 mass) {
  bool rest;
  return u >= 1.f ? mass - 1 : u > 0.f ? share_of(u, mass, rest) : 0ull;
}
__device__ __forceinline__ void write_token(const RowArgs& a, int t, int id, u64 x, u64 mass) {
  a.tokens[t] = id;
  if (a.logp) a.logp[t] = mass > x ? -log1pf((float)(mass - x) / (float)x) : 0.f;
}
__device__ __forceinline__ u64 share_up(float x, u64 mass) {
  bool rest;
  const u64 s = share_of(x, mass, rest);
  return s + rest;
}
__device__ __forceinline__ u64 top_p_target(float p, u64 mass) {
  return max(1ull, p > 0.f ? share_up(p, mass) : 0ull);
}
__device__ __forceinline__ u64 min_p_weight(float p, u64 top) {
  return p >= 1.f ? top : p > 0.f ? share_up(p, top) : 0ull;
}

// The first CTA alone: the draw from the list's n best entries, which hold the k first of the
// row's order (k entries or all there are).
template <typename E, bool HELD, int NT>
__device__ __forceinline__ void draw_listed(const RowArgs& a, Row<E, HELD, NT>& row, int t, int n,
                                            const Weights& w, float top_p, float min_p) {
  auto& sh = row.sh;
  const u64 least = min_p_weight(min_p, w(w.m));
  if (n <= 32) {
    // one warp, without barriers
    if (threadIdx.x >= 32) return;
    const int lane = threadIdx.x;
    const u64 e = lane < n ? sh.list[lane] : 0ull;
    const uint32_t id = 0xFFFFFFFFu - (uint32_t)e;
    u64 x = w(value_of(lane < n ? (uint32_t)(e >> 32) : kNoKey));
    x = lane < n ? x : 0ull;
    u64 in = warp_scan(x), all = __shfl_sync(0xFFFFFFFFu, in, 31);
    if (top_p < 1.f && in - x >= top_p_target(top_p, all)) x = 0;
    if (x < least) x = 0;
    all = warp_sum(x);
    u64 run = 0;
#pragma unroll 8
    for (int o = 0; o < n; ++o) {
      const u64 y = __shfl_sync(0xFFFFFFFFu, x, o);
      run += __shfl_sync(0xFFFFFFFFu, id, o) < id ? y : 0ull;
    }
    const u64 target = draw_target(a.uniform[t], all);
    if (target >= run && target < run + x) write_token(a, t, (int)id, x, all);
    return;
  }
  constexpr int kEach = Row<E, HELD, NT>::kEach, kThreads = NT;
  __shared__ int s_n;
  u64 x[kEach], all;
  if (top_p < 1.f) {
    const int each = row.list_each(n);
    u64 run = row.list_weights(n, w, [](u64 e) { return (uint32_t)(e >> 32); }, x, all);
    const u64 target = top_p_target(top_p, all);
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
      if (x[q] > 0 && run < target && run + x[q] >= target) s_n = (int)threadIdx.x * each + q + 1;
      run += x[q];
    }
    __syncthreads();
    n = s_n;
  }
  // the kept ones by id: (~id, key)
  for (int i = threadIdx.x; i < n; i += kThreads) sh.list[i] = sh.list[i] << 32 | sh.list[i] >> 32;
  __syncthreads();
  row.sort_list(n);
  u64 run = row.list_weights(n, w, [](u64 e) { return (uint32_t)e; }, x, all);
  if (least > 0) {
    u64 s = 0;
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
      x[q] = x[q] >= least ? x[q] : 0ull;
      s += x[q];
    }
    run = row.scan(s, all);
  }
  const int each = row.list_each(n);
  const u64 target = draw_target(a.uniform[t], all);
#pragma unroll
  for (int q = 0; q < kEach; ++q) {
    if (target >= run && target < run + x[q])
      write_token(a, t, (int)(0xFFFFFFFFu - (uint32_t)(sh.list[threadIdx.x * each + q] >> 32)), x[q],
                  all);
    run += x[q];
  }
}

template <typename E, bool TOP, bool HELD, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) rows_kernel(const RowArgs a) {
  extern __shared__ uint4 s_held[];
  using R = Row<E, HELD, NT>;
  constexpr int kList = R::kList, kThreads = NT, kWarps = NT / 32;
  __shared__ typename R::Sh sh;
  constexpr int VE = Vec<E>::n;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  R row(sh);
  const int rank = row.rank(), size = row.size(), t = HELD ? blockIdx.x / size : blockIdx.x % a.T;
  const int per = ((a.V + size - 1) / size + VE - 1) / VE * VE;
  auto& part = row.part;
  {
    part.i0 = min(a.V, rank * per);
    part.n = min(a.V, part.i0 + per) - part.i0;
    const E* g = (const E*)a.logits + (long long)t * a.ld + part.i0;
    part.lead = (int)((uintptr_t)g / sizeof(E) % VE);
    part.g = g - part.lead;
    part.nv = part.n > 0 ? (part.lead + part.n + VE - 1) / VE : 0;
    part.share = (part.nv + kWarps - 1) / kWarps;
    part.v0 = min(part.nv, warp * part.share);
    part.v1 = min(part.nv, part.v0 + part.share);
    part.held = s_held;
  }

  // the settings of this row
  float tau = a.temperature, top_p = a.top_p, min_p = a.min_p;
  int K = a.top_k;
  if (TOP) {
    tau = 1.f;
    K = a.k;
  } else {
    if (a.row_temperature) tau = a.row_temperature[t];
    if (a.row_top_p) top_p = a.row_top_p[t];
    if (a.row_min_p) min_p = a.row_min_p[t];
    if (a.row_top_k) K = a.row_top_k[t];
  }
  if (K <= 0 || K > a.V) K = a.V;
  const bool greedy = !TOP && (!(tau > 0.f) || K == 1);
  const bool cut_k = !greedy && K < a.V, cut_p = !TOP && !greedy && top_p < 1.f;
  const bool classes = cut_p && !cut_k;
  // (a row that no list serves takes ten times as long as one that does: those are begun first)
  if (!HELD && a.long_first && (!greedy && !cut_k) != (blockIdx.x < a.T)) return;
  if (tid == 0) {
    sh.count = sh.claim = 0;
    sh.least_id = 0xFFFFFFFFu;
  }
  if (classes)
    for (int i = tid; i < kBins; i += kThreads) sh.mass[i] = 0;
  if (tid < kWarps) sh.extra[tid] = 0;
  row.started();

  // the row, its maximum, and for the k largest its sum of exponentials: 2^(z log2(e) - ref), ref
  // the rounded log2(e) times a logit that the running maximum is at most 11 above.  (A sum that
  // takes every maximum as its reference is scaled, and rounded, at every vector of a rising row.)
  float top = -INFINITY, ref = 0.f, near_to = -INFINITY;
  LongSum sum;
  // one CTA a row, and rows long enough: one pass does the rest too, where a look at a part of
  // the row tells what to expect
  const bool ahead = !HELD && !greedy && !classes && part.share >= 3 * 32 * kRing && (K <= 256 || !(TOP || cut_k));
  Weights ahead_w = {};
  u64 ahead_sum = 0;
  int seen_octave = 0;
  uint32_t first = 0xFFFFFFFFu;                  // greedy: the lowest id of the maximum
  auto look = [&](int v, const uint4& x) {
    const float best = fmaxf(top, Vec<E>::top(x));
    if (TOP && a.lse) {
      if (best > near_to) {
        const float r = best * kLog2e;
        sum.scale(near_to > -INFINITY ? fast_exp2(ref - r) : 0.f);
        ref = r;
        near_to = best + 11.f;
      }
      float z[VE], s[4] = {};
      Vec<E>::get(x, z);
#pragma unroll
      for (int j = 0; j < VE; ++j) s[j % 4] += fast_exp2(fmaf(z[j], kLog2e, -ref));
      sum.add((s[0] + s[1]) + (s[2] + s[3]), chain_ends(v));
    }
    if (!TOP && greedy && best > top) {
      float z[VE];
      Vec<E>::get(x, z);
#pragma unroll
      for (int j = VE - 1; j >= 0; --j)
        if (z[j] == best) first = (uint32_t)part.id(v, j);
    }
    top = best;
  };
  if (HELD) {
    // a quarter of the warp's vectors at a time while the others are on their way
    const int step = (part.v1 - part.v0 + 127) / 128 * 32;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int end = min(part.v1, part.v0 + (q + 1) * step);
      for (int v = part.v0 + q * step + lane; v < end; v += 32) part.copy(v, s_held + v);
      part.copied();
    }
    auto quarter = [&](int q) {
      const int end = min(part.v1, part.v0 + (q + 1) * step);
#pragma unroll 2
      for (int v = part.v0 + q * step + lane; v < end; v += 32) look(v, s_held[v]);
    };
    part.template arrived<3>();
    quarter(0);
    part.template arrived<2>();
    quarter(1);
    part.template arrived<1>();
    quarter(2);
    part.template arrived<0>();
    quarter(3);
  } else if (!ahead) {
    part.each(look);
  } else {
    // a ninth or so of the row first, spread over it: what to expect of the rest
    const int some = min(part.v1, part.v0 + 32 * kRing);
    float best = -INFINITY;
    part.each(part.v0, some, [&](int, const uint4& x) { best = fmaxf(best, Vec<E>::top(x)); });
    // 32 maxima: of warps, or of half ones
    constexpr int kOfLanes = kWarps;
    float m = best;
#pragma unroll
    for (int o = 1; o < kOfLanes; o *= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (lane % kOfLanes == 0) sh.half_top[tid / kOfLanes] = m;
    __syncthreads();
    m = sh.half_top[lane];
    const float seen = warp_top(m);
    if (TOP || cut_k) {
      // The r-th largest of the 32 maxima: of n draws of a share f of the row, some
      // c = -32 ln(1 - r / 32) are not below it, and c / f of the row.  c is chosen four standard
      // deviations above K f, so that K are hardly ever missed.
      const float f = fminf(1.f, 32.f * kRing / (float)part.share), kf = (float)K * f;
      const float c = kf + 4.f * sqrtf(kf) + 4.f;
      const int r = min(32, (int)(32.f * (1.f - fast_exp2(c * (-kLog2e / 32.f)))) + 1);
      int above = 0;
#pragma unroll
      for (int o = 0; o < 32; ++o) {
        const float x = __shfl_sync(0xFFFFFFFFu, m, o);
        above += x > m || (x == m && o < lane);
      }
      const unsigned at = __ballot_sync(0xFFFFFFFFu, above == r - 1);
      const float z_lo = fmaxf(__shfl_sync(0xFFFFFFFFu, m, __ffs(at) - 1), value_of(kNoKey + 1));
      int n = 0;
      part.each([&](int v, const uint4& raw) {
        look(v, raw);
        n += row.put_from(v, raw, z_lo);
      });
      row.put_count(n);
    } else {
      ahead_w.set(seen, tau, a.V);             // (nothing seen: far)
      seen_octave = ahead_w.octave;
      if (!ahead_w.far) {
        part.each([&](int v, const uint4& raw) {
          if (Vec<E>::top(raw) > ahead_w.z_cap) ahead_sum >>= min(63, ahead_w.raise(Vec<E>::top(raw)));
          look(v, raw);
          float z[VE];
          Vec<E>::get(raw, z);
#pragma unroll
          for (int j = 0; j < VE; ++j) ahead_sum += ahead_w(z[j]);
        });
      } else {
        part.each(look);
      }
    }
  }
  // the least of the groups' maxima, of at least K groups of threads where there are as many
  uint32_t key = key_of(top), low = 0;
  {
    const int want = ((TOP || cut_k ? K : 1) + size - 1) / size;  // of this CTA
    int lanes = 32, warps = kWarps;
    while (warps > 1 && kWarps / warps < want) warps /= 2;
    while (lanes > 1 && kWarps * (32 / lanes) < want) lanes /= 2;
    uint32_t m = key;
    for (int o = 1; o < lanes; o *= 2) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const uint32_t least = __reduce_min_sync(0xFFFFFFFFu, m);
    if (lane == 0) sh.warp_key[warp] = least;                     // (lanes = 32: the maximum)
    const uint32_t best = __reduce_max_sync(0xFFFFFFFFu, key);
    if (lane == 0) sh.warp_top[warp] = best;
    __syncthreads();
    low = 0xFFFFFFFFu;
    uint32_t group = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      key = max(key, sh.warp_top[w]);
      // (merged warps hold maxima; single ones the least of theirs)
      group = max(group, sh.warp_key[w]);
      if ((w + 1) % warps == 0) {
        low = min(low, group);
        group = 0;
      }
    }
    // (sums are told with their reference)
    float all = 0.f, cta_ref = 0.f;
    if (TOP && a.lse) {
      cta_ref = value_of(key) * kLog2e;
      float s = top > -INFINITY ? sum.value() * fast_exp2(ref - cta_ref) : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      __syncthreads();
      if (lane == 0) sh.warp_f[warp] = s;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) all += sh.warp_f[w];
    }
    row.all_started();
    row.tell(__float_as_uint(all), 0, key, low);
    row.sync();
    const Slot* s = row.told();
    for (int r = 0; r < size; ++r) {
      key = max(key, s[r].c);
      low = min(low, s[r].d);
    }
    if (TOP && a.lse) {
      const float top_ref = value_of(key) * kLog2e;
      float total = 0.f;
      for (int r = 0; r < size; ++r)
        if (s[r].c > kNoKey)
          total += __uint_as_float((uint32_t)s[r].a) *
                   fast_exp2(value_of(s[r].c) * kLog2e - top_ref);
      const float m = value_of(key);
      const bool plain = fabsf(top_ref) < INFINITY && total > 0.f && total < INFINITY;
      if (key > kNoKey && !plain) {
        // a logit is no number, or so large that the reference is none: the sum of those that are,
        // from their distances
        LongSum own;
        part.each([&](int v, const uint4& raw) {
          float z[VE], s[4] = {};
          Vec<E>::get(raw, z);
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            const float x = z[j] == m ? 0.f : fmaxf(z[j] - m, -150.f);
            s[j % 4] += z[j] > -INFINITY ? fast_exp2(x * kLog2e) : 0.f;
          }
          own.add((s[0] + s[1]) + (s[2] + s[3]), chain_ends(v));
        });
        float s1 = own.value();
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s1 += __shfl_xor_sync(0xFFFFFFFFu, s1, o);
        __syncthreads();
        if (lane == 0) sh.warp_f[warp] = s1;
        __syncthreads();
        float cta = 0.f;
        for (int w = 0; w < kWarps; ++w) cta += sh.warp_f[w];
        row.tell(__float_as_uint(cta), 0, 0, 0);
        row.sync();
        const Slot* o = row.told();
        total = 0.f;
        for (int r = 0; r < size; ++r) total += __uint_as_float((uint32_t)o[r].a);
      }
      if (rank == 0 && tid == 0)
        a.lse[t] = key <= kNoKey ? -INFINITY
                   : plain       ? (top_ref + log2f(total)) * 0.693147181f
                                 : m + logf(total);
    }
  }
  const Border every = {kNoKey, -1};             // all but -infinity
  low = max(low, kNoKey + 1);
  if (key <= kNoKey) {
    // nothing to choose from
    if (rank != 0) return;
    if (!TOP && tid == 0) {
      a.tokens[t] = -1;
      if (a.logp) a.logp[t] = -INFINITY;
    }
    if (TOP)
      for (int i = tid; i < a.k; i += kThreads) {
        a.ids[(size_t)t * a.k + i] = -1;
        a.values[(size_t)t * a.k + i] = -INFINITY;
      }
    return;
  }
  if (greedy) {
    // the lowest id of the largest logit
    const uint32_t id = __reduce_min_sync(0xFFFFFFFFu, key_of(top) == key ? first : 0xFFFFFFFFu);
    if (lane == 0 && id != 0xFFFFFFFFu) atomicMin(row.of(&sh.least_id, 0), id);
    row.sync();
    if (rank == 0 && tid == 0) {
      a.tokens[t] = (int)sh.least_id;
      if (a.logp) a.logp[t] = 0.f;
    }
    return;
  }
  Weights w;
  if (!TOP) w.set(value_of(key), tau, a.V);

  Border b = every;
  if (TOP || cut_k) {
    if (ahead) {
      // (where the look was misleading: once more, with what is now known)
      const int n = (int)sh.count;
      if (n > kList || n < K) {
        __syncthreads();
        if (tid == 0) sh.count = sh.claim = 0;
        __syncthreads();
        row.collect(value_of(low));
      }
    } else {
      row.collect(value_of(low));
    }
    row.sync();
    int n = (int)sh.count;
    if (n <= kList && (n >= K || low == kNoKey + 1)) {
      if (rank != 0) return;
      row.sort_list(n);
    } else {
      const bool some = row.template locate<false>((u64)K, b, n >= K ? low : kNoKey, key, 0, w);
      if (TOP) {
        if (tid == 0) sh.count = sh.claim = 0;
        row.sync();
        row.collect(some ? b.key : kNoKey + 1, key, b);
        row.sync();
        if (rank != 0) return;
        n = (int)sh.count;
        row.sort_list(n);
      } else {
        n = -1;
      }
    }
    if (TOP) {
      for (int i = tid; i < a.k; i += kThreads) {
        const u64 e = i < n ? sh.list[i] : 0ull;
        a.ids[(size_t)t * a.k + i] = i < n ? (int)(0xFFFFFFFFu - (uint32_t)e) : -1;
        a.values[(size_t)t * a.k + i] = i < n ? value_of((uint32_t)(e >> 32)) : -INFINITY;
      }
      return;
    }
    if (n >= 0) {
      draw_listed(a, row, t, min(n, K), w, top_p, min_p);
      return;
    }
  }

  auto kept = [&](int v, const uint4& raw, u64 (&x)[VE]) {
    if (!__any_sync(0xFFFFFFFFu, Vec<E>::top(raw) >= value_of(b.key))) {
#pragma unroll
      for (int j = 0; j < VE; ++j) x[j] = 0;
      return;
    }
    float z[VE];
    Vec<E>::get(raw, z);
#pragma unroll
    for (int j = 0; j < VE; ++j) x[j] = w(z[j]);
    if (b.key == kNoKey) return;
#pragma unroll
    for (int j = 0; j < VE; ++j)
      if (!b.keeps(key_of(z[j]), part.id(v, j))) x[j] = 0;
  };
  u64 before = 0;
  const u64 least = min_p_weight(min_p, w(w.m));
  if (cut_p) {
    bool found = false;
    u64 target = 0, above = 0;
    if (classes) {
      // masses of the classes of weights in units of 2^-bits of a class's
      const Classes cl = {w.m, w.c_hi * 64.f};
      const int bits = min(16, __clz(max(1, a.V - 1)) - 1);
      part.each([&](int, const uint4& raw) { row.add_classes(raw, cl, (float)(1 << bits)); });
      __syncthreads();
      if (rank != 0)
        for (int i = tid; i < kBins; i += kThreads)
          if (sh.mass[i]) atomicAdd(row.of(&sh.mass[i], 0), sh.mass[i]);
      row.sync();
      if (rank == 0) {
        // the classes that the border may lie in
        constexpr int kOf = kBins / kThreads;
        float x[kOf], s = 0.f, all;
#pragma unroll
        for (int q = 0; q < kOf; ++q) {
          const int i = tid * kOf + q;
          x[q] = (float)sh.mass[i] * fast_exp2((float)i * (-1.f / 64.f));
          s += x[q];
        }
        float run = row.scan(s, all);
        const float slack = fmaxf(ldexpf(1.f, 2 - bits), 1e-5f);
        const float lo = top_p * all * (1.f - slack);
        const float hi = top_p * (all + (float)a.V * fast_exp2(-31.9f) * (float)(1 << bits)) * (1.f + slack);
        if (tid == 0) {
          sh.warp_key[0] = kBins;
          sh.warp_key[1] = kBins;
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kOf; ++q) {
          run += x[q];
          if (run >= lo) atomicMin(&sh.warp_key[0], (uint32_t)(tid * kOf + q));
          if (run >= hi) atomicMin(&sh.warp_key[1], (uint32_t)(tid * kOf + q));
        }
        __syncthreads();
        if (tid < size)
          *row.of(&sh.slot[row.phase % kSlots][0], tid) = {0, 0, sh.warp_key[0], sh.warp_key[1]};
      }
      row.sync();
      const Slot range = row.told()[0];
      const int c0 = (int)range.c, c1 = (int)range.d;
      // the logits of the range: the largest of class c0 or worse, the least of c1 or better
      uint32_t hi_key, lo_key;
      {
        uint32_t no = kNoKey;
        lo_key = key;
        while (lo_key - no > 1) {
          const uint32_t k = no + (lo_key - no) / 2;
          (Classes::of(cl.step(value_of(k))) <= c1 ? lo_key : no) = k;
        }
        hi_key = lo_key;
        no = key + 1;
        while (no - hi_key > 1) {
          const uint32_t k = hi_key + (no - hi_key) / 2;
          (Classes::of(cl.step(value_of(k))) >= c0 ? hi_key : no) = k;
        }
      }
      const float z_hi = value_of(hi_key), z_lo = value_of(lo_key);
      // bf16: the range has few different logits, of which there may be very many (a step of 1/16
      // from 8 on), and they are counted instead of listed
      constexpr int kKeys = kThreads;
      const uint32_t k_hi = hi_key >> 16;
      const bool by_key = sizeof(E) == 2 && k_hi - (lo_key >> 16) < (uint32_t)kKeys;
      uint32_t* key_n = reinterpret_cast<uint32_t*>(sh.list);
      u64* key_w = sh.list + kKeys;
      if (by_key) {
        const uint32_t k = k_hi - min(k_hi, (uint32_t)tid);
        key_n[tid] = 0;
        key_w[tid] = w(value_of(k & 0x8000u ? k << 16 : k << 16 | 0xFFFFu));
        __syncthreads();
      }
      // the exact mass, that above the range, and the list of those in it
      u64 mass = 0;
      int n = 0;
      part.each([&](int v, const uint4& raw) {
        float z[VE];
        Vec<E>::get(raw, z);
        unsigned take = 0;
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const u64 x = w(z[j]);
          mass += x;
          if (z[j] > z_hi) above += x;
          else if (z[j] >= z_lo) take |= 1u << j;
        }
        if (!by_key) {
          n += row.put(v, take);
        } else if (take) {
#pragma unroll
          for (int j = 0; j < VE; ++j)
            if (take >> j & 1) atomicAdd(&key_n[k_hi - (key_of(z[j]) >> 16)], 1u);
        }
      });
      row.put_count(n);
      mass = warp_sum(mass);
      const u64 own_above = warp_sum(above);
      mass = row.row_sum(mass, before);
      above = row.row_sum(own_above, before);
      target = top_p_target(top_p, mass);
      n = (int)sh.count;
      if constexpr (sizeof(E) == 2) if (by_key && above < target) {
        if (rank != 0 && key_n[tid]) atomicAdd(row.of(&key_n[tid], 0), key_n[tid]);
        if (rank == 0 && tid < size) *row.of(&sh.slot[row.phase % kSlots][0], tid) = {0, 0, 0, 0};
        row.sync();
        if (rank == 0) {
          const u64 x = key_n[tid] * key_w[tid], left = target - above;
          u64 all;
          const u64 run = row.scan(x, all);
          if (x > 0 && run < left && run + x >= left) {
            for (int r = 0; r < size; ++r)
              *row.of(&sh.slot[row.phase % kSlots][0], r) = {
                  (left - run + key_w[tid] - 1) / key_w[tid], 1, k_hi - (uint32_t)tid, 0};
          }
        }
        row.sync();
        const Slot s = row.told()[0];
        if (s.b != 0) {
          // the `nth` of the logits equal to `z_b` is the border: this warp's kept ones, and its id
          found = true;
          const u64 nth = s.a, w_b = key_w[k_hi - s.c];
          const uint32_t key_b = s.c & 0x8000u ? s.c << 16 : s.c << 16 | 0xFFFFu;
          const float z_b = value_of(key_b);
          u64 kept_mass = 0;
          uint32_t ties = 0;
          part.each([&](int, const uint4& raw) {
            if (!(Vec<E>::top(raw) >= z_b)) return;
            float z[VE];
            Vec<E>::get(raw, z);
#pragma unroll
            for (int j = 0; j < VE; ++j) {
              ties += z[j] == z_b;
              if (z[j] > z_b && z[j] <= z_hi) kept_mass += key_w[k_hi - (key_of(z[j]) >> 16)];
            }
          });
          const u64 own_ties = warp_sum((u64)ties);
          u64 ties_before;
          row.row_sum(own_ties, ties_before);
          row.find(nth - 1, ties_before, own_ties,
                   [&](int, const uint4& raw, u64 (&y)[VE]) {
                     float z[VE];
                     Vec<E>::get(raw, z);
#pragma unroll
                     for (int j = 0; j < VE; ++j) y[j] = z[j] == z_b;
                   },
                   [&](int id, u64, u64) {
                     row.tell_border((u64)key_b << 32 | (0xFFFFFFFFu - (uint32_t)id));
                   });
          b = row.told_border();
          if (w_b >= least) {
            const u64 kept_ties = nth > ties_before ? min(nth - ties_before, own_ties) : 0ull;
            const u64 own = own_above + warp_sum(kept_mass) + kept_ties * w_b;
            const u64 all = row.row_sum(own, before);
            row.find(draw_target(a.uniform[t], all), before, own, kept,
                     [&](int id, u64 x, u64) { write_token(a, t, id, x, all); });
            return;
          }
        }
      }
      // (exact: what the classes said was only where to look)
      if (!by_key && n > kList && above < target)
        found = row.template locate<true>(target, b, lo_key, hi_key, above, w);
      if (!by_key && n <= kList && above < target) {
        if (rank == 0) {
          row.sort_list(n);
          if (tid == 0) sh.claim = 0;
          __syncthreads();
          const int phase = row.phase;
          row.list_mass(n, w, target - above, [&](int i, u64, u64) {
            const u64 e = sh.list[i];
            for (int r = 0; r < size; ++r)
              *row.of(&sh.slot[phase % kSlots][0], r) = {0, 1, (uint32_t)(e >> 32),
                                                         0xFFFFFFFFu - (uint32_t)e};
            sh.claim = (uint32_t)i + 1;
          });
          __syncthreads();
          const int kept_n = (int)sh.claim;
          if (kept_n == 0 && tid < size) *row.of(&sh.slot[phase % kSlots][0], tid) = {0, 0, 0, 0};
          // the kept entries' masses, for the warps that hold them
          constexpr int kOf = R::kEach;
          u64 x[kOf], all;
          row.list_weights(kept_n, w, [](u64 e) { return (uint32_t)(e >> 32); }, x, all);
#pragma unroll
          for (int q = 0; q < kOf; ++q) {
            const int i = tid * row.list_each(kept_n) + q;
            if (q >= row.list_each(kept_n) || i >= kept_n) continue;
            const int id = (int)(0xFFFFFFFFu - (uint32_t)sh.list[i]), r = id / per;
            const E* g = (const E*)a.logits + (long long)t * a.ld + r * per;
            const int lead = (int)((uintptr_t)g / sizeof(E) % VE);
            const int held = min(a.V, (r + 1) * per) - r * per;
            const int share = ((lead + held + VE - 1) / VE + kWarps - 1) / kWarps;
            atomicAdd(row.of(&sh.extra[(id - r * per + lead) / VE / share], r), x[q]);
          }
        }
        row.sync();
        const Slot s = row.told()[0];
        if (s.b != 0) {
          found = true;
          b = {s.c, (int)s.d};
          if (w(value_of(b.key)) >= least) {
            // nothing that min_p would cut: the draw, from the sums there are
            const u64 own = own_above + sh.extra[warp];
            const u64 all = row.row_sum(own, before);
            row.find(draw_target(a.uniform[t], all), before, own, kept,
                     [&](int id, u64 x, u64) { write_token(a, t, id, x, all); });
            return;
          }
        }
      }
    } else {
      target = top_p_target(top_p, row.row_sum(row.own_sum(kept), before));
    }
    if (!found) row.template locate<true>(target, b, b.key, key, 0, w);
  }
  if (ahead && !cut_k && !cut_p && !(min_p > 0.f) && !ahead_w.far && !w.far) {
    // From the sums of the one pass.  Where the rest of the row had a larger logit (by an octave),
    // they began in finer units, and hold up to one unit more for each weight, whose cut-off parts
    // they add up: the exact mass, what lies before a token and the target are each less by 0 to
    // V.  A token that holds the target by more than that on both sides is the exact sums' too;
    // any other draw is made anew (and one that falls behind the last weight).
    const int down = w.octave - ahead_w.octave;
    const u64 own = warp_sum(down < 64 ? ahead_sum >> down : 0ull);
    const u64 mass = row.row_sum(own, before), slack = w.octave > seen_octave ? (u64)a.V : 0ull;
    if (tid == 0) sh.least_id = 0;
    __syncthreads();
    row.find(draw_target(a.uniform[t], mass), before, own, kept, [&](int id, u64 x, u64 past) {
      if (past < slack || x - past <= slack) return;
      write_token(a, t, id, x, mass);
      sh.least_id = 1;
    });
    __syncthreads();
    if (sh.least_id) return;
  }
  auto drawn = [&](int v, const uint4& raw, u64 (&x)[VE]) {
    kept(v, raw, x);
#pragma unroll
    for (int j = 0; j < VE; ++j) x[j] = x[j] >= least ? x[j] : 0ull;
  };
  const u64 own = row.own_sum(drawn), mass = row.row_sum(own, before);
  row.find(draw_target(a.uniform[t], mass), before, own, drawn,
           [&](int id, u64 x, u64) { write_token(a, t, id, x, mass); });
}

}  // namespace

cudaError_t launch_rows(const RowArgs& a) {
  const size_t es = a.dtype == 0 ? 4 : 2;
  auto bytes = [&](int c) {      // of one CTA's part, with a vector for the alignment
    return ((((size_t)a.V + c - 1) / c * es + 15) / 16 + 1) * 16;
  };
  // Held: parts that leave room for two CTAs a SM, and enough CTAs for the GPU where rows are few.
  // One CTA a row, which reads it again for every pass, where rows are many and do not fit one
  // CTA: the barriers of clusters then cost more than the memory's time.  (151936 fp32 logits, the
  // 64 largest: 17 rows 21 us held, 48 by one CTA each; 76 rows 46 and 37; 2048 rows 911 and 326.)
  int c = 1;
  while (c < kMaxCluster && (bytes(c) > 84 * 1024 || (a.T * c < 152 && a.V / c >= 4096))) c *= 2;
  const bool held = bytes(c) <= 196 * 1024 && (a.T < 64 || bytes(1) <= 84 * 1024);
  if (!held) c = 1;
  // Threads of a row that no cluster holds.  Two CTAs of 512 a SM overlap their barriers; where rows
  // that no list serves are few, one of 1024 has its row sooner.  (p 0.9, 152 rows of 151936 fp32
  // logits: 176 us with 512, 139 with 1024; 304 rows 248 and 273.  Rows of different settings, one
  // in five such, bf16: 544 rows 257 and 196, 1024 rows 308 and 325.)  The settings of rows lie on
  // the device, so the rule takes it that some are long; where none is, it costs: 544 bf16 rows of
  // top_k 20 take 98 us with an array of them and 55 with one for all, greedy ones 51 and 37.
  const bool own = a.row_temperature || a.row_top_p || a.row_top_k;
  int sms = 0;
  cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  const bool many = !held && a.tokens &&
                    (own ? a.T <= 4 * sms : a.T <= sms && a.top_k <= 0 && a.temperature > 0.f);
  const int nt = many ? 1024 : 512;
  const size_t smem = held ? bytes(c) : (size_t)kRing * nt * 16;
  auto pick = [&](auto e, auto top, auto in, auto threads) {
    return rows_kernel<typename decltype(e)::type, decltype(top)::value, decltype(in)::value,
                       decltype(threads)::value>;
  };
  auto of_type = [&](auto e) {
    using Yes = std::true_type;
    using No = std::false_type;
    using Some = std::integral_constant<int, 512>;
    using Many = std::integral_constant<int, 1024>;
    if (!a.tokens) return held ? pick(e, Yes{}, Yes{}, Some{}) : pick(e, Yes{}, No{}, Some{});
    return held   ? pick(e, No{}, Yes{}, Some{})
           : many ? pick(e, No{}, No{}, Many{})
                  : pick(e, No{}, No{}, Some{});
  };
  void (*kernel)(RowArgs) =
      a.dtype == 0 ? of_type(std::common_type<float>{}) : of_type(std::common_type<__nv_bfloat16>{});
  e = raise_smem_limit((const void*)kernel, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  // rows of different settings: one CTA each for the long ones, then one each for the others (2048
  // rows: 498 us instead of 577)
  RowArgs r = a;
  r.long_first = !held && own;
  cfg.gridDim = dim3((unsigned)a.T * (r.long_first ? 2 : c));
  cfg.blockDim = dim3((unsigned)nt);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, r);
}

}  // namespace dspark
