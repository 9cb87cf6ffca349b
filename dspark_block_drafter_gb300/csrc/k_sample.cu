// Draws from rows of logits, and their k largest.
//
// The order of a row's tokens is that of common.cuh: falling logits, equal ones by rising id.
// Every filter keeps a prefix of it, so the kept set is known by its border, the last (logit,
// id) kept:
//   top_k   the border is the k-th of the order
//   top_p   the first whose mass, with all before it, reaches p times the mass after top_k
//   min_p   the last whose weight is at least min_p times the largest's
// and the token is the first by id whose mass, with all kept ids below it, exceeds u times the
// kept mass.
//
// Weights are whole numbers: w = e^((z - max) / temperature) in units of 2^-S (S = 44 for a
// vocabulary of 2^18), each off by at most 2^-28 of itself and cut to whole units.  Sums of them are exact in 64 bits,
// in any order and by atomics too, so that the same row gives the same token however it is
// split, and a border of a long sum lies where the definition has it.  (An fp32 sum of 151936
// weights is off by some 1e-7 of itself: among as many tokens, that is the next token in one
// row of a hundred.)
//
// A row is held in the shared memory of one cluster of 1 to 8 CTAs (76 KB of each for 151936
// fp32 logits in 8, two CTAs a SM), so it is read from memory once, and every later pass is one
// over shared memory.  Passes: the maximum, while it is read; a list of the largest logits; the
// mass, where a filter needs it; the kept mass by id.  The list is what is not below the least
// of some groups' maxima: with at least k groups it holds the k largest, and some 600 entries
// of 151936 for 128 groups.  One CTA sorts it, and finds the borders of top_k and top_p there.
// Where it does not (more groups than fit, a flat nucleus, many equal logits) the border is
// found by histograms of the logits' order keys, 2048 bins at a time.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "tokens.h"

namespace dspark {

namespace {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048, kList = 2048;
constexpr int kMaxCluster = 8;
constexpr uint32_t kNoKey = 0x007FFFFFu;       // the order key of -infinity
constexpr int kSlots = 4;

// 2^(-j / 64) in units of 2^-30
__constant__ uint32_t kExp2[64] = {
    0x40000000u, 0x3f4f8303u, 0x3ea0ecb7u, 0x3df437ddu, 0x3d495f45u, 0x3ca05dcfu, 0x3bf92e67u, 0x3b53cc08u,
    0x3ab031bau, 0x3a0e5a94u, 0x396e41bau, 0x38cfe25du, 0x383337bbu, 0x37983d21u, 0x36feede6u, 0x36674571u,
    0x35d13f33u, 0x353cd6abu, 0x34aa0764u, 0x3418ccf7u, 0x33892305u, 0x32fb0540u, 0x326e6f62u, 0x31e35d32u,
    0x3159ca84u, 0x30d1b337u, 0x304b1333u, 0x2fc5e66eu, 0x2f4228e8u, 0x2ebfd6adu, 0x2e3eebd2u, 0x2dbf6479u,
    0x2d413ccdu, 0x2cc47105u, 0x2c48fd60u, 0x2bcede2bu, 0x2b560fbbu, 0x2ade8e6du, 0x2a6856adu, 0x29f364edu,
    0x297fb5aau, 0x290d456cu, 0x289c10c1u, 0x282c1444u, 0x27bd4c98u, 0x274fb66au, 0x26e34e6eu, 0x26781165u,
    0x260dfc14u, 0x25a50b4eu, 0x253d3beau, 0x24d68accu, 0x2470f4ddu, 0x240c7711u, 0x23a90e63u, 0x2346b7d7u,
    0x22e57079u, 0x2285355du, 0x222603a0u, 0x21c7d866u, 0x216ab0dau, 0x210e8a31u, 0x20b361a6u, 0x2059347du,
};

struct Slot {
  u64 a, b;
  uint32_t c;
  int32_t d;
};

struct Shared {
  union {
    struct {
      uint32_t cnt[kBins], lo[kBins], hi[kBins];
    } h;
    u64 list[kList];
  };
  u64 warp_sum[kWarps];
  Slot slot[kSlots];
  uint32_t exp2[64];
  uint32_t warp_key[kWarps], warp_low[kWarps];
  uint32_t count;
};

__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t u = __float_as_uint(z + 0.f);            // (-0 is 0)
  const uint32_t k = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return z == z ? k : kNoKey;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// The border of the kept set.
struct Border {
  uint32_t key;
  int id;
  __device__ __forceinline__ bool keeps(uint32_t k, int i) const {
    return (k > key) | ((k == key) & (i <= id));
  }
};

// The weights of a row.
struct Weights {
  float m, c_hi, c_lo;      // the maximum, log2(e) / temperature
  int shift;                // S - 30
  const uint32_t* table;

  // y = (m - z) log2(e) / t = n / 64 + f, |f| <= 2^-7, with the rounding errors of m - z and of
  // the product carried along; w = 2^-(n / 64) (1 + g), g = 2^-f - 1 to third order (off by
  // 2^-34).  T (1 + g) is cut to units of 2^-30.
  __device__ __forceinline__ u64 operator()(float z) const {
    float d = m - z;
    const float zb = m - d, db = d + zb;
    float e = (m - db) + (zb - z);
    if (z == m) d = e = 0.f;                   // (an infinite maximum too)
    const float p = d * c_hi;
    float r = fmaf(d, c_hi, -p);
    r = fmaf(d, c_lo, r);
    r = fmaf(e, c_hi, r);
    const float t = p + 196608.f;              // 1.5 * 2^17: steps of 1/64
    const int n = __float_as_int(t) - 0x48400000;
    const float f = (p - (t - 196608.f)) + r;
    float g = fmaf(f, -0.0555041087f, 0.240226507f);
    g = fmaf(f, g, -0.693147181f) * f;
    // g 2^29 as an integer
    const int gi = __float_as_int(fmaf(g, 536870912.f, 12582912.f)) - 0x4B400000;
    const uint32_t T = table[n & 63];
    const uint32_t w = T + (uint32_t)__mulhi((int)T, gi * 8);
    return p < 62.f ? ((u64)w << shift) >> (n >> 6) : 0ull;
  }
};

template <typename E>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int n = 4;
  static __device__ __forceinline__ void get(const uint4& v, float (&z)[4]) {
    z[0] = __uint_as_float(v.x); z[1] = __uint_as_float(v.y);
    z[2] = __uint_as_float(v.z); z[3] = __uint_as_float(v.w);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void get(const uint4& v, float (&z)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      z[2 * j] = __uint_as_float(w[j] << 16);
      z[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
};

// One CTA's part of a row: elements [i0, i0 + n), in vectors of 16 bytes of memory.  Vector
// elements that are not of the part read -infinity.
template <typename E>
struct Part {
  static constexpr int VE = Vec<E>::n;
  const E* g;               // the 16-byte boundary at or before element i0
  uint4* held;              // the vectors in shared memory, or NULL
  int i0, n, lead, nv;      // lead: elements before i0 in the first vector
  int v0, v1;               // this warp's vectors

  __device__ __forceinline__ uint4 load(int v) const {
    const int a = v * VE;
    if (a >= lead && a + VE <= lead + n) return __ldg(reinterpret_cast<const uint4*>(g) + v);
    alignas(16) E x[VE];
#pragma unroll
    for (int j = 0; j < VE; ++j)
      x[j] = a + j >= lead && a + j < lead + n ? g[a + j] : (E)-INFINITY;
    return *reinterpret_cast<const uint4*>(x);
  }
  __device__ __forceinline__ uint4 at(int v) const { return held ? held[v] : load(v); }
  __device__ __forceinline__ int id(int v, int j) const { return i0 + v * VE + j - lead; }

  // f(vector, its elements) over this warp's vectors, all lanes together; past the end
  // elements are -infinity
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    const int lane = threadIdx.x % 32;
#pragma unroll 2
    for (int b = v0; b < v1; b += 32) {
      const int v = b + lane;
      float z[VE];
      if (v < v1) {
        Vec<E>::get(at(v), z);
      } else {
#pragma unroll
        for (int j = 0; j < VE; ++j) z[j] = -INFINITY;
      }
      f(v, z);
    }
  }
};

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ u64 warp_scan(u64 v) {          // inclusive
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

template <typename E>
struct Row {
  static constexpr int VE = Vec<E>::n;
  Shared& sh;
  Part<E> part;
  int rank, size, phase;

  __device__ __forceinline__ Row(Shared& s) : sh(s), phase(0) {}

  __device__ __forceinline__ void sync() const {
    if (size > 1) cg::this_cluster().sync();
    else __syncthreads();
  }
  template <typename T>
  __device__ __forceinline__ T* of(T* p, int r) const {
    return size > 1 ? cg::this_cluster().map_shared_rank(p, r) : p;
  }
  // Every CTA's slot of a phase is written by one of its threads; after the sync all are read.
  // (A slot is written again four phases later: by then every CTA has read it.)
  __device__ __forceinline__ Slot& mine() { return sh.slot[phase % kSlots]; }
  __device__ __forceinline__ const Slot* theirs(int r) { return of(&sh.slot[phase % kSlots], r); }
  __device__ __forceinline__ void next() { ++phase; }

  // The sum of v over the threads before this one, and over all of the CTA.
  __device__ __forceinline__ u64 scan(u64 v, u64& all) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const u64 in = warp_scan(v);
    __syncthreads();
    if (lane == 31) sh.warp_sum[warp] = in;
    __syncthreads();
    u64 before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sh.warp_sum[w];
      all += sh.warp_sum[w];
    }
    return before + in - v;
  }

  // The sum of f(z, id) over the row; `before`: of all lower ids than this warp's, `own`: this
  // warp's.
  template <typename F>
  __device__ __forceinline__ u64 sum(F f, u64& before, u64& own) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    u64 s = 0;
    part.each([&](int v, const float (&z)[VE]) { s += f(v, z); });
    own = warp_sum(s);
    __syncthreads();
    if (lane == 0) sh.warp_sum[warp] = own;
    __syncthreads();
    before = 0;
    u64 all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sh.warp_sum[w];
      all += sh.warp_sum[w];
    }
    if (size == 1) return all;
    if (threadIdx.x == 0) mine().a = all;
    sync();
    all = 0;
    for (int r = 0; r < size; ++r) {
      const u64 x = theirs(r)->a;
      if (r < rank) before += x;
      all += x;
    }
    next();
    return all;
  }
  // The first id at which the running sum exceeds `target`: found(v, j, z) is called by one
  // thread of the cluster.  f as summed, and of one element.
  template <typename F, typename G, typename H>
  __device__ __forceinline__ void find(u64 target, u64 before, u64 own, F f, G one, H found) {
    if (target < before || target >= before + own) return;
    const int lane = threadIdx.x % 32;
    u64 left = target - before;
    bool done = false;
    part.each([&](int v, const float (&z)[VE]) {
      if (done) return;
      const u64 s = f(v, z), in = warp_scan(s);
      const u64 all = __shfl_sync(0xFFFFFFFFu, in, 31);
      if (left < all) {
        done = true;
        const u64 ex = in - s;
        if (left >= ex && left < in) {
          u64 run = ex;
          bool hit = false;
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            run += one(v, j, z[j]);
            if (!hit && left < run) {
              hit = true;
              found(v, j, z[j]);
            }
          }
        }
      } else {
        left -= all;
      }
    });
  }

  // Writes the elements with lo <= key <= hi that `b` keeps into the first CTA's list, as
  // (key, ~id), in no order; their number may be more than the list holds.
  __device__ __forceinline__ void collect(uint32_t lo, uint32_t hi, const Border& b) {
    const int lane = threadIdx.x % 32;
    uint32_t* count = of(&sh.count, 0);
    u64* list = of(sh.list, 0);
    part.each([&](int v, const float (&z)[VE]) {
      uint32_t k[VE];
      unsigned take = 0;
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        k[j] = key_of(z[j]);
        take |= (unsigned)((k[j] >= lo) & (k[j] <= hi) & b.keeps(k[j], part.id(v, j))) << j;
      }
      if (!__any_sync(0xFFFFFFFFu, take)) return;
      const int n = __popc(take);
      int in = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, in, o);
        if (lane >= o) in += y;
      }
      uint32_t at = 0;
      if (lane == 31) at = atomicAdd(count, (uint32_t)in);
      at = __shfl_sync(0xFFFFFFFFu, at, 31) + in - n;
#pragma unroll
      for (int j = 0; j < VE; ++j)
        if (take >> j & 1) {
          if (at < kList)
            list[at] = (u64)k[j] << 32 | (0xFFFFFFFFu - (uint32_t)part.id(v, j));
          ++at;
        }
    });
  }

  // Sorts the first n entries of this CTA's list, the best first.
  __device__ __forceinline__ void sort_list(int n) {
    int m = 32;
    while (m < n) m *= 2;
    for (int i = n + threadIdx.x; i < m; i += kThreads) sh.list[i] = 0;
    __syncthreads();
    for (int k = 2; k <= m; k *= 2)
      for (int j = k / 2; j > 0; j /= 2) {
        for (int q = threadIdx.x; q < m / 2; q += kThreads) {
          const int i = 2 * q - (q & (j - 1)), o = i + j;
          const u64 x = sh.list[i], y = sh.list[o];
          if ((x < y) == ((i & k) == 0)) {
            sh.list[i] = y;
            sh.list[o] = x;
          }
        }
        __syncthreads();
      }
  }

  // The first entry of this CTA's n sorted ones with which their mass reaches `target`, by one
  // thread: found(entry); returns the mass of all.
  template <typename F>
  __device__ __forceinline__ u64 list_mass(int n, const Weights& w, u64 target, F found) {
    constexpr int kEach = kList / kThreads;
    u64 x[kEach], s = 0, all;
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
      const int i = threadIdx.x * kEach + q;
      x[q] = i < n ? w(value_of((uint32_t)(sh.list[i] >> 32))) : 0ull;
      s += x[q];
    }
    u64 run = scan(s, all);
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
      if (x[q] > 0 && run < target && run + x[q] >= target) found(threadIdx.x * kEach + q);
      run += x[q];
    }
    return all;
  }

  // The border at which the kept elements' number (MASS: mass) reaches `target`, by histograms;
  // false, and b as it was, where all of them do not.  top: the largest key.
  template <bool MASS>
  __device__ __noinline__ bool locate(u64 target, Border& b, uint32_t top, const Weights w) {
    const Border in = b;
    uint32_t hi = top, lo = b.key;
    u64 above = 0;
    const int per = kBins / size;
    sync();                            // (the list and its count have been read)
    for (;;) {
      const uint32_t span = hi - lo;
      const int shift = max(0, 21 - __clz(span));
      for (int i = threadIdx.x; i < kBins; i += kThreads) sh.h.cnt[i] = sh.h.lo[i] = sh.h.hi[i] = 0;
      if (threadIdx.x == 0) sh.count = 0;
      __syncthreads();
      part.each([&](int v, const float (&z)[VE]) {
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const uint32_t k = key_of(z[j]);
          if (k < lo || k > hi || !in.keeps(k, part.id(v, j))) continue;
          const uint32_t bin = (hi - k) >> shift;
          atomicAdd(&sh.h.cnt[bin], 1u);
          if (MASS) {
            // 64 bits by two words: whoever wraps the low one carries
            const u64 x = w(z[j]);
            const uint32_t xl = (uint32_t)x, old = atomicAdd(&sh.h.lo[bin], xl);
            const uint32_t xh = (uint32_t)(x >> 32) + (old + xl < old);
            if (xh) atomicAdd(&sh.h.hi[bin], xh);
          }
        }
      });
      sync();
      // this CTA's share of the bins, summed over the cluster
      const int each = max(1, per / kThreads);
      u64 x[kBins / kThreads], s = 0;
      uint32_t c[kBins / kThreads];
#pragma unroll
      for (int q = 0; q < kBins / kThreads; ++q) {
        x[q] = 0;
        c[q] = 0;
        const int i = threadIdx.x * each + q;
        if (q >= each || i >= per) continue;
        for (int r = 0; r < size; ++r) {
          const Shared* o = of(&sh, r);
          const int at = rank * per + i;
          c[q] += o->h.cnt[at];
          if (MASS) x[q] += (u64)o->h.hi[at] << 32 | o->h.lo[at];
        }
        if (!MASS) x[q] = c[q];
        s += x[q];
      }
      u64 all;
      const u64 ex = scan(s, all);
      if (threadIdx.x == 0) mine().a = all;
      sync();
      u64 before = above, run = above;
      int owner = -1;
      for (int r = 0; r < size; ++r) {
        const u64 y = theirs(r)->a;
        if (owner < 0 && run + y >= target) owner = r;
        run += y;
        if (r < rank) before += y;
      }
      next();
      if (owner < 0) return false;
      if (owner == rank) {
        u64 at = before + ex;
#pragma unroll
        for (int q = 0; q < kBins / kThreads; ++q) {
          if (x[q] > 0 && at < target && at + x[q] >= target) {
            Slot& o = mine();
            o.a = at;
            o.c = c[q];
            o.d = rank * per + threadIdx.x * each + q;
          }
          at += x[q];
        }
      }
      sync();
      const Slot* o = theirs(owner);
      above = o->a;
      const uint32_t n = o->c;
      hi -= (uint32_t)o->d << shift;
      next();
      const uint32_t wide = (1u << shift) - 1;
      lo = hi - lo > wide ? hi - wide : lo;
      if (n <= kList) {
        collect(lo, hi, in);
        sync();
        if (rank == 0) {
          sort_list((int)n);
          if (MASS) {
            list_mass((int)n, w, target - above, [&](int i) { put_border(sh.list[i]); });
          } else if (threadIdx.x == 0) {
            put_border(sh.list[target - above - 1]);
          }
        }
        b = get_border();
        return true;
      }
      if (shift == 0) {
        // equal logits: the border is the `nth` of them by id
        const u64 x1 = MASS ? w(value_of(hi)) : 1ull;
        const u64 nth = (target - above + x1 - 1) / x1;
        auto one = [&](int v, int j, float z) -> u64 {
          const uint32_t k = key_of(z);
          return k == hi && in.keeps(k, part.id(v, j));
        };
        auto all_of = [&](int v, const float (&z)[VE]) {
          u64 t = 0;
#pragma unroll
          for (int j = 0; j < VE; ++j) t += one(v, j, z[j]);
          return t;
        };
        u64 first, own;
        sum(all_of, first, own);
        // (found by some CTA, told by the first)
        int* at = reinterpret_cast<int*>(of(&sh.count, 0));
        find(nth - 1, first, own, all_of, one, [&](int v, int j, float) { *at = part.id(v, j); });
        sync();
        if (rank == 0 && threadIdx.x == 0) {
          mine().c = hi;
          mine().d = (int)sh.count;
        }
        b = get_border();
        return true;
      }
    }
  }

  __device__ __forceinline__ void put_border(u64 entry) {
    mine().c = (uint32_t)(entry >> 32);
    mine().d = (int)(0xFFFFFFFFu - (uint32_t)entry);
  }
  // what one thread of the first CTA has put
  __device__ __forceinline__ Border get_border() {
    sync();
    const Slot* s = theirs(0);
    const Border b = {s->c, s->d};
    next();
    return b;
  }
};

template <typename E, bool TOP>
__global__ void __launch_bounds__(kThreads, 2) rows_kernel(const RowArgs a, int hold) {
  extern __shared__ uint4 s_held[];
  __shared__ Shared sh;
  constexpr int VE = Vec<E>::n;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  Row<E> row(sh);
  row.size = (int)cg::this_cluster().num_blocks();
  row.rank = (int)cg::this_cluster().block_rank();
  const int t = blockIdx.x / row.size;
  const int rank = row.rank;
  Part<E>& part = row.part;
  {
    const int per = ((a.V + row.size - 1) / row.size + VE - 1) / VE * VE;
    part.i0 = min(a.V, rank * per);
    part.n = min(a.V, part.i0 + per) - part.i0;
    const E* g = (const E*)a.logits + (long long)t * a.ld + part.i0;
    part.lead = (int)((uintptr_t)g / sizeof(E) % VE);
    part.g = g - part.lead;
    part.nv = part.n > 0 ? (part.lead + part.n + VE - 1) / VE : 0;
    const int share = (part.nv + kWarps - 1) / kWarps;
    part.v0 = min(part.nv, warp * share);
    part.v1 = min(part.nv, part.v0 + share);
    part.held = nullptr;
  }
  if (tid < 64) sh.exp2[tid] = kExp2[tid];
  if (tid == 0) sh.count = 0;

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
  const bool cut_p = !TOP && top_p < 1.f;

  // the row, and the maximum of every thread's part of it
  float top = -INFINITY;
  {
    constexpr int U = 4;
    for (int b = part.v0; b < part.v1; b += 32 * U) {
      uint4 x[U];
#pragma unroll
      for (int q = 0; q < U; ++q)
        if (b + 32 * q + lane < part.v1) x[q] = part.load(b + 32 * q + lane);
#pragma unroll
      for (int q = 0; q < U; ++q) {
        if (b + 32 * q + lane >= part.v1) continue;
        if (hold) s_held[b + 32 * q + lane] = x[q];
        float z[VE];
        Vec<E>::get(x[q], z);
#pragma unroll
        for (int j = 0; j < VE; ++j) top = fmaxf(top, z[j]);
      }
    }
    if (hold) part.held = s_held;
  }
  // the least of the groups' maxima, of at least K groups of lanes where there are as many
  uint32_t key = key_of(top), low;
  {
    const int want = K < a.V ? K : 128;
    int lanes = 32;
    while (lanes > 1 && kWarps * row.size * (32 / lanes) < want) lanes /= 2;
    uint32_t m = key;
    for (int o = 1; o < lanes; o *= 2) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    low = __reduce_min_sync(0xFFFFFFFFu, m);
    key = __reduce_max_sync(0xFFFFFFFFu, key);
    if (lane == 0) {
      sh.warp_key[warp] = key;
      sh.warp_low[warp] = low;
    }
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) {
      key = max(key, sh.warp_key[w]);
      low = min(low, sh.warp_low[w]);
    }
    if (tid == 0) {
      row.mine().c = key;
      row.mine().d = (int)low;
    }
    row.sync();
    for (int r = 0; r < row.size; ++r) {
      key = max(key, row.theirs(r)->c);
      low = min(low, (uint32_t)row.theirs(r)->d);
    }
    row.next();
  }
  const Border every = {kNoKey, -1};             // all but -infinity
  low = max(low, kNoKey + 1);
  const bool greedy = !TOP && !(tau > 0.f);
  if (key <= kNoKey) {
    // nothing to choose from
    if (!TOP && rank == 0 && tid == 0) {
      a.tokens[t] = -1;
      if (a.logp) a.logp[t] = -INFINITY;
    }
    if (TOP && rank == 0) {
      for (int i = tid; i < a.k; i += kThreads) {
        a.ids[(size_t)t * a.k + i] = -1;
        a.values[(size_t)t * a.k + i] = -INFINITY;
      }
      if (a.lse && tid == 0) a.lse[t] = -INFINITY;
    }
    row.sync();
    return;
  }
  Weights w;
  {
    w.m = value_of(key);
    const double c = 1.4426950408889634 / (double)(greedy ? 1.f : tau);
    w.c_hi = (float)fmin(c, 3e38);
    w.c_lo = c < 3e38 ? (float)(c - (double)w.c_hi) : 0.f;
    w.shift = 32 - (32 - __clz(max(1, a.V - 1)));
    w.table = sh.exp2;
  }
  const int S = w.shift + 30;

  Border b = every;
  const bool cut_k = K < a.V;
  bool listed = false;
  int n = 0;
  if (TOP || (!greedy && K > 1 && (cut_k || cut_p))) {
    row.collect(low, key, every);
    row.sync();
    n = (int)*row.of(&sh.count, 0);
    listed = n <= kList && (TOP || !cut_k || n >= K || low == kNoKey + 1);
    if (listed && rank == 0) row.sort_list(n);
  }

  if (TOP) {
    // the k largest, and the sum of all in fp32: its terms' errors are some 1e-7 of them
    if (a.lse) {
      float s = 0.f;
      part.each([&](int v, const float (&z)[VE]) {
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const float x = z[j] == w.m ? 0.f : z[j] - w.m;
          float y;
          asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.44269504f));
          s += z[j] == z[j] ? y : 0.f;
        }
      });
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      __syncthreads();
      if (lane == 0) sh.warp_key[warp] = __float_as_uint(s);
      __syncthreads();
      if (tid == 0) {
        float all = 0.f;
        for (int q = 0; q < kWarps; ++q) all += __uint_as_float(sh.warp_key[q]);
        row.mine().c = __float_as_uint(all);
      }
      row.sync();
      if (rank == 0 && tid == 0) {
        float all = 0.f;
        for (int r = 0; r < row.size; ++r) all += __uint_as_float(row.theirs(r)->c);
        a.lse[t] = w.m + logf(all);
      }
      row.next();
    }
    if (!listed || (n < K && low > kNoKey + 1)) {
      const bool some = row.template locate<false>((u64)K, b, key, w);
      if (rank == 0 && tid == 0) sh.count = 0;
      row.sync();
      row.collect(some ? b.key : kNoKey + 1, key, b);
      row.sync();
      n = (int)*row.of(&sh.count, 0);
      if (rank == 0) row.sort_list(n);
    }
    if (rank == 0) {
      for (int i = tid; i < a.k; i += kThreads) {
        const u64 e = i < n ? sh.list[i] : 0ull;
        a.ids[(size_t)t * a.k + i] = i < n ? (int)(0xFFFFFFFFu - (uint32_t)e) : -1;
        a.values[(size_t)t * a.k + i] = i < n ? value_of((uint32_t)(e >> 32)) : -INFINITY;
      }
    }
    row.sync();
    return;
  }

  if (greedy || K == 1) {
    // the lowest id of the largest logit
    auto one = [&](int v, int j, float z) -> u64 { return key_of(z) == key; };
    auto some = [&](int v, const float (&z)[VE]) {
      u64 s = 0;
#pragma unroll
      for (int j = 0; j < VE; ++j) s += one(v, j, z[j]);
      return s;
    };
    u64 before, own;
    row.sum(some, before, own);
    row.find(0, before, own, some, one, [&](int v, int j, float) {
      a.tokens[t] = part.id(v, j);
      if (a.logp) a.logp[t] = 0.f;
    });
    row.sync();
    return;
  }

  auto kept = [&](int v, int j, float z) -> u64 {
    return b.keeps(key_of(z), part.id(v, j)) ? w(z) : 0ull;
  };
  auto kept_all = [&](int v, const float (&z)[VE]) {
    u64 s = 0;
    bool any = false;
#pragma unroll
    for (int j = 0; j < VE; ++j) any |= key_of(z[j]) >= b.key;
    if (any) {
#pragma unroll
      for (int j = 0; j < VE; ++j) s += kept(v, j, z[j]);
    }
    return s;
  };
  u64 before, own;
  if (cut_k) {
    if (listed) {
      if (rank == 0 && tid == 0) {
        if (n >= K) {
          row.put_border(sh.list[K - 1]);
        } else {
          row.mine().c = kNoKey;
          row.mine().d = -1;
        }
      }
      b = row.get_border();
      n = min(n, K);
    } else {
      row.template locate<false>((u64)K, b, key, w);
    }
  }
  if (cut_p) {
    u64 mass = row.sum(kept_all, before, own);
    const double want = ceil(fmax((double)top_p, 0.) * (double)mass);
    const u64 target = min(mass, max(1ull, (u64)want));
    bool found = false;
    if (listed) {
      if (rank == 0) {
        if (tid == 0) row.mine().a = 0;
        __syncthreads();
        row.list_mass(n, w, target, [&](int i) {
          row.put_border(sh.list[i]);
          row.mine().a = 1;
        });
      }
      row.sync();
      const Slot* s = row.theirs(0);
      found = s->a != 0;
      if (found) b = {s->c, s->d};
      row.next();
    }
    if (!found) row.template locate<true>(target, b, key, w);
  }
  const u64 least = min_p > 0.f ? (u64)ceil(fmin((double)min_p, 1.) * (double)(1ull << S)) : 0ull;
  auto drawn = [&](int v, int j, float z) -> u64 {
    const u64 x = kept(v, j, z);
    return x >= least ? x : 0ull;
  };
  auto drawn_all = [&](int v, const float (&z)[VE]) {
    u64 s = 0;
    bool any = false;
#pragma unroll
    for (int j = 0; j < VE; ++j) any |= key_of(z[j]) >= b.key;
    if (any) {
#pragma unroll
      for (int j = 0; j < VE; ++j) s += drawn(v, j, z[j]);
    }
    return s;
  };
  const u64 mass = row.sum(drawn_all, before, own);
  const double u = (double)a.uniform[t];
  const u64 target = u > 0. ? min(mass - 1, (u64)(fmin(u, 1.) * (double)mass)) : 0ull;
  row.find(target, before, own, drawn_all, drawn, [&](int v, int j, float z) {
    a.tokens[t] = part.id(v, j);
    const u64 x = w(z);
    if (a.logp) a.logp[t] = -log1pf((float)(mass - x) / (float)x);
  });
  row.sync();
}

}  // namespace

cudaError_t launch_rows(const RowArgs& a) {
  const size_t es = a.dtype == 0 ? 4 : 2;
  auto bytes = [&](int c) {      // of one CTA's part, with a vector for the alignment
    return ((((size_t)a.V + c - 1) / c * es + 15) / 16 + 1) * 16;
  };
  // parts that leave room for two CTAs a SM, and enough CTAs for the GPU where rows are few
  int c = 1;
  while (c < kMaxCluster && (bytes(c) > 84 * 1024 || (a.T * c < 152 && a.V / c >= 4096))) c *= 2;
  int hold = bytes(c) <= 196 * 1024;
  const size_t smem = hold ? bytes(c) : 0;
  void (*kernel)(RowArgs, int) =
      a.tokens ? (a.dtype == 0 ? rows_kernel<float, false> : rows_kernel<__nv_bfloat16, false>)
               : (a.dtype == 0 ? rows_kernel<float, true> : rows_kernel<__nv_bfloat16, true>);
  cudaError_t e = raise_smem_limit((const void*)kernel, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.T * c);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, hold);
}

}  // namespace dspark
