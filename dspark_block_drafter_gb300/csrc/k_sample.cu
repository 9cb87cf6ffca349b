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
// vocabulary of 2^18), each off by at most 2^-27 of itself and cut to whole units.  Sums of them
// are exact in 64 bits, in any order and by atomics too, so that the same row gives the same
// token however it is split, and a border of a long sum lies where the definition has it.  (An
// fp32 sum of 151936 weights is off by some 1e-7 of itself: among as many tokens, that is the
// next token in one row of a hundred.)
//
// A row is held in the shared memory of one cluster of 1 to 8 CTAs (76 KB of each for 151936
// fp32 logits in 8, two CTAs a SM), so it is read from memory once, and every later pass is one
// over shared memory.  CTAs tell each other by stores into all of their shared memories before
// a barrier of the cluster, and read only their own after it.
//
//   top_k, and the k largest: a list of what is not below the least of some groups' maxima; with
//     at least k groups it holds the k largest (some 150 entries for 32 groups, 300 for 64).
//     The first CTA sorts it and does the rest alone.
//   top_p: masses by 2048 classes of weights, 1/64 of an octave wide, off by 2^-13 of themselves
//     (32-bit sums by shared memory atomics); then, in one pass, the exact mass, that of the
//     classes surely kept, and a list of the few classes that the border may lie in.
//   Where a list does not do (more entries than it holds, many equal logits): histograms of the
//     logits' order keys, 2048 bins at a time, with exact masses.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

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
constexpr float kLog2e = 1.44269504f;

// 2^(j / 32) in units of 2^-30
__constant__ uint32_t kExp2[32] = {
    0x40000000u, 0x4166c34cu, 0x42d561b4u, 0x444c0740u, 0x45cae0f2u, 0x47521cc6u, 0x48e1e9bau, 0x4a7a77d4u,
    0x4c1bf829u, 0x4dc69cddu, 0x4f7a9930u, 0x51382182u, 0x52ff6b55u, 0x54d0ad5au, 0x56ac1f75u, 0x5891fac1u,
    0x5a82799au, 0x5c7dd7a4u, 0x5e8451d0u, 0x60962665u, 0x62b39509u, 0x64dcdec3u, 0x6712460bu, 0x69540ec9u,
    0x6ba27e65u, 0x6dfddbccu, 0x70666f76u, 0x72dc8374u, 0x75606374u, 0x77f25cceu, 0x7a92be8bu, 0x7d41d96eu,
};

struct Slot {
  u64 a, b;
  uint32_t c, d;
};

struct Shared {
  union {
    struct {
      uint32_t cnt[kBins], lo[kBins], hi[kBins];
    } h;
    struct {
      u64 list[kList];
      uint32_t mass[kBins];         // of this CTA's elements, in the first CTA then of all
    };
  };
  Slot slot[kSlots][kMaxCluster];
  u64 warp_sum[kWarps], extra[kWarps];
  uint32_t warp_key[kWarps], warp_top[kWarps];
  float warp_f[kWarps], half_top[2 * kWarps];
  uint32_t count;                   // entries of the list, told to every CTA
  uint32_t claim;                   // entries that have a place in the first CTA's list
  uint32_t least_id;
};

__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t u = __float_as_uint(z + 0.f);            // (-0 is 0)
  const uint32_t k = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return z == z ? k : kNoKey;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The border of the kept set.
struct Border {
  uint32_t key;
  int id;
  __device__ __forceinline__ bool keeps(uint32_t k, int i) const {
    return (k > key) | ((k == key) & (i <= id));
  }
};

// The weights of a row, whole numbers: the largest is between 2^(S - 2) and 2^S.
struct Weights {
  float m, c_hi, c_lo;      // the maximum, log2(e) / temperature
  float z_low, z_cap;       // below z_low nothing is left; above z_cap an octave more is needed
  float magic;
  int octave, shift;        // weights are in units of 2^(octave - S)
  bool far;
  uint32_t t_lane;          // kExp2[lane]

  // (in pairs of fp32: fp64 runs at two lanes a clock)
  __device__ __forceinline__ void set(float top, float temperature, int V) {
    constexpr float kLo = 1.92596299e-8f;       // log2(e) - kLog2e
    m = top;
    c_hi = fminf(kLog2e / temperature, 3e38f);
    c_lo = (fmaf(-c_hi, temperature, kLog2e) + kLo) / temperature;
    if (!(c_hi < 3e38f) || !(fabsf(c_lo) < 1e30f) || c_hi == 0.f) c_lo = 0.f;
    far = !(fabsf(top * c_hi) < 60000.f) || !(c_hi > 1e-6f);
    shift = 32 - __clz(max(1, V - 1));          // ceil(log2 V): S = 62 - shift
    t_lane = kExp2[threadIdx.x % 32];
    raise(top);
  }
  // makes room for a logit of `top`; the octaves that this took
  __device__ __forceinline__ int raise(float top) {
    const int was = octave;
    // steps of 1/32 up to it, in whole octaves
    octave = far ? 1 : ((__float2int_ru(__fmul_rn(top, c_hi) * 32.f) + 2) >> 5) + 1;
    magic = 393216.f - (float)octave;           // 1.5 * 2^18 - octave: a sum's low bits count 1/32
    z_low = far ? -100.f : ((float)octave - 100.f) / c_hi;
    z_cap = far ? INFINITY : top;
    return octave - was;
  }
  // z log2(e) / t = octave + n / 32 + f, |f| <= 2^-6, with the rounding error of the product
  // carried along; w = 2^(n / 32) (1 + g), g = 2^f - 1 to third order (off by 2^-30), in steps of
  // 2^-28.  The table's entries lie in the lanes of the warp (from shared memory, 32 different
  // ones take 3.5 times as long), so all of them call this together.
  __device__ __forceinline__ u64 weight(float p, float r) const {
    const float t = __fadd_rn(p, magic);
    const float f = __fadd_rn(__fsub_rn(p, __fsub_rn(t, magic)), r);
    // g 2^28 as an integer
    float h = fmaf(f, 0.0555041087f * 268435456.f, 0.240226507f * 268435456.f);
    h = fmaf(h, f, 0.693147181f * 268435456.f);
    const int g = __float_as_int(fmaf(h, f, 12582912.f)) * 16 - (int)0xB4000000;
    const int n = __float_as_int(t) - 0x48C00000;
    const uint32_t T = __shfl_sync(0xFFFFFFFFu, t_lane, n & 31);
    const uint32_t w = T + (uint32_t)__mulhi((int)T, g);
    // w 2^(n >> 5) in the units
    u64 x;
    asm("shr.u64 %0, %1, %2;" : "=l"(x) : "l"((u64)w << 32), "r"(shift - (n >> 5)));
    return x;
  }
  // A row whose largest logit leaves the range of n takes the distance from it first.
  __device__ __forceinline__ u64 operator()(float z) const {
    if (far) {
      float d = m - z;
      const float zb = m - d, db = d + zb;
      float e = (m - db) + (zb - z);
      if (z == m) d = e = 0.f;                 // (an infinite maximum too)
      const float p = fmaxf(-d * c_hi, -100.f);
      return weight(p, p > -100.f ? -fmaf(e, c_hi, fmaf(d, c_lo, fmaf(d, c_hi, p))) : 0.f);
    }
    const float y = fmaxf(z, z_low);           // (NaN too)
    const float p = __fmul_rn(y, c_hi);
    return weight(p, fmaf(y, c_lo, fmaf(y, c_hi, -p)));
  }
};

// The classes of weights: 1/64 of an octave each, by rounding; the last takes the rest.  The
// class never falls as the logit does, whatever is rounded.
struct Classes {
  float m, c;               // where the first one is, 64 log2(e) / temperature
  __device__ __forceinline__ float step(float z) const {
    return fmaxf(fminf(__fmul_rn(__fsub_rn(m, z), c), (float)(kBins - 1)), 0.f);
  }
  static __device__ __forceinline__ int of(float y) {
    return __float_as_int(__fadd_rn(y, 12582912.f)) - 0x4B400000;
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
  static __device__ __forceinline__ float top(const uint4& v) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                 fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
  static __device__ __forceinline__ uint4 none() {
    return make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
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
  static __device__ __forceinline__ __nv_bfloat162 two(uint32_t w) {
    return *reinterpret_cast<const __nv_bfloat162*>(&w);
  }
  static __device__ __forceinline__ float top(const uint4& v) {
    const __nv_bfloat162 m = __hmax2(__hmax2(two(v.x), two(v.y)), __hmax2(two(v.z), two(v.w)));
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ uint4 none() {
    return make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
  }
};

// One CTA's part of a row: elements [i0, i0 + n), in vectors of 16 bytes of memory.  Vector
// elements that are not of the part read -infinity.
//
// HELD: they are in shared memory once they have been read; otherwise every pass reads them
// from memory again, through a ring of kRing places for each thread.
constexpr int kRing = 8;
template <typename E, bool HELD>
struct Part {
  static constexpr int VE = Vec<E>::n;
  const E* g;               // the 16-byte boundary at or before element i0
  uint4* held;              // the vectors in shared memory, or the ring
  int i0, n, lead, nv;      // lead: elements before i0 in the first vector
  int share;                // vectors of a warp
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
  // Vector v to `to` in shared memory, without waiting for it.
  __device__ __forceinline__ void copy(int v, uint4* to) const {
    const int a = v * VE;
    if (a >= lead && a + VE <= lead + n)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                       (uint32_t)__cvta_generic_to_shared(to)),
                   "l"(reinterpret_cast<const uint4*>(g) + v)
                   : "memory");
    else
      *to = load(v);
  }
  static __device__ __forceinline__ void copied() {
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // all but the last `left` groups of copies have arrived
  template <int left>
  static __device__ __forceinline__ void arrived() {
    asm volatile("cp.async.wait_group %0;" ::"n"(left) : "memory");
  }
  __device__ __forceinline__ int id(int v, int j) const { return i0 + v * VE + j - lead; }
  __device__ __forceinline__ float element(int v, int j) const {
    return to_f32(HELD ? reinterpret_cast<const E*>(held)[v * VE + j] : g[v * VE + j]);
  }

  // f(vector, its raw elements) over this warp's vectors, all lanes together; past the end
  // elements are -infinity
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    each(v0, v1, f);
  }
  // the same for its vectors [v0, v1)
  template <typename F>
  __device__ __forceinline__ void each(int v0, int v1, F f) const {
    const int lane = threadIdx.x % 32;
    if (HELD) {
#pragma unroll 2
      for (int b = v0; b < v1; b += 32) {
        const int v = b + lane;
        f(v, v < v1 ? held[v] : Vec<E>::none());
      }
      return;
    }
    uint4* ring = held + threadIdx.x;
#pragma unroll
    for (int q = 0; q < kRing; ++q) {
      if (v0 + 32 * q + lane < v1) copy(v0 + 32 * q + lane, ring + q * kThreads);
      copied();
    }
    // two at a time, so that their arithmetic overlaps
    int at = 0;
    for (int b = v0; b < v1; b += 64) {
      arrived<kRing - 2>();
      const int v = b + lane, far = v + 32 * kRing;
      const uint4 x = v < v1 ? ring[at] : Vec<E>::none();
      const uint4 y = v + 32 < v1 ? ring[at + kThreads] : Vec<E>::none();
      if (far < v1) copy(far, ring + at);
      copied();
      if (far + 32 < v1) copy(far + 32, ring + at + kThreads);
      copied();
      at = at == (kRing - 2) * kThreads ? 0 : at + 2 * kThreads;
      f(v, x);
      f(v + 32, y);
    }
    arrived<0>();
  }
};

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ float warp_top(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
template <typename T>
__device__ __forceinline__ T warp_scan(T v) {              // inclusive
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// HELD: a cluster of `size` CTAs; otherwise one CTA.
template <typename E, bool HELD>
struct Row {
  static constexpr int VE = Vec<E>::n;
  Shared& sh;
  Part<E, HELD> part;
  int phase;

  __device__ __forceinline__ Row(Shared& s) : sh(s), phase(0) {}
  __device__ __forceinline__ int size() const {
    return HELD ? (int)cg::this_cluster().num_blocks() : 1;
  }
  __device__ __forceinline__ int rank() const {
    return HELD ? (int)cg::this_cluster().block_rank() : 0;
  }

  __device__ __forceinline__ void sync() const {
    if (HELD) {
      __cluster_barrier_arrive();
      __cluster_barrier_wait();
    } else {
      __syncthreads();
    }
  }
  // No CTA touches another's shared memory before all have started.
  __device__ __forceinline__ void started() const {
    if (HELD) __cluster_barrier_arrive();
  }
  __device__ __forceinline__ void all_started() const {
    if (HELD) __cluster_barrier_wait();
  }
  template <typename T>
  __device__ __forceinline__ T* of(T* p, int r) const {
    return HELD ? cg::this_cluster().map_shared_rank(p, r) : p;
  }
  // Tells every CTA this one's slot (all threads call it with the same values); they read them
  // after the next sync.  A slot is written again four syncs later at the earliest, when every
  // CTA has read it.
  __device__ __forceinline__ void tell(u64 a, u64 b, uint32_t c, uint32_t d) {
    if ((int)threadIdx.x < size()) *of(&sh.slot[phase % kSlots][rank()], (int)threadIdx.x) = {a, b, c, d};
  }
  // The slots' values after a sync.
  __device__ __forceinline__ const Slot* told() { return sh.slot[phase++ % kSlots]; }

  // The sum of v over the threads before this one, and over all of the CTA.
  template <typename T>
  __device__ __forceinline__ T scan(T v, T& all) {
    T* s_warp = reinterpret_cast<T*>(sh.warp_sum);
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const T in = warp_scan(v);
    __syncthreads();
    if (lane == 31) s_warp[warp] = in;
    __syncthreads();
    T before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s_warp[w];
      all += s_warp[w];
    }
    return before + in - v;
  }

  // From each warp's sum `own`: the row's, and that of all lower ids than this warp's.
  __device__ __forceinline__ u64 row_sum(u64 own, u64& before) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
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
    if (size() == 1) return all;
    tell(all, 0, 0, 0);
    sync();
    const Slot* s = told();
    all = 0;
    for (int r = 0; r < size(); ++r) {
      if (r < rank()) before += s[r].a;
      all += s[r].a;
    }
    return all;
  }
  // The sum of a warp's elements; f(v, raw, x) gives each of a vector's.
  template <typename F>
  __device__ __forceinline__ u64 own_sum(F f) {
    u64 s = 0;
    part.each([&](int v, const uint4& raw) {
      u64 x[VE];
      f(v, raw, x);
#pragma unroll
      for (int j = 0; j < VE; ++j) s += x[j];
    });
    return warp_sum(s);
  }
  // The first id at which the running sum exceeds `target`: found(id, x) is called by one
  // thread of the cluster.
  template <typename F, typename H>
  __device__ __forceinline__ void find(u64 target, u64 before, u64 own, F f, H found) {
    if (target < before || target >= before + own) return;
    u64 left = target - before;
    bool done = false;
    part.each([&](int v, const uint4& raw) {
      if (done) return;
      u64 x[VE], s = 0;
      f(v, raw, x);
#pragma unroll
      for (int j = 0; j < VE; ++j) s += x[j];
      const u64 in = warp_scan(s), all = __shfl_sync(0xFFFFFFFFu, in, 31);
      if (left >= all) {
        left -= all;
        return;
      }
      done = true;
      if (left < in - s || left >= in) return;
      u64 run = in - s;
      bool hit = false;
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        run += x[j];
        if (!hit && left < run) {
          hit = true;
          found(part.id(v, j), x[j]);
        }
      }
    });
  }

  // Gives the lane's elements of `take` places in the first CTA's list, as (key, ~id), in no
  // order; their number may be more than the list holds.  Returns it.
  __device__ __forceinline__ int put(int v, unsigned take) {
    const int n = __popc(take);
    if (n == 0) return 0;
    // (a list that runs over by far, of equal logits, is not worth its atomics)
    if (!HELD && *(volatile uint32_t*)&sh.claim > kList) return n;
    uint32_t at = atomicAdd(of(&sh.claim, 0), (uint32_t)n);
    u64* list = of(sh.list, 0);
    for (; take && at < kList; take &= take - 1, ++at) {
      const int j = __ffs(take) - 1;
      list[at] = (u64)key_of(part.element(v, j)) << 32 | (0xFFFFFFFFu - (uint32_t)part.id(v, j));
    }
    return n;
  }
  // Tells every CTA of `n` more entries of this lane; they know the number after the next sync.
  __device__ __forceinline__ void put_count(int n) {
    const int lane = threadIdx.x % 32;
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if (lane < size() && n > 0) atomicAdd(of(&sh.count, lane), (uint32_t)n);
  }

  // Lists a vector's elements not below z_lo; their number.
  __device__ __forceinline__ int put_from(int v, const uint4& raw, float z_lo) {
    if (!(Vec<E>::top(raw) >= z_lo)) return 0;
    float z[VE];
    Vec<E>::get(raw, z);
    unsigned take = 0;
#pragma unroll
    for (int j = 0; j < VE; ++j) take |= (unsigned)(z[j] >= z_lo) << j;
    return put(v, take);
  }
  // Lists the elements not below z_lo.
  __device__ __forceinline__ void collect(float z_lo) {
    int n = 0;
    part.each([&](int v, const uint4& raw) { n += put_from(v, raw, z_lo); });
    put_count(n);
  }
  // Adds a vector's weights to the classes' masses, in units of 1 / unit of the class's.
  __device__ __forceinline__ void add_classes(const uint4& raw, const Classes& cl, float unit) {
    float z[VE];
    Vec<E>::get(raw, z);
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      const float y = cl.step(z[j]), c = __fadd_rn(y, 12582912.f);
      // 2^-(x / 64) for |x| <= 1/2, rounded to whole units.  (The last class, with -infinity and
      // NaN, is bounded by the number of all: its elements may be most of the row's.)
      const float q = fmaf(y - (c - 12582912.f), unit * -0.0108304247f, unit + 8388608.f);
      if (y < (float)(kBins - 1))
        atomicAdd(&sh.mass[__float_as_int(c) - 0x4B400000], __float_as_uint(q) - 0x4B000000u);
    }
  }
  // Lists the elements with lo <= key <= hi that `b` keeps.
  __device__ __forceinline__ void collect(uint32_t lo, uint32_t hi, const Border& b) {
    const float z_lo = lo > kNoKey ? value_of(lo) : -INFINITY;
    int n = 0;
    part.each([&](int v, const uint4& raw) {
      if (!(Vec<E>::top(raw) >= z_lo)) return;
      float z[VE];
      Vec<E>::get(raw, z);
      unsigned take = 0;
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const uint32_t k = key_of(z[j]);
        take |= (unsigned)((k >= lo) & (k <= hi) & b.keeps(k, part.id(v, j))) << j;
      }
      n += put(v, take);
    });
    put_count(n);
  }

  // Sorts the first n entries of this CTA's list, the largest first.  Up to one a thread, steps
  // within a warp need no barrier.
  __device__ __forceinline__ void sort_list(int n) {
    const int tid = threadIdx.x;
    int m = 32;
    while (m < n) m *= 2;
    if (m <= kThreads) {
      u64 x = tid < n ? sh.list[tid] : 0;
      for (int k = 2; k <= m; k *= 2)
        for (int j = k / 2; j > 0; j /= 2) {
          u64 y;
          if (j >= 32) {
            __syncthreads();
            sh.list[tid] = x;
            __syncthreads();
            y = sh.list[tid ^ j];
          } else {
            y = __shfl_xor_sync(0xFFFFFFFFu, x, j);
          }
          const bool larger = ((tid & j) == 0) == ((tid & k) == 0);
          x = larger == (x > y) ? x : y;
        }
      __syncthreads();
      sh.list[tid] = x;
      __syncthreads();
      return;
    }
    for (int i = n + tid; i < m; i += kThreads) sh.list[i] = 0;
    __syncthreads();
    for (int k = 2; k <= m; k *= 2)
      for (int j = k / 2; j > 0; j /= 2) {
        for (int q = tid; q < m / 2; q += kThreads) {
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

  // Weights of this CTA's first n list entries, kEach a thread in order, and the sum before the
  // thread's; key_at(entry) is an entry's order key.
  static constexpr int kEach = kList / kThreads;
  template <typename W, typename F>
  __device__ __forceinline__ u64 list_weights(int n, const W& w, F key_at, u64 (&x)[kEach],
                                              u64& all) {
    u64 s = 0;
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
      const int i = threadIdx.x * kEach + q;
      const u64 y = w(value_of(i < n ? key_at(sh.list[i]) : kNoKey));
      x[q] = i < n ? y : 0ull;
      s += x[q];
    }
    return scan(s, all);
  }
  // The first entry with which the mass of the sorted list reaches `target`, by one thread:
  // found(index, mass before it, its own).
  template <typename W, typename F>
  __device__ __forceinline__ void list_mass(int n, const W& w, u64 target, F found) {
    u64 x[kEach], all;
    u64 run = list_weights(n, w, [](u64 e) { return (uint32_t)(e >> 32); }, x, all);
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
      if (x[q] > 0 && run < target && run + x[q] >= target)
        found((int)threadIdx.x * kEach + q, run, x[q]);
      run += x[q];
    }
  }

  // The border at which the kept elements' number (MASS: mass) reaches `target`, by histograms;
  // false, and b as it was, where all of them do not.  It is looked for among the keys lo to hi;
  // `above`: the number or mass of the kept ones above hi.
  template <bool MASS>
  __device__ __noinline__ bool locate(u64 target, Border& b, uint32_t lo, uint32_t hi, u64 above,
                                      const Weights w) {
    const Border in = b;
    // (the keys of bf16 logits differ in their high halves)
    constexpr int kUnit = sizeof(E) == 2 ? 16 : 0;
    const uint32_t least = lo, most = hi;
    lo >>= kUnit;
    hi >>= kUnit;
    const int per = kBins / size();
    sync();                            // (the list and its count have been read)
    for (;;) {
      const uint32_t span = hi - lo;
      const int shift = max(0, 21 - __clz(span));
      for (int i = threadIdx.x; i < kBins; i += kThreads) sh.h.cnt[i] = sh.h.lo[i] = sh.h.hi[i] = 0;
      if (threadIdx.x == 0) sh.count = sh.claim = 0;
      __syncthreads();
      part.each([&](int v, const uint4& raw) {
        float z[VE];
        Vec<E>::get(raw, z);
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const uint32_t full = key_of(z[j]), k = full >> kUnit;
          const bool take = k >= lo && k <= hi && full >= least && full <= most &&
                            in.keeps(full, part.id(v, j));
          const uint32_t bin = (hi - k) >> shift;
          const unsigned m = __ballot_sync(0xFFFFFFFFu, take);
          if (!m) continue;
          const u64 x = MASS ? w(z[j]) : 0;
          // (equal logits, of which there may be very many, in one go)
          const int lead = __ffs(m) - 1;
          const uint32_t k_lead = __shfl_sync(0xFFFFFFFFu, k, lead);
          const bool same = __all_sync(0xFFFFFFFFu, !take | (k == k_lead));
          if (same ? (int)(threadIdx.x % 32) != lead : !take) continue;
          const uint32_t n = same ? __popc(m) : 1;
          atomicAdd(&sh.h.cnt[bin], n);
          if (MASS) {
            // 64 bits by two words: whoever wraps the low one carries
            const u64 y = x * n;
            const uint32_t yl = (uint32_t)y, old = atomicAdd(&sh.h.lo[bin], yl);
            const uint32_t yh = (uint32_t)(y >> 32) + (old + yl < old);
            if (yh) atomicAdd(&sh.h.hi[bin], yh);
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
        for (int r = 0; r < size(); ++r) {
          const Shared* o = of(&sh, r);
          const int at = rank() * per + i;
          c[q] += o->h.cnt[at];
          if (MASS) x[q] += (u64)o->h.hi[at] << 32 | o->h.lo[at];
        }
        if (!MASS) x[q] = c[q];
        s += x[q];
      }
      u64 all;
      const u64 ex = scan(s, all);
      tell(all, 0, 0, 0);
      sync();
      const Slot* t = told();
      u64 before = above, run = above;
      int owner = -1;
      for (int r = 0; r < size(); ++r) {
        if (owner < 0 && run + t[r].a >= target) owner = r;
        run += t[r].a;
        if (r < rank()) before += t[r].a;
      }
      if (owner < 0) return false;
      if (owner == rank()) {
        u64 at = before + ex;
#pragma unroll
        for (int q = 0; q < kBins / kThreads; ++q) {
          if (x[q] > 0 && at < target && at + x[q] >= target)
            for (int r = 0; r < size(); ++r)
              *of(&sh.slot[phase % kSlots][0], r) = {
                  at, 0, c[q], (uint32_t)(rank() * per + threadIdx.x * each + q)};
          at += x[q];
        }
      }
      sync();
      const Slot o = told()[0];
      above = o.a;
      const uint32_t n = o.c;
      hi -= o.d << shift;
      const uint32_t wide = (1u << shift) - 1;
      lo = hi - lo > wide ? hi - wide : lo;
      if (n <= kList) {
        collect(max(least, lo << kUnit), min(most, (hi << kUnit) | ((1u << kUnit) - 1u)), in);
        sync();
        if (rank() == 0) {
          sort_list((int)n);
          if (MASS) {
            list_mass((int)n, w, target - above, [&](int i, u64, u64) { tell_border(sh.list[i]); });
          } else if (threadIdx.x == 0) {
            tell_border(sh.list[target - above - 1]);
          }
        }
        b = told_border();
        return true;
      }
      if (shift == 0) {
        // equal logits: the border is the `nth` of them by id
        const uint32_t key = kUnit > 0 && !(hi & 0x8000u) ? (hi << kUnit) | 0xFFFFu : hi << kUnit;
        const u64 x1 = MASS ? w(value_of(key)) : 1ull;
        const u64 nth = (target - above + x1 - 1) / x1;
        auto ones = [&](int v, const uint4& raw, u64 (&y)[VE]) {
          float z[VE];
          Vec<E>::get(raw, z);
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            const uint32_t k = key_of(z[j]);
            y[j] = k == key && in.keeps(k, part.id(v, j));
          }
        };
        u64 first;
        const u64 own = own_sum(ones);
        row_sum(own, first);
        find(nth - 1, first, own, ones, [&](int id, u64) {
          tell_border((u64)key << 32 | (0xFFFFFFFFu - (uint32_t)id));
        });
        b = told_border();
        return true;
      }
    }
  }

  // One thread of the cluster tells all CTAs.
  __device__ __forceinline__ void tell_border(u64 entry) {
    for (int r = 0; r < size(); ++r)
      *of(&sh.slot[phase % kSlots][0], r) = {0, 0, (uint32_t)(entry >> 32),
                                             0xFFFFFFFFu - (uint32_t)entry};
  }
  __device__ __forceinline__ Border told_border() {
    sync();
    const Slot s = told()[0];
    return {s.c, (int)s.d};
  }
};

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
template <typename E, bool HELD>
__device__ __forceinline__ void draw_listed(const RowArgs& a, Row<E, HELD>& row, int t, int n,
                                            const Weights& w, float top_p, float min_p) {
  Shared& sh = row.sh;
  constexpr int kEach = Row<E, HELD>::kEach;
  __shared__ int s_n;
  u64 x[kEach], all;
  if (top_p < 1.f) {
    u64 run = row.list_weights(n, w, [](u64 e) { return (uint32_t)(e >> 32); }, x, all);
    const u64 target = top_p_target(top_p, all);
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
      if (x[q] > 0 && run < target && run + x[q] >= target) s_n = (int)threadIdx.x * kEach + q + 1;
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
  const u64 least = min_p_weight(min_p, w(w.m));
  if (least > 0) {
    u64 s = 0;
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
      x[q] = x[q] >= least ? x[q] : 0ull;
      s += x[q];
    }
    run = row.scan(s, all);
  }
  const u64 target = draw_target(a.uniform[t], all);
#pragma unroll
  for (int q = 0; q < kEach; ++q) {
    if (target >= run && target < run + x[q])
      write_token(a, t, (int)(0xFFFFFFFFu - (uint32_t)(sh.list[threadIdx.x * kEach + q] >> 32)), x[q],
                  all);
    run += x[q];
  }
}

template <typename E, bool TOP, bool HELD>
__global__ void __launch_bounds__(kThreads, 2) rows_kernel(const RowArgs a) {
  extern __shared__ uint4 s_held[];
  __shared__ Shared sh;
  constexpr int VE = Vec<E>::n;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  Row<E, HELD> row(sh);
  const int rank = row.rank(), size = row.size(), t = blockIdx.x / size;
  const int per = ((a.V + size - 1) / size + VE - 1) / VE * VE;
  Part<E, HELD>& part = row.part;
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
  if (tid == 0) {
    sh.count = sh.claim = 0;
    sh.least_id = 0xFFFFFFFFu;
  }
  if (classes)
    for (int i = tid; i < kBins; i += kThreads) sh.mass[i] = 0;
  if (tid < kWarps) sh.extra[tid] = 0;
  row.started();

  // the row, its maximum, and for the k largest its sum of exponentials: 2^(z log2(e) - ref), ref
  // the rounded log2(e) times the running maximum
  float top = -INFINITY, sum = 0.f, ref = 0.f;
  // one CTA a row, and rows long enough: one pass does the rest too, where a look at a part of
  // the row tells what to expect
  const bool ahead = !HELD && !greedy && !classes && part.share >= 3 * 32 * kRing && (K <= 256 || !(TOP || cut_k));
  Weights ahead_w = {};
  u64 ahead_sum = 0;
  uint32_t first = 0xFFFFFFFFu;                  // greedy: the lowest id of the maximum
  auto look = [&](int v, const uint4& x) {
    const float best = fmaxf(top, Vec<E>::top(x));
    if (TOP && a.lse) {
      if (best > top) {
        const float r = best * kLog2e;
        sum = top > -INFINITY ? sum * fast_exp2(ref - r) : 0.f;
        ref = r;
      }
      float z[VE], s[4] = {};
      Vec<E>::get(x, z);
#pragma unroll
      for (int j = 0; j < VE; ++j) s[j % 4] += fast_exp2(fmaf(z[j], kLog2e, -ref));
      sum += (s[0] + s[1]) + (s[2] + s[3]);
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
    // half a warp's maxima
    float m = best;
#pragma unroll
    for (int o = 1; o < 16; o *= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (lane % 16 == 0) sh.half_top[warp * 2 + lane / 16] = m;
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
      float s = top > -INFINITY ? sum * fast_exp2(ref - cta_ref) : 0.f;
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
      if (!(total >= 0.f)) {
        // a logit is no number, or infinite: the sum of those that are
        const float m = value_of(key);
        float s1 = 0.f;
        part.each([&](int v, const uint4& raw) {
          float z[VE];
          Vec<E>::get(raw, z);
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            const float x = z[j] == m ? 0.f : fmaxf(z[j] - m, -150.f);
            s1 += z[j] > -INFINITY ? fast_exp2(x * kLog2e) : 0.f;
          }
        });
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
        a.lse[t] = key <= kNoKey                ? -INFINITY
                   : value_of(key) == INFINITY ? INFINITY
                                               : (top_ref + log2f(total)) * 0.693147181f;
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
            const u64 nth = (left - run + key_w[tid] - 1) / key_w[tid];
            for (int r = 0; r < size; ++r)
              *row.of(&sh.slot[row.phase % kSlots][0], r) = {nth, 1, k_hi - (uint32_t)tid, 0};
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
                   [&](int id, u64) {
                     row.tell_border((u64)key_b << 32 | (0xFFFFFFFFu - (uint32_t)id));
                   });
          b = row.told_border();
          if (w_b >= least) {
            const u64 kept_ties = nth > ties_before ? min(nth - ties_before, own_ties) : 0ull;
            const u64 own = own_above + warp_sum(kept_mass) + kept_ties * w_b;
            const u64 all = row.row_sum(own, before);
            row.find(draw_target(a.uniform[t], all), before, own, kept,
                     [&](int id, u64 x) { write_token(a, t, id, x, all); });
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
          constexpr int kOf = Row<E, HELD>::kEach;
          u64 x[kOf], all;
          row.list_weights(kept_n, w, [](u64 e) { return (uint32_t)(e >> 32); }, x, all);
#pragma unroll
          for (int q = 0; q < kOf; ++q) {
            const int i = tid * kOf + q;
            if (i >= kept_n) continue;
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
                     [&](int id, u64 x) { write_token(a, t, id, x, all); });
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
    // from the sums of the one pass.  (A lane's may have lost a unit in every octave it rose:
    // where the draw falls behind all of them, it is made anew.)
    int down = w.octave - ahead_w.octave;
    const u64 own = warp_sum(down < 64 ? ahead_sum >> max(0, down) : 0ull);
    const u64 mass = row.row_sum(own, before);
    if (tid == 0) sh.least_id = 0;
    __syncthreads();
    row.find(draw_target(a.uniform[t], mass), before, own, kept, [&](int id, u64 x) {
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
           [&](int id, u64 x) { write_token(a, t, id, x, mass); });
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
  const size_t smem = held ? bytes(c) : kRing * kThreads * 16;
  auto pick = [&](auto e, auto top, auto in) {
    return rows_kernel<typename decltype(e)::type, decltype(top)::value, decltype(in)::value>;
  };
  auto of_type = [&](auto e) {
    using Yes = std::true_type;
    using No = std::false_type;
    return a.tokens ? (held ? pick(e, No{}, Yes{}) : pick(e, No{}, No{}))
                    : (held ? pick(e, Yes{}, Yes{}) : pick(e, Yes{}, No{}));
  };
  void (*kernel)(RowArgs) =
      a.dtype == 0 ? of_type(std::common_type<float>{}) : of_type(std::common_type<__nv_bfloat16>{});
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
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace dspark
