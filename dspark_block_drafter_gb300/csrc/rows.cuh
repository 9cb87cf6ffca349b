// A row of logits in the hands of one CTA, or of a cluster: its elements, its weights, and what is
// done over all of it (sums by id, lists of the largest, borders by histograms).
//
// Weights are whole numbers: w = e^((z - max) / temperature) in units of 2^-S of about the
// largest (S = 44 for a vocabulary of 2^18), each off by at most 2^-27 of itself and cut to whole
// units.  Sums of them are exact in 64 bits, in any order and by atomics too, so that the same row
// gives the same token however it is split, and a border of a long sum lies where the
// definition has it.  (An fp32 sum of 151936 weights is off by some 1e-7 of itself: among as many
// tokens, that is the next token in one row of a hundred.)  The one sum that is taken before the
// largest is known is in finer units; a draw from it counts where that cannot matter, and is made
// anew where it could (k_sample.cu).
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace dspark {

namespace {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

constexpr int kBins = 2048;
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

// LIST: entries of a list; NT: threads.
template <int LIST, int NT>
struct Shared {
  static constexpr int kList = LIST, kWarps = NT / 32;
  union {
    struct {
      uint32_t cnt[kBins], lo[kBins], hi[kBins];
    } h;
    struct {
      u64 list[LIST];
      uint32_t mass[kBins];         // of this CTA's elements, in the first CTA then of all
    };
  };
  Slot slot[kSlots][kMaxCluster];
  u64 warp_sum[kWarps], extra[kWarps];
  uint32_t warp_key[kWarps], warp_top[kWarps];
  float warp_f[kWarps], half_top[32];
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

// An fp32 sum of many values that is as good for many as for a few: chains of values, and the
// chains' sums with their rounding errors (Knuth's two-sum).  A plain sum of 4000 equal values,
// whose roundings go one way within an octave, was off by 5e-5 of itself.
struct LongSum {
  float sum = 0.f, err = 0.f, chain = 0.f;
  __device__ __forceinline__ void add(float x, bool last) {
    chain += x;
    if (!last) return;
    const float t = sum + chain, b = t - sum;
    err += (sum - (t - b)) + (chain - b);
    sum = t;
    chain = 0.f;
  }
  __device__ __forceinline__ void scale(float x) {
    sum *= x;
    err *= x;
    chain *= x;
  }
  __device__ __forceinline__ float value() const { return sum + (err + chain); }
};
// Whether a lane's vector v is the last of a chain of 32: alike in all lanes of its warp.
__device__ __forceinline__ bool chain_ends(int v) {
  return ((v - (int)(threadIdx.x % 32)) & 0x3E0) == 0x3E0;
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
    octave = 0;
    raise(top);
  }
  // makes room for a logit of `top`; the octaves that this took
  __device__ __forceinline__ int raise(float top) {
    const int was = octave;
    // steps of 1/32 up to it, in whole octaves (a row with one above 60000 is far, and what the
    // weights before it made is not used)
    octave = far ? 1 : ((__float2int_ru(fminf(__fmul_rn(top, c_hi), 65536.f) * 32.f) + 2) >> 5) + 1;
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
  float m, c;               // the maximum, 64 log2(e) / temperature
  __device__ __forceinline__ float step(float z) const {
    return fminf(__fmul_rn(__fsub_rn(m, z), c), (float)(kBins - 1));
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
template <typename E, bool HELD, int NT>
struct Part {
  static constexpr int VE = Vec<E>::n, kThreads = NT;
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
  static __device__ __forceinline__ void copy16(uint32_t to, const uint4* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  }
  // Vector v to `to` in shared memory, without waiting for it.
  __device__ __forceinline__ void copy(int v, uint4* to) const {
    const int a = v * VE;
    if (a >= lead && a + VE <= lead + n)
      copy16((uint32_t)__cvta_generic_to_shared(to), reinterpret_cast<const uint4*>(g) + v);
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
    // kRing / 2 pairs of vectors on their way; whole ones only (the first and the last of a row may
    // not be)
    constexpr uint32_t kSlot = kThreads * 16, kAll = kRing * kSlot;
    uint4* ring = held + threadIdx.x;
    const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
    const int whole = min(v1, (lead + n) / VE);
#pragma unroll
    for (int q = 0; q < kRing; ++q) {
      const int v = v0 + 32 * q + lane;
      if (v < whole) copy(v, ring + q * kThreads);
      if (q % 2) copied();
    }
    const uint4* src = reinterpret_cast<const uint4*>(g) + v0 + 32 * kRing + lane;
    uint32_t at = 0;
    // two at a time, so that their arithmetic overlaps
    for (int v = v0 + lane; v - lane < v1; v += 64, src += 64) {
      arrived<kRing / 2 - 1>();
      uint4 x = ring[at / 16], y = ring[(at + kSlot) / 16];
      if (v >= whole) x = v < v1 ? load(v) : Vec<E>::none();
      if (v + 32 >= whole) y = v + 32 < v1 ? load(v + 32) : Vec<E>::none();
      if (v + 32 * kRing < whole) copy16(ring_s + at, src);
      if (v + 32 * kRing + 32 < whole) copy16(ring_s + at + kSlot, src + 32);
      copied();
      at = (at + 2 * kSlot) % kAll;
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
template <typename E, bool HELD, int NT>
struct Row {
  static constexpr int VE = Vec<E>::n, kThreads = NT, kWarps = NT / 32;
  // (a CTA that holds no part of its row has room for a longer list)
  using Sh = Shared<HELD ? 2048 : 4096, NT>;
  static constexpr int kList = Sh::kList;
  Sh& sh;
  Part<E, HELD, NT> part;
  int phase;

  __device__ __forceinline__ Row(Sh& s) : sh(s), phase(0) {}
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
  // The first id at which the running sum exceeds `target`: found(id, x, past) is called by one
  // thread of the cluster; `past`: how far into this id's x the target lies.
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
          found(part.id(v, j), x[j], x[j] - (run - left));
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
    if (!(cl.step(Vec<E>::top(raw)) < (float)(kBins - 1))) return;       // all in the last class
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

  // Weights of this CTA's first n list entries, list_each(n) a thread in order, and the sum before the
  // thread's; key_at(entry) is an entry's order key.
  static constexpr int kEach = kList / kThreads;
  template <typename W, typename F>
  __device__ __forceinline__ u64 list_weights(int n, const W& w, F key_at, u64 (&x)[kEach],
                                              u64& all) {
    u64 s = 0;
    const int each = list_each(n);
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
      x[q] = 0;
      if (q >= each) continue;
      const int i = threadIdx.x * each + q;
      const u64 y = w(value_of(i < n ? key_at(sh.list[i]) : kNoKey));
      x[q] = i < n ? y : 0ull;
      s += x[q];
    }
    return scan(s, all);
  }
  static __device__ __forceinline__ int list_each(int n) { return n <= kThreads ? 1 : kEach; }
  // The first entry with which the mass of the sorted list reaches `target`, by one thread:
  // found(index, mass before it, its own).
  template <typename W, typename F>
  __device__ __forceinline__ void list_mass(int n, const W& w, u64 target, F found) {
    u64 x[kEach], all;
    u64 run = list_weights(n, w, [](u64 e) { return (uint32_t)(e >> 32); }, x, all);
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
      if (x[q] > 0 && run < target && run + x[q] >= target)
        found((int)threadIdx.x * list_each(n) + q, run, x[q]);
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
          const Sh* o = of(&sh, r);
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
        find(nth - 1, first, own, ones, [&](int id, u64, u64) {
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

}  // namespace

}  // namespace dspark
