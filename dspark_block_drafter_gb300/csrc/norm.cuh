// The norms around the end of a drafter block, and their gradient.
//
//   ry = 1 / sqrt(mean(y^2) + eps)   yn = y ry   p = s g yn (o + w_post)   (p = s g y without)
//   x' = x + p                       rx = 1 / sqrt(mean(x'^2) + eps)   xn = x' rx
//   h  = xn (o + w_pre)
//
// With a = dh (o + w_pre):
//   dx' = d_x_out + rx (a - xn mean(a xn))      dx = dx'     dw_pre = sum_t dh xn
//   dg = s dx' yn (o + w_post)                  du = s g dx'  dw_post = sum_t du yn
//   b = du (o + w_post)                         dy = ry (b - yn mean(b yn))
// where b yn = p dx', so that its mean too follows from sums over the row that need no dx':
//   sum p dx' = sum p d_x_out + rx sum p a - rx^2 mean(a xn) sum p x'
// A row takes two sums over the CTA: y^2, then the other five at once.
//
// Bound by memory: each input is read once and each output written once.  A CTA takes rows in
// turn, 8 or 16 elements a thread.  Each thread copies its own elements of the next row to
// shared memory (cp.async) while it works on this one's, which it reads there again after
// each sum instead of holding them in registers: two rows of 4096 are at work on an SM and
// two more on their way.  Everything is computed in fp32.  8192 rows of 4096, bf16, gate and
// both weights: 54 us forward (6.3 TB/s), 110 us backward with its sums (4.9 TB/s).  The gradient is
// bound by latency: registers and shared memory hold 16 warps on an SM, half the issue slots and 59%
// of the DRAM's time are used, and of the 7.6 cycles a warp takes for an instruction 1.4 are waits
// for rows on their way, 1.3 for shared memory and 0.9 for the sums' barriers.  (Its form for shared
// gate rows, with their sums in registers too, spills 22 words a thread.)
#pragma once

#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "launch.h"
#include "train.h"

namespace dspark {

namespace {

// Rows of one gate row that a CTA takes at a time: 16 in a large batch (their gate gradient
// is summed in registers), fewer where that would leave SMs without rows.
__host__ __device__ inline int norm_unit(int T) {
  return T >= 16 * 512 ? 16 : T >= 1024 ? T / 512 : 1;
}

// Threads of a row with `per` elements each.  Wide rows take 16 each, 512 threads at most: half
// the threads make half the shuffles of a sum, and their 128 registers hold what the gradient
// keeps (8192 rows of 4096, gradient: 512 threads at 64 registers 133 us, at 128 120 us; 256
// threads 108 us).
inline int row_per(int H) { return H > 2048 ? 16 : 8; }
inline int row_threads(int H) {
  const int n = row_per(H) * 32;
  return (H + n - 1) / n * 32;
}

// Two fp32 values in one 64-bit register, for the packed arithmetic (half the instructions).
struct F2 {
  unsigned long long v;
  __device__ __forceinline__ F2() {}
  __device__ __forceinline__ F2(float lo, float hi) {
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  }
  explicit __device__ __forceinline__ F2(float x) : F2(x, x) {}
  __device__ __forceinline__ float lo() const {
    float a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
    return a;
  }
  __device__ __forceinline__ float hi() const {
    float a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
    return b;
  }
};
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return d;
}

__device__ __forceinline__ F2 pair_of(const float* p) { return F2(p[0], p[1]); }
__device__ __forceinline__ F2 pair_of(const __nv_bfloat16* p) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
  return F2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// A thread's elements of one row of one tensor, as they lie in memory: vectors of VEC
// consecutive elements, the threads' vectors side by side.
template <typename E, int VEC, int kPer>
struct Part {
  struct alignas(sizeof(E) * VEC) Vec { E e[VEC]; };
  Vec v[kPer / VEC];

  static __device__ __forceinline__ int column(int e) {
    return ((e / VEC) * (int)blockDim.x + (int)threadIdx.x) * VEC + e % VEC;
  }
  // elements 2 q and 2 q + 1
  __device__ __forceinline__ void set(int q, F2 x) {
    if constexpr (sizeof(E) == 2 && VEC > 1) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x.lo(), x.hi());
      *reinterpret_cast<__nv_bfloat162*>(&v[2 * q / VEC].e[2 * q % VEC]) = b;
    } else {
      v[2 * q / VEC].e[2 * q % VEC] = (E)x.lo();
      v[(2 * q + 1) / VEC].e[(2 * q + 1) % VEC] = (E)x.hi();
    }
  }
  // stores the vectors that the pair ending in element e completes
  __device__ __forceinline__ void put(void* base, size_t row, int H, int e) const {
    E* p = (E*)base + row * H;
    if constexpr (VEC == 1) {
      if (column(e - 1) < H) *reinterpret_cast<Vec*>(p + column(e - 1)) = v[e - 1];
      if (column(e) < H) *reinterpret_cast<Vec*>(p + column(e)) = v[e];
    } else {
      const int q = e / VEC, c = column(q * VEC);
      if (e % VEC == VEC - 1 && c < H) *reinterpret_cast<Vec*>(p + c) = v[q];
    }
  }
};

// The current and the next row of N tensors in shared memory, and the two weight vectors
// (w_post, w_pre).  Vectors of 16, 8 or 4 bytes go to the thread's own places (so no barrier is
// needed).  bf16 rows that are not whole words (H odd, or an odd address) are copied word by
// word as they lie, and their threads meet at a barrier before they read single elements (a
// word may hold half a neighbouring row's element: in place it may be changing, and is not used).
template <typename E, int VEC, int N, int kPer>
struct Rows {
  static constexpr int kBytes = VEC * (int)sizeof(E);
  static constexpr bool kWords = kBytes < 4;
  static constexpr int kVecs = kPer / VEC;
  using P = Part<E, VEC, kPer>;
  using Vec = typename P::Vec;
  char* at;
  int H, stages;                              // 2: the next row is fetched ahead; 1: not
  int turn = 0;
  uint32_t odd = 0;                           // kWords: bit (stage N + n): the row lies one
                                              // element into its first word

  // bytes of one tensor's row
  static __host__ __device__ size_t row_bytes(int H, int threads) {
    return kWords ? (size_t)((H + 3) / 2) * 4 : (size_t)kPer * threads * sizeof(E);
  }
  static size_t smem(int H, int threads, int stages) {
    return (size_t)(stages * N + 2) * row_bytes(H, threads);
  }
  __device__ __forceinline__ char* row(int k) const { return at + k * row_bytes(H, blockDim.x); }
  __device__ __forceinline__ Vec* slot(int k, int q) const {
    return reinterpret_cast<Vec*>(row(k)) + q * blockDim.x + threadIdx.x;
  }
  // row k's element at column c (kWords)
  __device__ __forceinline__ float element(int k, int c) const {
    const E* e = reinterpret_cast<const E*>(row(k)) + ((odd >> k) & 1u);
    return c < H ? to_f32(e[c]) : 0.f;
  }
  __device__ __forceinline__ void init(char* smem_base, const NormArgs& a, int stages_) {
    at = smem_base;
    H = a.H;
    stages = stages_;
    if constexpr (!kWords) {                  // zeros past the row, for good
      Vec none;
#pragma unroll
      for (int j = 0; j < VEC; ++j) none.e[j] = (E)0.f;
#pragma unroll
      for (int q = 0; q < kVecs; ++q)
        if (P::column(q * VEC) >= H)
          for (int k = 0; k < stages * N + 2; ++k) *slot(k, q) = none;
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const E* base = (const E*)(w ? a.w_pre : a.w_post);
      if (!base) continue;
      if constexpr (kWords) {
        E* to = reinterpret_cast<E*>(row(stages * N + w));
        for (int c = threadIdx.x; c < H; c += blockDim.x) to[c] = base[c];
      } else {
        copy(stages * N + w, base);
      }
    }
  }
  // the thread's vectors of a row at p; they are there after the next next()
  __device__ __forceinline__ void copy(int k, const E* p) const {
#pragma unroll
    for (int q = 0; q < kVecs; ++q) {
      const int c = P::column(q * VEC);
      const uint32_t to = (uint32_t)__cvta_generic_to_shared(slot(k, q));
      if (c >= H) continue;
      if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p + c) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(p + c), "n"(kBytes)
                     : "memory");
    }
  }
  __device__ __forceinline__ bool ahead() const { return stages == 2; }
  // start on row r of tensor n, the next one when ahead.  `last`: nothing of the tensor follows
  __device__ __forceinline__ void fetch(int n, const void* base, size_t r, bool last) {
    const int k = (ahead() ? turn ^ 1 : 0) * N + n;
    const E* p = (const E*)base + r * H;
    if constexpr (kWords) {
      const int skip = (int)((uintptr_t)p >> 1) & 1;
      odd = (odd & ~(1u << k)) | (uint32_t)skip << k;
      E* to = reinterpret_cast<E*>(row(k));
      for (int w = threadIdx.x; 2 * w < H + skip; w += blockDim.x) {
        const int c = 2 * w - skip;           // the word holds columns c, c + 1
        if ((c < 0 && r == 0) || (c + 1 >= H && last)) {
          if (c >= 0) to[2 * w] = p[c];       // (the other half lies outside the tensor)
          if (c + 1 < H) to[2 * w + 1] = p[c + 1];
        } else {
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                           (uint32_t)__cvta_generic_to_shared(to + 2 * w)),
                       "l"(p + c)
                       : "memory");
        }
      }
    } else {
      copy(k, p);
    }
  }
  __device__ __forceinline__ void commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // the fetched row becomes the current one
  __device__ __forceinline__ void next() {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (ahead()) turn ^= 1;
    if (kWords) __syncthreads();
  }
  // elements [4 c, 4 c + 4) of the current row of tensor n, or of a weight vector
  __device__ __forceinline__ void four(F2 (&x)[2], int n, int c) const { place(x, turn * N + n, c); }
  __device__ __forceinline__ void weight_four(F2 (&x)[2], int w, int c) const {
    place(x, stages * N + w, c);
  }
  __device__ __forceinline__ void place(F2 (&x)[2], int k, int c) const {
    if constexpr (kWords) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        x[j] = F2(element(k, P::column(4 * c + 2 * j)), element(k, P::column(4 * c + 2 * j + 1)));
    } else if constexpr (VEC >= 4) {
      struct alignas(4 * sizeof(E)) Four { E e[4]; };
      const Four f = *(reinterpret_cast<const Four*>(slot(k, 4 * c / VEC)) + 4 * c % VEC / 4);
      x[0] = pair_of(f.e);
      x[1] = pair_of(f.e + 2);
    } else if constexpr (VEC == 2) {
#pragma unroll
      for (int j = 0; j < 2; ++j) x[j] = pair_of(slot(k, 2 * c + j)->e);
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        x[j] = F2(to_f32(slot(k, 4 * c + 2 * j)->e[0]), to_f32(slot(k, 4 * c + 2 * j + 1)->e[0]));
    }
  }
};

// Sums of up to five values over the CTA, in a fixed order.  Two buffers taken in turn make
// one barrier a sum enough.
struct RowSum {
  float (*s)[32][5];
  int turn;
  template <int N>
  __device__ __forceinline__ void operator()(float (&v)[N]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] += __shfl_xor_sync(0xFFFFFFFFu, v[j], o);
    const int warps = blockDim.x / 32, lane = threadIdx.x % 32;
    if (warps == 1) return;
    if (lane == 0)
#pragma unroll
      for (int j = 0; j < N; ++j) s[turn][threadIdx.x / 32][j] = v[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = lane < warps ? s[turn][lane][j] : 0.f;
    turn ^= 1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] += __shfl_xor_sync(0xFFFFFFFFu, v[j], o);
  }
};

extern __shared__ uint4 norm_smem[];     // (16-byte aligned)

template <typename E, int VEC, int kPer>
__global__ void __launch_bounds__(32 * kPer, 1) block_norm(const NormArgs a, int stages) {
  using P = Part<E, VEC, kPer>;
  __shared__ float s_sum[2][32][5];
  RowSum sum{s_sum, 0};
  pdl_wait();
  pdl_signal();
  const int H = a.H;
  const float inv_h = 1.f / (float)H;
  Rows<E, VEC, 3, kPer> rows;                 // x, y, gate
  rows.init((char*)norm_smem, a, stages);
  auto fetch = [&](int t) {
    if (t < a.T) {
      const bool last = t == a.T - 1;
      rows.fetch(0, a.x, t, last);
      if (a.y) rows.fetch(1, a.y, t, last);
      if (a.gate) rows.fetch(2, a.gate, t / a.span, t / a.span == (a.T - 1) / a.span);
    }
    rows.commit();
  };
  if (rows.ahead()) fetch(blockIdx.x);
  const F2 off(a.offset);
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    if (!rows.ahead()) fetch(t);
    rows.next();
    if (rows.ahead()) fetch(t + gridDim.x);
    F2 x[kPer / 2];
#pragma unroll
    for (int c = 0; c < kPer / 4; ++c) {
      F2 f[2];
      rows.four(f, 0, c);
      x[2 * c] = f[0];
      x[2 * c + 1] = f[1];
    }
    if (a.y) {
      float f = a.scale;
      if (a.w_post) {
        F2 s2(0.f);
#pragma unroll
        for (int c = 0; c < kPer / 4; ++c) {
          F2 y[2];
          rows.four(y, 1, c);
          s2 = fma2(y[0], y[0], s2);
          s2 = fma2(y[1], y[1], s2);
        }
        float ss[1] = {s2.lo() + s2.hi()};
        sum(ss);
        f *= rsqrtf(ss[0] * inv_h + a.eps);
      }
      const F2 f2(f);
#pragma unroll
      for (int c = 0; c < kPer / 4; ++c) {
        F2 y[2], g[2], w[2];
        rows.four(y, 1, c);
        if (a.gate) rows.four(g, 2, c);
        if (a.w_post) rows.weight_four(w, 0, c);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          F2 u = y[j];
          if (a.w_post) u = u * (off + w[j]);
          if (a.gate) u = u * g[j];
          x[2 * c + j] = fma2(f2, u, x[2 * c + j]);
        }
      }
    }
    P out;
    F2 s2(0.f);
#pragma unroll
    for (int q = 0; q < kPer / 2; ++q) {
      s2 = fma2(x[q], x[q], s2);              // (0 past the row)
      if (a.x_out) {
        out.set(q, x[q]);
        out.put(a.x_out, t, H, 2 * q + 1);
      }
    }
    float ss[1] = {s2.lo() + s2.hi()};
    sum(ss);
    const F2 rx2(rsqrtf(ss[0] * inv_h + a.eps));
#pragma unroll
    for (int c = 0; c < kPer / 4; ++c) {
      F2 w[2];
      rows.weight_four(w, 1, c);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        out.set(2 * c + j, x[2 * c + j] * rx2 * (off + w[j]));
        out.put(a.h, t, H, 2 * (2 * c + j) + 1);
      }
    }
  }
}

// A unit is up to norm_unit(T) consecutive rows of one gate row (one row without shared gate
// rows); a CTA takes units in turn and keeps its column sums in registers.
// GATE: 0 none, 1 a gate row for each row, 2 shared gate rows, whose gradients are sums too.
// FULL: y, w_post and d_x_out are all there (else what is there is looked up).
template <typename E, int VEC, int kPer, int GATE, bool FULL>
__global__ void __launch_bounds__(32 * kPer, 1) block_norm_backward(const NormArgs a, int units,
                                                               int per_span, int stages) {
  using P = Part<E, VEC, kPer>;
  constexpr bool kShared = GATE == 2;
  const bool has_y = FULL || a.y, has_post = FULL || a.w_post, has_up = FULL || a.d_x_out;
  __shared__ float s_sum[2][32][5];
  RowSum sum{s_sum, 0};
  pdl_wait();
  pdl_signal();
  const int H = a.H;
  const float inv_h = 1.f / (float)H;
  const F2 off(a.offset), zero2(0.f);
  F2 dw_pre[kPer / 2], dw_post[kPer / 2], dg[kShared ? kPer / 2 : 1];
#pragma unroll
  for (int e = 0; e < kPer / 2; ++e) {
    dw_pre[e] = dw_post[e] = zero2;
    if (kShared) dg[e] = zero2;
  }
  Rows<E, VEC, 5, kPer> rows;                       // x, dh, y, d_x_out, gate
  rows.init((char*)norm_smem, a, stages);
  // row t of rows [t, t1) of unit un
  int un = blockIdx.x, t = 0, t1 = 0;
  auto settle = [&]() {
    if (!kShared) {
      t = un;
      t1 = un + 1;
      return;
    }
    const int unit_rows = norm_unit(a.T);
    while (un < units) {
      const int row_g = un / per_span;
      t = row_g * a.span + un % per_span * unit_rows;
      t1 = min(min(a.T, (row_g + 1) * a.span), t + unit_rows);
      if (t < t1) break;
      // (the last gate row's last units may hold no row: their part of d_gate is zero)
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        if (P::column(e) < H) a.gate_part[(size_t)un * H + P::column(e)] = 0.f;
      un += gridDim.x;
    }
  };
  auto fetch = [&]() {
    if (un < units) {
      const bool last = t == a.T - 1;
      const int row_g = kShared ? un / per_span : t;
      rows.fetch(0, a.x, t, last);
      rows.fetch(1, a.d_h, t, last);
      if (has_y) rows.fetch(2, a.y, t, last);
      if (has_up) rows.fetch(3, a.d_x_out, t, last);
      if (GATE) rows.fetch(4, a.gate, row_g, row_g == (a.T - 1) / a.span);
    }
    rows.commit();
  };
  settle();
  if (rows.ahead()) fetch();
  while (un < units) {
    const int row = t, unit = un;
    if (!rows.ahead()) fetch();
    rows.next();
    if (++t == t1) {
      un += gridDim.x;
      settle();
    }
    if (rows.ahead()) fetch();
    float f = a.scale, ry = 1.f;              // p = f g y (o + w_post)
    if (has_post) {
      F2 s2 = zero2;
#pragma unroll
      for (int c = 0; c < kPer / 4; ++c) {
        F2 y[2];
        rows.four(y, 2, c);
        s2 = fma2(y[0], y[0], s2);
        s2 = fma2(y[1], y[1], s2);
      }
      float ss[1] = {s2.lo() + s2.hi()};
      sum(ss);
      ry = rsqrtf(ss[0] * inv_h + a.eps);
      f *= ry;
    }
    // Four elements at a time, read from shared memory when their turn comes (the fences keep
    // the compiler from reading ahead, which took more registers than there are).
    F2 v2[5] = {zero2, zero2, zero2, zero2, zero2};   // x'^2, a x', p x', p a, p d_x_out
    const F2 f2(f);
#pragma unroll
    for (int c = 0; c < kPer / 4; ++c) {
      F2 x[2], y[2], g[2], h[2], d[2], wo[2], wi[2];
      asm volatile("" ::: "memory");
      rows.four(x, 0, c);
      rows.four(h, 1, c);
      rows.weight_four(wi, 1, c);
      if (has_y) rows.four(y, 2, c);
      if (has_up) rows.four(d, 3, c);
      if (GATE) rows.four(g, 4, c);
      if (has_post) rows.weight_four(wo, 0, c);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        F2 p = zero2;
        if (has_y) {
          p = f2 * y[j];
          if (has_post) p = p * (off + wo[j]);
          if (GATE) p = p * g[j];
        }
        const F2 xx = x[j] + p, aa = h[j] * (off + wi[j]);
        v2[0] = fma2(xx, xx, v2[0]);
        v2[1] = fma2(aa, xx, v2[1]);
        v2[2] = fma2(p, xx, v2[2]);
        v2[3] = fma2(p, aa, v2[3]);
        if (has_up) v2[4] = fma2(p, d[j], v2[4]);
      }
    }
    float v[5];
#pragma unroll
    for (int j = 0; j < 5; ++j) v[j] = v2[j].lo() + v2[j].hi();
    sum(v);
    const float rx = rsqrtf(v[0] * inv_h + a.eps);
    const float mean = v[1] * inv_h * rx;                       // mean(a xn)
    const float mb = (v[4] + rx * v[3] - rx * rx * mean * v[2]) * inv_h;   // mean(b yn)
    const F2 rx2(rx), ry2(ry), m2(-mean), mb2(-mb), s2(a.scale);
    P o_dx, o_dy, o_dg;
#pragma unroll
    for (int c = 0; c < kPer / 4; ++c) {
      F2 x[2], y[2], g[2], h[2], d[2], wo[2], wi[2];
      asm volatile("" ::: "memory");
      rows.four(x, 0, c);
      rows.four(h, 1, c);
      rows.weight_four(wi, 1, c);
      if (has_y) rows.four(y, 2, c);
      if (has_up) rows.four(d, 3, c);
      if (GATE) rows.four(g, 4, c);
      if (has_post) rows.weight_four(wo, 0, c);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int q = 2 * c + j;
        F2 u = zero2, ow;                                       // u = s yn (o + w_post)
        if (has_y) u = f2 * y[j];
        if (has_post) {
          ow = off + wo[j];
          u = u * ow;
        }
        const F2 xn = (GATE ? fma2(g[j], u, x[j]) : x[j] + u) * rx2;
        dw_pre[q] = fma2(h[j], xn, dw_pre[q]);
        const F2 in = fma2(xn, m2, h[j] * (off + wi[j]));
        const F2 dx = has_up ? fma2(rx2, in, d[j]) : rx2 * in;
        o_dx.set(q, dx);
        o_dx.put(a.d_x, row, H, 2 * q + 1);
        if (kShared) {
          dg[q] = fma2(dx, u, dg[q]);
        } else if (GATE) {
          o_dg.set(q, dx * u);
          o_dg.put(a.d_gate, row, H, 2 * q + 1);
        }
        if (has_y) {
          const F2 du = GATE ? (s2 * g[j]) * dx : s2 * dx;
          F2 dy = du;
          if (has_post) {
            const F2 yn = y[j] * ry2;
            dw_post[q] = fma2(du, yn, dw_post[q]);
            dy = ry2 * fma2(yn, mb2, du * ow);
          }
          o_dy.set(q, dy);
          o_dy.put(a.d_y, row, H, 2 * q + 1);
        }
      }
    }
    if constexpr (kShared) {
      if (un != unit) {                       // the unit is done
#pragma unroll
        for (int q = 0; q < kPer / 2; ++q) {
          if (per_span == 1) {
            o_dg.set(q, dg[q]);
            o_dg.put(a.d_gate, unit, H, 2 * q + 1);
          } else {
            float* to = a.gate_part + (size_t)unit * H;
            if (P::column(2 * q) < H) to[P::column(2 * q)] = dg[q].lo();
            if (P::column(2 * q + 1) < H) to[P::column(2 * q + 1)] = dg[q].hi();
          }
          dg[q] = zero2;
        }
      }
    }
  }
  float* part = a.w_part + (size_t)blockIdx.x * H;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int c = P::column(e);
    if (c >= H) continue;
    part[c] = e & 1 ? dw_pre[e / 2].hi() : dw_pre[e / 2].lo();
    if (has_post)
      part[(size_t)gridDim.x * H + c] = e & 1 ? dw_post[e / 2].hi() : dw_post[e / 2].lo();
  }
}

// Column sums of part[rows][H] in a fixed order: 32 columns and 32 interleaved row lanes a CTA.
template <typename E>
__global__ void __launch_bounds__(1024) column_sums(const float* part, int rows, int H, E* out0,
                                                   E* out1) {
  __shared__ float s[32][33];
  pdl_wait();
  pdl_signal();
  const int c = blockIdx.x * 32 + threadIdx.x % 32, lane = threadIdx.x / 32;
  const float* p = part + (size_t)blockIdx.y * rows * H;
  float a = 0.f;
  if (c < H)
#pragma unroll 4
    for (int r = lane; r < rows; r += 32) a += p[(size_t)r * H + c];
  s[lane][threadIdx.x % 32] = a;
  __syncthreads();
  if (lane != 0 || c >= H) return;
  for (int j = 1; j < 32; ++j) a += s[j][threadIdx.x];
  (blockIdx.y == 0 ? out0 : out1)[c] = (E)a;
}

// d_gate rows of shared gate rows, from their parts in order: 256 of them at a time, then those sums
// (one chain over 65536 parts was off by 8e-6).
template <typename E>
__global__ void __launch_bounds__(128) gate_sums(const float* part, int per_span, int H, E* out) {
  pdl_wait();
  pdl_signal();
  const int c = blockIdx.y * 128 + threadIdx.x;
  if (c >= H) return;
  const float* p = part + (size_t)blockIdx.x * per_span * H + c;
  float a = 0.f;
  for (int j0 = 0; j0 < per_span; j0 += 256) {
    const int j1 = min(per_span, j0 + 256);
    float part_sum = 0.f;
#pragma unroll 8
    for (int j = j0; j < j1; ++j) part_sum += p[(size_t)j * H];
    a += part_sum;
  }
  out[(size_t)blockIdx.x * H + c] = (E)a;
}

// Bytes of a vector that every row of every tensor is made of: 16, 8, 4, or 2 (words with odd
// ends).  What narrow ones cost: 8192 bf16 rows of 4096, 4100, 4098 and 4097, gradient, take 115,
// 208, 278 and 562 us, forward 58, 64, 113 and 175 us (a row above 4096 also has its SM alone);
// loaded into registers, without a copy ahead, rows of 4955 took 693 us instead of 476, and 304
// instead of 154.  4096 fp32 rows of 4096, 4098 and 4097, gradient: 93, 181 and 293 us.
inline int vector_bytes(const NormArgs& a) {
  const int es = a.dtype == DSPARK_F32 ? 4 : 2;
  uintptr_t all = (uintptr_t)a.H * es;
  for (const void* p : {a.x, a.y, a.gate, a.w_post, a.w_pre, a.d_h, a.d_x_out,
                        (const void*)a.x_out, (const void*)a.h, (const void*)a.d_x,
                        (const void*)a.d_y, (const void*)a.d_gate})
    all |= (uintptr_t)p;
  return all % 16 == 0 ? 16 : all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : 2;
}

// CTAs that are resident at once, at most `items`.
inline cudaError_t resident(const void* kernel, int threads, size_t smem, int items, int* grid) {
  int sms = 0, per_sm = 0;
  cudaError_t e = device_sms(&sms);
  if (e == cudaSuccess && smem > 0) e = raise_smem_limit(kernel, smem);
  if (e == cudaSuccess) e = blocks_per_sm(kernel, threads, smem, &per_sm);
  *grid = std::min(items, std::max(1, per_sm) * sms);
  return e;
}

// Rows in flight: two where they fit (fp32 rows above 4608 with five tensors do not), else one.
constexpr size_t kSmemMost = 226 * 1024 - 1280;

template <typename E, int VEC, int kPer>
cudaError_t forward(const NormArgs& a) {
  using R = Rows<E, VEC, 3, kPer>;
  const int threads = row_threads(a.H);
  const int stages = R::smem(a.H, threads, 2) <= kSmemMost ? 2 : 1;
  const size_t smem = R::smem(a.H, threads, stages);
  int grid = 0;
  const cudaError_t e =
      resident((const void*)block_norm<E, VEC, kPer>, threads, smem, a.T, &grid);
  if (e != cudaSuccess) return e;
  return launch_after(block_norm<E, VEC, kPer>, grid, threads, smem, a.stream, a, stages);
}

template <typename E, int VEC, int kPer, int GATE, bool FULL>
cudaError_t backward(const NormArgs& a) {
  using R = Rows<E, VEC, 5, kPer>;
  const int threads = row_threads(a.H);
  const int stages = R::smem(a.H, threads, 2) <= kSmemMost ? 2 : 1;
  const size_t smem = R::smem(a.H, threads, stages);
  const int per_span = GATE == 2 ? norm_span_parts(a.T, a.span) : 1;
  const int units = GATE == 2 ? (a.T + a.span - 1) / a.span * per_span : a.T;
  const auto kernel = block_norm_backward<E, VEC, kPer, GATE, FULL>;
  int grid = 0;
  cudaError_t e = resident((const void*)kernel, threads, smem, units, &grid);
  if (e != cudaSuccess) return e;
  grid = std::min(grid, norm_max_ctas(a.H));
  e = launch_after(kernel, grid, threads, smem, a.stream, a, units, per_span, stages);
  if (e == cudaSuccess)
    e = launch_after(column_sums<E>, dim3((a.H + 31) / 32, a.w_post ? 2 : 1), 1024, 0, a.stream,
                     a.w_part, grid, a.H, (E*)a.d_w_pre, (E*)a.d_w_post);
  if (e == cudaSuccess && per_span > 1)
    e = launch_after(gate_sums<E>, dim3(units / per_span, (a.H + 127) / 128), 128, 0, a.stream,
                     a.gate_part, per_span, a.H, (E*)a.d_gate);
  return e;
}

template <typename E, int VEC, int kPer>
cudaError_t backward_of(const NormArgs& a) {
  constexpr bool kFull = VEC * sizeof(E) == 16;
  const bool full = kFull && a.y && a.w_post && a.d_x_out;
  if (!a.gate)
    return full ? backward<E, VEC, kPer, 0, kFull>(a) : backward<E, VEC, kPer, 0, false>(a);
  if (a.span == 1)
    return full ? backward<E, VEC, kPer, 1, kFull>(a) : backward<E, VEC, kPer, 1, false>(a);
  return full ? backward<E, VEC, kPer, 2, kFull>(a) : backward<E, VEC, kPer, 2, false>(a);
}

template <typename E, int VEC>
cudaError_t launch_of(const NormArgs& a, bool grad) {
  if (row_per(a.H) == 16) return grad ? backward_of<E, VEC, 16>(a) : forward<E, VEC, 16>(a);
  return grad ? backward_of<E, VEC, 8>(a) : forward<E, VEC, 8>(a);
}

}  // namespace

}  // namespace dspark
