// Rows of the embedding table, and the table's gradient.
//
//   out[t]     = s table[ids[t]]                                   (0 where ids[t] is no token)
//   d_table[v] = add[v] + s sum of d_out[t] over ids[t] = v
//
// Both are bound by memory.  The gradient sorts the rows by their token (a stable radix sort,
// so that a token's rows stay in their order and its sum is taken in that order whatever the
// launch looks like), cuts the sorted list into chunks of equal length, and sums the runs of
// equal tokens of each chunk in registers: frequent tokens then cost no more than others.  A run
// that ends in its chunk is written to the table; the parts of one that chunks share are
// joined by a last kernel, in order.  Rows of the table that no token asks for are written
// while one CTA sorts (up to kSortAll rows: each CTA finds out about its own rows of the table
// by looking at every token), or by a bit map of the tokens that occur.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "launch.h"
#include "tokens.h"

namespace dspark {

namespace {

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kSortAll = 16384;          // rows that one CTA sorts in its shared memory
constexpr int kTile = 4096;              // rows of one CTA of the sort of more
constexpr int kDigit = 8, kDigits = 1 << kDigit;
constexpr int kMaxChunk = 512;
constexpr int kSumThreads = 256;

template <typename E, int VE>
struct alignas(sizeof(E) * VE) Pack {
  E e[VE];
};

template <typename E>
__device__ __forceinline__ E rounded(float x);
template <>
__device__ __forceinline__ float rounded<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float x) {
  return __float2bfloat16(x);
}

// ------------------------------------------------------------------ lookup
// CTA (b, c): rows [b rows, ...) of columns of block c, `rows` loads of a thread in flight.
template <typename E, int VE, int ROWS>
__global__ void __launch_bounds__(256) embed_rows(const EmbedArgs a) {
  using P = Pack<E, VE>;
  pdl_wait();
  pdl_signal();
  const int per = a.H / VE, t0 = blockIdx.x * ROWS;
  const int c = blockIdx.y * blockDim.x + threadIdx.x;
  int id[ROWS];
#pragma unroll
  for (int q = 0; q < ROWS; ++q) id[q] = t0 + q < a.T ? a.ids[t0 + q] : -1;
  if (c >= per) return;
  P x[ROWS];
#pragma unroll
  for (int q = 0; q < ROWS; ++q) {
    if (id[q] >= 0 && id[q] < a.V) {
      x[q] = reinterpret_cast<const P*>(a.table)[(size_t)id[q] * per + c];
#pragma unroll
      for (int j = 0; j < VE; ++j) x[q].e[j] = rounded<E>(a.scale * to_f32(x[q].e[j]));
    } else {
#pragma unroll
      for (int j = 0; j < VE; ++j) x[q].e[j] = rounded<E>(0.f);
    }
  }
#pragma unroll
  for (int q = 0; q < ROWS; ++q)
    if (t0 + q < a.T) reinterpret_cast<P*>(a.out)[(size_t)(t0 + q) * per + c] = x[q];
}

// ------------------------------------------------------------------ sorting
// The sort key of row t: its token, or V (sorted last) where it has none.
__device__ __forceinline__ uint32_t sort_key(const EmbedArgs& a, int t) {
  const int id = a.ids[t];
  if (id >= a.V) flag_error(a.ctrl, kErrBadToken);
  return id >= 0 && id < a.V ? (uint32_t)id : (uint32_t)a.V;
}

// The exclusive sum over the CTA's threads.
__device__ __forceinline__ uint32_t block_before(uint32_t v, uint32_t* s_warp) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  uint32_t in = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, in, o);
    if (lane >= o) in += y;
  }
  if (lane == 31) s_warp[warp] = in;
  __syncthreads();
  uint32_t w = s_warp[lane];                       // (32 warps)
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, w, o);
    if (lane >= o) w += y;
  }
  const uint32_t before = warp > 0 ? __shfl_sync(0xFFFFFFFFu, w, warp - 1) : 0u;
  __syncthreads();
  return before + in - v;
}

// The places of R items a thread among the CTA's by their digit, equal digits in the items'
// order: warp w holds items [32 R w, 32 R (w + 1)), item r of a lane is 32 r + lane of those.
// cnt: [warps][kDigits]; afterwards place[r] + cnt[warp][digit] is an item's place.
template <int R>
__device__ __forceinline__ void rank_items(const uint32_t (&digit)[R], uint32_t (&place)[R],
                                           uint32_t* cnt, uint32_t* s_warp) {
  const int tid = threadIdx.x, lane = tid % 32;
  uint32_t* mine = cnt + (tid / 32) * kDigits;
  for (int i = tid; i < kSortWarps * kDigits; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    // (items past the end have a digit of their own, and are not counted)
    const unsigned peers = __match_any_sync(0xFFFFFFFFu, digit[r]);
    const bool in = digit[r] < kDigits;
    const uint32_t before = __popc(peers & ((1u << lane) - 1u));
    const uint32_t base = in ? mine[digit[r]] : 0u;
    __syncwarp();
    if (in && before == 0) mine[digit[r]] = base + __popc(peers);
    __syncwarp();
    place[r] = base + before;
  }
  __syncthreads();
  // counts become offsets, digit by digit and in each warp by warp: eight a thread
  static_assert(kSortWarps * kDigits == 8 * kSortThreads, "eight counts a thread");
  const int d = tid / 4, w0 = tid % 4 * 8;
  uint32_t x[8], s = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    x[q] = cnt[(w0 + q) * kDigits + d];
    s += x[q];
  }
  uint32_t at = block_before(s, s_warp);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    cnt[(w0 + q) * kDigits + d] = at;
    at += x[q];
  }
  __syncthreads();
}

// Sorts all rows, in shared memory: s_key, s_pos [1024 R] and the counts.
template <int R>
__device__ void sort_all(const EmbedArgs& a, uint32_t* smem) {
  __shared__ uint32_t s_warp[32];
  uint32_t* s_key = smem;
  uint32_t* s_pos = smem + kSortThreads * R;
  uint32_t* cnt = smem + 2 * kSortThreads * R;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  uint32_t key[R], pos[R], digit[R], place[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    pos[r] = warp * 32 * R + r * 32 + lane;
    key[r] = (int)pos[r] < a.T ? sort_key(a, (int)pos[r]) : 0u;
  }
  const int passes = (a.bits + kDigit - 1) / kDigit, width = (a.bits + passes - 1) / passes;
  for (int p = 0; p < passes; ++p) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int item = warp * 32 * R + r * 32 + lane;
      if (p > 0 && item < a.T) {
        key[r] = s_key[item];
        pos[r] = s_pos[item];
      }
      digit[r] = item < a.T ? key[r] >> (p * width) & ((1u << width) - 1u) : 1u << 20;
    }
    rank_items<R>(digit, place, cnt, s_warp);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (digit[r] >= kDigits) continue;
      const uint32_t to = cnt[warp * kDigits + digit[r]] + place[r];
      s_key[to] = key[r];
      s_pos[to] = pos[r];
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < a.T; i += kSortThreads) {
    a.key[0][i] = s_key[i];
    a.pos[0][i] = s_pos[i];
  }
}

// Row v of the table where no token asks for it: zeros, or what the gradient is added to.  By a
// warp.
template <typename E, int VE>
__device__ __forceinline__ void fill_row(const EmbedArgs& a, size_t v) {
  using P = Pack<E, VE>;
  const int per = a.H / VE, lane = threadIdx.x % 32;
  P* to = reinterpret_cast<P*>(a.d_table) + v * per;
  if (a.add) {
    const P* from = reinterpret_cast<const P*>(a.add) + v * per;
#pragma unroll 8
    for (int c = lane; c < per; c += 32) to[c] = from[c];
  } else {
    P none;
#pragma unroll
    for (int j = 0; j < VE; ++j) none.e[j] = rounded<E>(0.f);
#pragma unroll 4
    for (int c = lane; c < per; c += 32) to[c] = none;
  }
}

// CTA 0 sorts the rows; the others each fill their part of the table's rows that do not occur.
template <typename E, int VE, int R>
__global__ void __launch_bounds__(kSortThreads, 1) embed_sort_fill(const EmbedArgs a, int rows) {
  extern __shared__ uint32_t s_dyn[];
  pdl_wait();
  pdl_signal();
  if (blockIdx.x == 0) {
    sort_all<R>(a, s_dyn);
    return;
  }
  const int tid = threadIdx.x, warp = tid / 32;
  const int v0 = (blockIdx.x - 1) * rows, v1 = min(a.V, v0 + rows);      // (rows: whole words)
  for (int i = tid; i < rows / 32; i += kSortThreads) s_dyn[i] = 0;
  __syncthreads();
#pragma unroll 4
  for (int t = tid; t < a.T; t += kSortThreads) {
    const int id = a.ids[t];
    if (id >= v0 && id < v1) atomicOr(&s_dyn[(id - v0) / 32], 1u << (id - v0) % 32);
  }
  __syncthreads();
  for (int v = v0 + warp; v < v1; v += kSortWarps)
    if (!(s_dyn[(v - v0) / 32] >> (v - v0) % 32 & 1u)) fill_row<E, VE>(a, (size_t)v);
}

// --- more rows than one CTA sorts
__global__ void __launch_bounds__(256) embed_mark(const EmbedArgs a) {
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t >= a.T) return;
  const uint32_t k = sort_key(a, t);
  a.key[1][t] = k;
  a.pos[1][t] = (uint32_t)t;
  if (k < (uint32_t)a.V) atomicOr(&a.there[k / 32], 1u << k % 32);
}

template <typename E, int VE>
__global__ void __launch_bounds__(256) embed_fill(const EmbedArgs a) {
  const int warps = gridDim.x * 8;
  for (int v = blockIdx.x * 8 + threadIdx.x / 32; v < a.V; v += warps)
    if (!(a.there[v / 32] >> v % 32 & 1u)) fill_row<E, VE>(a, (size_t)v);
}

// Counts of the digits at `shift` of tile blockIdx.x.
__global__ void __launch_bounds__(kSortThreads) embed_digits(const EmbedArgs a, int from, int shift,
                                                             int width) {
  __shared__ uint32_t cnt[kDigits];
  const int tid = threadIdx.x;
  if (tid < kDigits) cnt[tid] = 0;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kTile / kSortThreads; ++q) {
    const int i = blockIdx.x * kTile + q * kSortThreads + tid;
    if (i < a.T) atomicAdd(&cnt[a.key[from][i] >> shift & ((1u << width) - 1u)], 1u);
  }
  __syncthreads();
  if (tid < kDigits) a.hist[(size_t)tid * gridDim.x + blockIdx.x] = cnt[tid];
}

// The counts' exclusive sums, in place; one CTA.
__global__ void __launch_bounds__(kSortThreads) embed_offsets(const EmbedArgs a, int n) {
  __shared__ uint32_t s_warp[32];
  const int per = (n + kSortThreads - 1) / kSortThreads;
  const int i0 = min(n, (int)threadIdx.x * per), i1 = min(n, i0 + per);
  uint32_t s = 0;
#pragma unroll 8
  for (int i = i0; i < i1; ++i) s += a.hist[i];
  uint32_t at = block_before(s, s_warp);
  for (int i = i0; i < i1; ++i) {
    const uint32_t c = a.hist[i];
    a.hist[i] = at;
    at += c;
  }
}

// Moves tile blockIdx.x's rows to their places by the digit at `shift`.
__global__ void __launch_bounds__(kSortThreads) embed_place(const EmbedArgs a, int from, int shift,
                                                            int width) {
  constexpr int R = kTile / kSortThreads;
  __shared__ uint32_t cnt[kSortWarps * kDigits];
  __shared__ uint32_t s_warp[32], first[kDigits];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  uint32_t key[R], pos[R], digit[R], place[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = blockIdx.x * kTile + warp * 32 * R + r * 32 + lane;
    key[r] = i < a.T ? a.key[from][i] : 0u;
    pos[r] = i < a.T ? a.pos[from][i] : 0u;
    digit[r] = i < a.T ? key[r] >> shift & ((1u << width) - 1u) : 1u << 20;
  }
  rank_items<R>(digit, place, cnt, s_warp);
  if (tid < kDigits) first[tid] = cnt[tid];        // warp 0's: where the digit starts
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint32_t d = digit[r];
    if (d >= kDigits) continue;
    const uint32_t to = a.hist[(size_t)d * gridDim.x + blockIdx.x] +
                        (cnt[warp * kDigits + d] - first[d]) + place[r];
    a.key[from ^ 1][to] = key[r];
    a.pos[from ^ 1][to] = pos[r];
  }
}

// ------------------------------------------------------------------ sums
template <typename E, int VE>
__device__ __forceinline__ void put_sum(const EmbedArgs& a, size_t v, int c, const float (&s)[VE]) {
  using P = Pack<E, VE>;
  const size_t at = v * (a.H / VE) + c;
  P o;
  if (a.add) {
    const P x = reinterpret_cast<const P*>(a.add)[at];
#pragma unroll
    for (int j = 0; j < VE; ++j) o.e[j] = rounded<E>(fmaf(a.scale, s[j], to_f32(x.e[j])));
  } else {
#pragma unroll
    for (int j = 0; j < VE; ++j) o.e[j] = rounded<E>(a.scale * s[j]);
  }
  reinterpret_cast<P*>(a.d_table)[at] = o;
}

template <int VE>
__device__ __forceinline__ void put_part(float* to, const float (&s)[VE]) {
#pragma unroll
  for (int j = 0; j < VE; ++j) to[j] = s[j];
}

// CTA (chunk, column block): a thread sums VE columns of the chunk's rows, run by run, eight
// rows' loads in flight.
template <typename E, int VE>
__global__ void __launch_bounds__(kSumThreads) embed_sum(const EmbedArgs a, int buf) {
  using P = Pack<E, VE>;
  pdl_wait();
  pdl_signal();
  __shared__ uint32_t s_key[kMaxChunk + 2], s_pos[kMaxChunk];
  const int tid = threadIdx.x, chunk = blockIdx.x, i0 = chunk * a.chunk;
  const int n = min(a.chunk, a.T - i0);
  const uint32_t V = (uint32_t)a.V;
  for (int i = tid; i < n + 2; i += kSumThreads) {      // with the neighbours before and after
    const int at = i0 + i - 1;
    s_key[i] = at >= 0 && at < a.T ? a.key[buf][at] : V;
    if (i < n) s_pos[i] = a.pos[buf][i0 + i];
  }
  __syncthreads();
  const uint32_t* key = s_key + 1;
  const int per = a.H / VE, c = blockIdx.y * kSumThreads + tid;
  const bool in = c < per;
  int tok[2] = {-1, -1};
  float acc[VE] = {};
  int start = 0;
  const P* d = reinterpret_cast<const P*>(a.d_out);
  for (int b = 0; b < n && key[b] < V; b += 8) {
    P x[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int i = b + q;
      if (in && i < n && key[i] < V) x[q] = d[(size_t)s_pos[i] * per + c];
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int i = b + q;
      if (i >= n || key[i] >= V) break;
#pragma unroll
      for (int j = 0; j < VE; ++j) acc[j] += to_f32(x[q].e[j]);
      const uint32_t k = key[i];
      const bool last = i == n - 1;
      if (!last && key[i + 1] == k) continue;
      // the run ends here, or goes on in the next chunk
      const bool shared_before = start == 0 && key[-1] == k;
      const bool shared_after = last && key[n] == k;
      if (shared_before || shared_after) {
        const int s = shared_before ? 0 : 1;
        tok[s] = (int)k;
        if (in) put_part<VE>(a.part + ((size_t)chunk * 2 + s) * a.H + (size_t)c * VE, acc);
      } else if (in) {
        put_sum<E, VE>(a, k, c, acc);
      }
#pragma unroll
      for (int j = 0; j < VE; ++j) acc[j] = 0.f;
      start = i + 1;
    }
  }
  if (tid < 2 && blockIdx.y == 0) a.part_tok[chunk * 2 + tid] = tok[tid];
}

// CTA (chunk, column block): the token whose run starts in this chunk and goes on in the next
// ones.  The parts' rounding errors are carried along.
template <typename E, int VE>
__global__ void __launch_bounds__(kSumThreads) embed_join(const EmbedArgs a) {
  pdl_wait();
  pdl_signal();
  const int chunk = blockIdx.x, v = a.part_tok[chunk * 2 + 1];
  if (v < 0) return;
  const int per = a.H / VE, c = blockIdx.y * kSumThreads + threadIdx.x;
  if (c >= per) return;
  float s[VE], e[VE];
  const float* p = a.part + (size_t)c * VE;
#pragma unroll
  for (int j = 0; j < VE; ++j) {
    s[j] = p[((size_t)chunk * 2 + 1) * a.H + j];
    e[j] = 0.f;
  }
  bool more = true;
  for (int q0 = chunk + 1; more && q0 < a.chunks; q0 += 4) {
    float x[4][VE];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      more = more && q0 + q < a.chunks && a.part_tok[(q0 + q) * 2] == v;
#pragma unroll
      for (int j = 0; j < VE; ++j) x[q][j] = more ? p[(size_t)(q0 + q) * 2 * a.H + j] : 0.f;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float t = s[j] + x[q][j], y = t - s[j];
        e[j] += (s[j] - (t - y)) + (x[q][j] - y);
        s[j] = t;
      }
  }
#pragma unroll
  for (int j = 0; j < VE; ++j) s[j] += e[j];
  put_sum<E, VE>(a, (size_t)v, c, s);
}

bool by16(const EmbedArgs& a, int es) {
  const uintptr_t all = (uintptr_t)a.table | (uintptr_t)a.out | (uintptr_t)a.d_out |
                        (uintptr_t)a.add | (uintptr_t)a.d_table;
  return all % 16 == 0 && a.H * (size_t)es % 16 == 0;
}

template <typename E, int VE>
cudaError_t lookup(const EmbedArgs& a) {
  const int per = a.H / VE, threads = std::min(256, (per + 31) / 32 * 32);
  const unsigned cols = (unsigned)((per + threads - 1) / threads);
  // four rows a thread once that leaves enough CTAs
  if ((long long)a.T * cols >= 4 * 1216)
    return launch_after(embed_rows<E, VE, 4>, dim3((unsigned)(a.T + 3) / 4, cols), threads, 0,
                        a.stream, a);
  return launch_after(embed_rows<E, VE, 1>, dim3((unsigned)a.T, cols), threads, 0, a.stream, a);
}

template <typename E, int VE, int R>
cudaError_t sort_fill(const EmbedArgs& a) {
  const size_t smem = sizeof(uint32_t) * (2 * kSortThreads * R + kSortWarps * kDigits);
  int sms = 0;
  cudaError_t e = device_sms(&sms);
  if (e == cudaSuccess) e = raise_smem_limit((const void*)embed_sort_fill<E, VE, R>, smem);
  if (e != cudaSuccess) return e;
  const bool fill = a.add != a.d_table;
  // whole words of rows for each of the other CTAs, as many as their bits have room for
  const int most = (int)(smem / 4) * 32;
  const int ctas = std::max(sms - 1, (a.V + most - 1) / most);
  const int rows = ((a.V + ctas - 1) / ctas + 31) / 32 * 32;
  return launch_after(embed_sort_fill<E, VE, R>, 1 + (fill ? (a.V + rows - 1) / rows : 0),
                      kSortThreads, smem, a.stream, a, rows);
}

template <typename E, int VE>
cudaError_t backward(const EmbedArgs& a) {
  cudaError_t e = cudaMemsetAsync(a.ctrl, 0, 256, a.stream);
  int buf = 0;
  if (e == cudaSuccess && a.T <= kSortAll) {
    e = a.T <= kSortThreads       ? sort_fill<E, VE, 1>(a)
        : a.T <= 4 * kSortThreads ? sort_fill<E, VE, 4>(a)
                                  : sort_fill<E, VE, 16>(a);
  } else if (e == cudaSuccess) {
    e = cudaMemsetAsync(a.there, 0, ((size_t)a.V + 31) / 32 * 4, a.stream);
    if (e != cudaSuccess) return e;
    embed_mark<<<(a.T + 255) / 256, 256, 0, a.stream>>>(a);
    if (a.add != a.d_table) embed_fill<E, VE><<<1216, 256, 0, a.stream>>>(a);
    const int tiles = (a.T + kTile - 1) / kTile;
    const int passes = (a.bits + kDigit - 1) / kDigit, width = (a.bits + passes - 1) / passes;
    int from = 1;
    for (int p = 0; p < passes; ++p, from ^= 1) {
      embed_digits<<<tiles, kSortThreads, 0, a.stream>>>(a, from, p * width, width);
      embed_offsets<<<1, kSortThreads, 0, a.stream>>>(a, tiles * kDigits);
      embed_place<<<tiles, kSortThreads, 0, a.stream>>>(a, from, p * width, width);
    }
    buf = from;
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  const int per = a.H / VE;
  const dim3 grid((unsigned)a.chunks, (unsigned)((per + kSumThreads - 1) / kSumThreads));
  e = launch_after(embed_sum<E, VE>, grid, kSumThreads, 0, a.stream, a, buf);
  if (e == cudaSuccess && a.chunks > 1)
    e = launch_after(embed_join<E, VE>, grid, kSumThreads, 0, a.stream, a);
  return e;
}

}  // namespace

void plan_embed(EmbedArgs* a) {
  a->bits = 0;
  while (a->V >> a->bits) ++a->bits;               // (V itself is a sort key)
  // chunks long enough that their shared parts, in fp32, stay a small share of the rows
  a->chunk = std::max(32, (a->T + 2431) / 2432);
  a->chunks = (a->T + a->chunk - 1) / a->chunk;
}

size_t embed_hist_words(const EmbedArgs& a) {
  return (size_t)kDigits * ((a.T + kTile - 1) / kTile);
}

cudaError_t launch_embed(const EmbedArgs& a) {
  if (a.dtype == 0) return by16(a, 4) ? lookup<float, 4>(a) : lookup<float, 1>(a);
  return by16(a, 2) ? lookup<__nv_bfloat16, 8>(a) : lookup<__nv_bfloat16, 1>(a);
}

cudaError_t launch_embed_backward(const EmbedArgs& a) {
  if (a.dtype == 0) return by16(a, 4) ? backward<float, 4>(a) : backward<float, 1>(a);
  return by16(a, 2) ? backward<__nv_bfloat16, 8>(a) : backward<__nv_bfloat16, 1>(a);
}

}  // namespace dspark
