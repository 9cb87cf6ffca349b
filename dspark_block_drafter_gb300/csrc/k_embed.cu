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
// beside the sort and the sums, which both wait for their loads more than they use the memory:
// by a map of the tokens, or before there is one by looking at every token.
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
constexpr int kDigitAll = 9;             // bits of a digit in one CTA's sort: two passes up to 2^18
constexpr int kDigit = 8, kDigits = 1 << kDigit;                 // and in the other
constexpr int kMaxChunk = 512;
constexpr int kSumThreads = 256;
constexpr int kFillRows = 64;            // rows of the table that one CTA beside the sums fills

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

// The places of R items a thread among the CTA's by their digit of D bits, equal digits in the
// items' order: warp w holds items [32 R w, 32 R (w + 1)), item r of a lane is 32 r + lane of those.
// cnt: [warps][2^D]; afterwards place[r] + cnt[warp][digit] is an item's place.
template <int R, int D>
__device__ __forceinline__ void rank_items(const uint32_t (&digit)[R], uint32_t (&place)[R],
                                           uint32_t* cnt, uint32_t* s_warp) {
  constexpr int kOf = 1 << D;
  const int tid = threadIdx.x, lane = tid % 32;
  uint32_t* mine = cnt + (tid / 32) * kOf;
  for (int i = tid; i < kSortWarps * kOf; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    // (items past the end have a digit of their own, and are not counted)
    const unsigned peers = __match_any_sync(0xFFFFFFFFu, digit[r]);
    const bool in = digit[r] < kOf;
    const uint32_t before = __popc(peers & ((1u << lane) - 1u));
    const uint32_t base = in ? mine[digit[r]] : 0u;
    __syncwarp();
    if (in && before == 0) mine[digit[r]] = base + __popc(peers);
    __syncwarp();
    place[r] = base + before;
  }
  __syncthreads();
  // counts become offsets, digit by digit and in each warp by warp: `each` a thread
  constexpr int each = kSortWarps * kOf / kSortThreads, per = kSortWarps / each;
  const int d = tid / per, w0 = tid % per * each;
  uint32_t x[each], s = 0;
#pragma unroll
  for (int q = 0; q < each; ++q) {
    x[q] = cnt[(w0 + q) * kOf + d];
    s += x[q];
  }
  uint32_t at = block_before(s, s_warp);
#pragma unroll
  for (int q = 0; q < each; ++q) {
    cnt[(w0 + q) * kOf + d] = at;
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
  const int passes = (a.bits + kDigitAll - 1) / kDigitAll, width = (a.bits + passes - 1) / passes;
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
    rank_items<R, kDigitAll>(digit, place, cnt, s_warp);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (digit[r] >> kDigitAll) continue;
      const uint32_t to = cnt[(warp << kDigitAll) + digit[r]] + place[r];
      s_key[to] = key[r];
      s_pos[to] = pos[r];
    }
    __syncthreads();
  }
  // the sorted list, and its tokens' places in the map
  for (int i = threadIdx.x; i < a.T; i += kSortThreads) {
    const uint32_t k = s_key[i];
    a.key[0][i] = k;
    a.pos[0][i] = s_pos[i];
    if (k < (uint32_t)a.V) a.there[k] = 1;
  }
}

// Row v of the table where no token asks for it: zeros, or what the gradient is added to.  By a
// warp, 16 bytes at a time between the ends that are not.
template <typename E>
__device__ __forceinline__ void fill_row(const EmbedArgs& a, size_t v) {
  constexpr int VE = 16 / sizeof(E);
  const int lane = threadIdx.x % 32;
  E* to = reinterpret_cast<E*>(a.d_table) + v * a.H;
  const E* from = a.add ? reinterpret_cast<const E*>(a.add) + v * a.H : nullptr;
  const bool alike = !from || ((uintptr_t)from - (uintptr_t)to) % 16 == 0;
  const int head = alike ? min(a.H, (int)((16 - (uintptr_t)to % 16) % 16 / sizeof(E))) : a.H;
  const int vecs = (a.H - head) / VE, tail = head + vecs * VE;
  uint4* tv = reinterpret_cast<uint4*>(to + head);
  if (from) {
    const uint4* fv = reinterpret_cast<const uint4*>(from + head);
    for (int c0 = lane; c0 < vecs; c0 += 32 * 8) {
      uint4 x[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (c0 + 32 * q < vecs) x[q] = __ldcs(fv + c0 + 32 * q);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (c0 + 32 * q < vecs) tv[c0 + 32 * q] = x[q];
    }
    for (int c = lane; c < head; c += 32) to[c] = from[c];
    for (int c = tail + lane; c < a.H; c += 32) to[c] = from[c];
  } else {
#pragma unroll 4
    for (int c = lane; c < vecs; c += 32) tv[c] = make_uint4(0, 0, 0, 0);
    for (int c = lane; c < head; c += 32) to[c] = rounded<E>(0.f);
    for (int c = tail + lane; c < a.H; c += 32) to[c] = rounded<E>(0.f);
  }
}

// CTA 0 sorts the rows; the others meanwhile fill the first ones of the table that do not occur,
// `rows` each (whole words of bits).  They find out which by looking at every token.
template <typename E, int R>
__global__ void __launch_bounds__(kSortThreads, 1) embed_sort(const EmbedArgs a, int rows) {
  extern __shared__ uint32_t s_dyn[];
  pdl_wait();
  pdl_signal();
  if (blockIdx.x == 0) {
    sort_all<R>(a, s_dyn);
    return;
  }
  const int v0 = (blockIdx.x - 1) * rows, v1 = min(a.V, v0 + rows), tid = threadIdx.x;
  for (int i = tid; i < rows / 32; i += kSortThreads) s_dyn[i] = 0;
  __syncthreads();
#pragma unroll 8
  for (int t = tid; t < a.T; t += kSortThreads) {
    const int id = a.ids[t];
    if (id >= v0 && id < v1) atomicOr(&s_dyn[(id - v0) / 32], 1u << (id - v0) % 32);
  }
  __syncthreads();
  for (int v = v0 + tid / 32; v < v1; v += kSortWarps)
    if (!(s_dyn[(v - v0) / 32] >> (v - v0) % 32 & 1u)) fill_row<E>(a, (size_t)v);
}

// --- more rows than one CTA sorts
__global__ void __launch_bounds__(256) embed_mark(const EmbedArgs a) {
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t >= a.T) return;
  const uint32_t k = sort_key(a, t);
  a.key[1][t] = k;
  a.pos[1][t] = (uint32_t)t;
  if (k < (uint32_t)a.V) a.there[k] = 1;
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
  for (int i = i0; i < i1; i += 8) {
    uint32_t c[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) c[q] = i + q < i1 ? a.hist[i + q] : 0u;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (i + q < i1) a.hist[i + q] = at;
      at += c[q];
    }
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
  rank_items<R, kDigit>(digit, place, cnt, s_warp);
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
// The table's row v from its sum, and `add`'s columns of it (NULL: none).
template <typename E, int VE>
__device__ __forceinline__ void put_sum(const EmbedArgs& a, size_t v, int c, const float (&s)[VE],
                                        const Pack<E, VE>* add) {
  Pack<E, VE> o;
#pragma unroll
  for (int j = 0; j < VE; ++j)
    o.e[j] = rounded<E>(add ? fmaf(a.scale, s[j], to_f32(add->e[j])) : a.scale * s[j]);
  reinterpret_cast<Pack<E, VE>*>(a.d_table)[v * (a.H / VE) + c] = o;
}

// VE sums of the workspace, in vectors of four where there are as many.
template <int VE>
__device__ __forceinline__ void put_part(float* to, const float (&s)[VE]) {
  if constexpr (VE == 1) {
    *to = s[0];
  } else {
#pragma unroll
    for (int j = 0; j < VE; j += 4)
      *reinterpret_cast<float4*>(to + j) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
  }
}
template <int VE>
__device__ __forceinline__ void get_part(const float* from, float (&s)[VE]) {
  if constexpr (VE == 1) {
    s[0] = *from;
  } else {
#pragma unroll
    for (int j = 0; j < VE; j += 4) {
      const float4 x = *reinterpret_cast<const float4*>(from + j);
      s[j] = x.x; s[j + 1] = x.y; s[j + 2] = x.z; s[j + 3] = x.w;
    }
  }
}

// One chunk and column block: a thread sums VE columns of the chunk's rows, run by run, the
// loads of several rows in flight.
template <typename E, int VE, bool ADD>
__device__ __forceinline__ void sum_chunk(const EmbedArgs& a, int buf, int chunk, int block,
                                          uint32_t* s_key, uint32_t* s_pos, Pack<E, VE>* s_add) {
  using P = Pack<E, VE>;
  constexpr int kAt = VE == 1 ? 16 : 8;
  constexpr uint32_t kEnd = 1u << 31;                   // the run ends with this row
  const int tid = threadIdx.x, i0 = chunk * a.chunk, size = min(a.chunk, a.T - i0);
  const uint32_t V = (uint32_t)a.V;
  for (int i = tid; i < size + 2; i += kSumThreads) {   // with the neighbours before and after
    const int at = i0 + i - 1;
    s_key[i] = at >= 0 && at < a.T ? a.key[buf][at] : V;
  }
  __syncthreads();
  const uint32_t* key = s_key + 1;
  for (int i = tid; i < size; i += kSumThreads) {
    const bool last = i == size - 1 || key[i + 1] != key[i];
    s_pos[i] = a.pos[buf][i0 + i] | (last ? kEnd : 0u);
  }
  // (rows with a token come first)
  int n = 0;
  if (key[size - 1] < V) {
    n = size;
  } else {
    for (int hi = size; n < hi;) {
      const int m = (n + hi) / 2;
      if (key[m] < V) n = m + 1;
      else hi = m;
    }
  }
  __syncthreads();
  const int per = a.H / VE, c = block * kSumThreads + tid;
  const bool in = c < per;
  const P* d = reinterpret_cast<const P*>(a.d_out) + (in ? c : 0);
  const P* add = reinterpret_cast<const P*>(a.add) + (in ? c : 0);
  bool first = true;                                    // of the chunk's runs
  int tok0 = -1, tok1 = -1;
  float acc[VE] = {};
#pragma unroll 1
  for (int b = 0; b < n; b += kAt) {
    P x[kAt];
    P y[ADD && VE == 1 ? kAt : 1];
#pragma unroll
    for (int q = 0; q < kAt; ++q) {
      const int i = min(b + q, n - 1);
      x[q] = d[(size_t)(s_pos[i] & ~kEnd) * per];
      // (what runs are added to: by way of shared memory where registers are short)
      if (ADD && VE == 1 && (s_pos[i] & kEnd)) y[q] = add[(size_t)key[i] * per];
      if (ADD && VE > 1 && (s_pos[i] & kEnd))
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                         (uint32_t)__cvta_generic_to_shared(&s_add[q * kSumThreads + tid])),
                     "l"(add + (size_t)key[i] * per)
                     : "memory");
    }
    if (ADD && VE > 1) asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int q = 0; q < kAt; ++q) {
      const int i = b + q;
      if (i >= n) continue;
#pragma unroll
      for (int j = 0; j < VE; ++j) acc[j] += to_f32(x[q].e[j]);
      if (!(s_pos[i] & kEnd)) continue;
      // the run ends here, or goes on in the next chunk
      const uint32_t k = key[i];
      const bool shared_before = first && key[-1] == k;
      const bool shared_after = i == size - 1 && key[size] == k;
      if (shared_before) tok0 = (int)k;
      else if (shared_after) tok1 = (int)k;
      if (in) {
        if (shared_before || shared_after)
          put_part<VE>(a.part + ((size_t)chunk * 2 + !shared_before) * a.H + (size_t)c * VE, acc);
        else
          put_sum<E, VE>(a, k, c, acc,
                         !ADD      ? nullptr
                         : VE == 1 ? &y[ADD && VE == 1 ? q : 0]
                                   : &s_add[q * kSumThreads + tid]);
      }
#pragma unroll
      for (int j = 0; j < VE; ++j) acc[j] = 0.f;
      first = false;
    }
  }
  if (tid == 0 && block == 0) {
    a.part_tok[chunk * 2] = tok0;
    a.part_tok[chunk * 2 + 1] = tok1;
  }
}

// The sums, which wait for their loads, and between them CTAs that fill the table's other rows
// from `v0` on, `fills` of them, which wait for nothing.
template <typename E, int VE, bool ADD>
__global__ void __launch_bounds__(kSumThreads, 4) embed_sum(const EmbedArgs a, int buf, int v0, int fills) {
  pdl_wait();
  pdl_signal();
  __shared__ uint32_t s_key[kMaxChunk + 2], s_pos[kMaxChunk];
  __shared__ Pack<E, VE> s_add[ADD && VE > 1 ? 8 * kSumThreads : 1];
  const long long b = blockIdx.x, all = gridDim.x;
  const int before = (int)(b * fills / all);            // fill CTAs before this one
  if ((int)((b + 1) * fills / all) > before) {
    const int first = v0 + before * kFillRows, end = min(a.V, first + kFillRows);
    for (int v = first + threadIdx.x / 32; v < end; v += kSumThreads / 32)
      if (!a.there[v]) fill_row<E>(a, (size_t)v);
    return;
  }
  const int i = (int)b - before, blocks = (a.H / VE + kSumThreads - 1) / kSumThreads;
  sum_chunk<E, VE, ADD>(a, buf, i / blocks, i % blocks, s_key, s_pos, s_add);
}

// CTA (chunk, column block): the token whose run starts in this chunk and goes on in the next
// ones.  Long runs are summed in thirds by three groups of threads, with their rounding errors,
// and the thirds are joined in order.  (A token in most of 16000 rows has some 300 parts: one
// thread for all of a column's took 75 us.)
constexpr int kJoinGroups = 3, kJoinThreads = kJoinGroups * kSumThreads;
constexpr int kJoinLong = 12;            // parts of a long run
template <int VE>
__device__ __forceinline__ void add_part(float (&s)[VE], float (&e)[VE], const float (&x)[VE]) {
#pragma unroll
  for (int j = 0; j < VE; ++j) {
    const float t = s[j] + x[j], y = t - s[j];
    e[j] += (s[j] - (t - y)) + (x[j] - y);
    s[j] = t;
  }
}
template <typename E, int VE>
__global__ void __launch_bounds__(kJoinThreads) embed_join(const EmbedArgs a) {
  pdl_wait();
  pdl_signal();
  __shared__ int s_end;
  __shared__ float s_sum[(kJoinGroups - 1) * kSumThreads * VE * 2];
  const int chunk = blockIdx.x, v = a.part_tok[chunk * 2 + 1], tid = threadIdx.x;
  if (v < 0) return;
  // the first chunk after the run
  int end = a.chunks;
  for (int q0 = chunk + 1; q0 < a.chunks && end == a.chunks; q0 += kJoinThreads) {
    __syncthreads();
    if (tid == 0) s_end = a.chunks;
    __syncthreads();
    const int q = q0 + tid;
    if (q < a.chunks && a.part_tok[q * 2] != v) atomicMin(&s_end, q);
    __syncthreads();
    end = s_end;
  }
  const int parts = end - chunk - 1, group = tid / kSumThreads, col = tid % kSumThreads;
  const bool split = parts >= kJoinLong;
  if (!split && group > 0) return;
  const int groups = split ? kJoinGroups : 1;
  const int q0 = chunk + 1 + (int)((long long)parts * group / groups);
  const int q1 = chunk + 1 + (int)((long long)parts * (group + 1) / groups);
  const int per = a.H / VE, c = blockIdx.y * kSumThreads + col;
  const bool in = c < per;
  float s[VE] = {}, e[VE] = {};
  const float* p = a.part + (size_t)(in ? c : 0) * VE;
  if (group == 0) get_part<VE>(p + ((size_t)chunk * 2 + 1) * a.H, s);
  constexpr int kAt = VE == 8 ? 4 : 8;
  for (int q = q0; q < q1; q += kAt) {
    float x[kAt][VE];
#pragma unroll
    for (int o = 0; o < kAt; ++o) get_part<VE>(p + (size_t)min(q + o, q1 - 1) * 2 * a.H, x[o]);
#pragma unroll
    for (int o = 0; o < kAt; ++o)
      if (q + o < q1) add_part<VE>(s, e, x[o]);
  }
  if (split) {
    // (value by value, so that neighbours' lie in different banks)
    float* mine = s_sum + (group - 1) * kSumThreads * VE * 2 + col;
    if (group > 0) {
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        mine[j * kSumThreads] = s[j];
        mine[(VE + j) * kSumThreads] = e[j];
      }
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 1; g < kJoinGroups; ++g) {
      const float* other = s_sum + (g - 1) * kSumThreads * VE * 2 + col;
      float x[VE];
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        x[j] = other[j * kSumThreads];
        e[j] += other[(VE + j) * kSumThreads];
      }
      add_part<VE>(s, e, x);
    }
  }
  if (!in) return;
#pragma unroll
  for (int j = 0; j < VE; ++j) s[j] += isfinite(s[j]) ? e[j] : 0.f;     // (inf - inf is in e)
  if (a.add) {
    const Pack<E, VE> x = reinterpret_cast<const Pack<E, VE>*>(a.add)[(size_t)v * per + c];
    put_sum<E, VE>(a, (size_t)v, c, s, &x);
  } else {
    put_sum<E, VE>(a, (size_t)v, c, s, nullptr);
  }
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

// Sorts the rows by their token in one CTA; the other SMs fill what rows of the table they can in
// the time that takes, up to row *filled.
template <typename E, int R>
cudaError_t sort_one(const EmbedArgs& a, bool fill, int* filled) {
  const size_t smem = sizeof(uint32_t) * (2 * kSortThreads * R + (kSortWarps << kDigitAll));
  int sms = 0;
  cudaError_t e = device_sms(&sms);
  if (e == cudaSuccess) e = raise_smem_limit((const void*)embed_sort<E, R>, smem);
  if (e != cudaSuccess) return e;
  // (580 MB take 100 us, and the sort of 16384 rows about 50: the sums beside the rest of a larger
  // table then read while it is written.  The gradient of 151936 x 4096 bf16 from 16384 rows: 249
  // us with 290 MB, 238 with 580, 240 with all of it beside the sort.)
  const size_t bytes = (size_t)a.H * sizeof(E) * (a.add ? 2 : 1);
  const int rows = (int)std::min((size_t)a.V, (size_t)580000000 / bytes);
  const int most = (int)(smem / 4) * 32;                // (bits that there is room for)
  const int each = std::max(32, std::min(most, ((rows + sms - 2) / std::max(1, sms - 1) + 31) / 32 * 32));
  const int ctas = fill ? std::min(sms - 1, (rows + each - 1) / each) : 0;
  *filled = std::min(a.V, ctas * each);
  return launch_after(embed_sort<E, R>, 1 + ctas, kSortThreads, smem, a.stream, a, each);
}

template <typename E, int VE>
cudaError_t backward(const EmbedArgs& a) {
  // (the map follows the control words)
  cudaError_t e = cudaMemsetAsync(a.ctrl, 0, 256 + (size_t)a.V, a.stream);
  const bool fill = a.add != a.d_table;
  int buf = 0, filled = 0;
  if (e == cudaSuccess && a.T <= kSortAll) {
    e = a.T <= kSortThreads       ? sort_one<E, 1>(a, fill, &filled)
        : a.T <= 4 * kSortThreads ? sort_one<E, 4>(a, fill, &filled)
        : a.T <= 8 * kSortThreads ? sort_one<E, 8>(a, fill, &filled)
                                  : sort_one<E, 16>(a, fill, &filled);
  } else if (e == cudaSuccess) {
    embed_mark<<<(a.T + 255) / 256, 256, 0, a.stream>>>(a);
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
  const unsigned blocks = (unsigned)((a.H / VE + kSumThreads - 1) / kSumThreads);
  const int fills = fill ? (a.V - filled + kFillRows - 1) / kFillRows : 0;
  e = launch_after(a.add ? embed_sum<E, VE, true> : embed_sum<E, VE, false>,
                   (unsigned)a.chunks * blocks + (unsigned)fills, kSumThreads, 0, a.stream, a, buf,
                   filled, fills);
  if (e == cudaSuccess && a.chunks > 1)
    e = launch_after(embed_join<E, VE>, dim3((unsigned)a.chunks, blocks), kJoinThreads, 0, a.stream, a);
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
