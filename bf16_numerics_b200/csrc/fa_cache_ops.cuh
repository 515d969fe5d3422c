// Writes to a paged key/value cache: new tokens' rows into their slots, and
// accepted drafted tokens' rows moved up behind the context.  Copies only:
// bound by memory traffic (2 x 4 d bytes per row of a key head), by launch
// latency when there are few.
//
// A slot outside the page table's reach, or whose page id is not a page of the
// pool, is skipped and reported in the device error word; nothing is written
// outside the pool.
#pragma once

#include "fa_cached.cuh"

namespace fa {

struct CachePool {
  uint4* k;          // [num_pages, Hkv, page, D / 8] (16 bytes = 8 bf16)
  uint4* v;
  const int* table;  // [B, width]
  const int* ctx_len;
  int Hkv, num_pages, page, width;
  // 16-byte index of chunk 0 of (sequence b, slot, head); -1 outside the cache
  template <int CH>
  __device__ __forceinline__ long long row(int b, long long slot, int hk, uint32_t site) const {
    if (slot >= 0 && slot < static_cast<long long>(width) * page) {
      const int s = static_cast<int>(slot);
      const int pg = s / page, id = __ldg(table + static_cast<long long>(b) * width + pg);
      if (id >= 0 && id < num_pages) return ((static_cast<long long>(id) * Hkv + hk) * page + (s - pg * page)) * CH;
    }
    report_page(site, b);
    return -1;
  }
};

// Token t of sequence b -> slot ctx_len[b] + t, for t < count[b] (null: all T).
// Threads walk the 16-byte chunks of one sequence in (token, head, chunk)
// order, U chunks of K and V each, all loads before any store.  Eight prompts of
// up to 4096 tokens, 8 heads, d = 128 (207 MB in all): 39.5 us with U = 2 and at
// most 8 blocks per SM, 41.5 us with U = 4 and 16, 47.9 us with U = 8.
template <int D>
__global__ void __launch_bounds__(256)
fa_cache_append_kernel(const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v, ViewStrides sk,
                       ViewStrides sv, const int* __restrict__ count, CachePool c, int B, int T) {
  constexpr int CH = D / 8, U = 2;
  grid_launch_dependents();
  grid_dependency_wait();
  for (int b = blockIdx.y; b < B; b += gridDim.y) {
    int n = T;
    if (count) {
      n = __ldg(count + b);
      if (n < 0 || n > T) {
        if (threadIdx.x == 0) report_page(3, b);
        n = 0;
      }
    }
    const long long ctx = __ldg(c.ctx_len + b);
    const int work = n * c.Hkv * CH;  // (the host keeps T * Hkv * CH below 2^31)
    const int stride = gridDim.x * 256;
    for (long long i0 = blockIdx.x * 256 + threadIdx.x; i0 < work; i0 += static_cast<long long>(stride) * U) {
      uint4 a[U], w[U];
      long long to[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long long i = i0 + static_cast<long long>(u) * stride;
        to[u] = -1;
        if (i < work) {
          const int r = static_cast<int>(i) / CH, ch = static_cast<int>(i) % CH;
          const int t = r / c.Hkv, hk = r - t * c.Hkv;
          to[u] = c.row<CH>(b, ctx + t, hk, 4);
          if (to[u] >= 0) {
            to[u] += ch;
            a[u] = __ldcs(reinterpret_cast<const uint4*>(k + b * sk.b + hk * sk.h + t * sk.n) + ch);
            w[u] = __ldcs(reinterpret_cast<const uint4*>(v + b * sv.b + hk * sv.h + t * sv.n) + ch);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (to[u] >= 0) {
          c.k[to[u]] = a[u];
          c.v[to[u]] = w[u];
        }
    }
  }
}

// Slot ctx_len[b] + i takes the row of slot ctx_len[b] + src[b, i], for
// i < count[b]: one block per (sequence, key head), every row into shared
// memory before any is written, so src may be in any order and name a row
// twice.
template <int D>
__global__ void __launch_bounds__(256)
fa_cache_compact_kernel(const int* __restrict__ src, const int* __restrict__ count, CachePool c, int B, int M) {
  constexpr int CH = D / 8;
  __shared__ uint4 rows[2][64][CH];
  grid_launch_dependents();
  grid_dependency_wait();
  for (long long item = blockIdx.x; item < static_cast<long long>(B) * c.Hkv; item += gridDim.x) {
    const int b = static_cast<int>(item / c.Hkv), hk = static_cast<int>(item % c.Hkv);
    int n = __ldg(count + b);
    if (n < 0 || n > M) {
      if (threadIdx.x == 0) report_page(5, b);
      n = 0;
    }
    const long long ctx = __ldg(c.ctx_len + b);
    for (int x = threadIdx.x; x < n * CH; x += 256) {
      const int i = x / CH, ch = x % CH, s = __ldg(src + static_cast<long long>(b) * M + i);
      if (s == i) continue;  // in its place already
      const long long at = s < 0 ? -1 : c.row<CH>(b, ctx + s, hk, 6);
      if (s < 0) report_page(6, b);
      if (at >= 0) {
        rows[0][i][ch] = c.k[at + ch];
        rows[1][i][ch] = c.v[at + ch];
      }
    }
    __syncthreads();
    for (int x = threadIdx.x; x < n * CH; x += 256) {
      const int i = x / CH, ch = x % CH, s = __ldg(src + static_cast<long long>(b) * M + i);
      if (s == i || s < 0) continue;
      // (the same check as above: a row that was not read is not written)
      if (c.row<CH>(b, ctx + s, hk, 6) < 0) continue;
      const long long to = c.row<CH>(b, ctx + i, hk, 7);
      if (to >= 0) {
        c.k[to + ch] = rows[0][i][ch];
        c.v[to + ch] = rows[1][i][ch];
      }
    }
    __syncthreads();
  }
}

}  // namespace fa
