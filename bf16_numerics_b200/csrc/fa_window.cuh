// Sliding window with sinks: which keys a query sees, by blocks and by bits.
//
//   key j is visible to query i  <=>  j <= i  and  (i - j < window or j < sinks)
//
// so a row sees its last `window` keys (itself included) and the first `sinks`
// keys of the sequence.  With window >= N this is plain causal attention.  H
// query heads share Hkv key/value heads in groups of G = H / Hkv: query head h
// reads key head h / G.
//
// The kernels work in 128 x 128 blocks.  Query block qb sees the key blocks
// [first_block(qb), qb] and the sink blocks below them; key block kb is seen by
// the query blocks [kb, last_query_block(kb)].  Blocks nothing of which is
// visible are never loaded; blocks that are visible in part are masked with one
// bit per (row, key): word(c0) holds 32 of them, built from at most three
// bounds with shifts, so that an element costs one bit test and one select.
#pragma once

#include <cstdint>
#include <type_traits>

namespace fa {

// bits [0, n) of a word (n clipped to [0, 32])
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : ((1u << n) - 1u));
}

// columns c of a run of keys (or queries) that are visible to one row:
// c < hi and (c >= lo or c < sk)
struct RowMask {
  int lo, hi, sk;
  // whether any of the first n columns is hidden
  __device__ __forceinline__ bool hides(int n) const { return hi < n || (lo > 0 && sk < n && sk < lo); }
  // bit i: column c0 + i is visible
  __device__ __forceinline__ uint32_t word(int c0) const {
    return bits_below(hi - c0) & (~bits_below(lo - c0) | bits_below(sk - c0));
  }
};

// Over a cache: the first context slot in the window of a new token that sees
// n of the new tokens, itself included (so it stands at ctx + n - 1); ctx + n
// and the window are below 2^31.  Not below slot 0: with a window of 2^31 - 1 the
// difference to a far slot would not fit.
__device__ __forceinline__ int window_first(int ctx, int n, int window) {
  const int first = ctx + n - window;
  return first > 0 ? first : 0;
}
// .. and how it sees the context in slots [key0, ..): not where key0 is beyond ctx
__device__ __forceinline__ RowMask context_mask(int ctx, int first, int sinks, int key0) {
  return RowMask{first - key0, ctx - key0, sinks - key0};
}
// whether n slots from key0 on hold any that it may not see
__device__ __forceinline__ bool context_hides(int ctx, int first, int sinks, int key0, int n) {
  return ctx - key0 < n || (key0 < first && sinks - key0 < n);
}

struct WindowShape {
  int H, G;            // query heads, query heads per key head
  int window, sinks;   // 1 <= window <= N, 0 <= sinks <= N (the host clips both)
  int n_sink_blk;      // ceil(sinks / 128)
  // first key block inside the window of query block qb's first row
  __device__ __forceinline__ int first_block(int qb) const {
    const int first = qb * 128 - window + 1;
    return first > 0 ? first / 128 : 0;
  }
  // last query block that sees a key of block kb
  __device__ __forceinline__ int last_query_block(int kb, int n_blk) const {
    if (kb < n_sink_blk) return n_blk - 1;
    const long long q = (static_cast<long long>(kb) * 128 + 127 + window - 1) / 128;
    return q < n_blk - 1 ? static_cast<int>(q) : n_blk - 1;
  }
  // keys [key0, ...) as query q sees them, N keys in all.  A row past the end
  // (the padding of a ragged last block, never stored) is treated as the last
  // one, so that it too sees a key of its diagonal block.
  __device__ __forceinline__ RowMask row_mask(int q, int key0, int N) const {
    const int rel = (q < N ? q : N - 1) - key0;  // column of the diagonal
    return RowMask{rel - window + 1, rel + 1, sinks - key0};
  }
  // queries [q0, ...) as they see key `key`: c is query q0 + c
  __device__ __forceinline__ RowMask column_mask(int key, int q0) const {
    const int rel = key - q0;  // column of the diagonal
    const long long end = static_cast<long long>(rel) + window;
    const int far = 1 << 30;   // above any column of a block
    return RowMask{rel, key < sinks || end > far ? far : static_cast<int>(end), 0};
  }
  // whether every (query, key) pair of the two blocks is visible
  __device__ __forceinline__ bool block_full(int qb, int kb) const {
    if (qb <= kb) return false;
    return static_cast<long long>(qb - kb) * 128 + 127 < window || static_cast<long long>(kb) * 128 + 128 <= sinks;
  }
};

}  // namespace fa
