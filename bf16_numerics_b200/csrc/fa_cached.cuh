// Attention of new tokens over a paged key/value cache.
//
// Per sequence b: ctx tokens are in the cache (slot j holds position j) and T
// new tokens (1 <= T <= 64) sit in slots ctx .. ctx+T-1.  Word t of the tree
// says which of the new tokens token t sees (bit u: token u; a chain sees
// itself and the ones before it).  Token t stands at position
// ctx + popcount(word) - 1 and sees
//   slot j < ctx  if  pos(t) - j < window or j < sinks,
//   token u       if  bit u is set and (pos(t) - pos(u) < window or pos(u) < sinks);
// a token whose word is zero is absent: its row is empty (o = 0, lse = -inf).
// The softmax is the forward's (fa_fwd.cuh), its shift rule applied to the keys
// a partial result has seen; partial results are joined with
//   M = max m_i,  l = sum l_i exp(m_i - M),  o = sum o_i exp(m_i - M) / l.
//
// What bounds it: every visible K and V row is read once for the G query heads
// that share it, 4 d bytes for 4 d T G flops, so up to T G ~ 250 rows the cost
// is the read from HBM and above it the tensor products.
//
// Layout.  The rows of one key head (T tokens of up to GT heads, R <= 128)
// fill the 128 lanes of a tcgen05 tile.  With few rows they are loaded C = 4
// (R <= 32) or C = 2 (R <= 64) times, and copy c of a row handles keys
// [c 128/C, (c+1) 128/C) of every 128-key tile: P_bar of its other keys is
// written as zero, so the four warps share the exponentials of a tile evenly
// and need no exchange; each copy is a partial result of its own.
//
// Work split: the (item, tile) pairs -- an item is a (sequence, key head, row
// tile) -- form one list, and every CTA (one per SM) takes an equal contiguous
// share of it, whatever the contexts' lengths.  The share of one item in one
// CTA is a segment; segment (item i, CTA c) is partial result i + c (a monotone
// path through items and CTAs, so no two share a number).  A second kernel
// joins the segments and copies of each row.  Lengths are read on the device, so a
// captured call follows them.
//
// Per CTA: two softmax warpgroups take the tiles of a segment alternately,
// each with its own S/P columns, O accumulator and running statistics (while
// one computes exponentials the other's products run); they join their two
// states through TMEM at the segment's end.  One warp loads (TMA: K and V
// through rings, one box per page, so a page may lie anywhere and be smaller
// than a tile), one issues products.
//   TMEM: S_t [128t, 128t+128), P_bar_t over its first 64 columns, O_t at 256 + D t.
// Pages that no row sees are not read (their place is filled with zeros by an
// out-of-range box); what lies in a read page behind the last token, or in the
// slot of an absent token, may be anything: its scores are masked and its V
// rows are overwritten with zeros in shared memory (0 * NaN would not be 0).
#pragma once

#include "fa_bwd.cuh"

namespace fa {

constexpr uint32_t kErrCached = 5;  // error word ids: a wait ran out ...
constexpr uint32_t kErrPage = 6;    // ... a page id, length or index outside the cache

__device__ __forceinline__ void report_page(uint32_t site, int b) {
  atomicCAS(&g_fa_error, 0u, (kErrPage << 24) | (site << 16) | (static_cast<uint32_t>(b) & 0xFFFFu));
}

struct CachedParams {
  const int* table;                  // [B, width] page ids
  const int* ctx_len;                // [B]
  const unsigned long long* tree;    // [B, T] or null: a chain
  float* part_o;                     // [slots][C * R][D]: O against the slot's own shift
  float2* part_ml;                   // [slots][C * R]: shift, sum
  long long* prefix;                 // [B + 1]: tiles of the sequences before b
  int B, H, Hkv, T;
  int GT, RT, R;                     // heads per row tile, row tiles, rows per row tile
  int page, width, num_pages;
  int window, sinks;
  int mode;
  float beta, scale;
};

// 128-slot tiles of one sequence that some row sees: the sink tiles below the
// window, then the window's first tile up to the last new token's.
struct CachedTiles {
  int ctx, total, lo, ns, n;  // n = 0: length outside the cache
  __device__ __forceinline__ void load(const CachedParams& p, int b) {
    ctx = __ldg(p.ctx_len + b);
    const long long cap = static_cast<long long>(p.width) * p.page;
    if (ctx < 0 || static_cast<long long>(ctx) + p.T > cap) {
      total = lo = ns = n = 0;
      return;
    }
    total = ctx + p.T;
    lo = ctx - p.window + 1;  // the root's first key; every other token's is no earlier
    lo = lo > 0 ? lo / 128 : 0;
    ns = p.sinks / 128 + (p.sinks % 128 != 0);
    if (ns > lo) ns = lo;
    n = (total - 1) / 128 - lo + 1 + ns;
  }
  __device__ __forceinline__ int tile(int i) const { return i < ns ? i : lo + i - ns; }
};

// The segments of one CTA.
struct CachedCursor {
  CachedTiles seq;
  int b, hr, i0, n;  // sequence, key head * RT + row tile, first tile, tiles of this segment
  long long left;    // tiles of the CTA's share from here on
  __device__ __forceinline__ void clip() {
    const int rest = seq.n - i0;
    n = left < rest ? static_cast<int>(left) : rest;
  }
  __device__ __forceinline__ bool valid() const { return left > 0; }
  __device__ __forceinline__ void next(const CachedParams& p) {
    left -= n;
    if (left <= 0) return;
    i0 = 0;  // a segment that is not the CTA's last ends its item
    if (++hr == p.Hkv * p.RT) {
      hr = 0;
      do {
        ++b;
        seq.load(p, b);
      } while (seq.n == 0);  // (tiles are left, so a sequence with some follows)
    }
    clip();
  }
  __device__ __forceinline__ int key_head(const CachedParams& p) const { return hr / p.RT; }
  __device__ __forceinline__ int row_tile(const CachedParams& p) const { return hr % p.RT; }
  __device__ __forceinline__ long long slot(const CachedParams& p) const {
    return static_cast<long long>(b) * (p.Hkv * p.RT) + hr + blockIdx.x;
  }
};

template <int D, int C>
struct CachedLayout {
  static constexpr int LR = 128 / C;                 // lanes (rows at most) per copy, and keys per copy and tile
  static constexpr int TILE = 128 * D * 2, HALF = 128 * 128;
  static constexpr int KVS = D == 64 ? 6 : 3;        // K and V ring stages
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = TILE, V_OFF = K_OFF + KVS * TILE;
  static constexpr int ML_OFF = V_OFF + KVS * TILE;  // [128] each: m of warpgroups 0 and 1, l of warpgroup 1
  static constexpr int CUR_OFF = ML_OFF + 3 * 128 * 4;
  static constexpr int BAR_OFF = CUR_OFF + 32;
  enum {
    Q_FULL = 0, Q_EMPTY, K_FULL, K_EMPTY = K_FULL + KVS, V_FULL = K_EMPTY + KVS, V_EMPTY = V_FULL + KVS,
    S_FULL = V_EMPTY + KVS, P_FULL = S_FULL + 2, O_READY = P_FULL + 2, TEARDOWN = O_READY + 2, NBAR
  };
  static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
  static constexpr int SMEM_BYTES = MISC_OFF + 16 + 1024;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr int THREADS = 320;
  __host__ __device__ static constexpr uint32_t s_col(int t) { return 128u * t; }
  __host__ __device__ static constexpr uint32_t o_col(int t) { return 256u + static_cast<uint32_t>(D) * t; }
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
};

template <int D, int C>
__global__ void __launch_bounds__(320, 1)
fa_cached_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const CachedParams p) {
  using L = CachedLayout<D, C>;
  constexpr int KVS = L::KVS, LR = L::LR;
  constexpr bool kRawCompare = (D == 64);  // scale is exactly 1/8
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw_addr);
  auto bar = [&](int i) { return base + L::BAR_OFF + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::MISC_OFF + 4);
  const uint64_t limit_ns = wait_limit_ns();
  const BoundedWait wait{abort_flag, kErrCached, limit_ns};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(bar(L::Q_FULL), 1);
    mbar_init(bar(L::Q_EMPTY), 1);
    for (int s = 0; s < KVS; ++s) {
      mbar_init(bar(L::K_FULL + s), 1);
      mbar_init(bar(L::K_EMPTY + s), 1);
      mbar_init(bar(L::V_FULL + s), 1);
      mbar_init(bar(L::V_EMPTY + s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(L::S_FULL + t), 1);
      mbar_init(bar(L::P_FULL + t), 128);
      mbar_init(bar(L::O_READY + t), 1);
    }
    mbar_init(bar(L::TEARDOWN), 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), L::TMEM_COLS);
    tmem_relinquish();
  }
  grid_launch_dependents();
  grid_dependency_wait();
  // this CTA's share of the list: [c U / G, (c+1) U / G) of U tiles, found by
  // one warp with two passes over the lengths (the second one from L1)
  int* cur_smem = reinterpret_cast<int*>(smem + L::CUR_OFF);
  if (warp == 8) {
    const int HR = p.Hkv * p.RT;
    long long sum = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      int n = 0;
      if (b0 + lane < p.B) {
        CachedTiles s;
        s.load(p, b0 + lane);
        n = s.n;
        if (n == 0 && blockIdx.x == 0) report_page(1, b0 + lane);
      }
      if (blockIdx.x == 0) {  // prefix sums for the joining kernel
        long long inc = n;
        for (int o = 1; o < 32; o <<= 1) {
          const long long x = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += x;
        }
        if (b0 + lane < p.B) p.prefix[b0 + lane + 1] = sum + inc;
        if (b0 == 0 && lane == 0) p.prefix[0] = 0;
        sum += __shfl_sync(0xffffffffu, inc, 31);
      } else {
        sum += __reduce_add_sync(0xffffffffu, static_cast<unsigned>(n));
      }
    }
    const long long U = sum * HR, G = gridDim.x < U ? gridDim.x : U;
    long long start = 0, left = 0;
    int b = 0, hr = 0, i0 = 0;
    if (static_cast<long long>(blockIdx.x) < G) {
      start = blockIdx.x * U / G;
      left = (blockIdx.x + 1) * U / G - start;
      long long before = 0;
      for (int b0 = 0; b0 < p.B; b0 += 32) {
        int n = 0;
        if (b0 + lane < p.B) {
          CachedTiles s;
          s.load(p, b0 + lane);
          n = s.n;
        }
        long long inc = n;
        for (int o = 1; o < 32; o <<= 1) {
          const long long x = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += x;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, start < (before + inc) * HR);
        if (hit) {
          const int at = __ffs(hit) - 1;
          const long long pre = before + __shfl_sync(0xffffffffu, inc - n, at);
          const int nt = __shfl_sync(0xffffffffu, n, at);
          const long long in = start - pre * HR;
          b = b0 + at;
          hr = static_cast<int>(in / nt);
          i0 = static_cast<int>(in - static_cast<long long>(hr) * nt);
          break;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
    if (lane == 0) {
      cur_smem[0] = b;
      cur_smem[1] = hr;
      cur_smem[2] = i0;
      *reinterpret_cast<long long*>(cur_smem + 4) = left;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  CachedCursor cur;
  cur.b = cur_smem[0];
  cur.hr = cur_smem[1];
  cur.i0 = cur_smem[2];
  cur.left = *reinterpret_cast<const long long*>(cur_smem + 4);
  cur.n = 0;
  if (cur.valid()) {
    cur.seq.load(p, cur.b);
    cur.clip();
  }

  auto teardown = [&]() {
    tc_fence_before();
    named_barrier_sync(2, L::THREADS);
    if (warp == 9) {
      tc_fence_after();
      volatile int never = 0;
      const BoundedWait drain{&never, kErrCached, limit_ns};
      drain(bar(L::TEARDOWN), 0, 30);
      tmem_dealloc(tmem, L::TMEM_COLS);
    }
  };

  if (warp == 8) {
    // -------------------------------------------------------------- TMA producer
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    const int rows = p.page < 128 ? p.page : 128;  // rows of a box
    const int boxes = 128 / rows;                  // boxes per tile: one lane each
    // page of this lane's box in tile i of the segment (num_pages, out of
    // range: the box is filled with zeros)
    auto page_of = [&](const CachedCursor& c, int i) -> int {
      if (lane >= boxes) return 0;
      const int first = c.seq.tile(c.i0 + i) * 128 + lane * rows;  // first slot
      const bool seen = first < c.seq.total &&
                        (first + rows > c.seq.ctx || first + rows > c.seq.ctx - p.window + 1 || first < p.sinks);
      if (!seen) return p.num_pages;
      const int id = __ldg(p.table + static_cast<long long>(c.b) * p.width + first / p.page);
      if (id < 0 || id >= p.num_pages) {
        report_page(2, c.b);
        return p.num_pages;
      }
      return id;
    };
    int k_issued = 0, v_issued = 0, segs = 0;
    bool ok = true;
    auto load = [&](const CUtensorMap& tm, uint32_t off, int full, int empty, int& issued, int tile, int hk,
                    int id) -> bool {
      const int s = issued % KVS, u = issued / KVS;
      if (u > 0 && !wait.warp(bar(empty + s), (u - 1) & 1, 2)) return false;
      if (lane == 0) mbar_expect_tx(bar(full + s), L::TILE);
      __syncwarp();
      if (lane < boxes) {
        const int row = p.page > 128 ? (tile * 128) % p.page : 0;
        for (int hh = 0; hh < D / 64; ++hh)
          tma_load_4d(base + off + s * L::TILE + hh * L::HALF + lane * rows * 128, &tm, bar(full + s), 64 * hh, row, hk,
                      id);
      }
      ++issued;
      return true;
    };
    for (; ok && cur.valid(); cur.next(p)) {
      const int hk = cur.key_head(p);
      int id = page_of(cur, 0);
      for (int i = 0; i < cur.n; ++i) {
        const int tile = cur.seq.tile(cur.i0 + i);
        const int next_id = i + 1 < cur.n ? page_of(cur, i + 1) : 0;
        ok = load(tm_k, L::K_OFF, L::K_FULL, L::K_EMPTY, k_issued, tile, hk, id);
        if (!ok) break;
        if (i == 0) {
          // the segment's rows, C copies, once the products that read the last one's are done
          ok = segs == 0 || wait.warp(bar(L::Q_EMPTY), (segs - 1) & 1, 1);
          if (!ok) break;
          if (lane == 0) {
            mbar_expect_tx(bar(L::Q_FULL), C * (D / 64) * p.R * 128);
            for (int c = 0; c < C; ++c)
              for (int hh = 0; hh < D / 64; ++hh)
                tma_load_4d(base + L::Q_OFF + hh * L::HALF + c * LR * 128, &tm_q, bar(L::Q_FULL), 64 * hh, 0,
                            hk * (p.H / p.Hkv) + cur.row_tile(p) * p.GT, cur.b);
          }
          ++segs;
          __syncwarp();
        }
        ok = load(tm_v, L::V_OFF, L::V_FULL, L::V_EMPTY, v_issued, tile, hk, id);
        if (!ok) break;
        id = next_id;
      }
    }
    // every load issued must have landed before the CTA may exit
    if (lane == 0) {
      volatile int never = 0;
      const BoundedWait drain{&never, kErrCached, limit_ns};
      for (int x = k_issued - KVS; x < k_issued; ++x)
        if (x >= 0) drain(bar(L::K_FULL + x % KVS), (x / KVS) & 1, 21);
      for (int x = v_issued - KVS; x < v_issued; ++x)
        if (x >= 0) drain(bar(L::V_FULL + x % KVS), (x / KVS) & 1, 22);
      if (segs > 0) drain(bar(L::Q_FULL), (segs - 1) & 1, 20);
    }
    __syncwarp();
    teardown();
    return;
  }
  if (warp == 9) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t IDESC_O = idesc_bf16_f32(128, D, false, true);
      const uint64_t dq = sdesc_sw128(base + L::Q_OFF, 16, 1024);
      const uint64_t dk0 = sdesc_sw128(base + L::K_OFF, 16, 1024);
      const uint64_t dv0 = sdesc_sw128(base + L::V_OFF, L::HALF, 1024);
      constexpr uint64_t kTile = L::TILE >> 4;
      int g0 = 0, segs = 0;
      int np[2] = {0, 0};  // P_bar tiles consumed per slot
      bool ok = true;
      auto issue_s = [&](int i, int n) -> bool {  // S of the segment's tile i into slot i & 1
        const int g = g0 + i, s = g % KVS;
        if (!wait(bar(L::K_FULL + s), (g / KVS) & 1, 5)) return false;
        tc_fence_after();
        const uint64_t kb = dk0 + kTile * static_cast<uint64_t>(s);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t koff = ((ks >> 2) * L::HALF + (ks & 3) * 32) >> 4;
          mma_ss(tmem + L::s_col(i & 1), dq + koff, kb + koff, IDESC_S, ks > 0 ? 1u : 0u);
        }
        tc_commit(bar(L::S_FULL + (i & 1)));
        tc_commit(bar(L::K_EMPTY + s));
        if (i + 1 == n) tc_commit(bar(L::Q_EMPTY));
        return true;
      };
      for (; ok && cur.valid(); cur.next(p), ++segs) {
        const int n = cur.n;
        ok = wait(bar(L::Q_FULL), segs & 1, 4) && issue_s(0, n) && (n < 2 || issue_s(1, n));
        for (int i = 0; ok && i < n; ++i) {
          const int t = i & 1, g = g0 + i, s = g % KVS;
          if (!wait(bar(L::P_FULL + t), np[t] & 1, 7) || !wait(bar(L::V_FULL + s), (g / KVS) & 1, 8)) {
            ok = false;
            break;
          }
          ++np[t];
          tc_fence_after();
          const uint64_t vd = dv0 + kTile * static_cast<uint64_t>(s);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_ts(tmem + L::o_col(t), tmem + L::s_col(t) + 8u * ks, vd + 128u * ks, IDESC_O,
                   (i > 1 || ks > 0) ? 1u : 0u);
          tc_commit(bar(L::O_READY + t));
          tc_commit(bar(L::V_EMPTY + s));
          // (products of one thread run in issue order: S may overwrite P_bar)
          if (i + 2 < n) ok = issue_s(i + 2, n);
        }
        g0 += n;
      }
      tc_commit(bar(L::TEARDOWN));
    }
    __syncwarp();
    teardown();
    return;
  }

  // -------------------------------------------------------- softmax warps 0..7
  const int t = warp >> 2;          // slot: tiles t, t+2, ... of a segment
  const int r = threadIdx.x & 127;  // TMEM lane
  const int copy = r / LR, row = r % LR;
  const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t s_addr = tmem + lane_base + L::s_col(t);
  const float cmp_scale = kRawCompare ? 1.f : p.scale;
  const float to_s = kRawCompare ? p.scale : 1.f;
  const float exp_c = (kRawCompare ? p.scale : 1.f) * kLog2e;
  const uint64_t EXPC2 = f2_pack(exp_c, exp_c);
  const unsigned long long all_new = p.T == 64 ? ~0ull : (1ull << p.T) - 1ull;
  // lanes past the last row hold whatever the Q buffer held: they follow a live
  // row's control flow, and nothing of theirs is read
  const int tok = row % p.T;
  const bool live = row < p.R;
  int gp[2] = {0, 0};  // products finished per slot before this segment
  int g0 = 0;
  bool ok = true;
  // Error discipline: the two warpgroups meet on named barrier 1 at the end of
  // each segment with an AND vote; a wait that gives up only clears `ok` and
  // takes its warp to that vote.
  for (; cur.valid(); cur.next(p)) {
    const int ctx = cur.seq.ctx, n = cur.n;
    // this row's new tokens, and the union over the rows (which slots hold one)
    unsigned long long bits = 0ull, any = 0ull;
    int lo = 0;
    if (p.tree == nullptr) {
      bits = (2ull << tok) - 1ull;  // tok = 63: all ones
      any = all_new;
    } else {
      const unsigned long long* words = p.tree + static_cast<long long>(cur.b) * p.T;
      for (int u = 0; u < p.T; ++u) any |= __ldg(words + u);
      any &= all_new;
      bits = __ldg(words + tok) & all_new;
    }
    const bool absent = bits == 0ull;
    lo = ctx + __popcll(bits) - p.window;  // first key of the window (pos - window + 1)
    if (p.window < p.T && !absent) {
      // some new tokens may be out of the window too
      const int pos = ctx + __popcll(bits) - 1;
      unsigned long long keep = 0ull;
      for (int u = 0; u < p.T; ++u) {
        const unsigned long long w =
            p.tree ? __ldg(p.tree + static_cast<long long>(cur.b) * p.T + u) & all_new : (2ull << u) - 1ull;
        const int pu = ctx + __popcll(w) - 1;
        if (pos - pu < p.window || pu < p.sinks) keep |= 1ull << u;
      }
      bits &= keep;
    }
    float rm_x = -INFINITY, m_run = -INFINITY, l = 0.f;
    int rs = 0;
    for (int i = t, k = 0; i < n; i += 2, ++k) {
      const int kv0 = cur.seq.tile(cur.i0 + i) * 128;
      ok = ok && wait.warp(bar(L::S_FULL + t), (gp[t] + k) & 1, 10);
      if (!ok) break;
      tc_fence_after();
      float x[LR];
      {
        uint32_t raw[LR];
        if constexpr (C == 1) {
          tmem_ld32x4(s_addr, raw);
        } else {
#pragma unroll
          for (int c0 = 0; c0 < LR; c0 += 32) tmem_ld32_nowait(s_addr + copy * LR + c0, &raw[c0]);
#pragma unroll
          for (int c0 = 0; c0 < LR; c0 += 32) tmem_wait_ld32(*reinterpret_cast<uint32_t(*)[32]>(&raw[c0]));
        }
#pragma unroll
        for (int c = 0; c < LR; ++c) x[c] = __uint_as_float(raw[c]);
      }
      const int key0 = kv0 + copy * LR;  // slot of x[0]
      if (absent || key0 + LR > ctx || (key0 < lo && key0 + LR > p.sinks)) {
        const RowMask mk{lo - key0, ctx - key0, p.sinks - key0};
#pragma unroll
        for (int w = 0; w < LR / 32; ++w) {
          uint32_t vis = mk.word(32 * w);
          const int s = ctx - key0 - 32 * w;  // column of the first new token
          if (s < 32 && s > -64) vis |= static_cast<uint32_t>(s >= 0 ? bits << s : bits >> -s);
          if (absent) vis = 0u;
#pragma unroll
          for (int c = 0; c < 32; ++c) x[32 * w + c] = (vis >> c) & 1u ? x[32 * w + c] * cmp_scale : -INFINITY;
        }
      } else if (!kRawCompare) {
#pragma unroll
        for (int c = 0; c < LR; ++c) x[c] *= cmp_scale;
      }
      float tmax;
      {
        float pm[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) pm[u] = fmaxf(x[2 * u], x[2 * u + 1]);
#pragma unroll
        for (int c = 16; c < LR; c += 16) {
#pragma unroll
          for (int u = 0; u < 8; ++u) pm[u] = fmax3(pm[u], x[c + 2 * u], x[c + 2 * u + 1]);
        }
        tmax = fmax3(fmax3(pm[0], pm[1], pm[2]), fmax3(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7]));
      }
      if (p.mode != 0) {
        int tcnt = 0;
        if (__any_sync(0xffffffffu, tmax >= rm_x)) {
          uint64_t cnt2[2] = {0ull, 0ull};
#pragma unroll
          for (int c = 0; c < LR; c += 2)
            cnt2[(c >> 1) & 1] = f2_add(cnt2[(c >> 1) & 1], f2_pack(feq(x[c], tmax), feq(x[c + 1], tmax)));
          float ca, cb;
          f2_unpack(f2_add(cnt2[0], cnt2[1]), ca, cb);
          tcnt = static_cast<int>(ca + cb);
        }
        rs = tmax > rm_x ? tcnt : (tmax == rm_x ? rs + tcnt : rs);
      }
      rm_x = fmaxf(rm_x, tmax);
      const float rm_s = rm_x * to_s;
      float m_new = rm_s;
      if (p.mode != 0 && rs > 1 && rm_s > -INFINITY) {
        m_new = (rm_s > 0.f) ? __fmul_rn(p.beta, rm_s) : ((rm_s < 0.f) ? 0.f : __fsub_rn(p.beta, 1.f));
        if (p.mode == 2 && __fsub_rn(m_new, rm_s) < kShiftMargin) m_new = __fadd_rn(rm_s, kShiftMargin);
      }
      // a row that has seen nothing yet keeps m = -inf; its P_bar is exp2(-inf) = 0
      const float nm = m_new > -INFINITY ? -m_new * kLog2e : 0.f;
      const uint64_t NM2 = f2_pack(nm, nm);
      uint64_t sum2[2] = {0ull, 0ull};
      uint32_t pk[LR / 2];
#pragma unroll
      for (int c = 0; c < LR; c += 2) {
        float y0, y1;
        f2_unpack(f2_fma(f2_pack(x[c], x[c + 1]), EXPC2, NM2), y0, y1);
        const float e0 = ex2_approx(y0), e1 = ex2_approx(y1);
        sum2[(c >> 1) & 1] = f2_add(sum2[(c >> 1) & 1], f2_pack(e0, e1));
        pk[c >> 1] = pack_bf16x2(e0, e1);
      }
      float psum;
      {
        float a, b;
        f2_unpack(f2_add(sum2[0], sum2[1]), a, b);
        psum = a + b;
      }
      // P_bar of this copy's keys, zeros for the other copies' keys
      if constexpr (C == 1) {
        tmem_st32(s_addr, *reinterpret_cast<const uint32_t(*)[32]>(&pk[0]));
        tmem_st32(s_addr + 32, *reinterpret_cast<const uint32_t(*)[32]>(&pk[32]));
      } else if constexpr (C == 2) {
        const uint32_t zero[32] = {};
        tmem_st32(s_addr + 32u * copy, pk);
        tmem_st32(s_addr + 32u * (1 - copy), zero);
      } else {
        const uint32_t zero[16] = {};
        tmem_st16(s_addr + 16u * copy, pk);
#pragma unroll
        for (int c = 1; c < 4; ++c) tmem_st16(s_addr + 16u * ((copy + c) & 3), zero);
      }
      // O of the previous tile of this slot is complete: rescale if the shift moved
      if (k > 0) {
        ok = wait.warp(bar(L::O_READY + t), (gp[t] + k - 1) & 1, 11);
        if (!ok) break;
        tc_fence_after();
        const bool changed = live && m_new != m_run;
        float alpha = 1.f;
        if (changed) {
          alpha = ex2_approx((m_run - m_new) * kLog2e);  // 0 from -inf
          l *= alpha;
        }
        if (__any_sync(0xffffffffu, changed)) {
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t v[32];
            tmem_ld32(tmem + lane_base + L::o_col(t) + c0, v);
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * alpha);
            tmem_st32(tmem + lane_base + L::o_col(t) + c0, v);
          }
        }
      }
      m_run = m_new;
      l += psum;
      // V rows of slots that hold no token: zeros (the tile's own slot r)
      if (kv0 + 128 > ctx) {
        const int s = (g0 + i) % KVS, u = kv0 + r - ctx;
        ok = wait.warp(bar(L::V_FULL + s), ((g0 + i) / KVS) & 1, 12);
        if (!ok) break;
        if (u >= 0 && (u >= p.T || !((any >> u) & 1ull))) {
          const uint32_t vr = base + L::V_OFF + s * L::TILE + r * 128;
#pragma unroll
          for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
            for (int c = 0; c < 8; ++c) sts128(vr + hh * L::HALF + 16 * c, 0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(bar(L::P_FULL + t));
    }
    // ------------------------------------------------------- end of a segment
    // the two warpgroups' states of lane r, joined: each warpgroup writes half of the columns
    const int n0 = (n + 1) / 2, n1 = n / 2;
    ok = ok && wait.warp(bar(L::O_READY + 0), (gp[0] + n0 - 1) & 1, 13);
    ok = ok && (n1 == 0 || wait.warp(bar(L::O_READY + 1), (gp[1] + n1 - 1) & 1, 14));
    const uint32_t ml = base + L::ML_OFF + r * 4;
    sts32(ml + t * 512, m_run);
    if (t == 1) sts32(ml + 1024, l);
    ok = named_barrier_and(1, 256, ok);
    if (!ok) break;
    tc_fence_after();
    const float m0 = lds32(ml), m1 = lds32(ml + 512);
    const float mm = fmaxf(m0, m1);
    const float w0 = m0 > -INFINITY ? ex2_approx((m0 - mm) * kLog2e) : 0.f;
    const float w1 = m1 > -INFINITY ? ex2_approx((m1 - mm) * kLog2e) : 0.f;
    const long long at = cur.slot(p) * (C * p.R) + copy * p.R + (live ? row : 0);
    float* dst = p.part_o + at * D + t * (D / 2);
#pragma unroll 1
    for (int c0 = 0; c0 < D / 2; c0 += 32) {
      uint32_t a[32], b[32];
      tmem_ld32x2(tmem + lane_base + L::o_col(0) + t * (D / 2) + c0, tmem + lane_base + L::o_col(1) + t * (D / 2) + c0,
                  a, b);
      if (live) {
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // (slot 1's accumulator holds nothing of this segment when it has one tile)
            v[e] = __uint_as_float(a[c + e]) * w0;
            if (n1 > 0) v[e] = fmaf(__uint_as_float(b[c + e]), w1, v[e]);
          }
          *reinterpret_cast<float4*>(dst + c0 + c) = make_float4(v[0], v[1], v[2], v[3]);
        }
      }
    }
    if (live && t == 0) p.part_ml[at] = make_float2(mm, l * w0 + lds32(ml + 1024) * w1);
    tc_fence_before();
    named_barrier_sync(1, 256);  // both have read: the next segment may overwrite O and the exchange
    gp[0] += n0;
    gp[1] += n1;
    g0 += n;
  }
  teardown();
}

// Joins the partial results of each row: one block per row of the output, the
// parts (segments x copies) dealt to its warps, then the warps' sums through
// shared memory.
struct JoinParams {
  __nv_bfloat16* o;
  ViewStrides so;
  float* lse;  // [B, H, T]
  int C, grid;
};
template <int D, int WARPS>
__global__ void __launch_bounds__(32 * WARPS)
fa_cached_join_kernel(const CachedParams p, const JoinParams q) {
  constexpr int V = D / 32;  // columns per lane
  __shared__ float sh_m[WARPS], sh_l[WARPS];
  __shared__ float sh_o[WARPS][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();
  const long long rows = static_cast<long long>(p.B) * p.H * p.T;
  const int HR = p.Hkv * p.RT, G = p.H / p.Hkv;
  for (long long id = blockIdx.x; id < rows; id += gridDim.x) {
    const int tok = static_cast<int>(id % p.T);
    const long long bh = id / p.T;
    const int h = static_cast<int>(bh % p.H), b = static_cast<int>(bh / p.H);
    const int hk = h / G, g = h - hk * G, rt = g / p.GT;
    const int row = (g - rt * p.GT) * p.T + tok, hr = hk * p.RT + rt;
    const long long before = __ldcg(p.prefix + b), nt = __ldcg(p.prefix + b + 1) - before;
    const long long U = __ldcg(p.prefix + p.B) * HR, grid = q.grid < U ? q.grid : U;
    float m = -INFINITY, l = 0.f, acc[V] = {};
    if (nt > 0) {
      const long long u0 = before * HR + hr * nt;
      // the CTA that holds unit u: the largest c with c U / grid <= u
      const long long c0 = ((u0 + 1) * grid - 1) / U, c1 = ((u0 + nt) * grid - 1) / U;
      const long long item = static_cast<long long>(b) * HR + hr;
      const int parts = static_cast<int>(c1 - c0 + 1) * q.C;
      for (int i = warp; i < parts; i += WARPS) {
        const long long at = (item + c0 + i / q.C) * (q.C * p.R) + (i % q.C) * p.R + row;
        const float2 ml = __ldcg(p.part_ml + at);
        float v[V];
        if constexpr (V == 4) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * D) + lane);
          v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
        } else {
          const float2 x = __ldcg(reinterpret_cast<const float2*>(p.part_o + at * D) + lane);
          v[0] = x.x; v[1] = x.y;
        }
        if (ml.x > -INFINITY) {
          const float mm = fmaxf(m, ml.x);
          const float wa = ex2_approx((m - mm) * kLog2e), wb = ex2_approx((ml.x - mm) * kLog2e);
          l = l * wa + ml.y * wb;
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] = acc[e] * wa + v[e] * wb;
          m = mm;
        }
      }
    }
    if (lane == 0) {
      sh_m[warp] = m;
      sh_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) sh_o[warp][lane * V + e] = acc[e];
    __syncthreads();
    if (warp == 0) {
      float mm = sh_m[0];
#pragma unroll
      for (int w = 1; w < WARPS; ++w) mm = fmaxf(mm, sh_m[w]);
      float ll = 0.f, out[V] = {};
      if (mm > -INFINITY) {
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          const float f = ex2_approx((sh_m[w] - mm) * kLog2e);
          ll += sh_l[w] * f;
#pragma unroll
          for (int e = 0; e < V; ++e) out[e] += sh_o[w][lane * V + e] * f;
        }
      }
      const float inv = mm > -INFINITY ? 1.f / ll : 0.f;
      __nv_bfloat16* dst = q.o + b * q.so.b + h * q.so.h + tok * q.so.n;
      if constexpr (V == 4)
        reinterpret_cast<uint2*>(dst)[lane] =
            make_uint2(pack_bf16x2(out[0] * inv, out[1] * inv), pack_bf16x2(out[2] * inv, out[3] * inv));
      else
        reinterpret_cast<uint32_t*>(dst)[lane] = pack_bf16x2(out[0] * inv, out[1] * inv);
      if (lane == 0) q.lse[id] = mm > -INFINITY ? mm + logf(ll) : -INFINITY;
    }
    __syncthreads();
  }
}

}  // namespace fa
