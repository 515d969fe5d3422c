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
// Per CTA: two slots take the tiles of a segment alternately, each with its own
// S/P columns, O accumulator, running statistics and softmax warpgroup (while one
// slot's exponentials are computed the other's products run), joined through
// TMEM at the segment's end.  With C = 1 a thread would hold 128 scores: there a
// slot has two warpgroups, which halve the columns of each row and exchange
// maxima and tie counts through shared memory.  Where a key head has more than
// 128 rows (PAIR) the slots hold two row tiles instead and both take every tile:
// K and V cross from L2 to the SM once for 256 rows (4 sequences of 64 tokens, 32
// heads over 4, contexts to 32768, d = 128: 135 us with a row tile at a time, 131
// us so).  One warp loads (TMA: K and V through rings, one box per page, so a page
// may lie anywhere and be smaller than a tile), one issues products.
//
// What bounds the full row tiles (the same case at 142 us): a step of a pair -- one
// 128-key tile for both row tiles -- takes 5300 cycles where its four products need
// 2048.  Clock stamps of one softmax thread in a copy of the kernel (5600 cycles a
// step with them): 2000 waiting for its scores (the slot's P V and next S, behind
// the other slot's), 1300 maximum, ties and the exchange of the halves, 1350
// exponentials, 230 waiting for O, 480 rescale, 250 reading scores and handing P_bar
// over.  These instances (two warpgroups per slot) also spill, about 300 bytes of
// stores and 400 of loads a thread.  With few rows the loads bind: 64 sequences to
// 8192, 16 heads over 4, d = 128 (675 MB): 119 us, of which 105 at 6.4 TB/s.
//   TMEM: S_t [128t, 128t+128), P_bar_t over its first 64 columns, O_t at 256 + D t.
// Pages that no row sees -- behind the window, or of absent tokens alone that no
// word names -- are not read (their place is filled with zeros by an
// out-of-range box); what lies in a read page behind the last token, or in the
// slot of an absent token, may be anything: its scores are masked and its V
// rows are overwritten with zeros in shared memory (0 * NaN would not be 0).
#pragma once

#include "fa_bwd.cuh"

namespace fa {

constexpr uint32_t kErrPage = 6;    // error word ids: a page id, length or index outside the cache ...
constexpr uint32_t kErrCached = 7;  // ... a wait of the split kernel ran out

__device__ __forceinline__ void report_page(uint32_t site, int b) {
  atomicCAS(&g_fa_error, 0u, (kErrPage << 24) | (site << 16) | (static_cast<uint32_t>(b) & 0xFFFFu));
}

struct CachedParams {
  const int* table;                  // [B, width] page ids
  const int* ctx_len;                // [B]
  const unsigned long long* tree;    // [B, T] or null: a chain
  // partial results: O against the partial's own shift; shift and sum.  C > 1:
  // [slots][C * R][D] and [slots][C * R].  Full row tiles: groups of eight rows, in runs of
  // four columns -- [slots][tiles of an item][R8 / 8][D / 4][8][4] and
  // [slots][tiles][R8], R8 = R rounded up to eights -- so that the rows of a warp fill
  // whole lines (128 rows of 512 B a thread each took 4 us to write)
  float* part_o;
  float2* part_ml;
  int* seg;                          // [items][2]: the CTAs that hold an item's first and last tile
  int B, H, Hkv, T;
  int GT, RT, R;                     // heads per row tile, items per key head (row tiles or pairs), rows per row tile
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

template <int D, int C, bool PAIR>
struct CachedLayout {
  static constexpr int LR = 128 / C;                 // lanes (rows at most) per copy, and keys per copy and tile
  static constexpr int HS = C == 1 ? 2 : 1;          // warpgroups per slot, each with LR / HS of a row's columns
  static constexpr int TILE = 128 * D * 2, HALF = 128 * 128;
  // ring stages: what is left beside the rows and the exchange
  static constexpr int KS = PAIR ? (D == 64 ? 5 : 2) : (D == 64 ? 6 : 3);
  static constexpr int VS = PAIR ? (D == 64 ? 5 : 2) : (D == 64 ? 6 : (HS == 2 ? 2 : 3));
  static constexpr int Q_OFF = 0;                    // PAIR: two row tiles
  static constexpr int K_OFF = (PAIR ? 2 : 1) * TILE, V_OFF = K_OFF + KS * TILE;
  static constexpr int ML_OFF = V_OFF + VS * TILE;   // [128] each: m of slots 0 and 1, l of the warpgroups but the first
  static constexpr int XCHG_OFF = ML_OFF + (1 + 2 * HS) * 128 * 4;  // HS = 2: [slot][parity][half][128] x 8 bytes
  static constexpr int CUR_OFF = XCHG_OFF + (HS == 2 ? 2 * 2 * 2 * 128 * 8 : 0);
  static constexpr int BAR_OFF = CUR_OFF + 32;
  enum {
    Q_FULL = 0, Q_EMPTY, K_FULL, K_EMPTY = K_FULL + KS, V_FULL = K_EMPTY + KS, V_EMPTY = V_FULL + VS,
    S_FULL = V_EMPTY + VS, P_FULL = S_FULL + 2, O_READY = P_FULL + 2, TEARDOWN = O_READY + 2, NBAR
  };
  static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
  static constexpr int SMEM_BYTES = MISC_OFF + 16 + 1024;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr int SOFT = 256 * HS;              // softmax threads; then a warpgroup: load, issue, idle, idle
  static constexpr int THREADS = SOFT + 128;
  // register budgets after setmaxnreg, against LAUNCH per thread at launch
  static constexpr uint32_t LAUNCH = HS == 2 ? 96 : 168;
  static constexpr uint32_t REGS_SOFT = HS == 2 ? 104 : 176, REGS_CTRL = HS == 2 ? 64 : 152;
  static_assert(2 * HS * REGS_SOFT + REGS_CTRL == (2 * HS + 1) * LAUNCH, "register split");
  static_assert(THREADS * LAUNCH <= 65536, "registers of an SM");
  __host__ __device__ static constexpr uint32_t s_col(int t) { return 128u * t; }
  __host__ __device__ static constexpr uint32_t o_col(int t) { return 256u + static_cast<uint32_t>(D) * t; }
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
};

template <int D, int C, bool PAIR>
__global__ void __launch_bounds__(CachedLayout<D, C, PAIR>::THREADS, 1)
fa_cached_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const CachedParams p) {
  using L = CachedLayout<D, C, PAIR>;
  constexpr int LR = L::LR, HS = L::HS;
  constexpr int LOAD_WARP = L::SOFT / 32, MMA_WARP = LOAD_WARP + 1;
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

  if (warp == MMA_WARP) {
    tmem_alloc(smem_u32(tmem_slot), L::TMEM_COLS);
    tmem_relinquish();
  }
  CachedCursor cur;
  cur.n = 0;
  grid_launch_dependents();
  int* cur_smem = reinterpret_cast<int*>(smem + L::CUR_OFF);
  if (warp == LOAD_WARP) {
    // The load warp prepares the barriers, finds this CTA's share of the list --
    // [c U / G, (c+1) U / G) of U tiles, with two passes over the lengths -- and
    // goes straight on to its loads; the others meet it at named barrier 4 (it
    // only arrives there).
    if (lane == 0) {
      mbar_init(bar(L::Q_FULL), 1);
      mbar_init(bar(L::Q_EMPTY), 1);
      for (int s = 0; s < L::KS; ++s) {
        mbar_init(bar(L::K_FULL + s), 1);
        mbar_init(bar(L::K_EMPTY + s), 1);
      }
      for (int s = 0; s < L::VS; ++s) {
        mbar_init(bar(L::V_FULL + s), 1);
        mbar_init(bar(L::V_EMPTY + s), 1);
      }
      for (int t = 0; t < 2; ++t) {
        mbar_init(bar(L::S_FULL + t), 1);
        mbar_init(bar(L::P_FULL + t), 128 * HS);
        mbar_init(bar(L::O_READY + t), 1);
      }
      mbar_init(bar(L::TEARDOWN), 1);
      *abort_flag = 0;
      mbar_fence_init();
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    grid_dependency_wait();
    // the pages may have been written by the grid before (fa_cache_append); the
    // loads below read them through the async proxy
    fence_proxy_async_all();
    const int HR = p.Hkv * p.RT;
    CachedTiles mine;  // sequence `lane` of the first 32
    mine.n = 0;
    long long sum = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      CachedTiles s;
      s.n = 0;
      if (b0 + lane < p.B) {
        s.load(p, b0 + lane);
        if (s.n == 0 && blockIdx.x == 0) report_page(1, b0 + lane);
      }
      if (b0 == 0) mine = s;
      sum += __reduce_add_sync(0xffffffffu, static_cast<unsigned>(s.n));
    }
    const long long U = sum * HR;
    const unsigned G = static_cast<unsigned>(gridDim.x < U ? gridDim.x : U), c = blockIdx.x;
    long long start = 0;
    cur.b = cur.hr = cur.i0 = 0;
    cur.left = 0;
    if (c < G) {
      if (U < (1 << 24)) {  // (at most kCachedGrid = 160 CTAs: the products fit in 32 bits)
        const unsigned u = static_cast<unsigned>(U), first = c * u / G;
        start = first;
        cur.left = (c + 1) * u / G - first;
      } else {
        start = c * U / G;
        cur.left = (c + 1) * U / G - start;
      }
      long long before = 0;
      for (int b0 = 0; b0 < p.B; b0 += 32) {
        CachedTiles s = mine;
        if (b0 > 0) {
          s.n = 0;
          if (b0 + lane < p.B) s.load(p, b0 + lane);
        }
        int inc = s.n;  // (32 sequences: below 2^31 tiles)
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += x;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, start < (before + inc) * HR);
        if (hit) {
          const int at = __ffs(hit) - 1;
          const long long in = start - (before + __shfl_sync(0xffffffffu, inc - s.n, at)) * HR;
          cur.seq.ctx = __shfl_sync(0xffffffffu, s.ctx, at);
          cur.seq.total = __shfl_sync(0xffffffffu, s.total, at);
          cur.seq.lo = __shfl_sync(0xffffffffu, s.lo, at);
          cur.seq.ns = __shfl_sync(0xffffffffu, s.ns, at);
          cur.seq.n = __shfl_sync(0xffffffffu, s.n, at);
          cur.b = b0 + at;
          if (in < (1ll << 31)) {
            cur.hr = static_cast<unsigned>(in) / static_cast<unsigned>(cur.seq.n);
            cur.i0 = static_cast<unsigned>(in) - static_cast<unsigned>(cur.hr) * cur.seq.n;
          } else {
            cur.hr = static_cast<int>(in / cur.seq.n);
            cur.i0 = static_cast<int>(in - static_cast<long long>(cur.hr) * cur.seq.n);
          }
          break;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
      }
      cur.clip();
    }
    if (lane == 0) {
      cur_smem[0] = cur.b;
      cur_smem[1] = cur.hr;
      cur_smem[2] = cur.i0;
      *reinterpret_cast<long long*>(cur_smem + 4) = cur.left;
    }
    __threadfence_block();
    __syncwarp();
    named_barrier_arrive(4, L::THREADS);
  } else {
    grid_dependency_wait();
    tc_fence_before();
    named_barrier_sync(4, L::THREADS);
    tc_fence_after();
    cur.b = cur_smem[0];
    cur.hr = cur_smem[1];
    cur.i0 = cur_smem[2];
    cur.left = *reinterpret_cast<const long long*>(cur_smem + 4);
    if (cur.valid()) {
      cur.seq.load(p, cur.b);
      cur.clip();
    }
  }
  // (the load warp has no use for the TMEM address)
  const uint32_t tmem = warp == LOAD_WARP ? 0u : *tmem_slot;

  auto teardown = [&]() {
    tc_fence_before();
    named_barrier_sync(2, L::THREADS);
    if (warp == MMA_WARP) {
      tc_fence_after();
      volatile int never = 0;
      const BoundedWait drain{&never, kErrCached, limit_ns};
      drain(bar(L::TEARDOWN), 0, 30);
      tmem_dealloc(tmem, L::TMEM_COLS);
    }
  };

  if (warp >= LOAD_WARP) warpgroup_reg_dealloc<L::REGS_CTRL>();
  if (warp > MMA_WARP) {
    teardown();
    return;
  }
  if (warp == LOAD_WARP) {
    // -------------------------------------------------------------- TMA producer
    const int rows = p.page < 128 ? p.page : 128;  // rows of a box
    const int boxes = 128 / rows;                  // boxes per tile: one lane each
    // what the rows of the current sequence see of it: the new tokens that a
    // word names (0: no row sees anything), and the first context slot in the
    // window of the row that reaches back furthest -- the one that sees the fewest
    // new tokens, which need not be the root: that one may be absent
    unsigned long long named = 0ull;
    int near = 0;
    auto look = [&](const CachedCursor& c) {
      const unsigned long long all_new = p.T == 64 ? ~0ull : (1ull << p.T) - 1ull;
      int fewest = 1;
      named = all_new;
      if (p.tree != nullptr) {
        const unsigned long long* words = p.tree + static_cast<long long>(c.b) * p.T;
        const unsigned long long w0 = lane < p.T ? __ldg(words + lane) & all_new : 0ull;
        const unsigned long long w1 = lane + 32 < p.T ? __ldg(words + lane + 32) & all_new : 0ull;
        const unsigned long long w = w0 | w1;
        named = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(w)) |
                static_cast<unsigned long long>(__reduce_or_sync(0xffffffffu, static_cast<unsigned>(w >> 32))) << 32;
        const unsigned n0 = w0 ? __popcll(w0) : 65, n1 = w1 ? __popcll(w1) : 65;
        fewest = static_cast<int>(__reduce_min_sync(0xffffffffu, n0 < n1 ? n0 : n1));
        if (named == 0ull) fewest = 1;
      }
      near = window_first(c.seq.ctx, fewest, p.window);
    };
    // first slot of this lane's box in tile i of the segment
    auto slot_of = [&](const CachedCursor& c, int i) { return c.seq.tile(c.i0 + i) * 128 + lane * rows; };
    // its entry of the page table, needed or not: asked for before the tree's
    // words arrive (8 sequences, trees of 16, 32 heads over 4, d = 128: 41.7 us
    // against 42.2 after them)
    auto entry_of = [&](const CachedCursor& c, int i) -> int {
      const int first = slot_of(c, i);
      if (lane >= boxes || first >= c.seq.total) return 0;
      return __ldg(p.table + static_cast<long long>(c.b) * p.width + first / p.page);
    };
    // the page to load for that entry (num_pages, out of range: the box is filled
    // with zeros)
    auto page_of = [&](const CachedCursor& c, int i, int id) -> int {
      if (lane >= boxes) return 0;
      const int ctx = c.seq.ctx, first = slot_of(c, i);
      if (first >= c.seq.total || named == 0ull) return p.num_pages;
      bool seen = first < ctx && (first < p.sinks || (ctx - first < rows ? ctx : first + rows) > near);
      const int u0 = first > ctx ? first - ctx : 0, n = rows - (ctx > first ? ctx - first : 0);  // new tokens [u0, u0 + n)
      if (n > 0 && u0 < 64) seen = seen || ((named >> u0) & (n < 64 ? (1ull << n) - 1ull : ~0ull)) != 0ull;
      if (!seen) return p.num_pages;
      if (id < 0 || id >= p.num_pages) {
        report_page(2, c.b);
        return p.num_pages;
      }
      return id;
    };
    int k_issued = 0, v_issued = 0, segs = 0;
    bool ok = true;
    auto load = [&](const CUtensorMap& tm, uint32_t off, int full, int empty, int stages, int& issued, int tile, int hk,
                    int id) -> bool {
      const int s = issued % stages, u = issued / stages;
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
    for (int b = -1; ok && cur.valid(); cur.next(p)) {
      const int hk = cur.key_head(p);
      const int entry = entry_of(cur, 0);
      if (cur.b != b) look(cur);
      b = cur.b;
      int id = page_of(cur, 0, entry);
      for (int i = 0; i < cur.n; ++i) {
        const int tile = cur.seq.tile(cur.i0 + i);
        const int next_id = i + 1 < cur.n ? page_of(cur, i + 1, entry_of(cur, i + 1)) : 0;
        ok = load(tm_k, L::K_OFF, L::K_FULL, L::K_EMPTY, L::KS, k_issued, tile, hk, id);
        if (!ok) break;
        if (i == 0) {
          // the segment's rows, C copies, once the products that read the last one's are done
          ok = segs == 0 || wait.warp(bar(L::Q_EMPTY), (segs - 1) & 1, 1);
          if (!ok) break;
          if (lane == 0) {
            constexpr int TILES = PAIR ? 2 : 1;
            mbar_expect_tx(bar(L::Q_FULL), TILES * C * (D / 64) * p.R * 128);
            for (int x = 0; x < TILES; ++x)  // (a head past the last one reads as zeros)
              for (int c = 0; c < C; ++c)
                for (int hh = 0; hh < D / 64; ++hh)
                  tma_load_4d(base + L::Q_OFF + x * L::TILE + hh * L::HALF + c * LR * 128, &tm_q, bar(L::Q_FULL),
                              64 * hh, 0, hk * (p.H / p.Hkv) + (cur.row_tile(p) * TILES + x) * p.GT, cur.b);
          }
          ++segs;
          __syncwarp();
        }
        ok = load(tm_v, L::V_OFF, L::V_FULL, L::V_EMPTY, L::VS, v_issued, tile, hk, id);
        if (!ok) break;
        id = next_id;
      }
    }
    // every load issued must have landed before the CTA may exit
    if (lane == 0) {
      volatile int never = 0;
      const BoundedWait drain{&never, kErrCached, limit_ns};
      for (int x = k_issued - L::KS; x < k_issued; ++x)
        if (x >= 0) drain(bar(L::K_FULL + x % L::KS), (x / L::KS) & 1, 21);
      for (int x = v_issued - L::VS; x < v_issued; ++x)
        if (x >= 0) drain(bar(L::V_FULL + x % L::VS), (x / L::VS) & 1, 22);
      if (segs > 0) drain(bar(L::Q_FULL), (segs - 1) & 1, 20);
    }
    __syncwarp();
    teardown();
    return;
  }
  if (warp == MMA_WARP) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t IDESC_O = idesc_bf16_f32(128, D, false, true);
      // descriptors as two 32-bit halves (see fa_bwd_pipe.cuh): the issuing
      // thread sits on the chain from P_bar to the next scores
      constexpr uint32_t HI = (1024u >> 4) | (1u << 14) | (2u << 29);
      const uint32_t lo_q = static_cast<uint32_t>(sdesc_sw128(base + L::Q_OFF, 16, 1024));
      const uint32_t lo_k = static_cast<uint32_t>(sdesc_sw128(base + L::K_OFF, 16, 1024));
      const uint32_t lo_v = static_cast<uint32_t>(sdesc_sw128(base + L::V_OFF, L::HALF, 1024));
      constexpr uint32_t kTile = L::TILE >> 4;
      int g0 = 0, segs = 0;
      int np[2] = {0, 0};  // P_bar tiles consumed per slot
      bool ok = true;
      // S of the segment's tile i into slot t (PAIR: both slots take every tile,
      // slot 0 first; otherwise slot i & 1 does)
      auto issue_s = [&](int i, int t, int n) -> bool {
        const int g = g0 + i, s = g % L::KS;
        if ((!PAIR || t == 0) && !wait(bar(L::K_FULL + s), (g / L::KS) & 1, 5)) return false;
        tc_fence_after();
        const uint32_t kb = lo_k + kTile * static_cast<uint32_t>(s), qa = lo_q + (PAIR ? kTile * static_cast<uint32_t>(t) : 0u);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t koff = ((ks >> 2) * L::HALF + (ks & 3) * 32) >> 4;
          mma_ss2(tmem + L::s_col(t), qa + koff, HI, kb + koff, HI, IDESC_S, ks > 0 ? 1u : 0u);
        }
        tc_commit(bar(L::S_FULL + t));
        if (!PAIR || t == 1) {
          tc_commit(bar(L::K_EMPTY + s));
          if (i + 1 == n) tc_commit(bar(L::Q_EMPTY));
        }
        return true;
      };
      // O_t (+)= P_bar_t V of the segment's tile i
      auto issue_pv = [&](int i, int t) -> bool {
        const int g = g0 + i, s = g % L::VS;
        if (!wait(bar(L::P_FULL + t), np[t] & 1, 7) || !wait(bar(L::V_FULL + s), (g / L::VS) & 1, 8)) return false;
        ++np[t];
        tc_fence_after();
        const uint32_t vd = lo_v + kTile * static_cast<uint32_t>(s);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_ts2(tmem + L::o_col(t), tmem + L::s_col(t) + 8u * ks, vd + 128u * ks, HI, IDESC_O,
                  (i >= (PAIR ? 1 : 2) || ks > 0) ? 1u : 0u);
        tc_commit(bar(L::O_READY + t));
        if (!PAIR || t == 1) tc_commit(bar(L::V_EMPTY + s));
        return true;
      };
      // (products of one thread run in issue order: the next S of a slot may
      // overwrite the P_bar that the product before it reads)
      for (; ok && cur.valid(); cur.next(p), ++segs) {
        const int n = cur.n;
        ok = wait(bar(L::Q_FULL), segs & 1, 4);
        if constexpr (PAIR) {
          ok = ok && issue_s(0, 0, n) && issue_s(0, 1, n);
          for (int i = 0; ok && i < n; ++i)
            for (int t = 0; ok && t < 2; ++t) ok = issue_pv(i, t) && (i + 1 >= n || issue_s(i + 1, t, n));
        } else {
          ok = ok && issue_s(0, 0, n) && (n < 2 || issue_s(1, 1, n));
          for (int i = 0; ok && i < n; ++i) ok = issue_pv(i, i & 1) && (i + 2 >= n || issue_s(i + 2, i & 1, n));
        }
        g0 += n;
      }
      tc_commit(bar(L::TEARDOWN));
    }
    __syncwarp();
    teardown();
    return;
  }

  // ------------------------------------------------------------ softmax warps
  warpgroup_reg_alloc<L::REGS_SOFT>();
  constexpr int CW = LR / HS;       // columns of a row and tile per thread
  const int t = (warp >> 2) / HS;   // slot: tiles t, t+2, ... of a segment (PAIR: all tiles, for row tile t)
  const int h = (warp >> 2) % HS;   // part of the slot's columns
  const int r = threadIdx.x & 127;  // TMEM lane
  const int copy = r / LR, row = r % LR;
  const int col = copy * LR + CW * h;  // this thread's first column
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
  const bool stall = t == 0 && inject_stall_here(kErrCached);  // test hook (fa_debug_inject_stall)
  // Error discipline: all softmax warps meet on named barrier 1 at the end of
  // each segment, and (HS = 2) the two warpgroups of a slot on barrier 3 + t in
  // each tile, with AND votes.  A wait that gives up only clears `ok`; its warp
  // goes on to the next of these meetings, which takes the others out too.
  for (; cur.valid(); cur.next(p)) {
    const int ctx = cur.seq.ctx, n = cur.n;
    // this row's new tokens, and the union over the rows (which slots hold one)
    unsigned long long bits = 0ull, any = 0ull;
    if (p.tree == nullptr) {
      bits = (2ull << tok) - 1ull;  // tok = 63: all ones
      any = all_new;
    } else {
      const unsigned long long* words = p.tree + static_cast<long long>(cur.b) * p.T;
      const int lane = threadIdx.x & 31;
      unsigned long long w = lane < p.T ? __ldg(words + lane) : 0ull;
      if (lane + 32 < p.T) w |= __ldg(words + lane + 32);
      any = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(w)) |
            static_cast<unsigned long long>(__reduce_or_sync(0xffffffffu, static_cast<unsigned>(w >> 32))) << 32;
      any &= all_new;
      bits = __ldg(words + tok) & all_new;
    }
    const bool absent = bits == 0ull;  // works like a row that sees the context; its result is put down as empty
    const int lo = window_first(ctx, __popcll(bits), p.window);
    if (p.window <= p.T && !absent) {
      // some new tokens may be out of the window too (positions of new tokens are
      // in [ctx - 1, ctx + T): an absent one's is ctx - 1)
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
    for (int i = PAIR ? 0 : t, k = 0; i < n; i += PAIR ? 1 : 2, ++k) {
      const int kv0 = cur.seq.tile(cur.i0 + i) * 128;
      ok = ok && wait.warp(bar(L::S_FULL + t), (gp[t] + k) & 1, 10);
      if (HS == 1 && !ok) break;
      tc_fence_after();
      float x[CW];
      {
        uint32_t raw[CW];
        if constexpr (CW == 64) {
          tmem_ld32x2(s_addr + col, s_addr + col + 32, *reinterpret_cast<uint32_t(*)[32]>(&raw[0]),
                      *reinterpret_cast<uint32_t(*)[32]>(&raw[32]));
        } else {
          tmem_ld32(s_addr + col, raw);
        }
#pragma unroll
        for (int c = 0; c < CW; ++c) x[c] = __uint_as_float(raw[c]);
      }
      const int key0 = kv0 + col;  // slot of x[0]
      if (__any_sync(0xffffffffu, context_hides(ctx, lo, p.sinks, key0, CW))) {
        const RowMask mk = context_mask(ctx, lo, p.sinks, key0);
#pragma unroll
        for (int w = 0; w < CW / 32; ++w) {
          uint32_t vis = mk.word(32 * w);
          const int s = ctx - key0 - 32 * w;  // column of the first new token
          if (s < 32 && s > -64) vis |= static_cast<uint32_t>(s >= 0 ? bits << s : bits >> -s);
#pragma unroll
          for (int c = 0; c < 32; ++c) x[32 * w + c] = (vis >> c) & 1u ? x[32 * w + c] * cmp_scale : -INFINITY;
        }
      } else if (!kRawCompare) {
#pragma unroll
        for (int c = 0; c < CW; c += 2) f2_unpack(f2_mul(f2_pack(x[c], x[c + 1]), f2_pack(cmp_scale, cmp_scale)), x[c], x[c + 1]);
      }
      float tmax;
      {
        float pm[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) pm[u] = fmaxf(x[2 * u], x[2 * u + 1]);
#pragma unroll
        for (int c = 16; c < CW; c += 16) {
#pragma unroll
          for (int u = 0; u < 8; ++u) pm[u] = fmax3(pm[u], x[c + 2 * u], x[c + 2 * u + 1]);
        }
        tmax = fmax3(fmax3(pm[0], pm[1], pm[2]), fmax3(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7]));
      }
      float cnt = 0.f;  // ties at tmax, where it can reach the running maximum
      if (p.mode != 0 && __any_sync(0xffffffffu, tmax >= rm_x)) {
        uint64_t cnt2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int c = 0; c < CW; c += 2)
          cnt2[(c >> 1) & 3] = f2_add(cnt2[(c >> 1) & 3], f2_pack(feq(x[c], tmax), feq(x[c + 1], tmax)));
        float ca, cb;
        f2_unpack(f2_add(f2_add(cnt2[0], cnt2[1]), f2_add(cnt2[2], cnt2[3])), ca, cb);
        cnt = ca + cb;
      }
      if constexpr (HS == 2) {
        // the row's other half (two buffers, by the parity of k)
        const uint32_t xa = base + L::XCHG_OFF + (((t * 2 + (k & 1)) * 2 + h) * 128 + r) * 8;
        sts32(xa, tmax);
        sts32(xa + 4, cnt);
        ok = named_barrier_and(3 + t, 256, ok);
        if (!ok) break;
        const uint32_t xb = base + L::XCHG_OFF + (((t * 2 + (k & 1)) * 2 + (1 - h)) * 128 + r) * 8;
        const float omax = lds32(xb), ocnt = lds32(xb + 4);
        const float both = fmaxf(tmax, omax);
        cnt = (tmax == both ? cnt : 0.f) + (omax == both ? ocnt : 0.f);
        tmax = both;
      }
      rs = tmax > rm_x ? static_cast<int>(cnt) : (tmax == rm_x ? rs + static_cast<int>(cnt) : rs);
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
      uint32_t pk[CW / 2];
#pragma unroll
      for (int c = 0; c < CW; c += 2) {
        const uint64_t y = f2_fma(f2_pack(x[c], x[c + 1]), EXPC2, NM2);
        float e0, e1;
        if (HS == 2 && (c >> 1) % 8 == 7) {
          // with full row tiles the MUFU (16 a clock) needs as long as the tensor
          // products: one pair in eight goes to the FMA pipe
          f2_unpack(exp2_poly_f2(y), e0, e1);
        } else {
          float y0, y1;
          f2_unpack(y, y0, y1);
          e0 = ex2_approx(y0);
          e1 = ex2_approx(y1);
        }
        sum2[(c >> 1) & 1] = f2_add(sum2[(c >> 1) & 1], f2_pack(e0, e1));
        pk[c >> 1] = pack_bf16x2(e0, e1);
      }
      float psum;
      {
        float a, b;
        f2_unpack(f2_add(sum2[0], sum2[1]), a, b);
        psum = a + b;
      }
      // P_bar of this copy's keys over the slot's first 64 columns (every thread
      // that reads scores there has them in registers), zeros for the other copies'
      if constexpr (C == 4) {
        const uint32_t zero[16] = {};
        tmem_st16(s_addr + 16u * copy, pk);
#pragma unroll
        for (int c = 1; c < 4; ++c) tmem_st16(s_addr + 16u * ((copy + c) & 3), zero);
      } else {
        tmem_st32(s_addr + col / 2, pk);
        if constexpr (C == 2) {
          const uint32_t zero[32] = {};
          tmem_st32(s_addr + 32u * (1 - copy), zero);
        }
      }
      // O of the previous tile of this slot is complete: rescale if the shift moved
      if (k > 0) {
        ok = wait.warp(bar(L::O_READY + t), (gp[t] + k - 1) & 1, 11);
        if (!ok) continue;
        tc_fence_after();
        const bool changed = live && m_new != m_run;
        float alpha = 1.f;
        if (changed) {
          alpha = ex2_approx((m_run - m_new) * kLog2e);  // 0 from -inf
          l *= alpha;
        }
        if (__any_sync(0xffffffffu, changed)) {
#pragma unroll 1
          for (int c0 = h * (D / HS); c0 < (h + 1) * (D / HS); c0 += 32) {
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
      // V rows of slots that hold no token: zeros (the tile's own slot r; PAIR:
      // slot 0 does it, whose product comes first)
      if (ctx - kv0 < 128 && (!PAIR || t == 0)) {
        const int s = (g0 + i) % L::VS, u = kv0 + r - ctx;
        ok = wait.warp(bar(L::V_FULL + s), ((g0 + i) / L::VS) & 1, 12);
        if (!ok) continue;
        if (h == 0 && u >= 0 && (u >= p.T || !((any >> u) & 1ull))) {
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
      if (!(stall && g0 + i == 0)) mbar_arrive(bar(L::P_FULL + t));
    }
    // ------------------------------------------------------- end of a segment
    // the two slots' states of lane r, joined, each warpgroup writing its part of
    // the columns; PAIR: each slot's on their own
    const int n0 = PAIR ? n : (n + 1) / 2, n1 = PAIR ? n : n / 2;
    if (!PAIR || t == 0) ok = ok && wait.warp(bar(L::O_READY + 0), (gp[0] + n0 - 1) & 1, 13);
    if (!PAIR || t == 1) ok = ok && (n1 == 0 || wait.warp(bar(L::O_READY + 1), (gp[1] + n1 - 1) & 1, 14));
    const uint32_t ml = base + L::ML_OFF + r * 4;
    if (absent) m_run = -INFINITY;
    if (h == 0) sts32(ml + t * 512, m_run);
    if (t * HS + h > 0) sts32(ml + 512 + (t * HS + h) * 512, l);
    ok = named_barrier_and(1, L::SOFT, ok);
    if (!ok) break;
    tc_fence_after();
    constexpr int TILES = PAIR ? 2 : 1;
    const int R8 = (p.R + 7) & ~7;
    const long long at = C > 1 ? cur.slot(p) * (C * p.R) + copy * p.R + (live ? row : 0)
                               : (cur.slot(p) * TILES + (PAIR ? t : 0)) * R8 + (live ? row : 0);
    // full row tiles: where this row's first four columns go; four more: 8 float4 on
    float4* dst8 = reinterpret_cast<float4*>(p.part_o) + (at & ~7ll) * (D / 4) + (at & 7);
    if constexpr (PAIR) {
      constexpr int CO = D / HS;  // columns per warpgroup
#pragma unroll 1
      for (int c0 = h * CO; c0 < (h + 1) * CO; c0 += 32) {
        uint32_t a[32];
        tmem_ld32(tmem + lane_base + L::o_col(t) + c0, a);
        if (live) {
#pragma unroll
          for (int c = 0; c < 32; c += 4)
            dst8[(c0 + c) * 2] = make_float4(__uint_as_float(a[c]), __uint_as_float(a[c + 1]),
                                             __uint_as_float(a[c + 2]), __uint_as_float(a[c + 3]));
        }
      }
      if (live && h == 0) p.part_ml[at] = make_float2(m_run, l + lds32(ml + 512 + (t * HS + 1) * 512));
    } else {
      const float m0 = lds32(ml), m1 = lds32(ml + 512);
      const float mm = fmaxf(m0, m1);
      const float w0 = m0 > -INFINITY ? ex2_approx((m0 - mm) * kLog2e) : 0.f;
      const float w1 = m1 > -INFINITY ? ex2_approx((m1 - mm) * kLog2e) : 0.f;
      constexpr int CO = D / (2 * HS);  // columns per warpgroup
      const int c_first = (t * HS + h) * CO;
      float* dst = p.part_o + at * D + c_first;
#pragma unroll 1
      for (int c0 = 0; c0 < CO; c0 += 16) {
        uint32_t a[16], b[16];
        tmem_ld16(tmem + lane_base + L::o_col(0) + c_first + c0, a);
        tmem_ld16(tmem + lane_base + L::o_col(1) + c_first + c0, b);
        if (live) {
#pragma unroll
          for (int c = 0; c < 16; c += 4) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // (slot 1's accumulator holds nothing of this segment when it has one tile)
              v[e] = __uint_as_float(a[c + e]) * w0;
              if (n1 > 0) v[e] = fmaf(__uint_as_float(b[c + e]), w1, v[e]);
            }
            if constexpr (C > 1)
              *reinterpret_cast<float4*>(dst + c0 + c) = make_float4(v[0], v[1], v[2], v[3]);
            else
              dst8[(c_first + c0 + c) * 2] = make_float4(v[0], v[1], v[2], v[3]);
          }
        }
      }
      if (live && t == 0 && h == 0) {
        float l0 = l, l1 = lds32(ml + 512 + HS * 512);
        if (HS == 2) {
          l0 += lds32(ml + 512 + 512);
          l1 += lds32(ml + 512 + 3 * 512);
        }
        p.part_ml[at] = make_float2(mm, l0 * w0 + l1 * w1);
      }
    }
    if (threadIdx.x == 0) {
      const long long item = cur.slot(p) - blockIdx.x;
      if (cur.i0 == 0) p.seg[2 * item] = blockIdx.x;
      if (cur.i0 + n == cur.seq.n) p.seg[2 * item + 1] = blockIdx.x;
    }
    tc_fence_before();
    named_barrier_sync(1, L::SOFT);  // all have read: the next segment may overwrite O and the exchange
    gp[0] += n0;
    gp[1] += n1;
    g0 += n;
  }
  teardown();
}

// Joins the partial results of each row of the output (C > 1).  A row's parts (segments
// x copies) are dealt to WPR warps; lane i of a warp holds its part i's shift and
// sum, the weights come from shuffles, and the loads of the parts' O depend on
// nothing but their addresses.  Bound by latency -- three loads, one after the
// other: the item's CTAs, the shifts, and (issued with them) the rows.  Few rows
// with many parts take eight warps per row, many rows with few parts one.
struct JoinParams {
  __nv_bfloat16* o;
  ViewStrides so;
  float* lse;  // [B, H, T]
  int C;        // parts of a row per segment
  int grid;     // CTAs of the split kernel
};
template <int D, int WPR>
__global__ void __launch_bounds__(WPR > 4 ? 32 * WPR : 128)
fa_cached_join_kernel(const CachedParams p, const JoinParams q) {
  constexpr int V = D / 32;  // columns per lane
  constexpr int WARPS = WPR > 4 ? WPR : 4, RPB = WARPS / WPR;  // rows per block
  __shared__ float sh_m[WARPS], sh_l[WARPS];
  __shared__ float sh_o[WARPS][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp % WPR;
  grid_launch_dependents();
  grid_dependency_wait();
  const int rows = p.B * p.H * p.T;  // (the host keeps it below 2^31)
  const int HR = p.Hkv * p.RT, G = p.H / p.Hkv;
  for (int r0 = blockIdx.x * RPB; r0 < rows; r0 += gridDim.x * RPB) {
    const int id = r0 + warp / WPR;
    const bool in = id < rows;
    const int bh = (in ? id : 0) / p.T, tok = (in ? id : 0) - bh * p.T;
    const int b = bh / p.H, h = bh - b * p.H;
    const int hk = h / G, row = (h - hk * G) * p.T + tok, hr = hk;  // (few rows: one row tile)
    const long long item = static_cast<long long>(b) * HR + hr;
    const int2 cta = __ldcg(reinterpret_cast<const int2*>(p.seg) + item);
    CachedTiles seq;
    seq.load(p, b);  // a sequence without tiles has no segments
    float m = -INFINITY, l = 0.f, acc[V] = {};
    // (a split kernel that gave up on a wait leaves entries of the workspace as
    // they were: what is no range of CTAs is not followed)
    if (in && seq.n > 0 && cta.x >= 0 && cta.x <= cta.y && cta.y < q.grid) {
      const int parts = (cta.y - cta.x + 1) * q.C;
      // C copies of R rows per segment: part i of the row is at first + i R
      const int stride = p.R;
      const long long first = (item + cta.x) * (q.C * stride) + row;
      const int share = (parts + WPR - 1) / WPR, begin = sub * share;
      const int end = begin + share < parts ? begin + share : parts;
      for (int i0 = begin; i0 < end; i0 += 32) {
        const int n = end - i0 < 32 ? end - i0 : 32;
        const long long at = first + static_cast<long long>(i0) * stride;
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < n) ml = __ldcg(p.part_ml + at + static_cast<long long>(lane) * stride);
        const float* src = p.part_o + at * D + lane * V;
        const long long step = static_cast<long long>(stride) * D;
        constexpr int U = 8;
        float v[U][V];
        auto fetch = [&](int i) {  // rows i .. i + U - 1
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if (i + u >= n) continue;
            if constexpr (V == 4) {
              const float4 x = __ldcg(reinterpret_cast<const float4*>(src + (i + u) * step));
              v[u][0] = x.x; v[u][1] = x.y; v[u][2] = x.z; v[u][3] = x.w;
            } else {
              const float2 x = __ldcg(reinterpret_cast<const float2*>(src + (i + u) * step));
              v[u][0] = x.x; v[u][1] = x.y;
            }
          }
        };
        fetch(0);
        float top = ml.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float mm = fmaxf(m, top);
        if (!(mm > -INFINITY)) continue;  // nothing seen in any of them
        const float w = ex2_approx((ml.x - mm) * kLog2e);  // 0 for a part that has seen nothing
        const float keep = ex2_approx((m - mm) * kLog2e);
        float sum = ml.y * w;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l = l * keep + sum;
        m = mm;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] *= keep;
        for (int i = 0; i < n; i += U) {
          if (i > 0) fetch(i);
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const float wi = __shfl_sync(0xffffffffu, w, (i + u) & 31);
            if (i + u >= n) continue;
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] = fmaf(v[u][e], wi, acc[e]);
          }
        }
      }
    }
    if constexpr (WPR > 1) {  // the warps' results, by the first
      __syncthreads();
      if (lane == 0) {
        sh_m[warp] = m;
        sh_l[warp] = l;
      }
#pragma unroll
      for (int e = 0; e < V; ++e) sh_o[warp][lane * V + e] = acc[e];
      __syncthreads();
      if (sub != 0) continue;
      float mm = m;
#pragma unroll
      for (int w = 1; w < WPR; ++w) mm = fmaxf(mm, sh_m[warp + w]);
      if (mm > -INFINITY) {
        const float a = ex2_approx((m - mm) * kLog2e);
        l *= a;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] *= a;
#pragma unroll
        for (int w = 1; w < WPR; ++w) {
          const float f = ex2_approx((sh_m[warp + w] - mm) * kLog2e);
          l = fmaf(sh_l[warp + w], f, l);
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] = fmaf(sh_o[warp + w][lane * V + e], f, acc[e]);
        }
        m = mm;
      }
    }
    if (!in) continue;
    const bool any = m > -INFINITY;
    const float inv = any ? 1.f / l : 0.f;
    __nv_bfloat16* dst = q.o + b * q.so.b + h * q.so.h + tok * q.so.n;
    if constexpr (V == 4)
      reinterpret_cast<uint2*>(dst)[lane] =
          make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
    else
      reinterpret_cast<uint32_t*>(dst)[lane] = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    if (lane == 0) q.lse[id] = any ? m + logf(l) : -INFINITY;
  }
}

// The same for full row tiles, whose partial results lie in groups of eight rows:
// a warp takes a group (lane: row lane & 7, columns 4 (lane >> 3) + 16 k), so that
// its loads are whole lines.  WPR warps share a group's segments.
template <int D, int WPR>
__global__ void __launch_bounds__(128)
fa_cached_join_tiles_kernel(const CachedParams p, const JoinParams q, int tiles) {
  constexpr int K = D / 16, GPB = 4 / WPR;
  __shared__ float sh_m[4][8], sh_l[4][8];
  __shared__ float sh_o[WPR > 1 ? 4 : 1][8][WPR > 1 ? D + 4 : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % WPR;
  const int r8 = lane & 7, cg = lane >> 3;
  grid_launch_dependents();
  grid_dependency_wait();
  const int HR = p.Hkv * p.RT, G = p.H / p.Hkv, RG = (p.R + 7) / 8;
  const long long groups = static_cast<long long>(p.B) * HR * tiles * RG;
  for (long long g0 = static_cast<long long>(blockIdx.x) * GPB; g0 < groups; g0 += static_cast<long long>(gridDim.x) * GPB) {
    const long long id = g0 + warp / WPR;
    const bool in = id < groups;
    const long long ti = (in ? id : 0) / RG, item = ti / tiles;  // (item, tile), item
    const int rg = static_cast<int>((in ? id : 0) - ti * RG), tile = static_cast<int>(ti - item * tiles);
    const int b = static_cast<int>(item / HR), hr = static_cast<int>(item - static_cast<long long>(b) * HR);
    const int hk = hr / p.RT, rt = (hr - hk * p.RT) * tiles + tile;
    const int row = rg * 8 + r8, g = rt * p.GT + row / p.T, tok = row % p.T;
    const int2 cta = __ldcg(reinterpret_cast<const int2*>(p.seg) + item);
    CachedTiles seq;
    seq.load(p, b);
    float m = -INFINITY, l = 0.f, acc[K][4] = {};
    if (in && seq.n > 0 && cta.x >= 0 && cta.x <= cta.y && cta.y < q.grid) {
      const int parts = cta.y - cta.x + 1, share = (parts + WPR - 1) / WPR;
      const int begin = sub * share, end = begin + share < parts ? begin + share : parts;
      for (int i = begin; i < end; ++i) {
        const long long at = ((item + cta.x + i) * tiles + tile) * (RG * 8) + rg * 8;
        // (rows past R of the last group hold nothing)
        const float2 ml = row < p.R ? __ldcg(p.part_ml + at + r8) : make_float2(-INFINITY, 0.f);
        const float4* src = reinterpret_cast<const float4*>(p.part_o) + at * (D / 4) + cg * 8 + r8;
        float4 v[K];
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = __ldcg(src + 32 * k);
        if (ml.x > -INFINITY) {
          const float mm = fmaxf(m, ml.x);
          const float a = ex2_approx((m - mm) * kLog2e), w = ex2_approx((ml.x - mm) * kLog2e);
          l = l * a + ml.y * w;
          m = mm;
#pragma unroll
          for (int k = 0; k < K; ++k) {
            acc[k][0] = fmaf(v[k].x, w, acc[k][0] * a);
            acc[k][1] = fmaf(v[k].y, w, acc[k][1] * a);
            acc[k][2] = fmaf(v[k].z, w, acc[k][2] * a);
            acc[k][3] = fmaf(v[k].w, w, acc[k][3] * a);
          }
        }
      }
    }
    if constexpr (WPR > 1) {  // the warps' results, by the first
      __syncthreads();
      if (cg == 0) {
        sh_m[warp][r8] = m;
        sh_l[warp][r8] = l;
      }
#pragma unroll
      for (int k = 0; k < K; ++k)
        *reinterpret_cast<float4*>(&sh_o[warp][r8][16 * k + 4 * cg]) =
            make_float4(acc[k][0], acc[k][1], acc[k][2], acc[k][3]);
      __syncthreads();
      if (sub != 0) continue;
#pragma unroll
      for (int w = 1; w < WPR; ++w) {
        const float mw = sh_m[warp + w][r8], mm = fmaxf(m, mw);
        if (!(mw > -INFINITY)) continue;
        const float a = ex2_approx((m - mm) * kLog2e), f = ex2_approx((mw - mm) * kLog2e);
        l = l * a + sh_l[warp + w][r8] * f;
        m = mm;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const float4 x = *reinterpret_cast<const float4*>(&sh_o[warp + w][r8][16 * k + 4 * cg]);
          acc[k][0] = fmaf(x.x, f, acc[k][0] * a);
          acc[k][1] = fmaf(x.y, f, acc[k][1] * a);
          acc[k][2] = fmaf(x.z, f, acc[k][2] * a);
          acc[k][3] = fmaf(x.w, f, acc[k][3] * a);
        }
      }
    }
    if (!in || row >= p.R || g >= G) continue;
    const int h = hk * G + g;
    const bool any = m > -INFINITY;
    const float inv = any ? 1.f / l : 0.f;
    __nv_bfloat16* dst = q.o + b * q.so.b + h * q.so.h + tok * q.so.n + 4 * cg;
#pragma unroll
    for (int k = 0; k < K; ++k)
      *reinterpret_cast<uint2*>(dst + 16 * k) =
          make_uint2(pack_bf16x2(acc[k][0] * inv, acc[k][1] * inv), pack_bf16x2(acc[k][2] * inv, acc[k][3] * inv));
    if (cg == 0) q.lse[(static_cast<long long>(b) * p.H + h) * p.T + tok] = any ? m + logf(l) : -INFINITY;
  }
}

}  // namespace fa
