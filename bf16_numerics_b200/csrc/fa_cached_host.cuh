// Host side of fa_cached_fwd, fa_cache_append and fa_cache_compact (included
// by fa_lib.cu, whose helpers and those of fa_window_host.cuh it uses).
#pragma once

namespace {

// How the T * G rows of a key head fill 128-row tiles: tiles of GT query heads
// each (the last may hold fewer), C copies of a tile's R = GT * T rows; with more
// than one tile (R is above 64 then) they are worked on in pairs.  RT: items, which
// are tiles or pairs of them.
struct CachedSplit {
  int GT, RT, R, C;
  bool pair;
};
CachedSplit cached_split(int G, int T) {
  CachedSplit s{};
  const int most = 128 / T;
  s.RT = (G + most - 1) / most;
  s.GT = (G + s.RT - 1) / s.RT;
  s.RT = (G + s.GT - 1) / s.GT;
  s.pair = s.RT > 1;
  if (s.pair) s.RT = (s.RT + 1) / 2;
  s.R = s.GT * T;
  s.C = s.R <= 32 ? 4 : (s.R <= 64 ? 2 : 1);
  return s;
}

constexpr int kCachedGrid = 160;  // most CTAs of the split kernel (one per SM)

struct CachedLayoutBytes {
  size_t seg_off, ml_off, o_off, bytes;
};
CachedLayoutBytes cached_layout(int B, int Hkv, int d, const CachedSplit& s) {
  CachedLayoutBytes l{};
  // rows per partial result: the copies', or the row tiles' in eights
  const size_t rows = s.C > 1 ? static_cast<size_t>(s.C) * s.R : static_cast<size_t>(s.pair ? 2 : 1) * ((s.R + 7) & ~7);
  const size_t parts = (static_cast<size_t>(B) * Hkv * s.RT + kCachedGrid) * rows;
  l.seg_off = 0;
  l.ml_off = round256(static_cast<size_t>(B) * Hkv * s.RT * 8);
  l.o_off = l.ml_off + round256(parts * 8);
  l.bytes = l.o_off + round256(parts * d * 4);
  return l;
}

// sizes that fa_cached_fwd and its workspace query share; *empty: nothing to do
fa_status cached_args(int B, int H, int Hkv, int T, int d, bool* empty) {
  if (!shape_ok(B, H, T, d) || Hkv < 0 || Hkv > H) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  *empty = static_cast<long long>(B) * H * T == 0;
  if (*empty) return FA_OK;
  if (Hkv == 0 || H % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (T > 64 || static_cast<long long>(B) * H * T >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// the pool and its page table
bool pool_ok(const void* k_pages, const void* v_pages, const int* table, const int* ctx_len, int Hkv, int d,
             int num_pages, int page_size, int table_width) {
  if (num_pages < 1 || table_width < 1) return false;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128 && page_size != 256) return false;
  if (static_cast<long long>(table_width) * page_size >= (1ll << 31)) return false;
  // TMA: a page of all heads below 2^40 bytes; 16-byte indices of the pool below 2^63
  if (static_cast<long long>(Hkv) * page_size * d >= (1ll << 39)) return false;
  if (!k_pages || !v_pages || !table || !ctx_len || !aligned16(k_pages) || !aligned16(v_pages)) return false;
  return !((reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(ctx_len)) & 3u);
}

bool encode_map_4d(CUtensorMap* map, const void* ptr, const cuuint64_t (&dims)[4], const cuuint64_t (&strides)[3],
                   const cuuint32_t (&box)[4]) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// pages [num_pages, Hkv, page, D], box 64 (d) x min(page, 128) slots x 1 x 1
bool make_map_pages(CUtensorMap* map, const void* ptr, int num_pages, int Hkv, int page, int D) {
  const cuuint64_t row = static_cast<cuuint64_t>(D) * 2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(page), static_cast<cuuint64_t>(Hkv),
                              static_cast<cuuint64_t>(num_pages)};
  const cuuint64_t strides[3] = {row, row * page, row * page * Hkv};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(page < 128 ? page : 128), 1, 1};
  return encode_map_4d(map, ptr, dims, strides, box);
}

template <int D, int C, bool PAIR>
fa_status launch_cached(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const fa::CachedParams& p,
                        const fa::JoinParams& j, int grid, cudaStream_t stream) {
  using L = fa::CachedLayout<D, C, PAIR>;
  static std::atomic<uint64_t> attr{0};
  if (!ensure_smem(fa::fa_cached_kernel<D, C, PAIR>, L::SMEM_BYTES, attr)) return FA_ERR_CUDA;
  cudaError_t e;
  e = launch_pdl(fa::fa_cached_kernel<D, C, PAIR>, dim3(static_cast<unsigned>(grid)), dim3(L::THREADS), L::SMEM_BYTES,
                 stream, mq, mk, mv, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail("fa_cached_kernel launch", e);
  if constexpr (C == 1) {
    // one warp per group of eight rows once there are some for every SM, else four
    constexpr int tiles = PAIR ? 2 : 1;
    const long long groups = static_cast<long long>(p.B) * p.Hkv * p.RT * tiles * ((p.R + 7) / 8);
    if (groups >= 4ll * grid)
      e = launch_pdl(fa::fa_cached_join_tiles_kernel<D, 1>, dim3(grid_for(groups, 4)), dim3(128), 0, stream, p, j, tiles);
    else
      e = launch_pdl(fa::fa_cached_join_tiles_kernel<D, 4>, dim3(grid_for(groups, 1)), dim3(128), 0, stream, p, j, tiles);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? FA_OK : cuda_fail("fa_cached_join_tiles_kernel launch", e);
  }
  const long long rows = static_cast<long long>(p.B) * p.H * p.T;
  // one warp per row once there are rows for every SM's warps, else eight
  if (rows >= 16ll * grid)
    e = launch_pdl(fa::fa_cached_join_kernel<D, 1>, dim3(grid_for(rows, 4)), dim3(128), 0, stream, p, j);
  else
    e = launch_pdl(fa::fa_cached_join_kernel<D, 8>, dim3(grid_for(rows, 1)), dim3(256), 0, stream, p, j);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : cuda_fail("fa_cached_join_kernel launch", e);
}

template <int D>
fa_status run_cached(const fa_view* q, const void* k_pages, const void* v_pages, const fa_view* o, fa::CachedParams p,
                     fa::JoinParams j, const CachedSplit& s, cudaStream_t stream) {
  const int n_sm = sm_count();
  if (n_sm <= 0) return cuda_fail("cudaDeviceGetAttribute(multiprocessor count)");
  const int grid = n_sm < kCachedGrid ? n_sm : kCachedGrid;
  j.C = s.C;
  j.grid = grid;
  j.so = strides_of(o);
  p.scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
  CUtensorMap mq, mk, mv;
  {
    auto bytes = [&](long long st, long long extent) { return static_cast<cuuint64_t>(extent > 1 ? st : D) * 2; };
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(p.T), static_cast<cuuint64_t>(p.H),
                                static_cast<cuuint64_t>(p.B)};
    const cuuint64_t strides[3] = {bytes(q->stride_n, p.T), bytes(q->stride_h, p.H), bytes(q->stride_b, p.B)};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(p.T), static_cast<cuuint32_t>(s.GT), 1};
    if (!encode_map_4d(&mq, q->ptr, dims, strides, box)) return cuda_fail("cuTensorMapEncodeTiled (q)");
  }
  if (!make_map_pages(&mk, k_pages, p.num_pages, p.Hkv, p.page, D) ||
      !make_map_pages(&mv, v_pages, p.num_pages, p.Hkv, p.page, D))
    return cuda_fail("cuTensorMapEncodeTiled (pages)");
  if (s.pair) return launch_cached<D, 1, true>(mq, mk, mv, p, j, grid, stream);
  if (s.C == 4) return launch_cached<D, 4, false>(mq, mk, mv, p, j, grid, stream);
  if (s.C == 2) return launch_cached<D, 2, false>(mq, mk, mv, p, j, grid, stream);
  return launch_cached<D, 1, false>(mq, mk, mv, p, j, grid, stream);
}

fa::CachePool cache_pool(void* k_pages, void* v_pages, const int* table, const int* ctx_len, int Hkv, int num_pages,
                         int page_size, int table_width) {
  return {static_cast<uint4*>(k_pages), static_cast<uint4*>(v_pages), table, ctx_len, Hkv, num_pages, page_size,
          table_width};
}

}  // namespace

extern "C" {

size_t fa_cached_workspace_bytes(int B, int H, int Hkv, int T, int d) {
  bool empty = false;
  if (cached_args(B, H, Hkv, T, d, &empty) != FA_OK || empty) return 0;
  return cached_layout(B, Hkv, d, cached_split(H / Hkv, T)).bytes;
}

fa_status fa_cached_fwd(const fa_view* q, const void* k_pages, const void* v_pages, const int32_t* page_table,
                        const int32_t* ctx_len, const uint64_t* tree, const fa_view* o, float* lse, void* workspace,
                        size_t workspace_bytes, int B, int H, int Hkv, int T, int d, int num_pages, int page_size,
                        int table_width, int window, int sinks, int softmax_mode, float beta, void* stream) {
  bool empty = false;
  const fa_status st = cached_args(B, H, Hkv, T, d, &empty);
  if (st != FA_OK) return st;
  if (window < 1 || sinks < 0 || !mode_ok(softmax_mode, beta)) return FA_ERR_INVALID_ARG;
  if (empty) return FA_OK;
  if (!pool_ok(k_pages, v_pages, page_table, ctx_len, Hkv, d, num_pages, page_size, table_width) ||
      !view_ok(q, B, H, T, d) || !view_ok(o, B, H, T, d) || !lse || (reinterpret_cast<uintptr_t>(lse) & 3u) ||
      (reinterpret_cast<uintptr_t>(tree) & 7u))
    return FA_ERR_INVALID_ARG;
  const CachedSplit s = cached_split(H / Hkv, T);
  const CachedLayoutBytes l = cached_layout(B, Hkv, d, s);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < l.bytes)
    return FA_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  fa::CachedParams p{};
  p.table = page_table;
  p.ctx_len = ctx_len;
  p.tree = reinterpret_cast<const unsigned long long*>(tree);
  p.seg = reinterpret_cast<int*>(ws + l.seg_off);
  p.part_ml = reinterpret_cast<float2*>(ws + l.ml_off);
  p.part_o = reinterpret_cast<float*>(ws + l.o_off);
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.T = T;
  p.GT = s.GT;
  p.RT = s.RT;
  p.R = s.R;
  p.page = page_size;
  p.width = table_width;
  p.num_pages = num_pages;
  p.window = window;
  p.sinks = sinks;
  p.mode = softmax_mode;
  p.beta = beta;
  fa::JoinParams j{};
  j.o = static_cast<__nv_bfloat16*>(o->ptr);
  j.lse = lse;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (d == 64) return run_cached<64>(q, k_pages, v_pages, o, p, j, s, cs);
  return run_cached<128>(q, k_pages, v_pages, o, p, j, s, cs);
}

fa_status fa_cache_append(const fa_view* k, const fa_view* v, void* k_pages, void* v_pages, const int32_t* page_table,
                          const int32_t* ctx_len, const int32_t* count, int B, int Hkv, int T, int d, int num_pages,
                          int page_size, int table_width, void* stream) {
  if (!shape_ok(B, Hkv, T, d)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * Hkv * T == 0) return FA_OK;
  if (static_cast<long long>(T) * Hkv * (d / 8) >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  if (!pool_ok(k_pages, v_pages, page_table, ctx_len, Hkv, d, num_pages, page_size, table_width) ||
      !view_ok(k, B, Hkv, T, d) || !view_ok(v, B, Hkv, T, d) || (reinterpret_cast<uintptr_t>(count) & 3u))
    return FA_ERR_INVALID_ARG;
  const fa::CachePool pool = cache_pool(k_pages, v_pages, page_table, ctx_len, Hkv, num_pages, page_size, table_width);
  // blocks: one chunk of K and V per thread until eight blocks per SM are there
  const long long work = static_cast<long long>(T) * Hkv * (d / 8);
  const int gy = B < 65535 ? B : 65535;
  const long long most = (8ll * (sm_count() > 0 ? sm_count() : 148) + gy - 1) / gy;
  long long gx = (work + 255) / 256;
  if (gx > most) gx = most;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const __nv_bfloat16* pk = static_cast<const __nv_bfloat16*>(k->ptr);
  const __nv_bfloat16* pv = static_cast<const __nv_bfloat16*>(v->ptr);
  cudaError_t e = d == 64 ? launch_pdl(fa::fa_cache_append_kernel<64>, grid, dim3(256), 0, s, pk, pv, strides_of(k),
                                       strides_of(v), count, pool, B, T)
                          : launch_pdl(fa::fa_cache_append_kernel<128>, grid, dim3(256), 0, s, pk, pv, strides_of(k),
                                       strides_of(v), count, pool, B, T);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : cuda_fail("fa_cache_append launch", e);
}

fa_status fa_cache_compact(void* k_pages, void* v_pages, const int32_t* page_table, const int32_t* ctx_len,
                           const int32_t* src, const int32_t* count, int B, int Hkv, int M, int d, int num_pages,
                           int page_size, int table_width, void* stream) {
  if (!shape_ok(B, Hkv, M, d)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * Hkv * M == 0) return FA_OK;
  if (M > 64) return FA_ERR_UNSUPPORTED;
  if (!pool_ok(k_pages, v_pages, page_table, ctx_len, Hkv, d, num_pages, page_size, table_width) || !src || !count ||
      ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(count)) & 3u))
    return FA_ERR_INVALID_ARG;
  const fa::CachePool pool = cache_pool(k_pages, v_pages, page_table, ctx_len, Hkv, num_pages, page_size, table_width);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(grid_for(static_cast<long long>(B) * Hkv, 1));
  cudaError_t e = d == 64 ? launch_pdl(fa::fa_cache_compact_kernel<64>, grid, dim3(256), 0, s, src, count, pool, B, M)
                          : launch_pdl(fa::fa_cache_compact_kernel<128>, grid, dim3(256), 0, s, src, count, pool, B, M);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : cuda_fail("fa_cache_compact launch", e);
}

}  // extern "C"
