// Host side of fa_window_fwd / fa_window_bwd (included by fa_lib.cu, whose
// helpers it uses).
#pragma once

namespace {

// A bf16 array [B, H, N, d] given by element strides, last axis contiguous.
// Valid: 16-byte aligned base; along every axis of more than one entry a
// positive stride that is a multiple of 8 elements (16 bytes: TMA, vector
// accesses) and below 2^39 (2^40 bytes: TMA); no two entries share memory
// (sorted by stride, every axis steps over the whole of the smaller ones).
bool view_ok(const fa_view* v, long long B, long long H, long long N, int d) {
  if (!v || !v->ptr || !aligned16(v->ptr)) return false;
  long long st[3] = {v->stride_b, v->stride_h, v->stride_n}, ext[3] = {B, H, N};
  long long span = d;  // elements covered by the axes taken so far
  bool used[3] = {false, false, false};
  for (int k = 0; k < 3; ++k) {
    int at = -1;
    for (int a = 0; a < 3; ++a)
      if (!used[a] && ext[a] > 1 && (at < 0 || st[a] < st[at])) at = a;
    if (at < 0) break;
    used[at] = true;
    if (st[at] < span || (st[at] & 7) || st[at] >= (1ll << 39)) return false;
    const __int128 s = static_cast<__int128>(st[at]) * (ext[at] - 1) + span;
    if (s >= (static_cast<__int128>(1) << 60)) return false;
    span = static_cast<long long>(s);
  }
  return true;
}

fa::ViewStrides strides_of(const fa_view* v) { return {v->stride_b, v->stride_h, v->stride_n}; }

// -> 4-D tensor map (d, N, H, B), box 64 (d) x 128 (rows) x 1 x 1, 128B
// swizzle; rows past N read as zeros and are not written.  An axis of one
// entry may carry any stride: a valid one is put in its place.
bool make_map_view(CUtensorMap* map, const fa_view* v, long long B, long long H, long long N, int D) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(H),
                        static_cast<cuuint64_t>(B)};
  auto bytes = [&](long long s, long long extent) { return static_cast<cuuint64_t>(extent > 1 ? s : D) * 2; };
  cuuint64_t strides[3] = {bytes(v->stride_n, N), bytes(v->stride_h, H), bytes(v->stride_b, B)};
  cuuint32_t box[4] = {64, 128, 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, v->ptr, dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

fa::WindowShape window_shape(int H, int Hkv, int N, int window, int sinks) {
  fa::WindowShape w{};
  w.H = H;
  w.G = H / Hkv;
  w.window = window < N ? window : N;
  w.sinks = sinks < N ? sinks : N;
  w.n_sink_blk = static_cast<int>((static_cast<long long>(w.sinks) + 127) / 128);
  return w;
}

bool mode_ok(int mode, float beta) {
  if (mode == FA_SOFTMAX_STANDARD) return true;
  return (mode == FA_SOFTMAX_STABILIZED || mode == FA_SOFTMAX_STABILIZED_MARGIN) && std::isfinite(beta) && beta > 1.0f;
}

// sizes, mode and window; *empty: nothing to do
fa_status window_args(int B, int H, int Hkv, int N, int d, int window, int sinks, int mode, float beta, bool* empty) {
  if (!shape_ok(B, H, N, d) || Hkv < 0 || Hkv > H || window < 1 || sinks < 0 || !mode_ok(mode, beta))
    return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  *empty = static_cast<long long>(B) * H * N == 0;
  if (!*empty && (Hkv == 0 || H % Hkv != 0)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

template <int D>
fa_status launch_window_fwd(const fa_view* q, const fa_view* k, const fa_view* v, const fa_view* o, float* lse,
                            const fa_row_stats* st, int B, int H, int Hkv, int N, int window, int sinks, int mode,
                            float beta, cudaStream_t stream) {
  CUtensorMap mq, mk, mv, mo;
  if (!make_map_view(&mq, q, B, H, N, D) || !make_map_view(&mk, k, B, Hkv, N, D) ||
      !make_map_view(&mv, v, B, Hkv, N, D) || !make_map_view(&mo, o, B, H, N, D))
    return cuda_fail("cuTensorMapEncodeTiled (q/k/v/o)");
  fa::FwdWinParams p{};
  p.lse = lse;
  if (st) {
    p.st_rm = st->rm;
    p.st_rs = st->rs;
    p.st_m = st->m;
    p.st_pbar_max = st->pbar_max;
  }
  p.BH = B * H;
  p.N = N;
  p.n_qblk = (N + 127) / 128;
  p.causal = 1;
  p.mode = mode;
  p.beta = beta;
  p.scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
  p.w = window_shape(H, Hkv, N, window, sinks);
  const int n_sm = sm_count();
  if (n_sm <= 0) return cuda_fail("cudaDeviceGetAttribute(multiprocessor count)");
  static std::atomic<uint64_t> attr{0};
  cudaError_t e;
  auto grid_of = [&](int nt, int ctas_per_sm) {
    const long long items = static_cast<long long>((p.n_qblk + nt - 1) / nt) * p.BH;
    const long long slots = static_cast<long long>(n_sm) * ctas_per_sm;
    return dim3(static_cast<unsigned>(items < slots ? items : slots));
  };
  if constexpr (D == 64) {
    using L = fa::FwdSplitLayout<64, false>;
    if (!ensure_smem(fa::fa_fwd_split_kernel<64, false, true>, L::SMEM_BYTES, attr)) return FA_ERR_CUDA;
    LaunchTimer tm(FA_KERNEL_FWD, stream);
    e = launch_pdl(fa::fa_fwd_split_kernel<64, false, true>, grid_of(1, L::CTAS_PER_SM), dim3(L::THREADS),
                   L::SMEM_BYTES, stream, mq, mk, mv, mo, p);
    tm.done();
  } else {
    using L = fa::FwdLayout<128, false>;
    if (!ensure_smem(fa::fa_fwd_kernel<128, false, true>, L::SMEM_BYTES, attr)) return FA_ERR_CUDA;
    LaunchTimer tm(FA_KERNEL_FWD, stream);
    e = launch_pdl(fa::fa_fwd_kernel<128, false, true>, grid_of(L::NT, 1), dim3(L::THREADS), L::SMEM_BYTES, stream,
                   mq, mk, mv, mo, p);
    tm.done();
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : cuda_fail("fa_window_fwd launch", e);
}

int sm_count_or_default() {
  const int n = sm_count();
  return n > 0 ? n : 148;
}
// How the backward's steps (128 x 128 block products) are cut into items.  A
// sink block has up to G * n_blk steps and another up to G * (window / 128 + 2);
// long items are waited for, many short ones pay for their ends.  For a series
// of longest pieces the time of the busiest SM is estimated -- an item costs its
// steps and two more, three if its result goes to a partial's place (K and V
// loads, first products and the epilogue do not overlap); the sink pieces go
// first, round by round, and each of the others to the SM that is free first; an
// eighth of the longest item stands for the spread -- and the smallest wins.
// Measured (forward + backward, one B200, pieces of a sink and of another block):
// N 4096, 8 heads over 1, d 128, window 512, sinks 4: 945 us uncut, 127 us with
// (22, 4), 155 with (32, 5), 148 with (11, 2); N 8192, 2 x 16 heads over 4, d 128,
// window 1024: 1600 us uncut, 955 us with (2, 1), 894 with (4, 1), 962 with (8, 2).
fa::WindowPieces window_pieces(int B, int H, int Hkv, int N, int window, int sinks, int n_sm) {
  constexpr long long kUnit = 16;  // times in sixteenths of a step
  const fa::WindowShape w = window_shape(H, Hkv, N, window, sinks);
  fa::WindowPieces best{1, 1, w.n_sink_blk, (N + 127) / 128};
  const long long n_blk = best.n_blk, nsb = best.nsb, G = w.G, BHk = static_cast<long long>(B) * Hkv;
  const long long rest = n_blk - nsb;
  const long long reach = (126ll + w.window) / 128 + 1;  // query blocks that see a block away from the row's end
  const long long wide = reach < rest ? reach : rest;    // .. the last ones: wide, wide - 1, .., 1
  const long long sink_steps = (nsb * n_blk - nsb * (nsb - 1) / 2) * G * BHk;
  const long long rest_steps = ((rest - wide) * wide + wide * (wide + 1) / 2) * G * BHk;
  const long long top = nsb > 0 ? G * n_blk : G * wide;
  long long best_time = -1;
  for (long long most = 4;; most += (most + 3) / 4) {
    auto cut = [&](long long steps, long long fewest) {
      const long long k = (steps + most - 1) / most;
      return k < 1 ? 1 : (k < fewest ? k : fewest);  // no piece without a step
    };
    const long long ps = nsb > 0 ? cut(G * n_blk, G * (n_blk - nsb + 1)) : 1, pw = rest > 0 ? cut(G * wide, G) : 1;
    // items of each kind, their mean cost and the longest one's
    const long long is = nsb * ps * BHk, iw = rest * pw * BHk;
    const long long es = (ps > 1 ? 3 : 2) * kUnit, ew = (pw > 1 ? 3 : 2) * kUnit;
    const long long ms = is > 0 ? sink_steps * kUnit / is + es : 1, mw = iw > 0 ? rest_steps * kUnit / iw + ew : 1;
    const long long ls = is > 0 ? G * n_blk * kUnit / ps + es : 0, lw = iw > 0 ? G * wide * kUnit / pw + ew : 0;
    const long long rounds = is / n_sm, more = is - rounds * n_sm;  // `more` SMs take one sink piece more
    const long long free_a = (rounds + 1) * ms, free_b = rounds * ms;
    auto started = [&](long long t) {  // others that have been started at time t
      return (t >= free_a ? ((t - free_a) / mw + 1) * more : 0) + (t >= free_b ? ((t - free_b) / mw + 1) * (n_sm - more) : 0);
    };
    long long lo = 0, hi = free_a + (iw / n_sm + 1) * mw;
    while (lo < hi) {  // when the last one starts
      const long long t = lo + (hi - lo) / 2;
      if (started(t) >= iw)
        hi = t;
      else
        lo = t + 1;
    }
    const long long longest = ls > lw ? ls : lw, sinks_end = more > 0 ? free_a : free_b;
    long long time = iw > 0 ? lo + lw : 0;
    if (time < sinks_end) time = sinks_end;
    if (time < longest) time = longest;
    time += longest / 8;
    if (best_time < 0 || time <= best_time) {  // of equals the fewest pieces
      best_time = time;
      best.ps = static_cast<int>(ps);
      best.pw = static_cast<int>(pw);
    }
    if (most >= top) break;
  }
  return best;
}

// workspace: delta | fp32 dQ accumulator | work-item counter | partial dV, dK
struct WindowBwdLayout {
  size_t acc_off, ctr_off, part_off, bytes;
};
WindowBwdLayout window_bwd_layout(int B, int H, int Hkv, int N, int d, const fa::WindowPieces& pc) {
  const size_t rows = static_cast<size_t>(B) * H * N;
  WindowBwdLayout l{};
  l.acc_off = round256(rows * 4);
  l.ctr_off = l.acc_off + rows * d * 4;  // a multiple of 256 past acc_off
  l.part_off = l.ctr_off + 256;
  l.bytes = l.part_off + static_cast<size_t>(pc.places(B * Hkv)) * 2 * 128 * d * 4;
  return l;
}

template <int D>
fa_status launch_window_bwd(const fa_view* q, const fa_view* k, const fa_view* v, const fa_view* o, const fa_view* dO,
                            const float* lse, const float* row_m, const fa_view* dq, const fa_view* dk,
                            const fa_view* dv, uint8_t* ws, int B, int H, int Hkv, int N, int window, int sinks,
                            int mode, cudaStream_t stream) {
  static std::atomic<uint64_t> attr{0};
  if constexpr (D == 64) {
    if (!ensure_smem(fa::fa_bwd_main_pipe_kernel<true>, fa::BwdPipeLayout::SMEM_BYTES, attr)) return FA_ERR_CUDA;
  } else {
    if (!ensure_smem(fa::fa_bwd_main_pipe128_kernel<true>, fa::BwdPipe128Layout::SMEM_BYTES, attr)) return FA_ERR_CUDA;
  }
  const int n_sm = sm_count();
  if (n_sm <= 0) return cuda_fail("cudaDeviceGetAttribute(multiprocessor count)");
  const int BH = B * H, n_blk = (N + 127) / 128;
  const fa::WindowPieces pieces = window_pieces(B, H, Hkv, N, window, sinks, n_sm);
  const WindowBwdLayout wl = window_bwd_layout(B, H, Hkv, N, D, pieces);
  float* delta = reinterpret_cast<float*>(ws);
  float* dq_acc = reinterpret_cast<float*>(ws + wl.acc_off);
  CUtensorMap mq, mk, mv, mdo, mdq, mdk, mdv;
  if (!make_map_view(&mq, q, B, H, N, D) || !make_map_view(&mk, k, B, Hkv, N, D) ||
      !make_map_view(&mv, v, B, Hkv, N, D) || !make_map_view(&mdo, dO, B, H, N, D) ||
      !make_map_view(&mdk, dk, B, Hkv, N, D) || !make_map_view(&mdv, dv, B, Hkv, N, D))
    return cuda_fail("cuTensorMapEncodeTiled (q/k/v/dO/dk/dv)");
  if (!make_map_dq(&mdq, dq_acc, BH, N, D)) return cuda_fail("cuTensorMapEncodeTiled (dQ accumulator)");
  {
    constexpr int rows_per_group = 2 * 32 / (D / 8);
    const int per_head = (N + rows_per_group - 1) / rows_per_group;
    const long long groups = static_cast<long long>(BH) * per_head;
    const long long clear4 = static_cast<long long>(wl.part_off - wl.acc_off) / 16;
    const dim3 grid(grid_for(groups, 4));
    LaunchTimer tm(FA_KERNEL_BWD_DELTA, stream);
    cudaError_t e = launch_pdl(fa::fa_window_delta_kernel<D>, grid, dim3(128), 0, stream,
                               static_cast<const __nv_bfloat16*>(o->ptr), static_cast<const __nv_bfloat16*>(dO->ptr),
                               strides_of(o), strides_of(dO), delta, reinterpret_cast<float4*>(dq_acc), clear4, H, N,
                               groups, per_head);
    tm.done();
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail("fa_window_delta_kernel launch", e);
  }
  {
    fa::BwdWinParams p{};
    p.lse = lse;
    p.row_m = row_m;
    p.delta = delta;
    p.dq_acc = dq_acc;
    p.item_ctr = reinterpret_cast<unsigned int*>(ws + wl.ctr_off);
    p.dk = static_cast<__nv_bfloat16*>(dk->ptr);
    p.dv = static_cast<__nv_bfloat16*>(dv->ptr);
    p.BH = B * Hkv;
    p.N = N;
    p.n_blk = n_blk;
    p.causal = 1;
    p.mode = mode;
    p.scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
    p.w = window_shape(H, Hkv, N, window, sinks);
    p.dk_strides = strides_of(dk);
    p.dv_strides = strides_of(dv);
    p.ps = pieces.ps;
    p.pw = pieces.pw;
    p.kv_part = reinterpret_cast<float*>(ws + wl.part_off);
    // d = 128 item order: key heads in groups whose fp32 dQ rows fit in 32 MB (see launch_bwd)
    const long long per_head = static_cast<long long>(N) * D * 4 * p.w.G;
    long long hg = (32ll << 20) / per_head;
    hg = hg < 1 ? 1 : (hg > p.BH ? p.BH : hg);
    p.head_group = static_cast<int>(hg);
    const long long items =
        (static_cast<long long>(p.w.n_sink_blk) * p.ps + static_cast<long long>(n_blk - p.w.n_sink_blk) * p.pw) * p.BH;
    const dim3 grid(static_cast<unsigned>(items < n_sm ? items : n_sm));
    LaunchTimer tm(FA_KERNEL_BWD_MAIN, stream);
    cudaError_t e;
    if constexpr (D == 64) {
      using L = fa::BwdPipeLayout;
      e = launch_pdl(fa::fa_bwd_main_pipe_kernel<true>, grid, dim3(L::THREADS), L::SMEM_BYTES, stream, mq, mk, mv, mdo,
                     mdq, mdk, mdv, p);
    } else {
      using L = fa::BwdPipe128Layout;
      e = launch_pdl(fa::fa_bwd_main_pipe128_kernel<true>, grid, dim3(L::THREADS), L::SMEM_BYTES, stream, mq, mk, mv,
                     mdo, mdq, p);
    }
    tm.done();
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail("fa_window_bwd main kernel launch", e);
  }
  {
    constexpr int rows_per_tile = 8192 / D;
    fa::ConvertParams p{};
    p.dq_acc = dq_acc;
    p.kv_part = reinterpret_cast<const float*>(ws + wl.part_off);
    p.dq = static_cast<__nv_bfloat16*>(dq->ptr);
    p.dk = static_cast<__nv_bfloat16*>(dk->ptr);
    p.dv = static_cast<__nv_bfloat16*>(dv->ptr);
    p.sdq = strides_of(dq);
    p.sdk = strides_of(dk);
    p.sdv = strides_of(dv);
    p.H = H;
    p.Hkv = Hkv;
    p.BHk = B * Hkv;
    p.N = N;
    p.dq_tiles_per_head = (N + rows_per_tile - 1) / rows_per_tile;
    p.dq_tiles = static_cast<long long>(BH) * p.dq_tiles_per_head;
    p.pieces = pieces;
    p.first_blk = pieces.ps > 1 ? 0 : pieces.nsb;
    p.n_blk_pieces = (pieces.pw > 1 ? n_blk : pieces.nsb) - p.first_blk;
    p.tiles = p.dq_tiles + static_cast<long long>(p.BHk) * p.n_blk_pieces * 2 * (128 / rows_per_tile);
    LaunchTimer tm(FA_KERNEL_BWD_DQ, stream);
    cudaError_t e = launch_pdl(fa::fa_window_convert_kernel<D>, dim3(grid_for(p.tiles, 1)), dim3(256), 0, stream, p);
    tm.done();
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail("fa_window_convert_kernel launch", e);
  }
  return FA_OK;
}

}  // namespace

extern "C" {

fa_status fa_window_fwd(const fa_view* q, const fa_view* k, const fa_view* v, const fa_view* o, float* lse,
                        const fa_row_stats* stats, int B, int H, int Hkv, int N, int d, int window, int sinks,
                        int softmax_mode, float beta, void* stream) {
  bool empty = false;
  const fa_status st = window_args(B, H, Hkv, N, d, window, sinks, softmax_mode, beta, &empty);
  if (st != FA_OK || empty) return st;
  if (!view_ok(q, B, H, N, d) || !view_ok(k, B, Hkv, N, d) || !view_ok(v, B, Hkv, N, d) || !view_ok(o, B, H, N, d) ||
      !lse || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return FA_ERR_INVALID_ARG;
  if (stats) {
    const void* ptrs[4] = {stats->rm, stats->rs, stats->m, stats->pbar_max};
    for (const void* sp : ptrs)
      if (sp && (reinterpret_cast<uintptr_t>(sp) & 3u)) return FA_ERR_INVALID_ARG;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 64)
    return launch_window_fwd<64>(q, k, v, o, lse, stats, B, H, Hkv, N, window, sinks, softmax_mode, beta, s);
  return launch_window_fwd<128>(q, k, v, o, lse, stats, B, H, Hkv, N, window, sinks, softmax_mode, beta, s);
}

size_t fa_window_bwd_workspace_bytes(int B, int H, int Hkv, int N, int d, int window, int sinks) {
  bool empty = false;
  if (window_args(B, H, Hkv, N, d, window, sinks, FA_SOFTMAX_STANDARD, 0.f, &empty) != FA_OK) return 0;
  if (empty) return 256;
  return window_bwd_layout(B, H, Hkv, N, d, window_pieces(B, H, Hkv, N, window, sinks, sm_count_or_default())).bytes;
}

fa_status fa_window_bwd(const fa_view* q, const fa_view* k, const fa_view* v, const fa_view* o, const fa_view* dO,
                        const float* lse, const float* row_m, const fa_view* dq, const fa_view* dk, const fa_view* dv,
                        void* workspace, size_t workspace_bytes, int B, int H, int Hkv, int N, int d, int window,
                        int sinks, int softmax_mode, float beta, void* stream) {
  bool empty = false;
  const fa_status st = window_args(B, H, Hkv, N, d, window, sinks, softmax_mode, beta, &empty);
  if (st != FA_OK || empty) return st;
  for (const fa_view* x : {q, o, dO, dq})
    if (!view_ok(x, B, H, N, d)) return FA_ERR_INVALID_ARG;
  for (const fa_view* x : {k, v, dk, dv})
    if (!view_ok(x, B, Hkv, N, d)) return FA_ERR_INVALID_ARG;
  if (!lse || (reinterpret_cast<uintptr_t>(lse) & 3u) || (reinterpret_cast<uintptr_t>(row_m) & 3u) ||
      (softmax_mode != FA_SOFTMAX_STANDARD && !row_m))
    return FA_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      workspace_bytes < fa_window_bwd_workspace_bytes(B, H, Hkv, N, d, window, sinks))
    return FA_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int mode = softmax_mode == FA_SOFTMAX_STANDARD ? 0 : 1;  // as in fa_bwd
  if (d == 64)
    return launch_window_bwd<64>(q, k, v, o, dO, lse, row_m, dq, dk, dv, ws, B, H, Hkv, N, window, sinks, mode, s);
  return launch_window_bwd<128>(q, k, v, o, dO, lse, row_m, dq, dk, dv, ws, B, H, Hkv, N, window, sinks, mode, s);
}

}  // extern "C"
