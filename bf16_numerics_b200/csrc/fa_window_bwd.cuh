// Delta preprocess and dQ convert of the windowed backward, for arrays given
// by strides (the main kernels are the WIN forms of fa_bwd_pipe.cuh and
// fa_bwd_pipe128.cuh).  Both are bound by memory traffic, like the contiguous
// forms in fa_bwd.cuh; the differences are the addressing (work comes in
// groups of rows of one head, so that the two divisions of a group's index are
// shared by its rows) and what the clear covers.
#pragma once

#include "fa_bwd.cuh"

namespace fa {

// delta[(b*H + h)*N + n] = sum_c dO * O in fp32, and `clear4` float4 starting at
// `clear` (the dQ accumulator and what follows it) zeroed: see
// fa_bwd_delta_kernel for why that comes last and why dependents launch only
// after the wait.
template <int D>
__global__ void __launch_bounds__(128, 16)
fa_window_delta_kernel(const __nv_bfloat16* __restrict__ o, const __nv_bfloat16* __restrict__ dO, ViewStrides so,
                       ViewStrides sdo, float* __restrict__ delta, float4* __restrict__ clear, long long clear4, int H,
                       int N, long long groups, int groups_per_head) {
  constexpr int LPR = D / 8;     // lanes per row (8 elements per lane)
  constexpr int RPW = 32 / LPR;  // rows per warp per pass
  constexpr int U = 2;           // passes per group: RPW * U rows, all loads before any use
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, li = lane % LPR;
  grid_dependency_wait();  // O comes from the forward grid
  grid_launch_dependents();
  const long long warp_global = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const long long n_warps = (static_cast<long long>(gridDim.x) * blockDim.x) >> 5;
  for (long long g = warp_global; g < groups; g += n_warps) {
    const long long bh = g / groups_per_head;
    const int n0 = static_cast<int>(g - bh * groups_per_head) * (RPW * U);
    const long long b = bh / H;
    const int h = static_cast<int>(bh - b * H);
    const __nv_bfloat16* po = o + b * so.b + h * so.h + 8 * li;
    const __nv_bfloat16* pd = dO + b * sdo.b + h * sdo.h + 8 * li;
    ORaw<__nv_bfloat16> a[U];
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long n = n0 + u * RPW + sub;
      if (n < N) {
        a[u].load(po + n * so.n);
        v[u] = __ldg(reinterpret_cast<const uint4*>(pd + n * sdo.n));
      } else {
        a[u].zero();
        v[u] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float acc = a[u].dot(v[u], 0.f);
#pragma unroll
      for (int off = LPR / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
      const long long n = n0 + u * RPW + sub;
      if (n < N && li == 0) delta[bh * N + n] = acc;
    }
  }
  const long long lo = clear4 * blockIdx.x / gridDim.x, hi = clear4 * (blockIdx.x + 1) / gridDim.x;
  for (long long i = lo + threadIdx.x; i < hi; i += blockDim.x) clear[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// dq = bf16(dq_acc), and dk, dv of the key blocks that were worked on in pieces
// = bf16(sum of the pieces, in order).  Tiles of 8192 elements of one head (256
// threads, four chunks of 8 elements each, loads first): the dq tiles, then two
// sets (dV, dK) of 128 * D / 8192 tiles per key block in pieces.
struct ConvertParams {
  const float* dq_acc;
  const float* kv_part;
  __nv_bfloat16 *dq, *dk, *dv;
  ViewStrides sdq, sdk, sdv;
  int H, Hkv, BHk, N;
  long long dq_tiles, tiles;
  int dq_tiles_per_head;
  int first_blk, n_blk_pieces;  // the key blocks in pieces: [first_blk, first_blk + n_blk_pieces)
  WindowPieces pieces;
};
template <int D>
__global__ void __launch_bounds__(256)
fa_window_convert_kernel(const ConvertParams p) {
  constexpr int U = 4, CPR = D / 8;    // chunks per row
  constexpr int ROWS = 256 * U / CPR;  // rows per tile
  constexpr int TPB = 128 / ROWS;      // tiles per key block
  grid_dependency_wait();  // the accumulator and the pieces are complete once the main grid is
  for (long long tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
    const float4* src;     // row n0 of what is converted
    __nv_bfloat16* dst;    // the same row of the output
    long long dst_n;       // its row stride
    int n0, parts = 1;
    if (tile < p.dq_tiles) {
      const long long bh = tile / p.dq_tiles_per_head, b = bh / p.H;
      n0 = static_cast<int>(tile - bh * p.dq_tiles_per_head) * ROWS;
      src = reinterpret_cast<const float4*>(p.dq_acc + (bh * p.N + n0) * D);
      dst = p.dq + b * p.sdq.b + (bh - b * p.H) * p.sdq.h;
      dst_n = p.sdq.n;
    } else {
      long long x = tile - p.dq_tiles;
      const int sub = static_cast<int>(x % TPB);
      x /= TPB;
      const int which = static_cast<int>(x & 1);  // 0: dV, 1: dK
      x >>= 1;
      const int bh = static_cast<int>(x / p.n_blk_pieces), kb = p.first_blk + static_cast<int>(x % p.n_blk_pieces);
      const int b = bh / p.Hkv;
      const ViewStrides& st = which == 0 ? p.sdv : p.sdk;
      n0 = kb * 128 + sub * ROWS;
      parts = p.pieces.of(kb);
      src = reinterpret_cast<const float4*>(
          p.kv_part + ((p.pieces.place(bh, p.BHk, kb, 0) * 2 + which) * 128 + sub * ROWS) * D);
      dst = (which == 0 ? p.dv : p.dk) + b * st.b + (bh - b * p.Hkv) * st.h;
      dst_n = st.n;
    }
    float4 x[U], y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = threadIdx.x + 256 * u;
      if (n0 + i / CPR < p.N) {
        x[u] = __ldcs(src + 2 * i);
        y[u] = __ldcs(src + 2 * i + 1);
      }
    }
    for (int k = 1; k < parts; ++k) {
      src += 2 * 128 * D / 4;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = threadIdx.x + 256 * u;
        if (n0 + i / CPR < p.N) {
          const float4 a = __ldcs(src + 2 * i), c = __ldcs(src + 2 * i + 1);
          x[u].x += a.x; x[u].y += a.y; x[u].z += a.z; x[u].w += a.w;
          y[u].x += c.x; y[u].y += c.y; y[u].z += c.z; y[u].w += c.w;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = threadIdx.x + 256 * u;
      const long long n = n0 + i / CPR;
      if (n < p.N) {
        uint4 w;
        w.x = pack_bf16x2(x[u].x, x[u].y);
        w.y = pack_bf16x2(x[u].z, x[u].w);
        w.z = pack_bf16x2(y[u].x, y[u].y);
        w.w = pack_bf16x2(y[u].z, y[u].w);
        *reinterpret_cast<uint4*>(dst + n * dst_n + 8 * (i % CPR)) = w;
      }
    }
  }
  grid_launch_dependents();
}

}  // namespace fa
