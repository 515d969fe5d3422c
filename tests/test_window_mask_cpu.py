"""The masks of fa_window.cuh compiled for the host (no GPU): every bit against the definition in 64 bits, with windows, sinks,
lengths and slots up to 2^31 - 1, in a program that stops at the first signed overflow or shift out of range."""

import os
import subprocess

import pytest

from bf16_numerics_b200.build import CSRC

HARNESS = r"""
#define __device__
#define __host__
#define __forceinline__ inline
#include "fa_window.cuh"
#include <cstdio>
#include <initializer_list>
using ll = long long;
constexpr int kTop = 2147483647;

static int fail(const char* what, ll a, ll b, ll c, ll d, ll e) {
  std::printf("%s: %lld %lld %lld %lld %lld\n", what, a, b, c, d, e);
  return 1;
}

// a token that sees n new tokens over ctx context slots, slots [key0, key0 + cols)
static int cached(int ctx, int n, int window, int sinks, int key0, int cols) {
  const int first = fa::window_first(ctx, n, window);
  const fa::RowMask m = fa::context_mask(ctx, first, sinks, key0);
  bool hidden = false;
  for (int w = 0; w < cols; w += 32) {
    const uint32_t word = m.word(w);
    for (int c = 0; c < 32; ++c) {
      const ll slot = ll(key0) + w + c, pos = ll(ctx) + n - 1;
      const bool sees = slot < ctx && (pos - slot < window || slot < sinks);
      hidden = hidden || !sees;
      if (((word >> c) & 1u) != (sees ? 1u : 0u)) return fail("cached", ctx, n, window, sinks, slot);
    }
  }
  if (hidden && !fa::context_hides(ctx, first, sinks, key0, cols)) return fail("hides", ctx, n, window, sinks, key0);
  return 0;
}

static int windowed(int N, int window, int sinks) {
  fa::WindowShape s{};
  s.H = s.G = 1;
  s.window = window < N ? window : N;
  s.sinks = sinks < N ? sinks : N;
  s.n_sink_blk = (s.sinks + 127) / 128;
  const int blocks = (N + 127) / 128;
  for (int qb = 0; qb < blocks; ++qb)
    for (int kb = 0; kb <= qb; ++kb) {
      bool any = false, all = true;
      for (int r = 0; r < 128; ++r) {
        const int q = qb * 128 + r;
        const fa::RowMask row = s.row_mask(q, kb * 128, N);
        bool hidden = false;
        for (int c = 0; c < 128; ++c) {
          const int k = kb * 128 + c, like = q < N ? q : N - 1;
          const bool sees = k <= like && (ll(like) - k < window || k < sinks);
          hidden = hidden || !sees;
          if (((row.word(c & ~31) >> (c & 31)) & 1u) != (sees ? 1u : 0u)) return fail("row", N, window, sinks, q, k);
          const fa::RowMask col = s.column_mask(k, qb * 128);
          const bool real = k <= q && (ll(q) - k < s.window || k < s.sinks);
          if (((col.word(r & ~31) >> (r & 31)) & 1u) != (real ? 1u : 0u)) return fail("column", N, window, sinks, q, k);
          if (q < N && k < N) any = any || sees, all = all && sees;
        }
        if (hidden && !row.hides(128)) return fail("row hides", N, window, sinks, q, kb);
      }
      if (s.block_full(qb, kb) && !all) return fail("full", N, window, sinks, qb, kb);
      if (any && kb < s.first_block(qb) && kb >= s.n_sink_blk) return fail("first", N, window, sinks, qb, kb);
      if (any && qb > s.last_query_block(kb, blocks)) return fail("last", N, window, sinks, qb, kb);
    }
  return 0;
}

int main() {
  for (int window : {1, 2, 5, 64, 127, 128, 129, 1000, 32768, kTop - 1, kTop})
    for (int sinks : {0, 1, 4, 127, 128, 130, 5000, kTop - 1, kTop})
      for (int ctx : {0, 1, 31, 127, 128, 129, 1000, 40000, kTop / 2, kTop - 300, kTop - 64, kTop - 1})
        for (int n : {1, 2, 13, 63, 64}) {
          if (ll(ctx) + n > kTop) continue;
          const ll last = (ll(ctx) + 63) / 128;  // no slot is at 2^31 - 1 or beyond
          for (ll tile : {0ll, 1ll, last - 1, last, (ll(ctx) - window) / 128, (ll(ctx) - window) / 128 + 1, ll(sinks) / 128})
            for (int cols : {32, 64})
              for (int col = 0; col < 128; col += cols)
                if (tile >= 0 && tile <= last && tile * 128 + 127 <= kTop && cached(ctx, n, window, sinks, int(tile * 128 + col), cols))
                  return 1;
        }
  for (int N : {1, 2, 127, 128, 129, 300, 700})
    for (int window : {1, 2, 64, 127, 128, 129, 255, 257, 700, kTop})
      for (int sinks : {0, 1, 4, 128, 129, 300, kTop})
        if (windowed(N, window, sinks)) return 1;
  return 0;
}
"""


def _compile(tmp_path, text):
    source, out = tmp_path / "mask.cpp", tmp_path / "mask"
    source.write_text(text)
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-fsanitize=signed-integer-overflow,shift",
                    "-fsanitize-undefined-trap-on-error", f"-I{CSRC}", "-x", "c++", str(source), "-o", str(out)], check=True)
    return out


def test_every_bit_of_the_masks(tmp_path):
    run = subprocess.run([str(_compile(tmp_path, HARNESS))], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stdout or f"stopped with {run.returncode}: a signed overflow or a shift out of range"


def test_an_overflow_stops_the_program(tmp_path):
    """The window's first slot without its bound at 0: the difference to a slot behind the context overflows."""
    text = HARNESS.replace("fa::window_first(ctx, n, window)", "ctx + n - window")
    assert text != HARNESS
    assert subprocess.run([str(_compile(tmp_path, text))], capture_output=True, timeout=300).returncode < 0
