"""The statistics that window_attention_forward allocates (GPU)."""

import pytest
import torch

import bf16_numerics_b200 as fa

pytestmark = pytest.mark.gpu


def test_the_shift_is_kept_without_the_other_statistics(cuda_device):
    """A training step keeps lse and m for its backward: neither keeps the memory of rm, rs and pbar_max."""
    q, k, v = (torch.randn(2, 3, 500, 64, device="cuda").to(torch.bfloat16) for _ in range(3))
    _, lse, st = fa.window_attention_forward(q, k, v, 100, 4)
    rows = 2 * 3 * 500 * 4
    for t in (lse, st.m):
        assert t.untyped_storage().nbytes() == rows
    want = fa.RowStats.empty(2, 3, 500, "cuda")
    o, again = torch.empty_like(q), torch.empty_like(lse)
    fa.fa_window_fwd(q, k, v, o, again, want, 100, 4)
    assert torch.equal(lse, again)
    for name in ("rm", "rs", "m", "pbar_max"):
        assert torch.equal(getattr(st, name), getattr(want, name)) and getattr(st, name).dtype == getattr(want, name).dtype
