"""Arguments that are no tensors, with and without a stream (no GPU): TypeError from every windowed and cached call."""

from types import SimpleNamespace

import pytest
import torch

import bf16_numerics_b200 as fa
from bf16_numerics_b200.build import build_library


@pytest.fixture(scope="module", autouse=True)
def built():
    build_library()


CALLS = [(fa.window_attention_forward, 3), (fa.window_attention_backward, 7), (fa.fa_window_fwd, 5), (fa.fa_window_bwd, 11),
         (fa.cached_attention, 5), (fa.fa_cached_fwd, 9), (fa.fa_cache_append, 6), (fa.fa_cache_compact, 6)]


@pytest.mark.parametrize("call,arguments", CALLS, ids=[c.__name__ for c, _ in CALLS])
@pytest.mark.parametrize("first", [None, "x", 3, [1.0]])
def test_the_first_argument_is_a_tensor(call, arguments, first):
    rest = [torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)] * (arguments - 1)
    stream = SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=0)
    for kw in ({}, {"stream": stream}):
        with pytest.raises(TypeError, match="must be a torch.Tensor"):
            call(first, *rest, **kw)


@pytest.mark.parametrize("call,arguments", CALLS, ids=[c.__name__ for c, _ in CALLS])
def test_the_stream_is_on_the_tensors_device(call, arguments):
    rest = [torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)] * arguments
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        call(*rest, stream=SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0))
