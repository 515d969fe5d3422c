"""No kernel writes global memory before its dependency wait (read from the sources, no GPU).

Every launch may start while the grids before it in the stream still work (programmatic dependent launch), and any
memory of an earlier call may be handed to a later one: as a shared scratch tensor, or by a stream-ordered allocator
that got the block back when the earlier call returned.  So nothing may be stored ahead of griddepcontrol.wait.
"""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bf16_numerics_b200", "csrc")
WAIT = "grid_dependency_wait();"


def _without_comments(text):
    return re.sub(r"//[^\n]*", "", text)


def _matching(text, at, pair):
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == pair[0]) - (text[i] == pair[1])
        if depth == 0:
            return i
    raise AssertionError("unbalanced source")


def kernels(text):
    """(name, parameter list, body) of every __global__ function."""
    text = _without_comments(text)
    for m in re.finditer(r"__global__", text):
        head = re.compile(r"(\w+_kernel)\s*\(").search(text, m.end())
        close = _matching(text, head.end() - 1, "()")
        begin = text.index("{", close)
        yield head.group(1), text[head.end():close], text[begin:_matching(text, begin, "{}") + 1]


def global_writes(params, code):
    """Stores through a pointer parameter, a pointer made from one or a member of a parameter struct; bulk stores, reductions
    and atomics."""
    names = set(re.findall(r"\*\s*(?:__restrict__\s*)?(\w+)\s*(?:,|$)", params))
    structs = set(re.findall(r"(?:Params|Args<\w+>|Pool)\s+(\w+)", params))
    source = lambda text: any(re.search(rf"\b{n}\b", text) for n in names | structs)
    for alias, value in re.findall(r"\*\s*(?:const\s+)?(\w+)\s*=\s*([^;]+);", code):
        if source(value):
            names.add(alias)
    found = []
    for line in code.split(";"):
        if re.search(r"tma_store|tma_reduce|atomic(Add|Exch|Max|CAS)|report_page|__stcs|__stcg", line):
            found.append(line.strip())
        for target in re.findall(r"([^=;{}]*[\w\])])\s*[+|]?=(?!=)", line):
            target = target.split(")", 1)[1] if target.count(")") > target.count("(") else target  # behind a loop's head
            if re.search(r"\]\s*$", target) and source(target.rsplit("[", 1)[0]) or \
                    re.search(r"^\s*\*", target) and source(target):
                found.append(line.strip())
    return found


SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cuh", ".cu")))


def test_the_reader_sees_the_kernels_and_their_stores():
    seen = {name for f in SOURCES for name, _, _ in kernels(open(os.path.join(CSRC, f)).read())}
    assert {"fa_bwd_delta_kernel", "fa_window_delta_kernel", "fa_cached_kernel", "fa_cached_join_kernel",
            "fa_cache_append_kernel", "fa_fwd_kernel", "fa_fwd_split_kernel", "fa_bwd_main_pipe128_kernel"} <= seen
    early = """__global__ void early_kernel(const float* x, float* __restrict__ acc, const CachePool c) {
      float4* acc4 = reinterpret_cast<float4*>(acc);
      float a[4];
      a[0] = x[0];
      if (x) for (int i = 0; i < 4; ++i) acc4[i] = zero;
      reinterpret_cast<int*>(acc + 4)[threadIdx.x] = 0;
      c.k[3] = a[0];
      grid_dependency_wait();
      acc[9] = 1.f; }"""
    (name, params, body), = kernels(early)
    assert name == "early_kernel" and len(global_writes(params, body.split(WAIT)[0])) == 3
    assert len(global_writes(params, body)) == 4


@pytest.mark.parametrize("source", SOURCES)
def test_nothing_is_written_before_the_wait(source):
    for name, params, body in kernels(open(os.path.join(CSRC, source)).read()):
        assert WAIT in body, f"{name} never waits for the grids before it"
        early = body.split(WAIT)[0]
        if name == "fa_bwd_main_pipe_kernel":
            # its loads run ahead: the delta kernel lets it start only when every earlier grid has completed, and what
            # it writes depends on vectors that its drain warps publish after their wait
            early = early.split("grid_launch_dependents();")[0]
        assert not global_writes(params, early), f"{name}: {global_writes(params, early)}"


@pytest.mark.parametrize("source,kernel", [("fa_bwd.cuh", "fa_bwd_delta_kernel"), ("fa_window_bwd.cuh", "fa_window_delta_kernel")])
def test_the_delta_kernels_let_dependents_start_after_their_wait(source, kernel):
    """What the d = 64 main kernel's early loads rest on."""
    body = {n: b for n, _, b in kernels(open(os.path.join(CSRC, source)).read())}[kernel]
    assert body.index(WAIT) < body.index("grid_launch_dependents();")
