"""Workspace queries: a workspace for T tokens serves every smaller batch too, so that a caller can keep one for the
largest."""
import ctypes

import pytest
import torch

from test_run_refusals import api  # noqa: F401 (fixture)

FMTS = range(5)
TOKENS = sorted({t + d for k in range(0, 4400, 48) for t in (k,) for d in (0, 1, 17)} |
                {1 << k for k in range(13, 20)} | {(1 << k) + 5 for k in range(13, 20)})


def sizes(fn, *args):
    n = ctypes.c_size_t()
    out = []
    for T in TOKENS:
        rc = fn(*[T if a == "T" else a for a in args], ctypes.byref(n))
        if rc == -4:  # more than a launch takes
            break
        assert rc == 0
        out.append(n.value)
    assert len(out) > 250
    return out


def never_falls(s):
    return all(a <= b for a, b in zip(s, s[1:]))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("inter,hidden", [(17408, 5120), (5632, 2048), (777, 512), (70, 256)])
@pytest.mark.parametrize("dtype", [0, 1])
def test_glu_sizes_never_fall(api, fmt, inter, hidden, dtype):  # noqa: F811
    L = api.lib()
    assert never_falls(sizes(L.iq_glu_workspace_size, fmt, inter, hidden, dtype, "T"))
    assert never_falls(sizes(L.iq_glu_backward_workspace_size, fmt, inter, hidden, dtype, "T"))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,cols", [(5120, 17408), (2048, 5632), (333, 768), (70, 256)])
@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("N,rank", [(0, 0), (1, 16), (4, 33)])
def test_linear_backward_sizes_never_fall(api, fmt, rows, cols, dtype, N, rank):  # noqa: F811
    assert never_falls(sizes(api.lib().iq_linear_backward_workspace_size, fmt, rows, cols, dtype, "T", N, rank))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [0, 1])
def test_sizes_of_running_never_fall(api, fmt, dtype):  # noqa: F811
    L = api.lib()
    for rows, cols in ((17408, 5120), (333, 768)):
        for rank in (0, 16, 100):
            assert never_falls(sizes(L.iq_linear_workspace_size, fmt, rows, cols, dtype, "T", rank))
    for E, k in ((8, 2), (128, 8)):
        assert never_falls(sizes(L.iq_moe_workspace_size, fmt, fmt, 2048, 768, E, dtype, "T", k))


def test_small_batches_need_little(api):  # noqa: F811
    """What is kept for sums of split rows goes with the batch, too: a token's backward pass takes no share of a large
    one's."""
    for f in FMTS:
        assert api.glu_backward_workspace_size(f, 17408, 5120, torch.bfloat16, 1) < 8 << 20
