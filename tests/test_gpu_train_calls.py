"""Calls of include/iq_train.h that a training loop makes in passing: one workspace for batches of all sizes, weights
with a scale that is not finite, infinite gradients."""
import numpy as np
import pytest

from ggml_iq_codebook_imatrix_amd import inputs
from test_gpu_run import FORMATS, decoded, dev, f64, payload
from test_gpu_train import DTYPES, tokens, upstream

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from ggml_iq_codebook_imatrix_amd import api as a
    a.lib()
    return a


@pytest.mark.parametrize("dtype", DTYPES)
def test_one_workspace_serves_smaller_batches(api, dtype):
    """The largest batch's workspace, with what the call before left in it, for ragged batches that split their sums."""
    print("[case] one workspace", dtype, flush=True)
    fmt, inter, nb, most, N, r = "IQ1_M", 900, 4, 1300, 2, 8
    g = inputs.rng(3)
    grid = dev(inputs.grid_for(fmt, 5))
    gate, up, down = (dev(payload(fmt, inter, nb, k)) for k in (6, 7, 8))
    a = dev(g.standard_normal((N, r, nb * 256), dtype=np.float32) * 0.05, dtype)
    b = dev(g.standard_normal((N, inter, r), dtype=np.float32) * 0.05, dtype)
    x, dh = tokens(most, nb, 1, dtype), upstream(most, inter, 2, dtype)
    ids = dev(g.integers(-1, N, most).astype(np.int32))
    n = max(api.glu_backward_workspace_size(fmt, inter, nb * 256, dtype, most),
            api.linear_backward_workspace_size(fmt, inter, nb * 256, dtype, most, N, r),
            api.glu_workspace_size(fmt, inter, nb * 256, dtype, most))
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN, whatever it is read as
    for T in (1300, 1, 7, 129, 250, 33, 700, 1024, 1041, 16):
        xs, d, i = x[:T].contiguous(), dh[:T].contiguous(), ids[:T].contiguous()
        lora = dict(x=xs, lora_a=a, lora_b=b, lora_ids=i)
        assert torch.equal(api.glu(fmt, gate, up, grid, xs, workspace=ws), api.glu(fmt, gate, up, grid, xs))
        assert torch.equal(api.glu_backward(fmt, gate, up, grid, xs, d, workspace=ws),
                           api.glu_backward(fmt, gate, up, grid, xs, d))
        for m, w in zip(api.linear_backward(fmt, down, grid, d, workspace=ws, **lora),
                        api.linear_backward(fmt, down, grid, d, **lora)):
            assert torch.equal(m, w) and bool(m.isfinite().all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FORMATS)
def test_an_infinite_scale_stays_infinite(api, orc, fmt, dtype):
    """An infinite block scale in the last row, which ends inside a chunk: its columns of dx become infinities of the
    weights' signs, the others keep their values."""
    print("[case] infinite scale", fmt, dtype, flush=True)
    rows, nb, T = 70, 3, 9
    grid, g = inputs.grid_for(fmt, 5), inputs.rng(4)
    d16 = np.full((rows, nb), 0x2000, np.uint16)
    clean = payload(fmt, rows, nb, 6, d16=d16)
    d16[-1, 1] = 0x7c00
    wild = payload(fmt, rows, nb, 6, d16=d16)
    dy = g.integers(-3, 4, (T, rows)).astype(np.float32)
    dy[:, -1] = 1 + np.arange(T) % 2
    want = f64(api.linear_backward(fmt, dev(clean), dev(grid), dev(dy, dtype)))
    got = f64(api.linear_backward(fmt, dev(wild), dev(grid), dev(dy, dtype)))
    sign = np.sign(decoded(orc, fmt, clean, grid)[-1, 256:512])
    assert np.array_equal(got[:, :256], want[:, :256]) and np.array_equal(got[:, 512:], want[:, 512:])
    assert np.all(sign != 0) and np.array_equal(got[:, 256:512], np.broadcast_to(sign * np.inf, (T, 256)))


@pytest.mark.parametrize("dtype", DTYPES)
def test_an_infinite_gradient_stays_infinite(api, orc, dtype):
    print("[case] infinite gradient", dtype, flush=True)
    fmt, rows, nb, T = "IQ2_XS", 70, 3, 9
    grid, p = inputs.grid_for(fmt, 5), payload(fmt, rows, nb, 6)
    dy = upstream(T, rows, 3, dtype)
    dy[4, 20] = float("-inf")
    got = f64(api.linear_backward(fmt, dev(p), dev(grid), dy))
    w = decoded(orc, fmt, p, grid)[20]
    assert np.all(w != 0) and np.array_equal(got[4], -np.sign(w) * np.inf)
    assert np.isfinite(np.delete(got, 4, 0)).all()
