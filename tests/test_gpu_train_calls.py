"""Calls of include/iq_train.h that a training loop makes in passing: one workspace for batches of all sizes."""
import numpy as np
import pytest

from ggml_iq_codebook_imatrix_amd import inputs
from test_gpu_run import dev, payload
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
