"""iq_linear and iq_moe without a GPU: the header's declarations, refusals before anything is enqueued (C ABI and
binding), workspace queries, and launch failures (every launch failed in turn against a stand-in for the runtime)."""
import ctypes
import glob
import os
import re
import subprocess

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F = ctypes.c_void_p(0x100000)  # stands for device memory; never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def api():
    from ggml_iq_codebook_imatrix_amd import api as a
    if not os.path.exists(a.LIB_PATH):
        from ggml_iq_codebook_imatrix_amd import build
        build.build()
    return a


@pytest.fixture(scope="module")
def stubbed(api, tmp_path_factory):
    objs = sorted(glob.glob(os.path.join(ROOT, "ggml_iq_codebook_imatrix_amd", "_build", "iq_*.hip.o")))
    assert objs, "build the library first"
    d = tmp_path_factory.mktemp("stub")
    so = str(d / "libiq_stubbed.so")
    subprocess.run(["gcc", "-O1", "-fPIC", "-c", os.path.join(ROOT, "tests", "hip_launch_stub.c"), "-o",
                    str(d / "stub.o")], check=True)
    subprocess.run(["gcc", "-shared", "-o", so, *objs, str(d / "stub.o"), "-L/opt/rocm/lib", "-lamdhip64",
                    "-Wl,-Bsymbolic", "-Wl,-rpath,/opt/rocm/lib"], check=True)
    L = ctypes.CDLL(so)
    for name, (args, res) in api.SIGNATURES.items():
        getattr(L, name).argtypes = args
        getattr(L, name).restype = res
    return L


def test_header_declares_the_calls(api):
    txt = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "iq_run.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(iq_\w+)\s*\(", txt, flags=re.M)))
    assert names == ["iq_linear", "iq_linear_workspace_size", "iq_moe", "iq_moe_workspace_size"]
    for n in names:
        assert n in api.SIGNATURES and hasattr(api.lib(), n)


def linear(L, fmt=1, packed=F, rows=64, cols=512, grid=F, x=F, dtype=1, T=5, a=F, b=F, scale=F, ids=F, N=2, rank=4,
           y=F, ws=F, wn=BIG, status=F):
    return L.iq_linear(fmt, packed, rows, cols, grid, x, dtype, T, a, b, scale, ids, N, rank, y, ws, wn, status, None)


def moe(L, fmt=0, down_fmt=2, gate=F, up=F, down=F, hidden=512, inter=256, E=8, grid=F, dgrid=F, x=F, dtype=1, T=5,
        router=F, rdtype=1, k=2, renorm=1, ids=F, weights=F, y=F, ws=F, wn=BIG, status=F):
    return L.iq_moe(fmt, down_fmt, gate, up, down, hidden, inter, E, grid, dgrid, x, dtype, T, router, rdtype, k,
                    renorm, ids, weights, y, ws, wn, status, None)


LINEAR_BAD = [
    (dict(fmt=5), -1), (dict(fmt=-1), -1), (dict(dtype=2), -2), (dict(grid=None), -3), (dict(packed=None), -3),
    (dict(x=None), -3), (dict(y=None), -3), (dict(a=None), -3), (dict(b=None), -3), (dict(ids=None), -3),
    (dict(ws=None), -3), (dict(cols=300), -4), (dict(cols=0), -4), (dict(rows=-1), -4), (dict(T=-1), -4),
    (dict(rows=1 << 40), -4), (dict(T=1 << 40), -4), (dict(cols=1 << 40), -4), (dict(rank=-1), -5),
    (dict(rank=1025), -5), (dict(N=0), -5), (dict(packed=ctypes.c_void_p(0x100001)), -5), (dict(wn=64), -7),
]
MOE_BAD = [
    (dict(fmt=5), -1), (dict(down_fmt=9), -1), (dict(dtype=3), -2), (dict(rdtype=7), -2), (dict(grid=None), -3),
    (dict(dgrid=None), -3), (dict(gate=None), -3), (dict(up=None), -3), (dict(down=None), -3), (dict(x=None), -3),
    (dict(ids=None), -3), (dict(weights=None), -3), (dict(y=None), -3), (dict(ws=None), -3), (dict(hidden=500), -4),
    (dict(inter=128), -4), (dict(inter=0), -4), (dict(T=-3), -4), (dict(T=1 << 40), -4), (dict(hidden=1 << 30), -4),
    (dict(E=0), -5), (dict(E=4097), -5), (dict(k=0), -5), (dict(k=65), -5), (dict(k=9), -5),
    (dict(gate=ctypes.c_void_p(0x100001)), -5), (dict(up=ctypes.c_void_p(0x100003)), -5),
    (dict(down=ctypes.c_void_p(0x100001)), -5), (dict(wn=100), -7),
]


@pytest.mark.parametrize("kw,rc", LINEAR_BAD)
def test_linear_refusals_enqueue_nothing(stubbed, kw, rc):
    stubbed.stub_reset(0)
    assert linear(stubbed, **kw) == rc
    assert stubbed.stub_launches() == 0


@pytest.mark.parametrize("kw,rc", MOE_BAD)
def test_moe_refusals_enqueue_nothing(stubbed, kw, rc):
    stubbed.stub_reset(0)
    assert moe(stubbed, **kw) == rc
    assert stubbed.stub_launches() == 0


def test_empty_calls_enqueue_nothing(stubbed):
    stubbed.stub_reset(0)
    assert linear(stubbed, T=0, x=None, y=None, ids=None, ws=None, wn=0) == 0
    assert linear(stubbed, rows=0, packed=None, y=None, b=None, ws=None, wn=0) == 0
    assert moe(stubbed, T=0, x=None, y=None, ids=None, weights=None, ws=None, wn=0) == 0
    assert stubbed.stub_launches() == 0


@pytest.mark.parametrize("kw", [dict(), dict(rank=0, N=0, a=None, b=None, ids=None), dict(T=700), dict(dtype=0),
                                dict(T=40, rows=5000, cols=5120), dict(T=4096, fmt=4, dtype=0)])
def test_linear_stops_at_the_first_failed_launch(stubbed, kw):
    for fmt in ([kw["fmt"]] if "fmt" in kw else range(5)):
        args = {**kw, "fmt": fmt}
        stubbed.stub_reset(0)
        assert linear(stubbed, **args) == 0
        for n in range(1, stubbed.stub_launches() + 1):
            stubbed.stub_reset(n)
            assert linear(stubbed, **args) == -6
            assert stubbed.stub_launches() == n


@pytest.mark.parametrize("kw", [dict(), dict(router=None), dict(T=1), dict(T=300), dict(dtype=0, rdtype=0)])
def test_moe_stops_at_the_first_failed_launch(stubbed, kw):
    for fmt in range(5):
        args = {**kw, "fmt": fmt, "down_fmt": 4 - fmt}
        stubbed.stub_reset(0)
        assert moe(stubbed, **args) == 0
        for n in range(1, stubbed.stub_launches() + 1):
            stubbed.stub_reset(n)
            assert moe(stubbed, **args) == -6
            assert stubbed.stub_launches() == n


def test_workspace_queries(api):
    L, n = api.lib(), ctypes.c_size_t()
    bf, f32 = torch.bfloat16, torch.float32
    assert api.linear_workspace_size("IQ2_XS", 0, 512, bf, 5) == 0
    assert api.linear_workspace_size("IQ2_XS", 64, 512, bf, 0) == 0
    assert api.linear_workspace_size("IQ2_XS", 64, 512, f32, 64) > api.linear_workspace_size("IQ2_XS", 64, 512, bf, 64)
    assert api.linear_workspace_size("IQ2_XS", 64, 512, bf, 64, 16) > api.linear_workspace_size("IQ2_XS", 64, 512, bf, 64)
    assert api.moe_workspace_size("IQ2_XS", 512, 256, 8, bf, 0, 2) == 0
    assert api.moe_workspace_size("IQ2_XS", 512, 256, 8, bf, 64, 2) > 64 * 2 * 256 * 2
    assert L.iq_linear_workspace_size(0, 64, 512, 1, 5, 0, None) == -3
    assert L.iq_linear_workspace_size(0, 64, 500, 1, 5, 0, ctypes.byref(n)) == -4
    assert L.iq_moe_workspace_size(0, 7, 512, 256, 8, 1, 5, 2, ctypes.byref(n)) == -1
    assert L.iq_moe_workspace_size(0, 0, 512, 256, 8, 1, 5, 2, None) == -3
    with pytest.raises(api.IQError):
        api.linear_workspace_size("IQ2_XS", 64, 512, torch.float16, 5)


# The binding checks shapes and types before it asks for a device, so CPU tensors reach every check.
def base_linear():
    return dict(fmt="IQ2_XXS", packed=torch.zeros((48, 2, 66), dtype=torch.uint8), grid=torch.zeros((256, 8)),
                x=torch.zeros((3, 512)), lora_a=torch.zeros((2, 4, 512)), lora_b=torch.zeros((2, 48, 4)),
                lora_scale=torch.ones(2), lora_ids=torch.zeros(3, dtype=torch.int32))


@pytest.mark.parametrize("kw", [
    dict(fmt="IQ3"), dict(packed=torch.zeros((48, 2, 74), dtype=torch.uint8)), dict(packed=torch.zeros((48, 2, 66))),
    dict(grid=torch.zeros((512, 8))), dict(grid=torch.zeros((256, 8), dtype=torch.float64)),
    dict(x=torch.zeros((3, 256))), dict(x=torch.zeros((3, 512), dtype=torch.float16)), dict(x=torch.zeros(512)),
    dict(lora_a=torch.zeros((2, 4, 256))), dict(lora_a=torch.zeros((2, 4, 512), dtype=torch.bfloat16)),
    dict(lora_a=torch.zeros((0, 4, 512))), dict(lora_b=torch.zeros((2, 4, 48))), dict(lora_b=None),
    dict(lora_scale=torch.ones(3)), dict(lora_ids=torch.zeros(3, dtype=torch.int64)), dict(lora_ids=None),
    dict(lora_ids=torch.zeros(2, dtype=torch.int32)), dict(lora_a=None), dict(out=torch.zeros((3, 47))),
    dict(out=torch.zeros((3, 48), dtype=torch.bfloat16)), dict(status=torch.zeros(1)), dict(),
])
def test_linear_binding_refuses(api, kw):
    with pytest.raises(api.IQError):  # the last one: CPU tensors
        api.linear(**{**base_linear(), **kw})


def base_moe():
    return dict(fmt="IQ2_XXS", gate=torch.zeros((4 * 256, 2, 66), dtype=torch.uint8),
                up=torch.zeros((4 * 256, 2, 66), dtype=torch.uint8),
                down=torch.zeros((4 * 512, 1, 66), dtype=torch.uint8), grid=torch.zeros((256, 8)),
                x=torch.zeros((3, 512)), num_experts=4, router=torch.zeros((4, 512)), top_k=2)


@pytest.mark.parametrize("kw", [
    dict(fmt="nope"), dict(down_fmt="nope"), dict(num_experts=0), dict(num_experts=3), dict(x=torch.zeros((3, 500))),
    dict(x=torch.zeros((3, 512), dtype=torch.float16)), dict(gate=torch.zeros((4 * 128, 2, 66), dtype=torch.uint8)),
    dict(up=torch.zeros((4 * 512, 2, 66), dtype=torch.uint8)), dict(down=torch.zeros((4 * 512, 2, 66), dtype=torch.uint8)),
    dict(down_fmt="IQ2_S"), dict(down_grid=torch.zeros((512, 8))), dict(router=torch.zeros((5, 512))),
    dict(router=torch.zeros((4, 512), dtype=torch.float16)), dict(top_k=0), dict(top_k=5), dict(top_k=None),
    dict(router=None), dict(router=None, ids=torch.zeros((3, 2), dtype=torch.int32)),
    dict(ids=torch.zeros((3, 2), dtype=torch.int64)), dict(ids=torch.zeros((3, 3), dtype=torch.int32)),
    dict(weights=torch.zeros((3, 1))), dict(out=torch.zeros((3, 500))), dict(),
])
def test_moe_binding_refuses(api, kw):
    with pytest.raises(api.IQError):
        api.moe(**{**base_moe(), **kw})


@pytest.mark.parametrize("name", ["x", "lora_a", "lora_b", "lora_scale"])
def test_linear_has_no_backward_pass(api, name):
    kw = base_linear()
    kw[name].requires_grad_()
    with pytest.raises(api.IQError, match="no backward pass"):
        api.linear(**kw)
    with torch.no_grad(), pytest.raises(api.IQError, match="device tensors"):
        api.linear(**kw)


@pytest.mark.parametrize("name", ["x", "router"])
def test_moe_has_no_backward_pass(api, name):
    kw = base_moe()
    kw[name].requires_grad_()
    with pytest.raises(api.IQError, match="no backward pass"):
        api.moe(**kw)
    with torch.no_grad(), pytest.raises(api.IQError, match="device tensors"):
        api.moe(**kw)


@pytest.fixture(scope="module")
def measured(api, tmp_path_factory):
    """The stand-in, which also keeps the largest dimensions that it was asked to launch."""
    objs = sorted(glob.glob(os.path.join(ROOT, "ggml_iq_codebook_imatrix_amd", "_build", "iq_*.hip.o")))
    d = tmp_path_factory.mktemp("measured")
    src, so = d / "measured.c", str(d / "libiq_measured.so")
    src.write_text(f"""
#define hipLaunchKernel base_launch
#include "{os.path.join(ROOT, 'tests', 'hip_launch_stub.c')}"
#undef hipLaunchKernel
static unsigned long long threads, rows, empty;
hipError_t hipLaunchKernel(const void *fn, dim3 grid, dim3 block, void **args, size_t shared, void *stream) {{
  unsigned long long n = (unsigned long long)grid.x * block.x;
  if (n > threads) threads = n;
  if (grid.y > rows) rows = grid.y;
  if (!grid.x || !grid.y || !block.x || block.x > 1024 || block.x % 64) empty = 1;
  return base_launch(fn, grid, block, args, shared, stream);
}}
void sizes_reset(void) {{ threads = rows = empty = 0; }}
unsigned long long most_threads(void) {{ return threads; }}
unsigned long long most_rows(void) {{ return rows; }}
unsigned long long bad_shape(void) {{ return empty; }}
""")
    subprocess.run(["gcc", "-O1", "-fPIC", "-c", str(src), "-o", str(d / "m.o")], check=True)
    subprocess.run(["gcc", "-shared", "-o", so, *objs, str(d / "m.o"), "-L/opt/rocm/lib", "-lamdhip64",
                    "-Wl,-Bsymbolic", "-Wl,-rpath,/opt/rocm/lib"], check=True)
    L = ctypes.CDLL(so)
    for name, (args, res) in api.SIGNATURES.items():
        getattr(L, name).argtypes = args
        getattr(L, name).restype = res
    for n in ("most_threads", "most_rows", "bad_shape"):
        getattr(L, n).restype = ctypes.c_ulonglong
    return L


def launches_fit(L, call):
    """call() either refuses the sizes before any launch, or launches what the hardware takes."""
    L.stub_reset(0)
    L.sizes_reset()
    rc = call()
    assert rc in (0, -4), rc
    if rc:
        assert L.stub_launches() == 0
    else:
        assert L.most_threads() < 1 << 32 and L.most_rows() <= 65535 and not L.bad_shape()
    return rc == 0


def test_linear_launches_fit_the_grid(measured):
    done = 0
    for rows in (1, 17, 640 * 16, 1 << 20, 1 << 27, (1 << 27) + 1, 1 << 31):
        for cols in (256, 1280, 2048, 1 << 24):
            for T in (1, 16, 17, 32, 33, 64, 65, 700, 5000, 1 << 20, 4 * 65535 * 16, 4 * 65535 * 16 + 1):
                for rank, dtype in ((0, 1), (1024, 1), (0, 0), (1024, 0)):
                    done += launches_fit(measured, lambda: linear(measured, rows=rows, cols=cols, T=T, rank=rank, N=1,
                                                                  dtype=dtype, wn=1 << 62))
    assert done > 500
    assert linear(measured, rows=1 << 27, wn=1 << 62) == 0 and linear(measured, rows=(1 << 27) + 1, wn=1 << 62) == -4


def test_moe_launches_fit_the_grid(measured):
    done = 0
    for E, k in ((1, 1), (8, 2), (256, 8), (300, 64), (4096, 64)):
        for hidden, inter in ((256, 256), (2048, 768), (1 << 18, 256), (256, 1 << 18), (1 << 24, 1 << 24)):
            for T in (1, 2, 8, 9, 16, 17, 700, 1 << 20, 1 << 24):
                for dtype in (0, 1):
                    done += launches_fit(measured, lambda: moe(measured, E=E, k=k, hidden=hidden, inter=inter, T=T,
                                                               dtype=dtype, wn=1 << 62))
    assert done > 200
    # 4,096 experts of 2^18 rows: 2^32 threads in a launch over whole rows
    assert moe(measured, E=4096, inter=1 << 18, T=700, wn=1 << 62) == -4


@pytest.mark.parametrize("name", ["grid", "down_grid", "weights"])
def test_codebooks_and_weights_have_no_backward_pass(api, name):
    """The output depends on the codebooks as well: a gradient through them is refused, not dropped."""
    kw = base_moe()
    kw.update(down_grid=torch.zeros((256, 8)))
    if name == "weights":
        kw.update(router=None, top_k=None, ids=torch.zeros((3, 2), dtype=torch.int32), weights=torch.zeros((3, 2)))
    kw[name].requires_grad_()
    with pytest.raises(api.IQError, match="no backward pass"):
        api.moe(**kw)
    with torch.no_grad(), pytest.raises(api.IQError, match="device tensors"):
        api.moe(**kw)
    if name == "grid":
        kw = base_linear()
        kw["grid"].requires_grad_()
        with pytest.raises(api.IQError, match="no backward pass"):
            api.linear(**kw)
        with torch.no_grad(), pytest.raises(api.IQError, match="device tensors"):
            api.linear(**kw)


@pytest.mark.parametrize("call, name", [("linear", n) for n in ("grid", "x", "lora_a", "lora_b", "lora_scale")] +
                         [("moe", n) for n in ("grid", "down_grid", "x", "router")])
def test_forward_mode_tangents_are_refused(api, call, name):
    """A dual tensor's tangent would be dropped: refused, under no_grad as well (which does not stop forward mode)."""
    kw = base_linear() if call == "linear" else {**base_moe(), "down_grid": torch.zeros((256, 8))}
    run = getattr(api, call)
    with torch.autograd.forward_ad.dual_level():
        with pytest.raises(api.IQError, match="device tensors"):
            run(**kw)
        kw[name] = torch.autograd.forward_ad.make_dual(kw[name], torch.ones_like(kw[name]))
        with pytest.raises(api.IQError, match="tangent"):
            run(**kw)
        with torch.no_grad(), pytest.raises(api.IQError, match="tangent"):
            run(**kw)
    if call == "linear":
        kw = base_linear()
        with pytest.raises(api.IQError, match="tangent"):
            torch.func.jvp(lambda t: run(**{**kw, name: t}), (kw[name],), (torch.ones_like(kw[name]),))


@pytest.mark.parametrize("router", [True, False])
def test_moe_ids_that_are_no_tensor(api, router):
    for ids in ([[0, 1]] * 3, 7, torch.zeros((3, 2), dtype=torch.int32).numpy()):
        kw = {**base_moe(), "ids": ids}
        if not router:
            kw.update(router=None, top_k=None, weights=torch.zeros((3, 2)))
        with pytest.raises(api.IQError, match="ids must be a tensor"):
            api.moe(**kw)


@pytest.mark.parametrize("call", ["linear", "moe"])
def test_out_that_requires_a_gradient(api, call):
    """A call into a tensor of a recorded graph would change it behind the graph's back."""
    kw = base_linear() if call == "linear" else base_moe()
    kw["out"] = torch.zeros((3, 48 if call == "linear" else 512), requires_grad=True)
    with pytest.raises(api.IQError, match="no backward pass"):
        getattr(api, call)(**kw)
    with torch.no_grad(), pytest.raises(api.IQError, match="device tensors"):
        getattr(api, call)(**kw)
