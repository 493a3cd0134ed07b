"""iq_glu, iq_glu_backward, iq_linear_backward, iq_checkpoint and iq_restore without a GPU: the header's declarations,
refusals before anything is enqueued (C ABI and binding), workspace queries, launch failures and launch sizes."""
import ctypes
import os
import re

import pytest

from test_run_refusals import BIG, F, ROOT, api, launches_fit, measured, stubbed  # noqa: F401 (fixtures)

torch = pytest.importorskip("torch")

ODD = ctypes.c_void_p(0x100001)


def test_header_declares_the_calls(api):  # noqa: F811
    txt = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "iq_train.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(iq_\w+)\s*\(", txt, flags=re.M)))
    assert names == ["iq_checkpoint", "iq_glu", "iq_glu_backward", "iq_glu_backward_workspace_size",
                     "iq_glu_workspace_size", "iq_linear_backward", "iq_linear_backward_workspace_size", "iq_restore"]
    for n in names:
        assert n in api.SIGNATURES and hasattr(api.lib(), n)


def checkpoint(L, x=F, dtype=1, T=5, cols=100, codes=F, ex=F, status=F):
    return L.iq_checkpoint(x, dtype, T, cols, codes, ex, status, None)


def restore(L, codes=F, ex=F, T=5, cols=100, y=F, dtype=1):
    return L.iq_restore(codes, ex, T, cols, y, dtype, None)


def glu(L, fmt=1, gate=F, up=F, inter=64, hidden=512, grid=F, x=F, dtype=1, T=5, act=0, h=F, ws=F, wn=BIG, status=F):
    return L.iq_glu(fmt, gate, up, inter, hidden, grid, x, dtype, T, act, h, ws, wn, status, None)


def glu_backward(L, fmt=1, gate=F, up=F, inter=64, hidden=512, grid=F, x=F, ex=None, dh=F, dtype=1, T=5, act=0, dx=F,
                 ws=F, wn=BIG, status=F):
    return L.iq_glu_backward(fmt, gate, up, inter, hidden, grid, x, ex, dh, dtype, T, act, dx, ws, wn, status, None)


def linear_backward(L, fmt=1, packed=F, rows=64, cols=512, grid=F, dy=F, x=F, ex=None, dtype=1, T=5, a=F, b=F, scale=F,
                    ids=F, N=2, rank=4, dx=F, da=F, db=F, ws=F, wn=BIG, status=F):
    return L.iq_linear_backward(fmt, packed, rows, cols, grid, dy, x, ex, dtype, T, a, b, scale, ids, N, rank, dx, da,
                                db, ws, wn, status, None)


CHECKPOINT_BAD = [(dict(dtype=2), -2), (dict(T=-1), -4), (dict(cols=-1), -4), (dict(cols=1 << 25), -4),
                  (dict(T=1 << 25), -4), (dict(T=1 << 24, cols=8193), -4), (dict(codes=None), -3), (dict(ex=None), -3)]
GLU_BAD = [(dict(fmt=5), -1), (dict(fmt=-1), -1), (dict(dtype=2), -2), (dict(grid=None), -3), (dict(gate=None), -3),
           (dict(up=None), -3), (dict(x=None), -3), (dict(ws=None), -3), (dict(hidden=300), -4), (dict(hidden=0), -4),
           (dict(inter=-1), -4), (dict(T=-1), -4), (dict(T=1 << 40), -4), (dict(inter=1 << 40), -4),
           (dict(hidden=1 << 40), -4), (dict(act=-1), -5), (dict(act=3), -5), (dict(gate=ODD), -5), (dict(up=ODD), -5),
           (dict(wn=64), -7)]
BACK_BAD = [(dict(fmt=5), -1), (dict(dtype=2), -2), (dict(grid=None), -3), (dict(packed=None), -3), (dict(dy=None), -3),
            (dict(x=None), -3), (dict(a=None), -3), (dict(b=None), -3), (dict(ids=None), -3), (dict(da=None), -3),
            (dict(db=None), -3), (dict(ws=None), -3), (dict(cols=300), -4), (dict(cols=0), -4), (dict(rows=-1), -4),
            (dict(T=-1), -4), (dict(rows=1 << 40), -4), (dict(T=1 << 40), -4), (dict(cols=1 << 40), -4),
            (dict(rank=-1), -5), (dict(rank=1025), -5), (dict(N=0), -5), (dict(N=65536), -4), (dict(packed=ODD), -5),
            (dict(wn=64), -7)]


@pytest.mark.parametrize("call,kw,rc", [(checkpoint, *c) for c in CHECKPOINT_BAD + [(dict(x=None), -3)]] +
                         [(restore, *c) for c in CHECKPOINT_BAD + [(dict(y=None), -3)]] +
                         [(glu, *c) for c in GLU_BAD + [(dict(h=None), -3)]] +
                         [(glu_backward, *c) for c in GLU_BAD + [(dict(dx=None), -3), (dict(dh=None), -3)]] +
                         [(linear_backward, *c) for c in BACK_BAD])
def test_refusals_enqueue_nothing(stubbed, call, kw, rc):  # noqa: F811
    stubbed.stub_reset(0)
    assert call(stubbed, **kw) == rc
    assert stubbed.stub_launches() == 0


def test_empty_calls(stubbed):  # noqa: F811
    stubbed.stub_reset(0)
    assert checkpoint(stubbed, T=0, x=None, codes=None, ex=None) == 0 == checkpoint(stubbed, cols=0, x=None, ex=None)
    assert restore(stubbed, T=0, y=None, codes=None, ex=None) == 0 == restore(stubbed, cols=0, y=None, ex=None)
    assert glu(stubbed, T=0, x=None, h=None, ws=None, wn=0) == 0
    assert glu(stubbed, inter=0, gate=None, up=None, h=None, ws=None, wn=0) == 0
    assert glu_backward(stubbed, T=0, x=None, dh=None, dx=None, ws=None, wn=0) == 0
    assert linear_backward(stubbed, dx=None, rank=0, N=0, a=None, b=None, ids=None, x=None, da=None, db=None, ws=None,
                           wn=0) == 0  # nothing is wanted
    assert stubbed.stub_launches() == 0
    # outputs that are empty sums are zeros: one launch each
    none = dict(ws=None, wn=0, x=None)
    for n, call in ((1, lambda: glu_backward(stubbed, inter=0, gate=None, up=None, dh=None, **none)),
                    (2, lambda: linear_backward(stubbed, rows=0, packed=None, dy=None, b=None, db=None, **none)),
                    (2, lambda: linear_backward(stubbed, T=0, packed=None, dy=None, ids=None, dx=None, **none)),
                    (1, lambda: linear_backward(stubbed, rows=0, packed=None, dy=None, rank=0, N=0, **none))):
        stubbed.stub_reset(0)
        assert call() == 0 and stubbed.stub_launches() == n
        for k in range(1, n + 1):
            stubbed.stub_reset(k)
            assert call() == -6 and stubbed.stub_launches() == k


SIZES = [dict(), dict(T=1), dict(T=40), dict(T=700), dict(T=300, dtype=0)]


@pytest.mark.parametrize("call,kw", [(checkpoint, {}), (restore, {}), (checkpoint, dict(cols=64))] +
                         [(c, kw) for c in (glu, glu_backward) for kw in SIZES] +
                         [(glu_backward, dict(ex=F, dtype=0)), (glu_backward, dict(ex=F, T=40, inter=4000))] +
                         [(linear_backward, kw) for kw in SIZES + [
                             dict(rank=0, N=0, a=None, b=None, ids=None, x=None, da=None, db=None), dict(dx=None),
                             dict(rank=100), dict(ex=F), dict(rows=4000, T=40, scale=None)]])
def test_stops_at_the_first_failed_launch(stubbed, call, kw):  # noqa: F811
    for fmt in range(1 if call in (checkpoint, restore) else 5):
        args = kw if call in (checkpoint, restore) else {**kw, "fmt": fmt}
        stubbed.stub_reset(0)
        assert call(stubbed, **args) == 0
        for n in range(1, stubbed.stub_launches() + 1):
            stubbed.stub_reset(n)
            assert call(stubbed, **args) == -6
            assert stubbed.stub_launches() == n


def test_launches_fit_the_grid(measured):  # noqa: F811
    done = 0
    for T in (1, 16, 17, 33, 65, 129, 700, 5000, 1 << 20, 4 * 65535 * 16, 4 * 65535 * 16 + 1, 1 << 24):
        for cols in (256, 1280, 5120, 1 << 18, 1 << 24):
            done += launches_fit(measured, lambda: checkpoint(measured, T=T, cols=cols + 1))
            done += launches_fit(measured, lambda: restore(measured, T=T, cols=cols))
            for rows in (1, 17, 5000, 1 << 20, 1 << 24):
                for dtype in (0, 1):
                    kw = dict(T=T, dtype=dtype, wn=1 << 62)
                    done += launches_fit(measured, lambda: glu(measured, inter=rows, hidden=cols, **kw))
                    done += launches_fit(measured, lambda: glu_backward(measured, inter=rows, hidden=cols, **kw))
                    for N, rank in ((1, 1), (1, 1024), (65535, 16)):
                        done += launches_fit(measured, lambda: linear_backward(measured, rows=rows, cols=cols, N=N,
                                                                               rank=rank, **kw))
    assert done > 1000


def test_workspace_queries(api):  # noqa: F811
    L, n = api.lib(), ctypes.c_size_t()
    bf, f32 = torch.bfloat16, torch.float32
    assert api.glu_workspace_size("IQ2_XS", 0, 512, bf, 5) == 0 == api.glu_workspace_size("IQ2_XS", 64, 512, bf, 0)
    assert api.glu_workspace_size("IQ2_XS", 64, 512, f32, 64) > api.glu_workspace_size("IQ2_XS", 64, 512, bf, 64)
    assert api.glu_backward_workspace_size("IQ2_XS", 64, 512, bf, 64) > 64 * 2 * 64 * 2
    assert api.glu_backward_workspace_size("IQ2_XS", 0, 512, bf, 5) == 0
    assert api.linear_backward_workspace_size("IQ2_XS", 64, 512, bf, 0) == 0
    assert api.linear_backward_workspace_size("IQ2_XS", 64, 512, bf, 64, 3, 16) > \
        api.linear_backward_workspace_size("IQ2_XS", 64, 512, bf, 64)
    for fn in ("iq_glu_workspace_size", "iq_glu_backward_workspace_size"):
        assert getattr(L, fn)(0, 64, 512, 1, 5, None) == -3 and getattr(L, fn)(0, 64, 500, 1, 5, ctypes.byref(n)) == -4
    assert L.iq_linear_backward_workspace_size(0, 64, 512, 1, 5, 0, 0, None) == -3
    assert L.iq_linear_backward_workspace_size(0, 64, 512, 1, 5, 0, 4, ctypes.byref(n)) == -5
    for call in (lambda: api.glu_workspace_size("IQ2_XS", 64, 512, torch.float16, 5),
                 lambda: api.glu_backward_workspace_size("IQ2_XS", 64, 512, torch.float16, 5),
                 lambda: api.linear_backward_workspace_size("IQ2_XS", 64, 512, torch.float16, 5)):
        with pytest.raises(api.IQError):
            call()


# The binding checks shapes and types before it asks for a device, so CPU tensors reach every check.
def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def base_glu():
    return dict(fmt="IQ2_XXS", gate=u8(48, 2, 66), up=u8(48, 2, 66), grid=torch.zeros((256, 8)), x=torch.zeros((3, 512)))


def base_glu_backward():
    return {**base_glu(), "dh": torch.zeros((3, 48))}


def base_linear_backward():
    return dict(fmt="IQ2_XXS", packed=u8(48, 2, 66), grid=torch.zeros((256, 8)), dy=torch.zeros((3, 48)),
                x=torch.zeros((3, 512)), lora_a=torch.zeros((2, 4, 512)), lora_b=torch.zeros((2, 48, 4)),
                lora_scale=torch.ones(2), lora_ids=torch.zeros(3, dtype=torch.int32))


CODES, EX = torch.zeros((3, 512), dtype=torch.int8), u8(3, 16)
BAD_KEPT = [dict(x=None), dict(x=torch.zeros((3, 256))), dict(x=torch.zeros((3, 512), dtype=torch.bfloat16)),
            dict(x=(CODES,)), dict(x=(CODES, EX, EX)), dict(x=(CODES, u8(3, 15))), dict(x=(EX, CODES)),
            dict(x=(CODES[:2], EX)), dict(x=(CODES, None))]


@pytest.mark.parametrize("kw", [
    dict(fmt="IQ3"), dict(gate=u8(48, 2, 74)), dict(up=u8(47, 2, 66)), dict(up=u8(48, 1, 66)), dict(up=None),
    dict(grid=torch.zeros((512, 8))), dict(x=torch.zeros((3, 256))), dict(x=torch.zeros((3, 512), dtype=torch.float16)),
    dict(x=torch.zeros(512)), dict(x=(CODES, EX)), dict(activation="relu"), dict(activation=0), dict(activation=None),
    dict(out=torch.zeros((3, 47))), dict(out=torch.zeros((3, 48), dtype=torch.bfloat16)), dict(status=torch.zeros(1)),
    dict()])
def test_glu_binding_refuses(api, kw):  # noqa: F811
    with pytest.raises(api.IQError):  # the last one: CPU tensors
        api.glu(**{**base_glu(), **kw})


@pytest.mark.parametrize("kw", BAD_KEPT + [
    dict(gate=u8(48, 2, 74)), dict(dh=torch.zeros((3, 47))), dict(dh=torch.zeros((4, 48))),
    dict(dh=torch.zeros((3, 48), dtype=torch.float16)), dict(dh=None), dict(activation="tanh"),
    dict(out=torch.zeros((3, 48))), dict(x=(CODES, EX)), dict()])
def test_glu_backward_binding_refuses(api, kw):  # noqa: F811
    with pytest.raises(api.IQError):
        api.glu_backward(**{**base_glu_backward(), **kw})


@pytest.mark.parametrize("kw", BAD_KEPT + [
    dict(fmt="IQ3"), dict(packed=u8(48, 2, 74)), dict(grid=torch.zeros((512, 8))), dict(dy=torch.zeros((3, 47))),
    dict(dy=torch.zeros((3, 48), dtype=torch.float16)), dict(dy=torch.zeros((2, 48))), dict(lora_a=torch.zeros((2, 4, 256))),
    dict(lora_a=torch.zeros((0, 4, 512))), dict(lora_a=torch.zeros((2, 4, 512), dtype=torch.bfloat16)), dict(lora_b=None),
    dict(lora_b=torch.zeros((2, 4, 48))), dict(lora_scale=torch.ones(3)), dict(lora_ids=None),
    dict(lora_ids=torch.zeros(3, dtype=torch.int64)), dict(lora_a=None), dict(grad_a=torch.zeros((2, 4, 48))),
    dict(grad_b=torch.zeros((2, 48, 4), dtype=torch.bfloat16)), dict(out=torch.zeros((3, 48))),
    dict(out=torch.zeros((3, 512)), need_dx=False), dict(x=(CODES, EX)), dict()])
def test_linear_backward_binding_refuses(api, kw):  # noqa: F811
    with pytest.raises(api.IQError):
        api.linear_backward(**{**base_linear_backward(), **kw})


def test_checkpoint_binding_refuses(api):  # noqa: F811
    x = torch.zeros((3, 512))
    for kw in (dict(x=x[0]), dict(x=x.half()), dict(x=None), dict(codes=EX), dict(codes=CODES[:2]), dict(exponents=CODES),
               dict(exponents=u8(3, 15)), dict(status=torch.zeros(1)), dict()):
        with pytest.raises(api.IQError):
            api.checkpoint(**{"x": x, **kw})
    for kw in (dict(codes=EX), dict(codes=CODES[0]), dict(exponents=u8(3, 15)), dict(dtype=torch.float16),
               dict(out=x[:2]), dict(out=x.half()), dict()):
        with pytest.raises(api.IQError):
            api.restore(**{"codes": CODES, "exponents": EX, **kw})


@pytest.mark.parametrize("call,name", [("glu", n) for n in ("x", "grid", "out")] +
                         [("glu_backward", n) for n in ("x", "dh", "grid", "out")] +
                         [("linear_backward", n) for n in ("dy", "x", "grid", "lora_a", "lora_b", "lora_scale", "out",
                                                           "grad_a", "grad_b")] + [("checkpoint", "x"), ("restore", "out")])
def test_gradients_and_tangents_are_refused(api, call, name):  # noqa: F811
    """These calls are a program's own backward pass; what autograd would record or carry along is refused."""
    base = {"glu": base_glu, "glu_backward": base_glu_backward, "linear_backward": base_linear_backward,
            "checkpoint": lambda: dict(x=torch.zeros((3, 512))),
            "restore": lambda: dict(codes=CODES, exponents=EX)}[call]()
    shapes = {("glu", "out"): (3, 48), ("linear_backward", "grad_a"): (2, 4, 512),
              ("linear_backward", "grad_b"): (2, 48, 4)}
    t = base.get(name, torch.zeros(shapes.get((call, name), (3, 512))))
    run = getattr(api, call)
    with pytest.raises(api.IQError, match="no backward pass"):
        run(**{**base, name: t.clone().requires_grad_()})
    with torch.no_grad(), pytest.raises(api.IQError, match="device tensors"):
        run(**{**base, name: t.clone().requires_grad_()})
    with torch.autograd.forward_ad.dual_level(), torch.no_grad():
        with pytest.raises(api.IQError, match="tangent"):
            run(**{**base, name: torch.autograd.forward_ad.make_dual(t, torch.ones_like(t))})
