"""Refusals of the layer's and the gradients' entry points: arguments are checked before anything is queued, so none of
this needs a GPU."""
import ctypes as C

import pytest
import torch

from collective_communication_schedules_gb300 import hoc

P = 4096  # a non-NULL, aligned address that no refused call may follow


def arr(*v):
    return (C.c_void_p * len(v))(*v)


def groups(k=1, experts=2, sources=1, seg=P, rows=(8,)):
    cap = (C.c_size_t * len(rows))(*rows)
    return C.byref(hoc._RowGroups(k, experts, sources, seg, cap))


def mm(g=None, x=arr(P), w=arr(P), b=None, inp=64, out=64, act=0, y=arr(P), pre=None, status=P):
    return hoc.lib().hoc_expert_mm(g if g is not None else groups(), x, w, b, inp, out, act, y, pre, status, None)


def linear(rows=4, x=P, ldx=64, w=P, b=None, r=None, ldr=0, inp=64, out=64, act=0, y=P, ldy=64, pre=None, status=P):
    return hoc.lib().hoc_linear(rows, x, ldx, w, b, r, ldr, inp, out, act, y, ldy, pre, status, None)


@pytest.mark.parametrize("bad", [
    dict(g=groups(k=0)), dict(g=groups(k=17, rows=(1,) * 17)), dict(g=groups(experts=0)), dict(g=groups(sources=0)),
    dict(g=groups(seg=None)), dict(g=groups(rows=(2 ** 31,))), dict(x=arr(None)), dict(x=arr(P + 1)), dict(w=arr(None)),
    dict(b=arr(None)), dict(y=arr(None)), dict(pre=arr(None)), dict(inp=0), dict(out=-1), dict(inp=2 ** 21), dict(act=5),
    dict(act=-1), dict(status=None), dict(x=None), dict(g=groups(rows=(2 ** 30,)), out=2 ** 20, act=4),
])
def test_expert_forward_refuses(bad):
    assert mm(**bad) == hoc.ERR_INVALID_ARG
    assert hoc.last_error_detail()


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(ldx=63), dict(ldy=8), dict(r=P, ldr=2), dict(inp=0), dict(act=9), dict(status=None), dict(x=None),
    dict(w=None), dict(y=None), dict(x=P + 1), dict(b=P + 1), dict(pre=P + 1),
])
def test_linear_refuses(bad):
    assert linear(**bad) == hoc.ERR_INVALID_ARG


def test_gradients_refuse():
    lib = hoc.lib()
    bad = hoc.ERR_INVALID_ARG
    g = groups()
    dgrad = lambda act=0, pre=None, dx=arr(P): lib.hoc_expert_mm_dgrad(g, arr(P), arr(P), 64, 64, act, pre, dx, P, None)  # noqa: E731
    assert dgrad(act=3) == bad and dgrad(act=3, pre=arr(None)) == bad and dgrad(dx=arr(None)) == bad
    wgrad = lambda dt=hoc.BFLOAT16, dw=arr(P), db=None: lib.hoc_expert_mm_wgrad(g, arr(P), arr(P), 64, 64, dt, 0, dw, db, P, None)  # noqa: E731
    assert wgrad(dt=hoc.INT32) == bad and wgrad(dw=arr(None)) == bad and wgrad(db=arr(None)) == bad
    assert wgrad(dt=hoc.FLOAT32, dw=arr(P + 2)) == bad
    assert lib.hoc_linear_dgrad(4, P, 8, P, 64, 64, 0, None, P, P, None) == bad
    assert lib.hoc_linear_dgrad(4, P, 64, P, 64, 64, 2, None, P, P, None) == bad
    assert lib.hoc_linear_wgrad(4, P, 64, P, 8, 64, 64, hoc.BFLOAT16, 0, P, None, P, None) == bad
    assert lib.hoc_linear_wgrad(4, P, 64, P, 64, 64, 64, hoc.FLOAT32, 0, P + 2, None, P, None) == bad
    assert lib.hoc_act_grad(4, 8, 0, P, P, P, None) == bad and lib.hoc_act_grad(4, 8, 2, P, None, P, None) == bad
    assert lib.hoc_ep_segments(2, arr(P, P), 4, 2, 3, P, None) == bad
    assert lib.hoc_ep_segments(2, arr(P, None), 4, 2, 4, P, None) == bad
    assert lib.hoc_ep_segments(2, arr(P, P), 4, 2, 4, None, None) == bad


def test_combine_gradient_refuses():
    lib = hoc.lib()
    cap = (C.c_size_t * 1)(64)
    call = lambda k=1, dy=arr(P), rows=arr(P), dr=arr(P), dw=arr(P), e=2, status=P: lib.hoc_ep_combine_grad(  # noqa: E731
        k, dy, rows, cap, arr(P), arr(P), P, arr(P), 1, 1, 8, e, dr, dw, status, None)
    for bad in (dict(k=0), dict(dy=None), dict(dy=arr(None)), dict(rows=arr(None)), dict(dr=arr(None)), dict(dw=arr(None)),
                dict(e=0), dict(status=None)):
        assert call(**bad) == hoc.ERR_INVALID_ARG


def test_tensor_lists_refuse():
    lib = hoc.lib()
    h = C.c_void_p()
    one = (C.c_size_t * 1)(4)
    make = lambda n=1, ptr=arr(P), count=one, dt=hoc.FLOAT32: lib.hoc_tensor_list_create(C.byref(h), n, ptr, count, dt)  # noqa: E731
    for bad in (dict(n=-1), dict(ptr=None), dict(count=None), dict(dt=hoc.INT32), dict(ptr=arr(None)), dict(ptr=arr(P + 2)),
                dict(count=(C.c_size_t * 1)(2 ** 42))):
        assert make(**bad) == hoc.ERR_INVALID_ARG and not h.value
    if not torch.cuda.is_available():
        assert make() == hoc.ERR_NO_DEVICE and not h.value
    assert lib.hoc_tensor_list_destroy(None) == hoc.ERR_INVALID_ARG
    assert lib.hoc_grad_workspace(None, C.byref(C.c_size_t())) == hoc.ERR_INVALID_ARG
    assert lib.hoc_grad_norm(None, P, P, 8, None) == hoc.ERR_INVALID_ARG
    assert lib.hoc_grad_clip(None, None, C.byref(C.c_float(1)), P, P, 8, None) == hoc.ERR_INVALID_ARG


def test_the_binding_names_what_is_wrong():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.bfloat16)
    y, st = torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="x: must be a CUDA tensor"):
        hoc.linear(x, w, y, status=st)
    with pytest.raises(TypeError, match="x: expected a bfloat16 tensor"):
        hoc.linear(x.float(), w, y, status=st)
    with pytest.raises(ValueError, match="act is one of"):
        hoc.linear(x, w, y, status=st, act="tanh")
    with pytest.raises(ValueError, match="swiglu needs an even number"):
        hoc.linear(x, w[:31], y, status=st, act="swiglu")
    seg = torch.zeros(1, 4, dtype=torch.int64)
    with pytest.raises(ValueError, match="seg: expected shape"):
        hoc.expert_mm([x], [w.view(2, 16, 64)], seg, [y], status=st)
    with pytest.raises(ValueError, match="pre is given exactly when"):
        hoc.expert_mm_dgrad([y], [w.view(1, 32, 64)], seg[:, :2], [x], status=st, act="gelu")
    with pytest.raises(TypeError, match="one dtype"):
        hoc.TensorList([x, x.float()])


def test_only_errors_of_the_call_itself_are_reported(tmp_path):
    """The library's own objects over a fake CUDA runtime (tests/c/fake_cudart.cpp): an error that an earlier call left
    is neither reported nor cleared, a failed launch is reported and leaves none."""
    import os
    import subprocess

    from collective_communication_schedules_gb300 import build

    objs = [os.path.join(build.BUILD, n + ".o") for n in ("layer", "mm_any", "mm_few", "mm_tc")]
    if not all(os.path.exists(o) for o in objs):
        pytest.skip("the library was not built here")
    here = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c")
    out = str(tmp_path / "launches")
    cmd = [build.nvcc()] + build.ARCH + ["-O1", "-std=c++17", "-cudart", "none", "-I", build.INCLUDE, "-I", here,
                                         os.path.join(here, "launches.cpp"), os.path.join(here, "fake_cudart.cpp")]
    r = subprocess.run(cmd + objs + ["-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([out], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "LAUNCHES OK" in r.stdout, r.stdout + r.stderr


def test_trimming_without_scratch():
    with pytest.raises(ValueError, match="keep"):
        hoc.layer_trim(-1)
    if not torch.cuda.is_available():
        assert hoc.lib().hoc_layer_trim(0) == hoc.ERR_NO_DEVICE


def test_the_products_that_run_on_realigned_copies(tmp_path):
    """The rule's two sides (sizes in tests/c/realign.cpp), by the launches of a call over the fake CUDA runtime."""
    import os
    import subprocess

    from collective_communication_schedules_gb300 import build

    objs = [os.path.join(build.BUILD, n + ".o") for n in ("layer", "mm_any", "mm_few", "mm_tc")]
    if not all(os.path.exists(o) for o in objs):
        pytest.skip("the library was not built here")
    here = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c")
    out = str(tmp_path / "realign")
    cmd = [build.nvcc()] + build.ARCH + ["-O1", "-std=c++17", "-cudart", "none", "-I", build.INCLUDE, "-I", here,
                                         os.path.join(here, "realign.cpp"), os.path.join(here, "fake_cudart.cpp")]
    r = subprocess.run(cmd + objs + ["-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([out], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "REALIGN OK" in r.stdout, r.stdout + r.stderr


def test_lists_and_experts_that_are_missing():
    """An empty list of weights, and weights of no expert, are refused by name."""
    x, y = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 32, dtype=torch.bfloat16)
    st, seg = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 3, dtype=torch.int64)
    none = torch.zeros(0, 32, 64, dtype=torch.bfloat16)
    for w, what in (([], "weight|dw"), ([none], "expert")):
        with pytest.raises(ValueError, match=what):
            hoc.expert_mm([x], w, seg, [y], status=st)
        with pytest.raises(ValueError, match=what):
            hoc.expert_mm_dgrad([y], w, seg, [x], status=st)
        with pytest.raises(ValueError, match=what):
            hoc.expert_mm_wgrad([y], [x], seg, w, status=st)
