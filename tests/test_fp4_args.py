"""Refusals of the 4-bit operators: wrong arguments return an error before
anything is enqueued (no GPU needed), and the Python layer names what is wrong."""
import ctypes

import pytest

from hbm_expert_slot_amd import binding as B

P = 0x10000     # stands for a device pointer: never followed


def _m(fmt=B.SC_FP4_NV, rows=8, cols=64, codes=P, scales=P, gs=P):
    return B.sc_fp4_matrix(fmt, rows, cols, codes, scales, gs)


def _fails(f, *args, status=B.SC_E_ARG):
    with pytest.raises(B.SlotCacheError) as e:
        f(*args)
    assert e.value.status == status and str(e.value)


BAD_MATRICES = [
    _m(fmt=2), _m(rows=-1), _m(cols=0), _m(cols=24), _m(cols=-16), _m(fmt=B.SC_FP4_MX, cols=48),
    _m(cols=(1 << 20) + 16), _m(codes=None), _m(scales=None), _m(codes=P + 8), _m(scales=P + 1), _m(gs=P + 2),
    _m(rows=2 ** 31 - 1, cols=1 << 20),
]


@pytest.mark.parametrize("m", BAD_MATRICES)
def test_matrices_that_are_refused(m):
    r = ctypes.byref(m)
    _fails(B.fp4_linear, r, P, B.SC_DTYPE_BF16, 1 << 21, 1, None, P, B.SC_DTYPE_F32, 2 ** 31, None)
    _fails(B.fp4_dequantize, r, P, B.SC_DTYPE_F32, 1 << 21, None)
    _fails(B.fp4_quantize, P, B.SC_DTYPE_F32, 1 << 21, r, 1, None, None)


def test_null_matrix():
    _fails(B.fp4_linear, None, P, B.SC_DTYPE_BF16, 64, 1, None, P, B.SC_DTYPE_F32, 8, None)


@pytest.mark.parametrize("change", [
    dict(x=None), dict(y=None), dict(x=P + 1), dict(y=P + 2), dict(xt=B.SC_DTYPE_F32), dict(xt=7), dict(yt=3),
    dict(ldx=63), dict(ldy=7), dict(M=-1), dict(bias=P + 2),
])
def test_linear_arguments_that_are_refused(change):
    a = dict(x=P, xt=B.SC_DTYPE_BF16, ldx=64, M=1, bias=None, y=P, yt=B.SC_DTYPE_F32, ldy=8)
    a.update(change)
    _fails(B.fp4_linear, ctypes.byref(_m()), a["x"], a["xt"], a["ldx"], a["M"], a["bias"], a["y"], a["yt"], a["ldy"],
           None)


@pytest.mark.parametrize("change", [
    dict(w=None), dict(w=P + 2), dict(t=9), dict(ld=63), dict(ws=None), dict(ws=P + 2), dict(gs=None),
])
def test_quantize_arguments_that_are_refused(change):
    a = dict(w=P, t=B.SC_DTYPE_F32, ld=64, ws=P, gs=P)
    a.update(change)
    _fails(B.fp4_quantize, a["w"], a["t"], a["ld"], ctypes.byref(_m(gs=a["gs"])), 0, a["ws"], None)


def test_nothing_to_do():
    m = ctypes.byref(_m(rows=0))
    B.fp4_linear(m, P, B.SC_DTYPE_BF16, 64, 3, None, P, B.SC_DTYPE_F32, 8, None)
    B.fp4_linear(ctypes.byref(_m()), None, B.SC_DTYPE_BF16, 64, 0, None, None, B.SC_DTYPE_F32, 8, None)
    B.fp4_dequantize(m, None, B.SC_DTYPE_F32, 64, None)
    B.fp4_quantize(None, B.SC_DTYPE_F32, 64, m, 0, P, None)


def test_python_refusals():
    import torch

    from hbm_expert_slot_amd import ops
    with pytest.raises(ValueError, match="GPU"):
        ops.fp4_quantize(torch.zeros(4, 32))
    with pytest.raises(ValueError, match="type"):
        ops.fp4_quantize(torch.zeros(4, 32, dtype=torch.int32))
    with pytest.raises(ValueError, match="dimensions"):
        ops.fp4_quantize(torch.zeros(32))
    with pytest.raises(ValueError, match="GPU"):
        ops.FP4Weight(torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(ValueError, match="format"):
        ops.FP4Weight.empty(4, 32, "int4")
    with pytest.raises(ValueError, match="multiple"):
        ops.FP4Weight.empty(4, 40)


def _made(cls, **attributes):
    """An object with attributes as its constructor leaves them (the constructor needs a GPU)."""
    q = cls.__new__(cls)
    for name, value in attributes.items():
        setattr(q, name, value)
    return q


def test_what_a_weight_was_made_of_cannot_be_exchanged():
    """The library has the tensors' addresses: another tensor would be ignored, and the old one's memory freed."""
    from hbm_expert_slot_amd import ops
    made = dict(codes=1, scales=2, global_scale=None, fmt="nvfp4", rows=4, cols=16, device="cuda:0")
    q = _made(ops.FP4Weight, **made)
    for name, value in made.items():
        with pytest.raises(AttributeError, match=name):
            setattr(q, name, 5)
        with pytest.raises(AttributeError, match=name):
            delattr(q, name)
        assert getattr(q, name) == value
    q.name = "mine"
    q.name = "other"
    del q.name


def test_what_a_layer_was_made_of_cannot_be_exchanged():
    from hbm_expert_slot_amd import ops
    made = dict(hidden=64, inter=64, n_experts=8, top_k=2, shared_inter=0, max_rows=16, device="cuda:0", workspace=3)
    layer = _made(ops.MoELayer, **made)
    for name, value in made.items():
        with pytest.raises(AttributeError, match=name):
            setattr(layer, name, 5)
        assert getattr(layer, name) == value


def test_going_backward_through_an_operator_raises():
    import torch

    from hbm_expert_slot_amd import ops
    x = torch.ones(3, requires_grad=True)
    y = ops._ForInference.apply("fp4_linear", lambda: torch.zeros(2), x, None)
    y.add_(1)
    with pytest.raises(NotImplementedError, match="fp4_linear is for inference"):
        (y.sum() + x.sum()).backward()
    assert ops._wants_grad(None, x) and not ops._wants_grad(None, x.detach())
    with torch.no_grad():
        assert not ops._wants_grad(x)


def test_a_torch_without_the_raw_stream_call(monkeypatch):
    import importlib.util

    import torch

    from hbm_expert_slot_amd import ops
    if hasattr(torch._C, "_cuda_getCurrentRawStream"):
        assert ops._raw_stream is torch._C._cuda_getCurrentRawStream
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    spec = importlib.util.spec_from_file_location("hbm_expert_slot_amd.ops_again", ops.__file__)
    again = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(again)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: type("Stream", (), {"cuda_stream": 77 + index})())
    assert again._raw_stream(3) == 80


def test_a_weights_shape_is_no_attribute_to_set():
    from hbm_expert_slot_amd import ops
    q = _made(ops.FP4Weight, rows=4, cols=16)
    with pytest.raises(AttributeError):
        q.shape = (8, 16)
    assert q.shape == (4, 16) and "shape" not in vars(q)
