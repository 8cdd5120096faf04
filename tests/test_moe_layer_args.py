"""Refusals of the whole MoE layer (no GPU needed: nothing is enqueued) and its workspace size."""
import ctypes

import pytest

from hbm_expert_slot_amd import binding as B

P = 0x100000     # stands for a device pointer: never followed


def _cfg(**kw):
    d = dict(hidden=256, inter=128, n_experts=16, top_k=2, shared_inter=128, max_rows=4, score=0, routed_scale=1.0)
    d.update(kw)
    return B.sc_moe_config(*[d[n] for n, _ in B.sc_moe_config._fields_])


def _fails(f, *args):
    with pytest.raises(B.SlotCacheError) as e:
        f(*args)
    assert e.value.status == B.SC_E_ARG and str(e.value)


BAD = [dict(hidden=0), dict(hidden=96), dict(hidden=32832), dict(inter=-64), dict(inter=100), dict(inter=65536),
       dict(n_experts=1), dict(n_experts=1025), dict(top_k=0), dict(top_k=33, n_experts=64), dict(shared_inter=-64),
       dict(shared_inter=65), dict(max_rows=0), dict(max_rows=17), dict(score=2)]


@pytest.mark.parametrize("bad", BAD, ids=str)
def test_configurations_that_are_refused(bad):
    c = ctypes.byref(_cfg(**bad))
    w = ctypes.byref(B.sc_moe_weights(P, None, P, P, P, P))
    _fails(B.moe_layer_workspace_bytes, c)
    _fails(B.moe_layer_prepare, c, P, None)
    _fails(B.moe_layer_forward, c, w, P, P, 1 << 20, 1, P, B.SC_DTYPE_F32, 1 << 20, None, None, None)


def test_workspace_holds_the_picks_rows():
    n = B.moe_layer_workspace_bytes(ctypes.byref(_cfg()))
    assert n >= 4 * 2 * (128 + 256) * 4 + 4 * (128 + 256) * 4
    assert B.moe_layer_workspace_bytes(ctypes.byref(_cfg(max_rows=16))) > n


@pytest.mark.parametrize("change", [
    dict(router=None), dict(blobs=None), dict(gs=None), dict(shared=None), dict(sgs=None), dict(router=P + 8),
    dict(blobs=P + 4), dict(shared=P + 8), dict(gs=P + 2), dict(bias=P + 1), dict(ws=None), dict(ws=P + 128),
    dict(x=None), dict(y=None), dict(x=P + 1), dict(y=P + 2), dict(ldx=255), dict(ldy=255), dict(M=-1), dict(M=5),
    dict(yt=B.SC_DTYPE_F16), dict(yt=5), dict(ids=P + 2), dict(wo=P + 1),
], ids=str)
def test_arguments_that_are_refused(change):
    a = dict(router=P, bias=None, blobs=P, gs=P, shared=P, sgs=P, ws=P, x=P, ldx=256, M=1, y=P, yt=B.SC_DTYPE_F32,
             ldy=256, ids=None, wo=None)
    a.update(change)
    w = B.sc_moe_weights(a["router"], a["bias"], a["blobs"], a["gs"], a["shared"], a["sgs"])
    _fails(B.moe_layer_forward, ctypes.byref(_cfg()), ctypes.byref(w), a["ws"], a["x"], a["ldx"], a["M"], a["y"],
           a["yt"], a["ldy"], a["ids"], a["wo"], None)


def test_null_structures():
    w = ctypes.byref(B.sc_moe_weights(P, None, P, P, P, P))
    _fails(B.moe_layer_forward, None, w, P, P, 256, 1, P, 0, 256, None, None, None)
    _fails(B.moe_layer_forward, ctypes.byref(_cfg()), None, P, P, 256, 1, P, 0, 256, None, None, None)
    _fails(B.moe_layer_prepare, ctypes.byref(_cfg()), None, None)


def test_no_rows():
    w = ctypes.byref(B.sc_moe_weights(P, None, P, P, P, P))
    B.moe_layer_forward(ctypes.byref(_cfg()), w, P, None, 256, 0, None, 0, 256, None, None, None)


def test_python_refusals():
    import torch

    from hbm_expert_slot_amd import ops
    r = torch.zeros(4, 64, dtype=torch.bfloat16)
    b = torch.zeros(4, ops.blob_bytes(64, 64), dtype=torch.uint8)
    g = torch.zeros(4, 2)
    with pytest.raises(ValueError, match="GPU"):
        ops.MoELayer(64, 64, 2, r, b, g)
    with pytest.raises(ValueError, match="score"):
        ops.MoELayer(64, 64, 2, r, b, g, score="max")
    with pytest.raises(ValueError, match="router"):
        ops.MoELayer(128, 64, 2, r, b, g)
    with pytest.raises(ValueError, match="blob"):
        ops.expert_matrices(b[0, 1:], 64, 64, g[0])


def test_places_of_the_control_words(tmp_path):
    """The GPU test of a call that gives up marks a word of the one-row kernel, whose place it spells out: the sources
    agree with it (on another word the mark would do something else)."""
    import os
    import shutil
    import subprocess

    from hbm_expert_slot_amd import build
    cc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(cc):
        pytest.skip("hipcc not available")
    claims = 5 * 16 * 32 + 2 * 32 + (513 + 32) // 32 * 32 + 1024 + 513 * 32
    with open(os.path.join(os.path.dirname(__file__), "test_gpu_moe_layer.py")) as f:
        assert "5 * 16 * 32 + 2 * 32 + (513 + 32) // 32 * 32 + 1024 + 513 * 32" in f.read()
    for name, claim in (("moe_layer", "sc::kLayerWords == %d" % claims),
                        ("moe_layer", "offsetof(sc::MoeWs, ctl) == 0"), ("moe_one", "sc::moe::O_CLAIM == 0")):
        src = tmp_path / "places.hip"
        src.write_text('#include "%s.hip"\nstatic_assert(%s, "");\n' % (name, claim))
        r = subprocess.run([cc] + build.FLAGS + ["-I" + os.path.join(build.HERE, "csrc"), "--cuda-device-only",
                                                 "-fsyntax-only", str(src)],
                           stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
        assert r.returncode == 0, (claim, r.stdout[-2000:])


def test_place_of_the_count_that_a_test_marks(tmp_path):
    import os
    import shutil
    import subprocess

    from hbm_expert_slot_amd import build
    from test_gpu_moe_layer import H_DONE
    cc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(cc):
        pytest.skip("hipcc not available")
    src = tmp_path / "places.hip"
    src.write_text('#include "moe_layer.hip"\nstatic_assert(sc::C_HDONE == %d && sc::C_HDONE < sc::C_TILES, "");\n' % H_DONE)
    r = subprocess.run([cc] + build.FLAGS + ["-I" + os.path.join(build.HERE, "csrc"), "--cuda-device-only",
                                             "-fsyntax-only", str(src)],
                       stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout[-2000:]
