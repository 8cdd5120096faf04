"""No matrix instruction of the 4-bit kernels writes its result over an operand.

The compiler allows that for results of four registers; kernels of this library
that had it in the 16x16x32 form have given wrong outputs.  Results either lie in
the accumulation registers, or the operands are kept alive past the instruction."""
import os
import re
import shutil
import subprocess

import pytest

from hbm_expert_slot_amd import build as B


def _range(operand):
    m = re.fullmatch(r"([av])\[(\d+):(\d+)\]", operand) or re.fullmatch(r"([av])(\d+)", operand)
    if m is None:
        return None
    g = m.groups()
    return g[0], int(g[1]), int(g[-1])


def _assembly(name, tmp_path):
    cc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(cc):
        pytest.skip("hipcc not available")
    out = str(tmp_path / (name + ".s"))
    cmd = [cc] + B.FLAGS + ["-I" + os.path.join(B.HERE, "csrc"), "--cuda-device-only", "-S",
                            os.path.join(B.HERE, "csrc", name + ".hip"), "-o", out]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout[-2000:]
    with open(out) as f:
        return f.read()


@pytest.mark.parametrize("name,kernels", [("moe_layer", 2), ("moe_one", 1)])
def test_the_layer_writes_through(name, kernels, tmp_path):
    """No store of the layer's kernels stays in an L2: the NaN of a call that was given up, written by the block that
    leaves last, is then the last that reaches y."""
    kernel, seen, stores = None, set(), 0
    for line in _assembly(name, tmp_path).splitlines():
        label = re.match(r"(_Z\w+):", line)
        if label:
            kernel = label.group(1)
        m = re.match(r"\s*((?:global|flat|buffer)_store\w*)(.*)", line)
        if m and "k_moe_clear" not in kernel:
            assert re.search(r"\bsc1\b", m.group(2).split(";")[0]), (kernel, line)
            stores += 1
            if re.search(r"k_moe_(layer|one)", kernel):
                seen.add(kernel)
    assert len(seen) == kernels and stores > 40


@pytest.mark.parametrize("name", ["fp4_linear", "moe_layer", "moe_one"])
def test_no_matrix_instruction_writes_over_its_operands(name, tmp_path):
    cc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(cc):
        pytest.skip("hipcc not available")
    out = str(tmp_path / (name + ".s"))
    cmd = [cc] + B.FLAGS + ["-I" + os.path.join(B.HERE, "csrc"), "--cuda-device-only", "-S",
                            os.path.join(B.HERE, "csrc", name + ".hip"), "-o", out]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout[-2000:]
    with open(out) as f:
        found = re.findall(r"^\s*(v_mfma\S*)\s+([^,\s]+),\s*([^,\s]+),\s*([^,\s]+),", f.read(), flags=re.M)
    assert len(found) > 100
    for op, d, x, w in found:
        rd = _range(d)
        for o in (_range(x), _range(w)):
            assert rd[0] != o[0] or o[2] < rd[1] or rd[2] < o[1], (op, d, x, w)
