"""No matrix instruction of the attention kernels writes its result over an operand
(kernels of this library that had that in the 16x16x32 form have given wrong
outputs), and what goes straight to LDS is waited for before it is read."""
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


@pytest.mark.parametrize("name", ["kv4_attend", "prompt_attention"])
def test_no_matrix_instruction_writes_over_its_operands(name, tmp_path):
    found = re.findall(r"^\s*(v_mfma\S*)\s+([^,\s]+),\s*([^,\s]+),\s*([^,\s]+),", _assembly(name, tmp_path), flags=re.M)
    assert len(found) > 100
    for op, d, x, w in found:
        rd = _range(d)
        for o in (_range(x), _range(w)):
            assert rd[0] != o[0] or o[2] < rd[1] or rd[2] < o[1], (op, d, x, w)


def test_loads_to_lds_are_waited_for(tmp_path):
    """After every load to LDS each path to a barrier has a wait for all loads; in program order it is enough that
    the next barrier behind one has such a wait between."""
    waiting, loads = False, 0
    for line in _assembly("prompt_attention", tmp_path).splitlines():
        line = line.strip()
        if re.match(r"buffer_load_dwordx4 .*\blds\b", line):
            waiting, loads = True, loads + 1
        elif re.match(r"s_waitcnt\b.*vmcnt\(0\)", line):
            waiting = False
        elif line.startswith("s_barrier"):
            assert not waiting, line
    assert loads > 50


def test_kernels_that_load_to_lds_have_no_other_lds(tmp_path):
    """The address that such a load takes has 16 bits, and the tiles have all of them."""
    text = _assembly("prompt_attention", tmp_path)
    kernels = re.findall(r"\.amdhsa_kernel (\S*k_promptI\S*).*?\.amdhsa_group_segment_fixed_size (\d+)", text, flags=re.S)
    assert len(kernels) > 10
    for name, size in kernels:
        assert size == "0", name
