"""Tiles of the 8-bit calls whose operands go through LDS stages that buffer loads
fill: behind a barrier a stage is loaded again that the step before it has read, so
no wave may pass the barrier with operand reads under way.  Shown in the assembly of
the sources, compiled here: LDS operations end in the order they are issued, and an
lgkmcnt(n) leaves the last n of them."""
import concurrent.futures as cf
import os
import re
import shutil
import subprocess

import pytest

from bit_nf4_quantized_07_amd import build as b

SOURCES = ["int8_adapter_kernels.hip", "int8_fwd_kernels.hip", "int8_dx_kernels.hip"]

if not (os.path.exists("/opt/rocm/bin/hipcc") or shutil.which("hipcc")):
    pytest.skip("needs hipcc", allow_module_level=True)


def _assembly(src, out):
    subprocess.run([b.hipcc(), *b.COMMON, "-S", "--offload-device-only", "-o", str(out),
                    os.path.join(b.CSRC, src)], check=True, capture_output=True)
    return out.read_text()


def _kernels(text):
    """name -> instructions of every kernel that loads into LDS."""
    found = {}
    for name in re.findall(r"^\s*\.amdhsa_kernel (\S+)", text, re.M):
        body = re.search(rf"^{re.escape(name)}:.*?^\.Lfunc_end", text, re.M | re.S).group(0)
        if re.search(r"buffer_load_\w+ .*\blds\b", body):
            found[name] = [l.strip() for l in body.splitlines()]
    return found


def reads_under_way(instructions):
    """For every barrier, the LDS reads that the wave has not waited for."""
    pending, at = [], []
    for i in instructions:
        if i.startswith("ds_"):
            pending.append(i)
        elif i.startswith("s_waitcnt"):
            n = re.search(r"lgkmcnt\((\d+)\)", i)
            if n:
                pending = pending[max(0, len(pending) - int(n.group(1))):]
        elif i.startswith("s_barrier"):
            at.append([p for p in pending if p.startswith("ds_read")])
    return at


def test_the_scan_itself():
    read, wait = "ds_read_b128 v[0:3], v4", "s_waitcnt vmcnt(6) lgkmcnt(1)"
    assert reads_under_way([read, "s_waitcnt lgkmcnt(0)", "s_barrier"]) == [[]]
    assert reads_under_way([read, "s_waitcnt vmcnt(6)", "s_barrier"]) == [[read]]
    assert reads_under_way([read, read, wait, "s_barrier"]) == [[read]]
    assert reads_under_way([read, "ds_write_b32 v0, v1", wait, "s_barrier"]) == [[]]
    assert reads_under_way([read, "s_waitcnt lgkmcnt(4)", "s_barrier"]) == [[read]]


def test_no_operand_read_crosses_a_barrier(tmp_path):
    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        texts = list(ex.map(lambda s: _assembly(s, tmp_path / (s + ".s")), SOURCES))
    checked = 0
    for src, text in zip(SOURCES, texts):
        kernels = _kernels(text)
        assert kernels, src
        for name, body in kernels.items():
            at = reads_under_way(body)
            assert at, (src, name)
            checked += len(at)
            assert not any(at), (src, name, [a for a in at if a])
    assert checked
