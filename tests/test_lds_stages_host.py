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


def loads_under_way(instructions):
    """For every barrier, the loads into LDS that the wave has not waited for."""
    pending, at = [], []
    for i in instructions:
        if re.match(r"(buffer|global|flat|scratch)_(load|store|atomic)", i):
            pending.append(i)
        elif i.startswith("s_waitcnt"):
            n = re.search(r"vmcnt\((\d+)\)", i)
            if n:
                pending = pending[max(0, len(pending) - int(n.group(1))):]
        elif i.startswith("s_barrier"):
            at.append([p for p in pending if re.search(r"\blds\b", p)])
    return at


def test_the_scan_itself():
    read, wait = "ds_read_b128 v[0:3], v4", "s_waitcnt vmcnt(6) lgkmcnt(1)"
    assert reads_under_way([read, "s_waitcnt lgkmcnt(0)", "s_barrier"]) == [[]]
    assert reads_under_way([read, "s_waitcnt vmcnt(6)", "s_barrier"]) == [[read]]
    assert reads_under_way([read, read, wait, "s_barrier"]) == [[read]]
    assert reads_under_way([read, "ds_write_b32 v0, v1", wait, "s_barrier"]) == [[]]
    assert reads_under_way([read, "s_waitcnt lgkmcnt(4)", "s_barrier"]) == [[read]]
    fill, load = "buffer_load_dwordx4 v2, s[28:31], 0 offen lds", "buffer_load_dwordx4 v[6:9], v2, s[24:27], 0 offen"
    assert loads_under_way([fill, load, "s_waitcnt vmcnt(1)", "s_barrier"]) == [[]]
    assert loads_under_way([fill, load, "s_waitcnt vmcnt(2) lgkmcnt(0)", "s_barrier"]) == [[fill]]
    assert loads_under_way([load, fill, "s_waitcnt vmcnt(1)", "s_barrier"]) == [[fill]]


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """source -> its kernels that load into LDS"""
    d = tmp_path_factory.mktemp("assembly")
    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        texts = ex.map(lambda s: _assembly(s, d / (s + ".s")), SOURCES)
    return {src: _kernels(text) for src, text in zip(SOURCES, texts)}


@pytest.mark.parametrize("src", SOURCES)
def test_no_operand_read_crosses_a_barrier(kernels, src):
    assert kernels[src]
    for name, body in kernels[src].items():
        at = reads_under_way(body)
        assert at and not any(at), (name, [a for a in at if a])


def test_single_tokens_have_landed(kernels):
    """The tokens' columns are waited for by counting the weight's loads behind them:
    those have to have been issued by then."""
    found = {n: b for n, b in kernels["int8_fwd_kernels.hip"].items() if "gemv" in n}
    assert len(found) == 4
    for name, body in found.items():
        at = loads_under_way(body)
        assert at and not any(at), (name, [a for a in at if a])
