"""The k loops of the 8-bit product and of the products grouped by expert, as compiled (CPU,
hipcc): one full wait for the global->LDS loads per tile of the contraction, at the barrier.  A
read of LDS that the compiler cannot tell apart from those loads' target (a transposing read, or
a byte, without alias information) makes it wait for them again at every such read, with
identical results and up to half the speed -- so no parity test would notice."""

import os
import re
import shutil
import subprocess

import pytest

from collective_overlap_amd import build


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    """The device assembly of a source, compiled once."""
    done = {}

    def get(name):
        if name not in done:
            done[name] = _asm(tmp_path_factory.mktemp("asm"), name)
        return done[name]
    return get


def _asm(tmp, name):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("no hipcc")
    out = tmp / (name + ".s")
    cmd = [hipcc, *build.COMMON, "-x", "hip", "-S", "--cuda-device-only",
           os.path.join(build.CSRC, name + ".hip"), "-o", str(out)]
    r = subprocess.run([c for c in cmd if c != "-fPIC"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return out.read_text()


def _body(text, name):
    i = text.index("\n" + name + ":")
    return text[i:text.index(".Lfunc_end", i)]


def _loop_blocks(body, mfmas):
    """The kernel's blocks with matrix instructions: its k loop, in one or a few pieces."""
    blocks = [b for b in re.split(r"^\.LBB\S+:.*$", body, flags=re.M) if "v_mfma" in b]
    assert sum(b.count("v_mfma") for b in blocks) == mfmas
    return blocks


@pytest.mark.parametrize("source,kernel,tile,mfmas", [
    ("ragged", "ragged_kernel", "Li256ELi256E", 64), ("ragged", "ragged_kernel", "Li128ELi128E", 16),
    ("gemm8", "gemm8_kernel", "Li256ELi256E", 32), ("gemm8", "gemm8_kernel", "Li128ELi128E", 8)])
def test_one_full_wait_per_tile(asm, source, kernel, tile, mfmas):
    text = asm(source)
    names = [n for n in re.findall(r"^(_ZN3cce12_GLOBAL__N_1\S+):", text, re.M) if kernel + "I" + tile in n]
    assert len(names) >= 2
    for name in names:
        waits = []
        for block in _loop_blocks(_body(text, name), mfmas):
            first = block.index("v_mfma")     # (the wait of the stage before belongs to the prologue)
            waits += re.findall(r"s_waitcnt [^\n]*vmcnt\((\d+)\)", block[first:])
        assert waits in (["0"], []), f"{name}: {waits}"
