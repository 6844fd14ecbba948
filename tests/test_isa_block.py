"""What the block operators' compiled kernels rely on (CPU only: hipcc cross-compiles gfx950 device code): the
direct-to-LDS loads' hand-counted waits, and register stages that stay in registers.

A direct load writes M0 and is not counted by the compiler, so M0 belongs to inline assembly alone.  The router's
tile kernel waits with loads of later stages in flight, so no other vector-memory load may stand among its
own.  A kernel that spills, or loads its pointers through memory in its loop, drains the ring it streams with.
"""
import os
import re
import subprocess

import pytest

from routed_expert_grouped_amd import build
from test_isa import _VMEM, _code

pytestmark = pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="hipcc not available")

FILES = ("moe_norm.hip", "moe_router.hip", "moe_few.hip", "moe_linear.hip")
LDS = 160 * 1024


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    out = {}
    procs = []
    for f in FILES:
        src, dst = os.path.join(build.CSRC, f), tmp_path_factory.mktemp("isa") / (f + ".s")
        procs.append((dst, subprocess.Popen([build.HIPCC, *build.flags_for(src), "-S", "--cuda-device-only", "-o",
                                             str(dst), src], stderr=subprocess.DEVNULL)))
    for dst, p in procs:
        assert p.wait() == 0, dst
        out[dst.name[:-2]] = dst.read_text()
    return out


def functions(text):
    return {m.group(1): m.group(2).splitlines()
            for m in re.finditer(r"^(_Z\w+):[^\n]*\n(.*?)^\.Lfunc_end", text, re.S | re.M)}


def test_no_spills_and_lds_within_a_cu(asm):
    kernels = 0
    for f, text in asm.items():
        for m in re.finditer(r"\.group_segment_fixed_size: (\d+)(.*?)\.vgpr_spill_count: (\d+)", text, re.S):
            kernels += 1
            assert int(m.group(1)) <= LDS and int(m.group(3)) == 0, f
        assert not re.search(r"\bscratch_(load|store)", text), f
    assert kernels >= 40


def test_m0_only_in_inline_asm(asm):
    checked = 0
    for f in ("moe_router.hip", "moe_linear.hip"):
        for name, lines in functions(asm[f]).items():
            bad = [t for t, inasm in _code(lines) if not inasm and re.search(r"\bm0\b", t)]
            assert not bad, (name, bad[:5])
            checked += any(t.startswith("global_load_lds") for t, _ in _code(lines))
    assert checked == 6  # three widths of the router's tiles, three of the projection's


def test_router_tiles_have_no_other_loads_among_the_direct_ones(asm):
    checked = 0
    for name, lines in functions(asm["moe_router.hip"]).items():
        if "router_dma_kernel" not in name:
            continue
        checked += 1
        code = [t for t, _ in _code(lines)]
        dma = [i for i, t in enumerate(code) if t.startswith("global_load_lds")]
        inside = [t for t in code[dma[0]:dma[-1] + 1] if _VMEM.match(t) and not t.startswith("global_load_lds")
                  and not re.match(r"(global|buffer|flat)_store", t)]
        assert not inside, (name, inside[:5])
    assert checked == 3


def test_streams_take_their_pointers_from_registers(asm):
    """No flat loads in the streaming kernels: a pointer chosen by value is a global-memory pointer."""
    checked = 0
    for f, kernel in (("moe_few.hip", "few_"), ("moe_linear.hip", "linear_stream_kernel")):
        for name, lines in functions(asm[f]).items():
            if kernel in name:
                checked += 1
                bad = [t for t, _ in _code(lines) if t.startswith("flat_load")]
                assert not bad, (name, bad[:3])
    assert checked == 6 + 18 + 9
