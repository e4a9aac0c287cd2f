"""The built device code against the wait states that inline assembly has to
keep by itself (tests/isa.py)."""
import os
import shutil

import pytest

import isa

pytestmark = [pytest.mark.cpu,
              pytest.mark.skipif(shutil.which(isa.OBJDUMP) is None, reason="needs llvm-objdump")]


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    from precision_rl_amd import build
    if not os.path.exists(build.LIB):
        build.build()
    return isa.disassemble(build.LIB, str(tmp_path_factory.mktemp("isa")))


def _listing(*lines):
    """A kernel of four-byte instructions."""
    return isa.parse("0 <k>:\n" + "".join(f"\t{t} // {4 * i:012X}: 0\n" for i, t in enumerate(lines)))[0][1]


def test_checker_sees_missing_wait_states():
    copy = "global_load_lds_dword v1, s[2:3]"
    assert [h[0] for h in isa.hazards(_listing("s_mov_b32 m0, s7", copy))] == ["M0"]
    assert not isa.hazards(_listing("s_mov_b32 m0, s7", "s_nop 0", copy))
    assert not isa.hazards(_listing("s_mov_b32 m0, s7", copy.replace("_lds", "")))   # reads no M0
    assert [h[0] for h in isa.hazards(_listing("v_readfirstlane_b32 s3, v0", "s_nop 3", copy))] == ["vector write"]
    assert not isa.hazards(_listing("v_readfirstlane_b32 s3, v0", "s_nop 4", copy))
    assert not isa.hazards(_listing("v_readfirstlane_b32 s4, v0", copy))
    # along a jump: the write at the end of a loop, the copy at its start
    assert [h[0] for h in isa.hazards(_listing(copy, "s_nop 7", "s_mov_b32 m0, s7", "s_cbranch_scc1 65532"))] == []
    assert [h[0] for h in isa.hazards(_listing(copy, "s_nop 7", "v_readfirstlane_b32 s3, v0",
                                               "s_cbranch_scc1 65532"))] == ["vector write"]


def test_copies_to_lds_keep_their_wait_states(kernels):
    copying = {n: c for n, c in kernels if any("_lds_" in i[1] for i in c)}
    assert len(copying) > 20
    bad = {n: h for n, c in copying.items() if (h := isa.hazards(c))}
    assert not bad, "\n".join(f"{n}: {len(h)} places, first {h[0]}" for n, h in bad.items())


def test_checker_sees_lds_reads_behind_a_barrier():
    read, wait = "ds_read_b128 v[0:3], v4", "s_waitcnt lgkmcnt(0)"
    assert isa.lds_outstanding_at_barriers(_listing(read, "s_barrier")) == [4]
    assert isa.lds_outstanding_at_barriers(_listing(read, read, "s_waitcnt lgkmcnt(1)", "s_barrier")) == [12]
    assert not isa.lds_outstanding_at_barriers(_listing(read, wait, "s_barrier"))
    # a read at the end of a loop whose barrier stands at its start
    assert isa.lds_outstanding_at_barriers(_listing("s_barrier", read, "s_cbranch_scc1 65533")) == [0]


def test_lds_reads_are_done_at_barriers(kernels):
    """Of every kernel that copies to LDS; in the dense MX product, whose next copies overwrite what
    was read last, by a wait directly in front of each barrier, which no order that the compiler gives
    the matrix instructions (and the waits for their operands) can open."""
    bad = {n: a for n, c in kernels if any("_lds_" in i[1] for i in c) and (a := isa.lds_outstanding_at_barriers(c))}
    assert not bad
    products = [(n, c) for n, c in kernels if "mx_linear_kernel" in n]
    assert len(products) >= 10
    for n, c in products:
        before = [c[k - 1] for k, i in enumerate(c) if i[1] == "s_barrier"]
        assert before and all(i[1] == "s_waitcnt" and "lgkmcnt(0)" in i[2] for i in before), n
