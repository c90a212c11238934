"""The int8 tile kernels on the compiler's gfx950 assembly (no GPU): their hand-set memory waits,
and what the large 2:4 kernel keeps the compiler from knowing.

A ring of NST stages has the requests of NST - 1 steps outstanding, each wave L of them a step.
Requests complete in issue order, so a wait before a step may leave at most the requests
issued after that step's: those of the NST - 2 steps behind it.  The loops are replayed and every
vmcnt wait is held against that count.

A stage is requested into again one barrier after it was read, so at every barrier of a loop all
LDS reads before it must have been waited for (lgkmcnt(0)).

k_i8_big multiplies in inline assembly on the accumulator half of the register file.  Its loop
must hold every sum where it is (no move between the register halves, no scratch), and the first
read of a sum after the loop must lie 19 issue slots (a 16-pass matrix instruction's latency
towards a vector instruction) behind the last product.
"""
import re

import pytest

from test_wait_counts_cpu import _assembly, _check_ring_loop, _functions, _loops, _template_ints


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    return _assembly("gemm_i8.hip", tmp_path_factory.mktemp("asm"))


def _events(body):
    ev = []
    for line in body:
        t = line.split(";")[0].strip()
        if t.startswith("global_load_lds_") or (t.startswith("buffer_load_") and t.endswith(" lds")):
            ev.append(("load",))
        elif t.startswith("s_barrier"):
            ev.append(("bar",))
        elif t.startswith("s_waitcnt"):
            m = re.search(r"vmcnt\((\d+)\)", t)
            if m:
                ev.append(("wait", int(m.group(1))))
        elif t.startswith(("global_", "buffer_", "flat_", "scratch_")):
            ev.append(("vload",))
    return ev


def _reads_at_barriers(body):
    """LDS reads that no lgkmcnt wait has covered when a barrier is reached, the most of any."""
    out, most = 0, 0
    for line in body * 2:
        t = line.split(";")[0].strip()
        if t.startswith("ds_read"):
            out += 1
        elif t.startswith("s_waitcnt"):
            m = re.search(r"lgkmcnt\((\d+)\)", t)
            if m:
                out = min(out, int(m.group(1)))
        elif t.startswith("s_barrier"):
            most = max(most, out)
    return most


def test_reads_are_complete_at_barriers(asm):
    n = 0
    for name, body in _functions(asm, "k_i8_tileI") + _functions(asm, "k_i8_bigI"):
        assert _reads_at_barriers(body) == 0, name
        for lp in _loops(body):
            assert _reads_at_barriers(lp) == 0, name
        n += 1
    assert n == 20


def _rings(body):
    """Events of the loops that request into LDS and wait at barriers, three steps or more a trip."""
    evs = [_events(lp) for lp in _loops(body)]
    return [e for e in evs if ("load",) in e and e.count(("bar",)) >= 3]


def test_ring_waits_cover_their_stage(asm):
    # <BM, BN, WM, WN, SP, GLU, NST>
    kernels = [(n, b) for n, b in _functions(asm, "k_i8_tileI") if _template_ints(n)[6] >= 3]
    assert len(kernels) == 16   # four tile shapes, dense and 2:4, one weight and two
    for name, body in kernels:
        bm, bn, wm, wn, sp, _, nst = _template_ints(name)
        nw = wm * wn
        per_step = bm // (16 if sp else 8) // nw + bn // 8 // nw + sp
        rings = _rings(body)
        assert len(rings) == 1, name
        ev = rings[0]
        assert ev.count(("bar",)) == nst and ev.count(("load",)) == nst * per_step, name
        assert ("vload",) not in ev, f"{name}: another memory operation in the loop"
        assert sum(e[0] == "wait" for e in ev) >= nst
        assert _check_ring_loop(ev, nst, name) >= nst


def test_large_sparse_loop(asm):
    kernels = _functions(asm, "k_i8_bigI")
    assert len(kernels) == 2
    for name, body in kernels:
        loops = [lp for lp in _loops(body) if sum("v_smfmac" in ln for ln in lp) == 96]   # three steps of 32
        assert len(loops) == 1, name
        ev = _events(loops[0])
        # 13 requests a step; a step's wait comes before its own, so the loads since the last
        # barrier are those of the stage after the one it waits for
        assert ev.count(("load",)) == 39 and ev.count(("bar",)) == 3 and ("vload",) not in ev
        assert _check_ring_loop(ev, 3, name) >= 3
        for ln in loops[0]:
            assert "accvgpr" not in ln and "scratch_" not in ln, (name, ln)
        code = [ln.split(";")[0].strip() for ln in body]
        code = [ln for ln in code if ln and not ln.startswith((".", "s_cbranch"))]
        last = max(i for i, ln in enumerate(code) if ln.startswith("v_smfmac"))
        reads = [i for i, ln in enumerate(code) if ln.startswith("v_accvgpr_read")]
        assert reads and min(reads) > last, f"{name}: a sum read before the last product"
        slots = sum(1 + (int(ln.split()[1]) if ln.startswith("s_nop") else 0) for ln in code[last + 1:reads[0]])
        assert slots >= 19, (name, slots)


def test_products_follow_no_vector_write_at_once(asm):
    """Two issue slots lie between any product of k_i8_big and the instruction before it (an
    operand it reads may just have been written)."""
    for name, body in _functions(asm, "k_i8_bigI"):
        code = [ln.split(";")[0].strip() for ln in body]
        code = [ln for ln in code if ln and not ln.startswith(".")]
        at = [i for i, ln in enumerate(code) if ln.startswith("v_smfmac")]
        assert at and all(code[i - 1] == "s_nop 1" for i in at), name
