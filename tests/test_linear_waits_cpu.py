"""The bf16 tile kernels with an epilogue on the compiler's gfx950 assembly (no GPU): their hand-set
memory waits, and what the large kernels keep the compiler from knowing.

Requests complete in issue order.  A ring of NST stages waits, each step, for all but the requests
of the NST - 2 steps behind the one it reads next, L a wave and step.  k_lin_big waits, each of a
step's four phases, for all but the four requests of each of the last six phases: the region that
the next phase reads was requested in the seventh.  k_lin_big24 waits for all but one step's.

A stage or region is requested into again one barrier after it was read, so at every barrier all LDS
reads before it must have been waited for (lgkmcnt(0)).  (A row that ends inside a piece is made up
in LDS before its step is read: a branch of each loop, with waits and barriers of its own.)

The large kernels multiply in inline assembly on the accumulator half of the register file: their
loops must hold every sum where it is, an operand must be two issue slots old, and the first read
of a sum must lie 19 issue slots (a 16-pass matrix instruction's latency towards a vector
instruction) behind the last product."""
import re

import pytest

from test_i8_waits_cpu import _reads_at_barriers
from test_wait_counts_cpu import _assembly, _functions, _loops, _template_ints


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    return _assembly("linear_tile.hip", tmp_path_factory.mktemp("asm"))


def _code(lines):
    out = [ln.split(";")[0].strip() for ln in lines]
    return [ln for ln in out if ln and not ln.startswith(".")]


def _regions(lines):
    """Code of every loop: from a label to a branch back to it, the smallest first.  (The branch that makes
    up a ragged row has loops of its own inside.)"""
    at, out = {}, []
    for i, ln in enumerate(lines):
        m = re.match(r"^(\.LBB\w+):", ln)
        if m:
            at[m.group(1)] = i
        m = re.match(r"^\s*s_c?branch\w*\s+(\.LBB\w+)", ln)
        if m and m.group(1) in at:
            out.append(lines[at[m.group(1)] + 1:i + 1])
    return [_code(c) for c in sorted(out, key=len)]


def _requests(code):
    return sum(ln.startswith("global_load_lds_") or (ln.startswith("buffer_load_") and ln.endswith(" lds")) for ln in code)


def _vm_waits(code):
    return [int(m.group(1)) for ln in code for m in [re.search(r"s_waitcnt.*vmcnt\((\d+)\)", ln)] if m]


def _other_memory(code):
    return [ln for ln in code if ln.startswith(("global_", "buffer_", "flat_", "scratch_"))
            and not (ln.startswith("global_load_lds_") or ln.endswith(" lds"))]


def test_reads_are_complete_at_barriers(asm):
    kernels = _functions(asm, "k_lin_tileI") + _functions(asm, "k_lin_big")
    assert len(kernels) == 10
    for name, body in kernels:
        assert _reads_at_barriers(body) == 0, name
        for lp in _loops(body):
            assert _reads_at_barriers(lp) == 0, name


def test_ring_waits_cover_their_stage(asm):
    # <BM, BN, WM, WN, SP, NST, KM>
    kernels = _functions(asm, "k_lin_tileI")
    assert len(kernels) == 8    # four tile shapes, dense and 2:4
    for name, body in kernels:
        bm, bn, wm, wn, sp, nst, km = _template_ints(name)
        per_step = km * (bm // (16 if sp else 8) // (wm * wn) + bn // 8 // (wm * wn)) + sp
        rings = [c for c in _regions(body) if _requests(c)]
        assert rings, name
        ring = rings[0]
        assert _requests(ring) == nst * per_step, (name, _requests(ring))
        waits = _vm_waits(ring)
        assert waits and all(n <= per_step * (nst - 2) for n in waits), (name, waits)
        assert len([n for n in waits if n == per_step * (nst - 2)]) >= nst, (name, waits)
        assert not _other_memory(ring), name


def _large(asm, name, product, products):
    kernels = [(n, b) for n, b in _functions(asm, name) if n.count("k_lin_big24") == (name == "k_lin_big24")]
    assert len(kernels) == 1
    body = kernels[0][1]
    loops = [c for c in _regions(body) if any(product in ln for ln in c)]
    assert loops and sum(product in ln for ln in loops[0]) == products
    assert not _other_memory(loops[0]) and not any("accvgpr" in ln for ln in loops[0])
    code = _code(body)
    at = [i for i, ln in enumerate(code) if ln.startswith(product)]
    assert all(code[i - 1] == "s_nop 1" for i in at)
    reads = [i for i, ln in enumerate(code) if ln.startswith("v_accvgpr_read")]
    assert reads and min(reads) > max(at), "a sum read before the last product"
    slots = sum(1 + (int(ln.split()[1]) if ln.startswith("s_nop") else 0) for ln in code[max(at) + 1:reads[0]])
    assert slots >= 19, slots
    assert not any(ln.startswith("scratch_") for ln in code)
    return loops[0]


def test_large_dense_loop(asm):
    loop = _large(asm, "k_lin_big", "v_mfma", 128)             # two steps of 64
    assert _requests(loop) == 2 * 4 * 4
    waits = _vm_waits(loop)
    assert all(n <= 24 for n in waits) and waits.count(24) == 8, waits


def test_large_sparse_loop(asm):
    loop = _large(asm, "k_lin_big24", "v_smfmac", 96)          # three steps of 32
    assert _requests(loop) == 3 * 14
    waits = _vm_waits(loop)
    assert all(n <= 14 for n in waits) and waits.count(14) == 3, waits
