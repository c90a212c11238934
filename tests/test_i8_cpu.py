"""The int8 layers without a GPU: refusals of every entry point with the documented status
(before any HIP call), the workspace query, and pins of the oracle's quantizer, positions and
products that do not use its own code."""
import math
from fractions import Fraction

import numpy as np
import pytest

import oracle as O
import semi_structured_sparse_amd as S
import synth

P, Q, R = 1 << 20, 1 << 24, 1 << 28     # fake, aligned, never dereferenced
MIS = P + 4


def quant(**kw):
    a = dict(x=P, q=Q, scale=R, n=0, m=0, ns=2, rows=4, k=64, ldx=64, ldq=64)
    a.update(kw)
    return S.nm_quant_i8(a.pop("x"), a.pop("q"), a.pop("scale"), a.pop("n"), a.pop("m"), a.pop("ns"), stream=0,
                         check=False, **a)


def test_quant_refusals():
    assert quant(rows=0) == S.NM_OK
    assert quant(x=None) == S.NM_EINVAL
    assert quant(q=None) == S.NM_EINVAL
    assert quant(scale=None) == S.NM_EINVAL
    assert quant(m=-4) == S.NM_EINVAL
    assert quant(m=4, n=0) == S.NM_EINVAL
    assert quant(m=4, n=5) == S.NM_EINVAL
    assert quant(ns=1) == S.NM_EINVAL
    assert quant(ns=9) == S.NM_EINVAL
    assert quant(m=6, n=2) == S.NM_EUNSUPPORTED
    assert quant(m=8, n=4, ns=4) == S.NM_EUNSUPPORTED
    assert quant(rows=-1) == S.NM_ESHAPE
    assert quant(k=-1) == S.NM_ESHAPE
    assert quant(k=60, m=8, n=4) == S.NM_ESHAPE
    assert quant(k=60, ns=4) == S.NM_ESHAPE
    assert quant(ldx=56) == S.NM_ESHAPE
    assert quant(ldq=48) == S.NM_ESHAPE
    assert quant(k=50, ldx=56, ldq=48) == S.NM_ESHAPE            # rounded up to 16: 64
    assert quant(ns=4, ldq=80) == S.NM_ESHAPE                     # lifted: 96
    assert quant(rows=1 << 62, ldx=1 << 20) == S.NM_ESHAPE
    assert quant(ldx=68) == S.NM_EALIGN
    assert quant(ldq=72) == S.NM_EALIGN
    assert quant(x=MIS) == S.NM_EALIGN
    assert quant(q=MIS) == S.NM_EALIGN
    assert quant(scale=MIS) == S.NM_EALIGN
    assert quant(k=65552, ldx=65552, ldq=65552) == S.NM_EUNSUPPORTED
    assert quant(rows=1 << 31) == S.NM_EUNSUPPORTED


def test_meta_block_refusals():
    f = lambda meta, o, kc, out: S.nm_meta_block(meta, o, kc, out, stream=0, check=False)  # noqa: E731
    assert f(P, 0, 64, Q) == S.NM_OK
    assert f(P, 4, 0, Q) == S.NM_OK
    assert f(None, 4, 64, Q) == S.NM_EINVAL
    assert f(P, 4, 64, None) == S.NM_EINVAL
    assert f(P, 4, 62, Q) == S.NM_ESHAPE
    assert f(P, -1, 64, Q) == S.NM_ESHAPE
    assert f(P, 4, -4, Q) == S.NM_ESHAPE
    assert f(MIS, 4, 64, Q) == S.NM_EALIGN
    assert f(P, 4, 64, MIS) == S.NM_EALIGN
    assert S.nm_meta_block_bytes(5, 128) == 80 and S.nm_meta_block_bytes(5, 132) == 160
    assert S.nm_meta_block_bytes(0, 128) == 0 and S.nm_meta_block_bytes(5, 0) == 0


def spmm(**kw):
    a = dict(x=P, x_scale=P, w=Q, w_scale=P, y=R, t=4, o=8, k=64, ldx=64, ldw=64, ldy=8, y_dtype=0, stream=0, check=False)
    a.update(kw)
    return S.nm_spmm_i8(a.pop("x"), a.pop("x_scale"), a.pop("w"), a.pop("w_scale"), a.pop("y"), **a)


def glu(**kw):
    a = dict(x=P, x_scale=P, wg=Q, gs=P, wu=Q, us=P, y=R, t=4, inter=8, k=64, ldx=64, ldw=64, ldy=8, y_dtype=0, stream=0,
             check=False)
    a.update(kw)
    return S.nm_glu_i8(a.pop("x"), a.pop("x_scale"), a.pop("wg"), a.pop("gs"), a.pop("wu"), a.pop("us"), a.pop("y"), **a)


@pytest.mark.parametrize("call,weight", [(spmm, "w"), (glu, "wg")])
def test_product_refusals(call, weight):
    o = "o" if call is spmm else "inter"
    assert call(t=0) == S.NM_OK
    assert call(**{o: 0}) == S.NM_OK
    for name in ("x", "x_scale", weight, "y") + (("w_scale",) if call is spmm else ("gs", "us", "wu")):
        assert call(**{name: None}) == S.NM_EINVAL, name
        assert call(**{name: MIS}) == S.NM_EALIGN, name
    assert call(y_dtype=2) == S.NM_EINVAL
    assert call(t=-1) == S.NM_ESHAPE
    assert call(k=-1) == S.NM_ESHAPE
    assert call(**{o: -1}) == S.NM_ESHAPE
    assert call(ldx=48) == S.NM_ESHAPE
    assert call(ldw=48) == S.NM_ESHAPE
    assert call(ldy=7) == S.NM_ESHAPE
    assert call(t=1 << 61, ldx=1 << 10) == S.NM_ESHAPE
    assert call(workspace=P, workspace_bytes=-1) == S.NM_ESHAPE
    assert call(ldx=72) == S.NM_EALIGN
    assert call(ldw=72) == S.NM_EALIGN
    assert call(workspace=MIS, workspace_bytes=64) == S.NM_EALIGN
    big = S.NM_I8_MAX_K + 1
    assert call(k=big, ldx=big, ldw=big) == S.NM_EUNSUPPORTED
    assert call(t=S.NM_I8_MAX_ROWS + 1) == S.NM_EUNSUPPORTED
    assert call(**{o: S.NM_I8_MAX_ROWS + 1, "ldy": 1 << 31, "t": 1}) == S.NM_EUNSUPPORTED
    assert call(t=1 << 31) == S.NM_EUNSUPPORTED
    assert call(**{o: 1 << 31, "ldy": 1 << 31, "t": 1}) == S.NM_EUNSUPPORTED


def test_product_refusals_of_one_call():
    assert spmm(accumulate=2) == S.NM_EINVAL
    assert spmm(accumulate=1, y_dtype=S.NM_Y_BF16) == S.NM_EUNSUPPORTED
    assert spmm(row_shift=P) == S.NM_EINVAL
    assert spmm(col_shift=MIS) == S.NM_EALIGN
    assert spmm(row_shift=MIS, col_shift=P) == S.NM_EALIGN
    assert spmm(w_meta=MIS) == S.NM_EALIGN
    assert spmm(w_meta=P, k=62) == S.NM_ESHAPE
    assert spmm(w_meta=P, ldw=16) == S.NM_ESHAPE              # 32 values a row
    assert glu(act=2) == S.NM_EINVAL
    assert glu(gate_meta=P) == S.NM_EINVAL                    # both weights 2:4, or neither
    assert glu(up_meta=P) == S.NM_EINVAL
    assert glu(gate_meta=P, up_meta=MIS) == S.NM_EALIGN


def test_workspace_query():
    for sparse in (False, True):
        for is_glu in (False, True):
            q = lambda t, o, k: S.nm_i8_workspace_size(t, o, k, sparse, is_glu)  # noqa: E731,B023
            assert q(0, 8, 64) == 0 and q(4, 0, 64) == 0 and q(4, 8, 0) == 0
            assert q(4, 8, S.NM_I8_MAX_K + 1) == 0 and q(1 << 62, 1 << 62, 64) == 0
            for t in (1, 17, 64, 200, 1000, 8192):
                for o in (1, 100, 1024, 4096):
                    n = q(t, o, 14336)
                    mats = 2 if is_glu else 1
                    per = mats * t * (-(-o // 4) * 4) * 4       # one split's partial sums
                    assert n % per == 0 and n // per != 1, (t, o, n, per)


# ------------------------------------------------------------------- pins of the oracle ---

def test_codes_are_the_exact_quotients_rounded_half_even():
    rng = np.random.default_rng(5)
    rows = [synth.student_t_bf16(rng, (6, 96), 4.0, 0.5)]
    # every significand pair: 127 a / b for all 128 x 128 of them, a few exponents apart
    a = (np.arange(128, dtype=np.uint16) + 0x3F80)
    for e in (0, 1, 2, 7):
        for b in range(0, 128, 9):
            row = (a - np.uint16(e * 128)).copy()
            row = np.minimum(row, np.uint16(0x3F80 + b))
            row[0] = 0x3F80 + b
            rows.append(np.pad(row, (0, 0))[None, :96])
            rows.append(row[None, 32:])
    tiny = np.array([[0x0001, 0x8001, 0x0002, 0x0000] * 24, [0x7F7F, 0xFF7F, 0x3F80, 0x0001] * 24], np.uint16)
    rows.append(tiny)
    ties = 0
    for block in rows:
        codes, scale = O.quantize_rows_i8(block)
        vals = O.bf16_to_f64(block)
        for r in range(block.shape[0]):
            top = max(abs(Fraction(float(v))) for v in vals[r])
            for c, v in zip(codes[r], vals[r]):
                ex = 127 * Fraction(float(v)) / top
                ties += (2 * ex).denominator == 1 and ex.denominator == 2
                assert int(c) == round(ex)                     # Python rounds halves to even
            assert abs(Fraction(float(scale[r])) - top / 127) <= top / 127 * Fraction(1, 1 << 24) + Fraction(1, 1 << 150)
    assert ties > 10


def test_zero_and_nonfinite_rows():
    x = np.array([[0, 0x8000, 0, 0], [0x7F80, 0x3F80, 0, 0], [0x7FC0, 0xFF80, 0x3F80, 0], [0x3F80, 0xBF80, 0, 0]], np.uint16)
    q, s = O.quantize_rows_i8(x)
    assert (q[:3] == 0).all() and q[3].tolist() == [127, -127, 0, 0]
    assert s[0] == 1 and np.isinf(s[1]) and np.isnan(s[2]) and s[3] == np.float32(1 / 127)


def test_selected_and_lifted_codes():
    rng = np.random.default_rng(6)
    x = synth.student_t_bf16(rng, (3, 48), 4.0, 0.5)
    q, s = O.quantize_rows_i8(x)
    sx, _ = O.sparsify(x, 8, 16)
    qs, ss = O.quantize_rows_i8(x, 8, 16)
    qz, sz = O.quantize_rows_i8(sx)               # the selection keeps the largest: same scale
    assert (qs == qz).all() and (ss == sz).all() and (s == ss).all()
    ql, sl = O.quantize_rows_i8(x, ns=4)
    for t in range(3):
        for j in range(ql.shape[1]):
            g, r = divmod(j, 12)
            assert ql[t, j] == q[t, 8 * g + 2 * (r // 4) + r % 4]
    assert ql.shape[1] == 72 and (sl == s).all()


def test_blocked_positions_and_expanded_weights():
    rng = np.random.default_rng(7)
    for kc in (4, 60, 128, 132, 260):
        w = synth.normal_bf16(rng, (5, kc))
        v, idx = O.compress(w, 2, 4)
        meta = O.pack_meta_2bit(idx)
        blk = O.block_meta(meta, kc)
        assert blk.shape == (math.ceil(kc / 128), 5, 16)
        flat = np.transpose(blk, (1, 0, 2)).reshape(5, -1)
        slots = np.stack([(flat >> (2 * i)) & 3 for i in range(4)], axis=2).reshape(5, -1)
        assert (slots[:, :kc // 2] == idx).all()
        assert (slots[:, kc // 2:].reshape(5, -1, 2) == [0, 1]).all()
        codes, _ = O.quantize_rows_i8(v)
        dense = O.expand_24(codes, idx, kc)
        back = O.decompress(v, idx, 2, 4, kc)
        assert ((dense != 0) <= (O.bf16_to_f64(back) != 0)).all()
        keep = O.select_keep(w, 2, 4)
        assert (dense[~keep] == 0).all()
        assert (np.sort(np.abs(dense[keep])) == np.sort(np.abs(codes.astype(np.int64)).ravel())).all()


def test_sums_are_exact_integers():
    rng = np.random.default_rng(8)
    x = rng.integers(-128, 128, (3, 50)).astype(np.int8)
    w = rng.integers(-128, 128, (4, 50)).astype(np.int8)
    got = O.sums_i8(x, w)
    for t in range(3):
        for o in range(4):
            assert int(got[t, o]) == sum(int(a) * int(b) for a, b in zip(x[t], w[o]))
    g = np.array([-3.0, 0.0, 2.0])
    for v, z in zip(g, O.glu_gate(g, "gelu")):
        assert abs(z - 0.5 * v * (1 + math.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))) < 1e-15


def test_binding_refuses_tensors_that_are_not_on_the_gpu_or_do_not_fit():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError, match="current GPU"):
        S.nm_quant_i8(x, q, s, stream=0)
    with pytest.raises(ValueError, match="current GPU"):
        S.nm_spmm_i8(q, s, q, s, torch.zeros(4, 4), stream=0)
    with pytest.raises(ValueError, match="current GPU"):
        S.nm_glu_i8(q, s, q, s, q, s, torch.zeros(4, 4), stream=0)
    with pytest.raises(ValueError, match="current GPU"):
        S.nm_meta_block(q, 4, 64, q, stream=0)


def test_errors_raise_by_default():
    with pytest.raises(S.NMError, match="NM_EINVAL"):
        S.nm_spmm_i8(P, None, Q, P, R, t=1, o=1, k=16, ldx=16, ldw=16, ldy=1, stream=0)
    with pytest.raises(S.NMError, match="NM_EALIGN"):
        S.nm_quant_i8(MIS, Q, R, rows=1, k=16, ldx=16, ldq=16, stream=0)
