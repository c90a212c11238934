"""The norm to int8 codes and the routing of experts without a GPU: refusals with the documented
status, what the binding accepts of its tensors (the library replaced by a recorder), and pins of
the oracle that do not use its own code."""
import math
from fractions import Fraction

import numpy as np
import pytest

import oracle as O
import semi_structured_sparse_amd as S
from test_i8_binding_cpu import Recorder, bf16, calls, i8, refused, taken  # noqa: F401

torch = pytest.importorskip("torch")

P, Q, R, U, V, W = (1 << 20), (1 << 24), (1 << 28), (1 << 30), (1 << 31), (1 << 32)   # fake, never dereferenced
MIS = P + 4


def norm(**kw):
    a = dict(x=P, weight=W, q=Q, scale=R, residual=U, sum_out=V, y=P + 4096, rows=4, k=64, ldx=64, ldr=64, lds=64, ldy=64,
             ldq=64)
    a.update(kw)
    return S.nm_rmsnorm_i8(a.pop("x"), a.pop("weight"), a.pop("q"), a.pop("scale"), stream=0, check=False, **a)


def test_norm_refusals():
    assert norm(rows=0) == S.NM_OK
    for name in ("x", "q", "scale"):
        assert norm(**{name: None}) == S.NM_EINVAL, name
    assert norm(residual=None) == S.NM_EINVAL                    # a sum without a residual
    assert norm(x_dtype=2) == S.NM_EINVAL
    assert norm(stream_dtype=-1) == S.NM_EINVAL
    for eps in (0.0, -1e-6, math.inf, math.nan):
        assert norm(eps=eps) == S.NM_EINVAL, eps
    assert norm(m=-4) == S.NM_EINVAL
    assert norm(m=4, n=0) == S.NM_EINVAL
    assert norm(m=4, n=5) == S.NM_EINVAL
    assert norm(ns=1) == S.NM_EINVAL
    assert norm(ns=9) == S.NM_EINVAL
    assert norm(m=6, n=2) == S.NM_EUNSUPPORTED
    assert norm(m=8, n=4, ns=4) == S.NM_EUNSUPPORTED
    assert norm(rows=-1) == S.NM_ESHAPE
    assert norm(k=-1) == S.NM_ESHAPE
    assert norm(k=60, m=8, n=4) == S.NM_ESHAPE
    assert norm(k=60, ns=4) == S.NM_ESHAPE
    for name in ("ldx", "ldr", "lds", "ldy", "ldq"):
        assert norm(**{name: 48}) == S.NM_ESHAPE, name
        assert norm(**{name: 68}) == S.NM_EALIGN, name
    assert norm(k=50, ldq=48) == S.NM_ESHAPE                      # rounded up to 16: 64
    assert norm(ns=4, ldq=80) == S.NM_ESHAPE                      # lifted: 96
    assert norm(rows=1 << 62, ldx=1 << 20) == S.NM_ESHAPE
    for name in ("x", "weight", "q", "scale", "residual", "sum_out", "y"):
        assert norm(**{name: MIS}) == S.NM_EALIGN, name
    far = {name: 32776 for name in ("k", "ldx", "ldr", "lds", "ldy")}
    assert norm(ldq=32784, **far) == S.NM_EUNSUPPORTED
    assert norm(rows=1 << 31) == S.NM_EUNSUPPORTED


def route(**kw):
    a = dict(logits=P, ids=Q, weights=R, kind=S.NM_ROUTER_SIGMOID, bias=U, t=4, experts=64, top=8, ldl=64)
    a.update(kw)
    return S.nm_moe_route(a.pop("logits"), a.pop("ids"), a.pop("weights"), a.pop("kind"), stream=0, check=False, **a)


def test_route_refusals():
    assert route(t=0) == S.NM_OK
    for name in ("logits", "ids", "weights"):
        assert route(**{name: None}) == S.NM_EINVAL, name
        assert route(**{name: MIS}) == S.NM_EALIGN, name
    assert route(bias=MIS) == S.NM_EALIGN
    assert route(kind=2) == S.NM_EINVAL
    assert route(scale=math.inf) == S.NM_EINVAL
    assert route(scale=math.nan) == S.NM_EINVAL
    assert route(top=0) == S.NM_EINVAL
    assert route(top=65) == S.NM_ESHAPE
    assert route(experts=65) == S.NM_ESHAPE                       # ldl
    assert route(t=-1) == S.NM_ESHAPE
    assert route(t=1 << 61, experts=64) == S.NM_ESHAPE
    assert route(kind=S.NM_ROUTER_SOFTMAX) == S.NM_EUNSUPPORTED   # with a bias
    assert route(experts=1025, ldl=1025) == S.NM_EUNSUPPORTED
    assert route(top=33) == S.NM_EUNSUPPORTED
    assert route(t=(1 << 25) + 1) == S.NM_EUNSUPPORTED


# ------------------------------------------------------------------------------ the binding ---

def test_norm_binding(calls):  # noqa: F811
    x, r, w, q, s = bf16(4, 64), torch.zeros(4, 64), torch.ones(64), i8(4, 64), torch.zeros(4)
    a = taken(calls, S.nm_rmsnorm_i8, x, w, q, s, r, torch.zeros(4, 64), bf16(4, 64))
    assert a[1] == S.NM_Y_BF16 and a[2:5] == (4, 64, 64) and a[6] == 64 and a[9] == S.NM_Y_F32
    a = taken(calls, S.nm_rmsnorm_i8, x.float(), None, q, s)
    assert a[1] == S.NM_Y_F32 and a[5] is None and a[7] is None and a[10] is None
    # rows of 60 values in rows of 64
    a = taken(calls, S.nm_rmsnorm_i8, x, w, q, s, k=60)
    assert a[3] == 60 and a[4] == 64
    # a view of 60 columns: its rows are readable up to 64, but for a last row that ends the storage
    taken(calls, S.nm_rmsnorm_i8, bf16(5, 64)[:4, :60], w, q, s)
    for bad in (lambda: S.nm_rmsnorm_i8(x.half(), w, q, s), lambda: S.nm_rmsnorm_i8(x, w.double(), q, s),
                lambda: S.nm_rmsnorm_i8(x, w[:60], q, s), lambda: S.nm_rmsnorm_i8(x, w, x, s),
                lambda: S.nm_rmsnorm_i8(x, w, q[:3], s), lambda: S.nm_rmsnorm_i8(x, w, q[:, :60], s),
                lambda: S.nm_rmsnorm_i8(x, w, q, s[:3]), lambda: S.nm_rmsnorm_i8(x, w, q, s.half()),
                lambda: S.nm_rmsnorm_i8(x.t(), w, q, s), lambda: S.nm_rmsnorm_i8(x, w, q, s, r[:3]),
                lambda: S.nm_rmsnorm_i8(x, w, q, s, r[:, :56]), lambda: S.nm_rmsnorm_i8(x, w, q, s, r, bf16(4, 64)),
                lambda: S.nm_rmsnorm_i8(x, w, q, s, r, torch.zeros(3, 64)),
                lambda: S.nm_rmsnorm_i8(x, w, q, s, y=torch.zeros(4, 64)),
                lambda: S.nm_rmsnorm_i8(x, w, q, s, y=bf16(4, 60)), lambda: S.nm_rmsnorm_i8(x, w[::2], q, s, k=32),
                lambda: S.nm_rmsnorm_i8(x, w, q, s, ns=4), lambda: S.nm_rmsnorm_i8(x, w, q, s, rows=5),
                lambda: S.nm_rmsnorm_i8(x, w, q, s, k=72), lambda: S.nm_rmsnorm_i8(bf16(4, 60), torch.ones(60), q, s),
                lambda: S.nm_rmsnorm_i8(x, w, q, s, ldx=72), lambda: S.nm_rmsnorm_i8(x, w, q, s, ldq=80)):
        refused(calls, bad)


def test_norm_binding_refuses_rows_past_a_view(calls):  # noqa: F811
    """Columns behind a view's last one may hold anything: a longer row must not read them, where they
    complete a piece of 8 either."""
    x, r, q, s = bf16(5, 64)[:4], torch.zeros(5, 64)[:4], i8(4, 64), torch.zeros(4)
    taken(calls, S.nm_rmsnorm_i8, x[:, :60], None, q, s, r[:, :60])
    taken(calls, S.nm_rmsnorm_i8, x[:, :60], None, q, s, r)
    taken(calls, S.nm_rmsnorm_i8, x, None, q, s, r[:, :60], k=60)
    for bad in (lambda: S.nm_rmsnorm_i8(x, None, q, s, r[:, :60]), lambda: S.nm_rmsnorm_i8(x[:, :60], None, q, s, k=64),
                lambda: S.nm_rmsnorm_i8(x[:, :60], None, q, s, k=61)):
        refused(calls, bad)


def test_route_binding(calls):  # noqa: F811
    l, ids, w = torch.zeros(4, 60), torch.zeros(4, 8, dtype=torch.int32), torch.zeros(4, 8)
    a = taken(calls, S.nm_moe_route, l, ids, w)
    assert a[1:4] == (4, 60, 60) and a[4] is None and a[6:8] == (8, 1)
    assert taken(calls, S.nm_moe_route, torch.zeros(4, 64)[:, :60], ids, w)[3] == 64
    for bad in (lambda: S.nm_moe_route(l.bfloat16(), ids, w), lambda: S.nm_moe_route(l, ids.long(), w),
                lambda: S.nm_moe_route(l, ids, w.half()), lambda: S.nm_moe_route(l, ids, w[:3]),
                lambda: S.nm_moe_route(l, ids[:3], w), lambda: S.nm_moe_route(l, ids, w, bias=torch.zeros(59)),
                lambda: S.nm_moe_route(l, ids[:, ::2], w), lambda: S.nm_moe_route(l.t(), ids, w),
                lambda: S.nm_moe_route(l, ids, w, t=5), lambda: S.nm_moe_route(l, ids, w, experts=61)):
        refused(calls, bad)


def test_route_binding_refuses_rows_of_other_lengths(calls):  # noqa: F811
    l, ids, w = torch.zeros(4, 60), torch.zeros(4, 8, dtype=torch.int32), torch.zeros(4, 8)
    taken(calls, S.nm_moe_route, l, ids.reshape(-1), w.reshape(-1), top=8)
    taken(calls, S.nm_moe_route, l, torch.zeros(5, 8, dtype=torch.int32), w)
    for bad in (lambda: S.nm_moe_route(l, ids, torch.zeros(4, 16)), lambda: S.nm_moe_route(l, ids, w, top=4),
                lambda: S.nm_moe_route(l, ids.reshape(2, 16), w, top=8)):
        refused(calls, bad)


# ------------------------------------------------------------------------- pins of the oracle ---

def test_oracle_norm_codes_are_the_exact_quotient():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((6, 48)).astype(np.float32)
    w = rng.standard_normal(48).astype(np.float32)
    r = rng.standard_normal((6, 48)).astype(np.float32)
    q, scale, s, y = O.rmsnorm_i8(x, r, "f32", w, 1e-5)
    for i in range(6):
        assert [Fraction(float(v)) for v in s[i]] == [Fraction(float(np.float32(a + b))) for a, b in zip(x[i], r[i])]
        p = [Fraction(float(np.float32(a * b))) for a, b in zip(s[i], w)]
        top = max(abs(v) for v in p)
        assert list(q[i]) == [round(127 * v / top) for v in p]    # Fraction rounds half to even
        rms = math.sqrt(sum(float(v) ** 2 for v in s[i]) / 48 + float(np.float32(1e-5)))
        assert scale[i] == pytest.approx(float(top) / 127 / rms, rel=1e-14)
        assert list(y[i]) == pytest.approx([float(v) / rms for v in p], rel=1e-14)


def test_oracle_norm_codes_next_to_a_half():
    n = np.arange(66054, 131000, 997, dtype=np.int64)
    for side in (-1, 1):
        x = np.stack([256 * (127 * n + side), 128 * n + side], axis=1).astype(np.float32)
        q, _, _, _ = O.rmsnorm_i8(x)
        for row, code in zip(x, q):
            exact = 127 * Fraction(float(row[1])) / Fraction(float(row[0]))
            assert 0 < abs(exact - Fraction(1, 2)) < Fraction(1, 2 ** 30)
            assert int(code[1]) == round(exact) == (side < 0)


def test_oracle_norm_selection_and_rows_without_a_value():
    x = np.array([[3, -3, 1, 2, 0, 0, 0, 0], [0] * 8, [1, np.inf, 0, 0, 0, 0, 0, 0]], np.float32)
    q, scale, _, _ = O.rmsnorm_i8(x, n=1, m=4)
    assert q[0].tolist() == [127, 0, 0, 0, 0, 0, 0, 0]
    assert q[1].tolist() == [0] * 8 and scale[1] == 1 and q[2].tolist() == [0] * 8 and scale[2] == np.inf
    q, _, _, _ = O.rmsnorm_i8(x[:1], ns=4)
    assert q.tolist() == [[127, -127, 42, 85, 42, 85, 0, 0, 0, 0, 0, 0]]


def test_oracle_route():
    inf = np.inf
    l = np.array([[0, 2, 1, 2], [-inf, -1, np.nan, -inf], [-inf] * 4, [inf, 0, inf, 1]], np.float32)
    ids, w = O.moe_route(l, 3, renormalize=False)
    assert ids.tolist() == [[1, 3, 2], [1, -1, -1], [-1, -1, -1], [0, 2, 3]]
    e = math.e
    whole = 1 + 2 * e ** 2 + e
    assert w[0].tolist() == pytest.approx([e ** 2 / whole, e ** 2 / whole, e / whole])
    assert w[1].tolist() == [1, 0, 0] and w[2].tolist() == [0, 0, 0] and w[3].tolist() == [0.5, 0.5, 0]
    ids, w = O.moe_route(l[:1], 2, sigmoid=True, bias=np.array([1, 0, 0, 0.5], np.float32), scale=2.0)
    assert ids.tolist() == [[0, 3]]                                # 1.5 and 1.38 against 0.88, 0.73
    a, b = 0.5, 1 / (1 + e ** -2)
    assert w[0].tolist() == pytest.approx([2 * a / (a + b), 2 * b / (a + b)])
