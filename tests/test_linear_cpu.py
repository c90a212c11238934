"""The bf16 linear layer with its epilogue without a GPU: refusals with the documented status, the
workspace query, what the binding accepts of its tensors, and a pin of the oracle."""
import math

import numpy as np
import pytest

import linear_plan as P
import oracle as O
import semi_structured_sparse_amd as S
from test_i8_binding_cpu import Recorder, bf16, calls, i8, refused, taken  # noqa: F401

torch = pytest.importorskip("torch")

A = [(i + 1) << 20 for i in range(8)]     # fake, aligned, never dereferenced


def lin(**kw):
    a = dict(x=A[0], w=A[1], y=A[2], bias=A[3], residual=A[4], workspace=A[5], t=4, o=32, k=64, ldx=64, ldw=64, ldr=32,
             ldy=32, workspace_bytes=0)
    a.update(kw)
    return S.nm_linear(a.pop("x"), a.pop("w"), a.pop("y"), stream=0, check=False, **a)


def test_refusals():
    assert lin(t=0) == S.NM_OK
    assert lin(o=0) == S.NM_OK
    for name in ("x", "w", "y"):
        assert lin(**{name: None}) == S.NM_EINVAL, name
    for name in ("x", "w", "y", "bias", "residual", "workspace", "w_meta"):
        assert lin(**{name: A[0] + 8}) == S.NM_EALIGN, name
    assert lin(fn=4) == S.NM_EINVAL
    assert lin(fn=-1) == S.NM_EINVAL
    assert lin(y_dtype=2) == S.NM_EINVAL
    for name in ("t", "o", "k", "workspace_bytes"):
        assert lin(**{name: -1}) == S.NM_ESHAPE, name
    assert lin(k=62, w_meta=A[6]) == S.NM_ESHAPE
    for name, v in (("ldx", 56), ("ldw", 56), ("ldr", 31), ("ldy", 31)):
        assert lin(**{name: v}) == S.NM_ESHAPE, name
    assert lin(ldw=24, w_meta=A[6]) == S.NM_ESHAPE
    for name in ("ldx", "ldw"):
        assert lin(**{name: 68}) == S.NM_EALIGN, name
    assert lin(t=1 << 60) == S.NM_ESHAPE
    big = (1 << 24) + 8
    assert lin(k=big, ldx=big, ldw=big) == S.NM_EUNSUPPORTED
    assert lin(t=(1 << 27) + 1) == S.NM_EUNSUPPORTED


def test_workspace_size():
    f = S.nm_linear_workspace_size
    assert f(0, 8, 8) == 0 and f(8, 0, 8) == 0 and f(8, 8, 0) == 0
    assert f(8192, 14336, 4096) == 0                               # whole tiles
    assert f(1, 64, 16384) >= 2 * 64 * 4                           # few rows, a long reduction: split
    assert f(40, 256, 14336) >= 2 * 40 * 256 * 4


def test_plan_agrees_with_the_workspace():
    """The tests' own account of the dispatch, by which they choose sizes: reduction ranges as the library
    asks for them."""
    rng = np.random.default_rng(1)
    for _ in range(4000):
        t, o, k = (int(2 ** rng.uniform(0, top)) for top in (12, 14, 14.5))
        sparse = bool(rng.integers(2))
        if sparse:
            k = max(4, k // 4 * 4)
        for route in (None, "few_stream", "few_tile", "tile_lds"):
            got = S.nm_linear_workspace_size(t, o, k, sparse, S.route_bits(route) if route else 0)
            assert got == P.workspace(t, o, k, sparse, route), (t, o, k, sparse, route)


def test_every_instance_is_run():
    """The sizes of test_linear_gpu.py's test_every_instance and test_rounds_of_large_tiles reach every
    kernel that nm_linear has, split and whole, with every count of waves."""
    few = [(1, 4, 4, False), (1, 2, 4, False), (2, 2, 4, False)]
    for tb in (1, 2, 4):
        few += [(tb, 1, 4, False), (tb, 1, 8, False), (tb, 1, 8, True)] + [(tb, 1, 16, False)] * (tb < 4)
    every = {("few", *f) for f in few} | {("tile", shape, split) for shape in range(4) for split in (False, True)}
    for sparse, sizes in ((False, P.DENSE), (True, P.SPARSE)):
        run = {P.instance(P.plan(t, o, k, sparse, route), sparse)[1:] for t, o, k, route in sizes}
        assert run == every, (every - run, run - every)
        for t, o, k in P.LARGE:
            assert P.plan(t, o, k, sparse) == ("large",)
            bands = -(-o // 256)
            assert bands > 8 and bands % 8 and bands * -(-t // 256) > 256


def test_binding(calls):  # noqa: F811
    x, w, y = bf16(4, 64), bf16(32, 64), bf16(4, 32)
    a = taken(calls, S.nm_linear, x, w, y, bias=torch.zeros(32), residual=bf16(4, 40)[:, :32], fn=S.NM_FN_SILU)
    assert a[1:4] == (4, 64, 64) and a[5:7] == (32, 64) and a[7] is None and a[9] == S.NM_FN_SILU and a[11] == 40
    assert a[13:15] == (32, S.NM_Y_BF16)
    a = taken(calls, S.nm_linear, x, bf16(32, 32), torch.zeros(4, 32), w_meta=i8(1, 32, 16), k=60)
    assert a[2] == 60 and a[14] == S.NM_Y_F32
    taken(calls, S.nm_linear, bf16(5, 64)[:4, :60], w, y)
    m = i8(1, 32, 16)
    for bad in (lambda: S.nm_linear(x.float(), w, y), lambda: S.nm_linear(x, w.float(), y), lambda: S.nm_linear(x, w, y.half()),
                lambda: S.nm_linear(x, w, y[:3]), lambda: S.nm_linear(x, w, y[:, :31]), lambda: S.nm_linear(x, w[:, :56], y),
                lambda: S.nm_linear(x, w, y, residual=torch.zeros(4, 32)), lambda: S.nm_linear(x, w, y, residual=bf16(3, 32)),
                lambda: S.nm_linear(x, w, y, residual=bf16(4, 31)), lambda: S.nm_linear(x, w, y, bias=torch.zeros(31)),
                lambda: S.nm_linear(x, w, y, bias=bf16(32)), lambda: S.nm_linear(x, w.t(), y),
                lambda: S.nm_linear(x, bf16(32, 24), y, w_meta=m), lambda: S.nm_linear(x, w, y, w_meta=m[:, :31]),
                lambda: S.nm_linear(x, w, y, t=5), lambda: S.nm_linear(x, w, y, o=33), lambda: S.nm_linear(x, w, y, k=72),
                lambda: S.nm_linear(bf16(4, 60), bf16(32, 60), y), lambda: S.nm_linear(x, w, y, ldx=72),
                lambda: S.nm_linear(x, w, y, ldy=40), lambda: S.nm_linear(x, w, y, workspace=i8(64)[::2]),
                lambda: S.nm_linear(x, w, y, y_dtype=S.NM_Y_F32)):
        refused(calls, bad)


def test_binding_refuses_reductions_past_a_view(calls):  # noqa: F811
    """Columns behind a view's last one may hold anything: a longer reduction must not read them, where
    they complete a piece of 8 either."""
    x, w, y = bf16(5, 64)[:4], bf16(33, 64)[:32], bf16(4, 32)
    taken(calls, S.nm_linear, x[:, :60], w[:, :60], y)
    taken(calls, S.nm_linear, x[:, :60], w, y)
    taken(calls, S.nm_linear, x, w[:, :60], y, k=60)
    taken(calls, S.nm_linear, x, bf16(33, 32)[:32, :30], y, w_meta=i8(1, 32, 16), k=60)
    for bad in (lambda: S.nm_linear(x, w[:, :60], y), lambda: S.nm_linear(x[:, :60], w, y, k=64),
                lambda: S.nm_linear(x[:, :60], w[:, :60], y, k=61),
                lambda: S.nm_linear(x, bf16(33, 32)[:32, :30], y, w_meta=i8(1, 32, 16))):
        refused(calls, bad)


def test_oracle():
    x, w = np.array([[1.0, 2.0], [0.0, -1.0]]), np.array([[1.0, 1.0], [2.0, -3.0], [0.0, 0.5]])
    y, size = O.linear(x, w, np.array([0.0, 1.0, -1.0]), "silu", np.ones((2, 3)))
    s = [[3.0, -3.0, 0.0], [-1.0, 4.0, -1.5]]
    want = [[1 + v / (1 + math.exp(-v)) for v in r] for r in s]
    assert y == pytest.approx(np.array(want), rel=1e-15) and size.tolist() == [[3, 8, 1], [1, 3, 0.5]]
    assert O.linear(x, w, None, "relu")[0].tolist() == [[3, 0, 1], [0, 3, 0]]
    v = np.array([[1.0, 2.0], [3.0, 4.0]])
    assert O.expand_24_values(v, np.array([[0, 3], [1, 2]]), 4).tolist() == [[1, 0, 0, 2], [0, 3, 4, 0]]
