"""The int8 mixture-of-experts layer without a GPU: refusals with the documented status, what the
binding accepts of its tensors, and a pin of the oracle that does not use its own code."""
import math

import numpy as np
import pytest

import oracle as O
import semi_structured_sparse_amd as S
from test_i8_binding_cpu import Recorder, bf16, calls, i8, refused, taken  # noqa: F401

torch = pytest.importorskip("torch")

A = [(i + 1) << 20 for i in range(20)]     # fake, aligned, never dereferenced


def moe(**kw):
    a = dict(x=A[0], x_scale=A[1], ids=A[2], weights=A[3], w_gate=A[4], gate_scale=A[5], w_up=A[6], up_scale=A[7],
             w_down=A[8], down_scale=A[9], y=A[10], residual=A[11], workspace=A[12], t=4, experts=8, top=2, hidden=64,
             inter=32, ldx=64, ldw=64, ldd=32, ldr=64, ldy=64, workspace_bytes=1 << 20)
    a.update(kw)
    names = ("x", "x_scale", "ids", "weights", "w_gate", "gate_scale", "w_up", "up_scale", "w_down", "down_scale", "y")
    return S.nm_moe_i8(*[a.pop(n) for n in names], stream=0, check=False, **a)


META = dict(gate_meta=A[13], up_meta=A[14], down_meta=A[15])


def test_refusals():
    assert moe(t=0) == S.NM_OK
    assert moe(hidden=0) == S.NM_OK
    for name in ("x", "x_scale", "ids", "weights", "w_gate", "gate_scale", "w_up", "up_scale", "w_down", "down_scale", "y",
                 "workspace"):
        assert moe(**{name: None}) == S.NM_EINVAL, name
        assert moe(**{name: A[0] + 4}) == S.NM_EALIGN, name
    assert moe(residual=A[0] + 8) == S.NM_EALIGN
    assert moe(act=2) == S.NM_EINVAL
    assert moe(y_dtype=2) == S.NM_EINVAL
    assert moe(top=0) == S.NM_EINVAL
    assert moe(experts=0) == S.NM_EINVAL
    for part in META:                                             # all or none
        assert moe(**{part: META[part]}) == S.NM_EINVAL
        assert moe(**{**META, part: None}) == S.NM_EINVAL
    for name in ("t", "hidden", "inter"):
        assert moe(**{name: -1}) == S.NM_ESHAPE, name
    assert moe(hidden=62, **META) == S.NM_ESHAPE
    assert moe(inter=30, **META) == S.NM_ESHAPE
    for name in ("ldx", "ldw", "ldr", "ldy"):
        assert moe(**{name: 48}) == S.NM_ESHAPE, name
    assert moe(ldd=16) == S.NM_ESHAPE
    for name in ("ldx", "ldw", "ldd"):
        assert moe(**{name: 72}) == S.NM_EALIGN, name
    assert moe(t=1 << 60) == S.NM_ESHAPE
    assert moe(inter=1 << 60, ldd=1 << 60) == S.NM_ESHAPE
    assert moe(hidden=131088, ldx=131088, ldw=131088, ldr=131088, ldy=131088) == S.NM_EUNSUPPORTED
    assert moe(inter=65552, ldd=65552) == S.NM_EUNSUPPORTED
    assert moe(experts=1025) == S.NM_EUNSUPPORTED
    assert moe(top=33) == S.NM_EUNSUPPORTED
    need = S.nm_moe_i8_workspace_size(4, 8, 2, 64, 32)
    assert need > 0
    assert moe(workspace_bytes=need - 1) == S.NM_EINVAL


def test_workspace_size():
    f = S.nm_moe_i8_workspace_size
    assert f(0, 8, 2, 64, 32) == 0 and f(4, 8, 2, 0, 32) == 0
    assert f(64, 8, 2, 64, 32) == f(1000, 8, 2, 64, 32)            # passes of 64 tokens
    assert f(1, 8, 2, 64, 32) < f(64, 8, 2, 64, 32)
    assert f(4, 2000, 2, 64, 32) == 0 and f(4, 8, 33, 64, 32) == 0


def test_binding(calls):  # noqa: F811
    e, h, i, t = 3, 60, 20, 4

    def parts(sparse=False):
        kh, ki = (h // 2, i // 2) if sparse else (h, i)
        p = dict(x=i8(t, 64), x_scale=torch.zeros(t), ids=torch.zeros(t, 2, dtype=torch.int32), weights=torch.zeros(t, 2),
                 w_gate=i8(e, i, kh + -kh % 16), gate_scale=torch.zeros(e, i), w_up=i8(e, i, kh + -kh % 16),
                 up_scale=torch.zeros(e, i), w_down=i8(e, h, ki + -ki % 16), down_scale=torch.zeros(e, h), y=bf16(t, h),
                 workspace=i8(4096))
        if sparse:
            p.update(gate_meta=i8(e, 1, i, 16), up_meta=i8(e, 1, i, 16), down_meta=i8(e, 1, h, 16))
        return p

    a = taken(calls, S.nm_moe_i8, **parts())[0]
    assert (a.t, a.hidden, a.inter, a.experts, a.top) == (t, h, i, e, 2)
    assert (a.ldx, a.ldw, a.ldd, a.ldy, a.y_dtype) == (64, 64, 32, h, S.NM_Y_BF16)
    a = taken(calls, S.nm_moe_i8, **{**parts(True), "y": torch.zeros(t, h), "residual": torch.zeros(t, 64)[:, :h]})[0]
    assert (a.ldw, a.ldd, a.ldr, a.y_dtype) == (32, 16, 64, S.NM_Y_F32)
    taken(calls, S.nm_moe_i8, **{**parts(), "w_gate": i8(e * i, 64)}, experts=e, inter=i)
    for bad in (dict(x=i8(t, 48)), dict(x=i8(3, 64), t=t), dict(x_scale=torch.zeros(3)), dict(x_scale=torch.zeros(t).half()),
                dict(ids=torch.zeros(t, 2)), dict(ids=torch.zeros(3, 2, dtype=torch.int32)), dict(weights=torch.zeros(t, 1)),
                dict(w_gate=i8(e, i, 48)), dict(w_gate=i8(e, i, 80)), dict(w_up=i8(e, 19, 64)), dict(w_up=i8(2, i, 64)),
                dict(w_up=i8(e, 2 * i, 64)[:, :i]), dict(w_gate=bf16(e, i, 64)), dict(w_down=i8(e, h, 16)),
                dict(w_down=i8(e, 59, 32)), dict(gate_scale=torch.zeros(e, 19)), dict(up_scale=torch.zeros(2, i)),
                dict(down_scale=torch.zeros(e, h)[:, ::2]), dict(y=bf16(3, h)), dict(y=bf16(t, h).half()),
                dict(residual=torch.zeros(t, h)), dict(residual=bf16(t, 59)), dict(residual=bf16(3, h)),
                dict(workspace=i8(4096)[::2])):
        p = {**parts(), **bad}
        refused(calls, S.nm_moe_i8, **{**p, "hidden": h})
    for bad in (dict(gate_meta=i8(e, 1, 19, 16)), dict(down_meta=i8(2, 1, h, 16))):
        refused(calls, S.nm_moe_i8, **{**parts(True), **bad})


def test_binding_refuses_rows_of_other_lengths(calls):  # noqa: F811
    """Choices, weights and scales follow each other without a gap: a matrix whose rows are longer than
    the call's would be read across them."""
    e, h, i, t = 3, 64, 100, 4
    parts = dict(x=i8(t, 64), x_scale=torch.zeros(t), ids=torch.zeros(t, 2, dtype=torch.int32), weights=torch.zeros(t, 2),
                 w_gate=i8(e, i, 64), gate_scale=torch.zeros(e, i), w_up=i8(e, i, 64), up_scale=torch.zeros(e, i),
                 w_down=i8(e, h, 112), down_scale=torch.zeros(e, h), y=bf16(t, h), workspace=i8(4096))
    taken(calls, S.nm_moe_i8, **parts)
    flat = {n: parts[n].reshape(-1) for n in ("ids", "weights", "gate_scale", "up_scale", "down_scale")}
    taken(calls, S.nm_moe_i8, **{**parts, **flat}, top=2)
    taken(calls, S.nm_moe_i8, **{**parts, "gate_scale": torch.zeros(e, i, 1), "up_scale": torch.zeros(e + 1, i)})
    taken(calls, S.nm_moe_i8, **{**parts, "ids": torch.zeros(t + 1, 2, dtype=torch.int32)})
    for bad in (dict(weights=torch.zeros(t, 4)), dict(ids=torch.zeros(t, 4, dtype=torch.int32)), dict(top=1),
                dict(gate_scale=torch.zeros(e, 112)), dict(up_scale=torch.zeros(i, e)), dict(down_scale=torch.zeros(e, 112)),
                # a matrix of all experts' rows says nothing of an expert's
                dict(w_gate=i8(e * i, 64), w_up=i8(e * i, 64), experts=e)):
        refused(calls, S.nm_moe_i8, **{**parts, **bad})


def test_oracle():
    x = np.array([[1, -2], [3, 0]], np.int8)
    xs = np.array([0.5, 0.25], np.float32)
    gate = (np.array([[[1, 1]], [[4, 0]]], np.int8), np.ones((2, 1), np.float32))
    up = (np.array([[[2, 1]], [[1, 1]]], np.int8), np.full((2, 1), 2.0, np.float32))
    down = (np.array([[[3], [-1]], [[1], [2]]], np.int8), np.ones((2, 2), np.float32))
    ids = np.array([[0, -1], [1, 1]], np.int32)
    w = np.array([[0.5, 9.0], [0.25, 0.5]], np.float32)
    y, far, size = O.moe_i8(x, xs, ids, w, gate, up, down, residual=np.array([[1.0, 2.0], [0.0, 0.0]]))
    # token 0, expert 0: g = -0.5, u = 0: nothing; token 1, expert 1 (twice): g = 3, u = 1.5
    assert y[0].tolist() == [1.0, 2.0]
    h = float(O.bf16_round(np.array([3 / (1 + math.exp(-3)) * 1.5], np.float32))[0])
    assert y[1].tolist() == pytest.approx([0.75 * h, 1.5 * h], rel=1e-6)
    assert size[1].tolist() == pytest.approx([0.75 * h, 1.5 * h], rel=1e-6) and (far >= 0).all()
