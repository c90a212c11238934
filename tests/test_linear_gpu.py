"""The bf16 linear layer with its epilogue on the GPU against the oracle's 64-bit definition, on every
route."""
import ctypes

import numpy as np
import pytest

import linear_plan as P
import oracle as O
import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import semi_structured_sparse_amd as S  # noqa: E402

U = 2.0 ** -24            # half a step of fp32, relative
UB = 2.0 ** -8            # half a step of bf16, relative
# What a gate may lose of a value next to nothing: (|v| / 4) / (1/4 + e^-z / 4) by a reciprocal that is 0
# where its operand passes 2^126, so where e^-z > 2^128, z < -88.7; |v| <= |z| + 0.8 there (gelu's z
# grows faster than v), and |z| e^z falls with |z|: at most 89.5 * 2^-128 < 2^-121.
GATE_LOST = 2.0 ** -121
ROUTES = {"auto": 0, "stream": S.route_bits("few_stream"), "split": S.route_bits("few_tile"),
          "tile": S.route_bits("tile_lds")}
FNS = {"none": S.NM_FN_NONE, "relu": S.NM_FN_RELU, "silu": S.NM_FN_SILU, "gelu": S.NM_FN_GELU_TANH}


def sync():
    torch.cuda.synchronize()


def up(v, m):
    return -(-v // m) * m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def padded(v, ld):
    """bf16-valued rows in rows of ld, NaN past each of them."""
    t = torch.full((v.shape[0], max(ld, 8)), float("nan"), dtype=torch.bfloat16, device="cuda")
    t[:, :v.shape[1]] = dev(v.astype(np.float32)).bfloat16()
    return t


class Case:
    def __init__(self, seed, t, o, k, sparse=False, fn="none", bias=True, res=True, kind=torch.bfloat16, pad=0, far=1.0):
        rng = np.random.default_rng(seed)
        self.t, self.o, self.k, self.sparse, self.fn, self.kind, self.pad = t, o, k, sparse, fn, kind, pad
        self.x = O.f32_from_bf16(synth.normal_bf16(rng, (t, k), far))
        if sparse:
            vals = O.f32_from_bf16(synth.normal_bf16(rng, (o, k // 2), 0.1))
            idx = np.sort(rng.random((o, k // 4, 4)).argsort(2)[..., :2], axis=2).reshape(o, k // 2).astype(np.uint8)
            self.meta = torch.zeros(max(1, S.nm_meta_block_bytes(o, k)), dtype=torch.uint8, device="cuda")
            if k and o:
                S.nm_meta_block(dev(O.pack_meta_2bit(idx)), o, k, self.meta)
            self.w, stored, self.idx = O.expand_24_values(vals, idx, k), vals, idx
        else:
            self.w, self.meta = O.f32_from_bf16(synth.normal_bf16(rng, (o, k), 0.1)), None
            stored = self.w
        self.xd, self.wd = padded(self.x, up(k, 8) + pad), padded(stored, up(stored.shape[1], 8) + pad)
        self.bias = rng.standard_normal(o).astype(np.float32) if bias else None
        self.res = O.bf16_round(rng.standard_normal((t, o)).astype(np.float32)) if res else None
        self.ref = None

    def run(self, route="auto", in_place=False, ws=True, **kw):
        t, o = self.t, self.o
        ldy = o + self.pad
        y = torch.full((t + 1, ldy + 4 if self.pad else ldy), 7.0, dtype=self.kind, device="cuda")[:, :max(ldy, 1)]
        r = None
        if self.res is not None:
            r = y if in_place else torch.full((t, ldy), float("nan"), dtype=self.kind, device="cuda")
            r[:t, :o] = dev(self.res).to(self.kind)
        n = S.nm_linear_workspace_size(t, o, self.k, self.sparse, ROUTES[route])
        wsd = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda") if ws else None
        taken = ctypes.c_uint32(0)
        S.nm_linear(self.xd, self.wd, y, self.meta, None if self.bias is None else dev(self.bias), FNS[self.fn], r, wsd, t=t,
                    o=o, k=self.k, ldx=self.xd.stride(0), ldw=self.wd.stride(0), route=ROUTES[route], taken=taken, **kw)
        sync()
        assert (y[t] == 7.0).all() and (y[:, o:] == 7.0).all()
        return y[:t, :o].double().cpu().numpy(), S.taken_names(taken.value)

    def check(self, got):
        if self.ref is None:
            self.ref = O.linear(self.x, self.w, self.bias, self.fn, self.res)
        y, size = self.ref
        # the sum in fp32, in whatever order: at most k additions of at most U of all magnitudes each
        # (products of bf16 are exact); the matrix unit may truncate instead of rounding (2 U)
        err = 2 * U * (self.k + 1) * size
        pre = np.abs(y if self.res is None else y - self.res)
        if self.bias is not None:
            err = err + U * (size + np.abs(self.bias)[None, :])
        if self.fn in ("silu", "gelu"):
            # slopes of silu and gelu stay below 1.13; their own fp32 evaluation: the exponent's
            # rounding (|z| U, where the gate is within its limits: |z| < 104) and a few steps
            err = 1.13 * err + (2 * 104 + 16) * U * pre + GATE_LOST
        err = err + 2 * U * (np.abs(y) + pre)
        if self.kind == torch.bfloat16:
            err = err + UB * (np.abs(y) + err)
        assert np.isfinite(got).all()
        worst = (np.abs(got - y) - err - 1e-38).max() if got.size else 0
        assert worst <= 0, worst
        if got.size > 64:
            assert np.linalg.norm(got - y) <= (3e-3 if self.kind == torch.bfloat16 else 3e-6) * np.linalg.norm(y)


SIZES = [(1, 1, 4), (1, 16, 64), (1, 100, 132), (3, 70, 260), (5, 33, 1000), (16, 256, 512), (17, 130, 96), (31, 4, 36),
         (33, 300, 68), (64, 64, 128), (65, 129, 192), (100, 257, 388), (128, 512, 256), (200, 96, 1028), (257, 300, 64),
         (300, 520, 60), (513, 258, 132), (48, 64, 4096), (2, 40, 20000)]


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("size", SIZES)
def test_sizes_on_every_route(size, sparse):
    for n, (fn, kind, pad) in enumerate([("none", torch.float32, 0), ("gelu", torch.bfloat16, 8), ("silu", torch.float32, 24)]):
        c = Case(11 * n + size[0], *size, sparse=sparse, fn=fn, kind=kind, pad=pad, bias=n != 1, res=n != 2)
        for r in ROUTES:
            print("linear", size, sparse, fn, r, flush=True)
            c.check(c.run(r)[0])


@pytest.mark.parametrize("k", [1, 2, 3, 7, 9, 31, 33, 63, 65, 127, 129, 199, 1999])
def test_odd_reductions(k):
    """Rows that end inside a piece, with NaN right behind their last value."""
    for t, o in ((3, 37), (70, 131), (300, 259)):
        for pad in (0, 8):
            c = Case(k, t, o, k, kind=torch.float32, fn="relu", pad=pad)
            for r in ROUTES:
                print("linear odd", t, o, k, r, flush=True)
                c.check(c.run(r)[0])


@pytest.mark.parametrize("k", [4, 8, 12, 20, 28, 60, 68, 124, 132, 140, 1996])
def test_odd_sparse_reductions(k):
    for t, o in ((3, 37), (70, 131), (300, 259)):
        c = Case(k, t, o, k, sparse=True, kind=torch.float32, pad=8 * (k % 3))
        for r in ROUTES:
            print("linear odd 2:4", t, o, k, r, flush=True)
            c.check(c.run(r)[0])


@pytest.mark.parametrize("fn", list(FNS))
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_epilogues(fn, kind):
    for sparse in (False, True):
        for bias in (False, True):
            for res in (False, True):
                for t, o, pad in ((9, 70, 0), (40, 64, 2), (130, 260, 3), (260, 131, 0), (260, 260, 8)):
                    c = Case(5, t, o, 128, sparse=sparse, fn=fn, bias=bias, res=res, kind=kind, pad=0, far=3.0)
                    c.pad = pad      # rows of y and of the residual: aligned or not
                    for r in ("stream", "split", "tile"):
                        c.check(c.run(r)[0])


def test_split_reductions():
    for sparse in (False, True):
        for t, o, k, route in ((4, 48, 16384, "stream"), (40, 192, 8192, "split"), (100, 130, 12288, "split"), (7, 33, 9000, "stream")):
            print("linear split", t, o, k, route, flush=True)
            for fn, kind, pad in (("gelu", torch.bfloat16, 0), ("none", torch.float32, 3)):
                c = Case(t, t, o, k, sparse=sparse, fn=fn, kind=kind)
                c.pad = pad
                got, taken = c.run(route)
                assert "reduce" in taken, taken
                c.check(got)
                got, taken = c.run(route, ws=False)
                assert "reduce" not in taken, taken
                c.check(got)


def test_residual_in_place():
    for route in ROUTES:
        for kind in (torch.float32, torch.bfloat16):
            for t, o in ((5, 100), (300, 260), (300, 259)):
                c = Case(6, t, o, 192, fn="silu", kind=kind)
                assert np.array_equal(c.run(route)[0], c.run(route, in_place=True)[0])


def test_no_reduction_and_no_outputs():
    c = Case(7, 5, 40, 0, fn="silu", kind=torch.float32)
    c.check(c.run()[0])
    x, w = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    S.nm_linear(x, w, torch.zeros(0, 8, device="cuda"))
    S.nm_linear(w, x, torch.zeros(8, 0, device="cuda"))
    sync()


def test_values_that_are_not_finite_stay_in_their_row_and_column():
    for sparse in (False, True):
        for t, o in ((6, 40), (300, 300)):
            c = Case(8, t, o, 256, sparse=sparse, fn="silu", kind=torch.float32)
            want = {r: c.run(r)[0] for r in ROUTES}
            c.xd[1, 5], c.xd[4, 0] = float("nan"), float("inf")
            c.wd[7, 3] = float("nan")
            for r in ROUTES:
                got = c.run(r)[0]
                clean = np.ones((t, o), bool)
                clean[[1, 4]] = clean[:, 7] = False
                assert np.array_equal(got[clean], want[r][clean])
                assert np.isnan(got[1]).all() if not sparse else True
                assert np.isnan(got[:, 7]).all()


def test_extreme_activations():
    """Sums far out in the gates: limits, no NaN."""
    x = torch.full((4, 8), 1.0, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(40, 8, dtype=torch.bfloat16, device="cuda")
    v = np.concatenate([np.linspace(-120, 120, 32), [3e38, -3e38, 1e-30, -1e-30, 0.0, -88.5, 89.5, 20.0]]).astype(np.float32)
    y = torch.empty(4, 40, device="cuda")
    for fn in ("silu", "gelu"):
        for r in ROUTES:
            S.nm_linear(x, w, y, bias=dev(v), fn=FNS[fn], route=ROUTES[r])
            sync()
            with np.errstate(over="ignore"):
                ref = O.glu_gate(v.astype(np.float64), fn)
            got = y.double().cpu().numpy()
            assert (np.abs(got - ref[None]) <= (2 * 104 + 16) * U * np.abs(ref) + GATE_LOST).all()


def test_repeated_calls_give_the_same_bits():
    for sparse in (False, True):
        for t, o, k, route in ((40, 256, 8192, "split"), (400, 512, 1024, "tile"), (200, 300, 2048, "split"), (5, 64, 16384, "stream")):
            c = Case(9, t, o, k, sparse=sparse)
            want = c.run(route)[0]
            for _ in range(8):
                assert np.array_equal(c.run(route)[0], want)


def test_large_products():
    """Several rounds of 256 x 256 tiles: a row of every 64 against the oracle, every output written."""
    for sparse in (False, True):
        t, o, k = 2100, 4200, 1024
        print("linear large", sparse, flush=True)
        c = Case(10, t, o, k, sparse=sparse, fn="gelu", kind=torch.float32)
        got, taken = c.run("auto")
        assert "tile_lds" in taken
        rows = np.unique(np.r_[np.arange(0, t, 61), t - 1])
        c.x, c.res, c.t = c.x[rows], c.res[rows], len(rows)
        assert np.isfinite(got).all()
        c.check(got[rows])


def test_offsets_past_32_bits():
    k = 128
    for sparse in (False, True):
        for t, o, ldx, ldw, ldy in ((1100, 70, 1 << 21, 256, 70), (300, 1100, 256, 1 << 21, 1100), (1100, 70, 256, 256, 1 << 20),
                                    (40, 70, 1 << 23, 256, 70)):
            print("linear far", sparse, t, o, ldx, ldw, ldy, flush=True)
            c = Case(12, t, o, k, sparse=sparse, kind=torch.float32)
            wk = c.wd.shape[1] if sparse else k
            x, w = torch.empty(t, ldx, dtype=torch.bfloat16, device="cuda"), torch.empty(o, ldw, dtype=torch.bfloat16, device="cuda")
            x[:, :k], w[:, :wk] = c.xd[:, :k], c.wd[:, :wk]
            y, r = torch.empty(t, ldy, device="cuda"), torch.empty(t, ldy, device="cuda")
            r[:, :o] = dev(c.res)
            for route in ROUTES:
                y[:, :o] = float("nan")
                S.nm_linear(x, w, y, c.meta, dev(c.bias), S.NM_FN_NONE, r, t=t, o=o, k=k, route=ROUTES[route])
                sync()
                c.check(y[:, :o].double().cpu().numpy())
            del x, w, y, r
            torch.cuda.empty_cache()


def test_captured_streams_and_a_shared_workspace():
    rng = np.random.default_rng(13)
    cases = [Case(14 + n, 20, 96, 16384, sparse=bool(n)) for n in range(2)]
    n = max(S.nm_linear_workspace_size(20, 96, 16384, s) for s in (False, True))
    assert n > 0
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    graphs, want, outs, kws = [], [], [], []
    for c in cases:
        y = torch.zeros(20, 96, dtype=c.kind, device="cuda")
        kw = dict(w_meta=c.meta, bias=dev(c.bias), residual=dev(c.res).to(c.kind), workspace=ws, k=c.k)
        S.nm_linear(c.xd, c.wd, y, **kw)
        sync()
        want.append(y.clone())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            S.nm_linear(c.xd, c.wd, y, **kw)
        graphs.append(g), outs.append(y), kws.append(kw)
    for i in (0, 1, 1, 0, 1, 0):
        outs[i].fill_(float("nan"))
        graphs[i].replay()
        sync()
        assert torch.equal(outs[i], want[i])
        torch.randn(100, 100, device="cuda").sum().item()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = torch.zeros_like(outs[0])
    side.wait_stream(torch.cuda.current_stream())
    S.nm_linear(cases[0].xd, cases[0].wd, y, stream=side, **kws[0])
    side.synchronize()
    assert torch.equal(y, want[0])
    for bad in (lambda: S.nm_linear(cases[0].xd.cpu(), cases[0].wd, y), lambda: S.nm_linear(cases[0].xd, cases[0].wd, y.cpu(), stream=side)):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("sparse,size", [(False, s) for s in P.DENSE] + [(True, s) for s in P.SPARSE])
def test_every_instance(sparse, size):
    """Each kernel instance that the dispatch has, with outputs in rows that keep the alignment of four
    and in rows that do not."""
    t, o, k, route = size
    route = {None: "auto", "few_stream": "stream"}[route]
    plan = P.plan(*size[:3], sparse, size[3])
    print("linear instance", sparse, size, plan, flush=True)
    for n, (fn, kind, pad) in enumerate([("gelu", torch.bfloat16, -o % 4), ("none", torch.float32, 1 + -o % 4)]):
        c = Case(20 + n, t, o, k, sparse=sparse, fn=fn, kind=kind)
        c.pad = pad
        got, taken = c.run(route)
        assert ("few_stream" in taken) == (plan[0] == "few") and ("reduce" in taken) == (plan[-1] > 1), taken
        c.check(got)


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("size", P.LARGE)
def test_rounds_of_large_tiles(sparse, size):
    """More tiles of 256 x 256 than the chip runs at once: the call by shape against the same kernel by hint
    (a row's bits do not depend on its place), hundreds of rows against a call of few tiles, a row of
    every 61 against the oracle."""
    t, o, k = size
    assert P.plan(t, o, k, sparse) == ("large",)
    k = k if sparse or k % 8 else k - 1                # dense: a row that ends inside a piece
    k = k - 4 if sparse else k
    for kind, pad in ((torch.float32, 0), (torch.bfloat16, 3)):
        print("linear large", sparse, size, k, kind, flush=True)
        c = Case(30, t, o, k, sparse=sparse, fn="silu", kind=kind)
        c.pad = pad
        got, taken = c.run("auto")
        assert "tile_lds" in taken and "reduce" not in taken
        assert np.array_equal(got, c.run("tile")[0])
        rows = np.r_[0:70, 251:262, 1000:1300, 4090:4200]
        part = Case(31, 1, 1, 4, kind=kind)
        part.__dict__.update(c.__dict__)
        part.t, part.x, part.xd, part.res = len(rows), c.x[rows], c.xd[torch.from_numpy(rows).cuda()].contiguous(), c.res[rows]
        assert np.array_equal(part.run("tile")[0], got[rows])
        rows = np.unique(np.r_[np.arange(0, t, 61), t - 1])
        part.t, part.x, part.res = len(rows), c.x[rows], c.res[rows]
        part.check(got[rows])


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("fn", ["none", "silu"])
def test_infinities_and_nan_reach_what_multiplies_them(sparse, fn):
    """A NaN or an infinity in X makes those outputs so whose weight row keeps its position, with the
    weight's sign, and leaves the others' bits; a NaN in W its output of every token."""
    for t, o, k in ((6, 40, 256), (40, 70, 260), (300, 300, 260)):
        c = Case(9, t, o, k, sparse=sparse, fn=fn, kind=torch.float32)
        kept = np.ones((o, k), bool)
        if sparse:
            kept = O.expand_24_values(np.ones((o, k // 2), bool), c.idx, k)
        want = {r: c.run(r)[0] for r in ROUTES}
        c.xd[1, 5], c.xd[4, k - 1], c.xd[2, 0] = float("nan"), float("inf"), float("-inf")
        c.wd[7, 3] = float("nan")
        for r in ROUTES:
            print("linear not finite", sparse, fn, t, o, k, r, flush=True)
            got = c.run(r)[0]
            expect = want[r].copy()
            expect[1, kept[:, 5]] = np.nan
            for row, pos, sign in ((4, k - 1, 1.0), (2, 0, -1.0)):
                v = np.where(c.w[:, pos] == 0, np.nan, np.copysign(np.inf, sign * c.w[:, pos]))
                if fn == "silu":                                     # the limit 0 at -inf
                    v = np.where(v == -np.inf, c.res[row], v)
                expect[row, kept[:, pos]] = v[kept[:, pos]]
            expect[:, 7] = np.nan
            assert np.array_equal(got, expect, equal_nan=True)
