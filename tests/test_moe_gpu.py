"""The int8 mixture-of-experts layer on the GPU against the oracle's 64-bit definition, and against
nm_glu_i8, nm_quant_i8 and nm_spmm_i8 run expert by expert."""
import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import semi_structured_sparse_amd as S  # noqa: E402

U = 2.0 ** -24            # half a step of fp32, relative
UB = 2.0 ** -8            # half a step of bf16, relative


def sync():
    torch.cuda.synchronize()


def up(v, m):
    return -(-v // m) * m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def expert_weights(rng, e, rows, k, sparse, extra=0):
    """(device codes [e][rows][ld], device scales, device positions or None, dense values [e][rows][k],
    scales): pad bytes of a row hold anything."""
    wk = k // 2 if sparse else k
    codes = rng.integers(-127, 128, (e, rows, wk)).astype(np.int8)
    wide = rng.integers(-127, 128, (e, rows, up(wk, 16) + extra)).astype(np.int8)
    wide[:, :, :wk] = codes
    scale = (0.5 + rng.random((e, rows))).astype(np.float32) * np.float32(0.02 / 127)
    if not sparse:
        return dev(wide), dev(scale), None, codes, scale
    idx = np.sort(rng.random((e, rows, k // 4, 4)).argsort(3)[..., :2], axis=3).reshape(e, rows, k // 2).astype(np.uint8)
    meta = torch.zeros(e, -(-k // 128), rows, 16, dtype=torch.uint8, device="cuda")
    for i in range(e):
        if rows and k:
            S.nm_meta_block(dev(O.pack_meta_2bit(idx[i])), rows, k, meta[i])
    vals = np.stack([O.expand_24(codes[i], idx[i], k) for i in range(e)]) if e else codes
    return dev(wide), dev(scale), meta, vals, scale


class Case:
    def __init__(self, seed, t, e, top, h, i, sparse=False, act="silu", kind=torch.bfloat16, res=True, ids=None, extra=0):
        rng = np.random.default_rng(seed)
        self.sizes, self.act, self.kind, self.sparse = (t, e, top, h, i), act, kind, sparse
        self.x = rng.integers(-127, 128, (t, h)).astype(np.int8)
        wide = np.zeros((t, up(h, 16) + 16), np.int8)
        wide[:, :h] = self.x
        self.xd = dev(wide)
        self.xs = (rng.random(t) + 0.5).astype(np.float32) / np.float32(30)
        if ids is None:
            ids = np.stack([rng.permutation(e)[:top] for _ in range(t)]) if t else np.zeros((0, top))
        self.ids = np.asarray(ids, np.int32).reshape(t, top)
        self.w = rng.random((t, top)).astype(np.float32)
        self.gate, self.up, self.down = (expert_weights(rng, e, r, k, sparse, extra) for r, k in ((i, h), (i, h), (h, i)))
        self.res = O.bf16_round(rng.standard_normal((t, h)).astype(np.float32)) if res else None

    def run(self, ws=None, y=None, into_residual=False, **kw):
        t, e, top, h, i = self.sizes
        guard = 8
        if y is None:
            y = torch.full((t + 1, h + guard), 7.0, dtype=self.kind, device="cuda")
        r = None
        if self.res is not None:
            r = y if into_residual else torch.full((t, h + 3), float("nan"), dtype=self.kind, device="cuda")
            r[:t, :h] = dev(self.res).to(self.kind)
        if ws is None:
            n = S.nm_moe_i8_workspace_size(t, e, top, h, i, self.sparse)
            ws = torch.full((max(n, 16) + 64,), 0x7F, dtype=torch.uint8, device="cuda")   # NaN as bf16 or fp32
            ws = ws[:max(n, 16)]
        S.nm_moe_i8(self.xd, dev(self.xs), dev(self.ids), dev(self.w), self.gate[0], self.gate[1], self.up[0], self.up[1],
                    self.down[0], self.down[1], y, S.NM_GLU_SILU if self.act == "silu" else S.NM_GLU_GELU_TANH,
                    self.gate[2], self.up[2], self.down[2], residual=r, workspace=ws, t=t, experts=e, top=top, hidden=h,
                    inter=i, **kw)
        sync()
        assert (y[t] == 7.0).all() and (y[:, h:] == 7.0).all()
        return y[:t, :h].double().cpu().numpy()

    def check(self, got):
        t, e, top, h, i = self.sizes
        y, far, size = O.moe_i8(self.x, self.xs, self.ids, self.w, self.gate[3:], self.up[3:], self.down[3:], self.act,
                                self.res)
        # fp32: a part's sum, its two scales and weight (4), its place among the parts of up to `top`
        # experts and 16 waves and the residual (top + 34); then y's own rounding
        bound = far + size * U * (top + 40)
        if self.kind == torch.bfloat16:
            bound = bound + UB * (np.abs(y) + bound)
        assert np.isfinite(got).all()
        worst = (np.abs(got - y) - bound - 1e-30).max() if got.size else 0
        assert worst <= 0, worst
        # and as a whole far nearer than that
        if got.size and far.max() < 1:
            assert np.linalg.norm(got - y) <= (4e-3 if self.kind == torch.bfloat16 else 1e-3) * np.linalg.norm(y)


SIZES = [  # t, experts, top, hidden, inter
    (1, 1, 1, 16, 16), (1, 8, 2, 256, 128), (2, 3, 3, 100, 36), (3, 64, 8, 512, 132), (5, 5, 1, 1028, 4),
    (16, 16, 4, 320, 64), (17, 4, 2, 260, 260), (33, 8, 2, 128, 192), (64, 4, 2, 64, 68), (64, 2, 2, 132, 128),
    (64, 130, 3, 96, 40), (20, 1000, 5, 64, 16), (7, 9, 9, 4, 4), (40, 6, 1, 2048, 8), (30, 3, 2, 36, 1500),
]


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("sizes", SIZES)
def test_sizes(sizes, sparse):
    for n, (act, kind, res) in enumerate([("silu", torch.float32, True), ("gelu", torch.bfloat16, False)]):
        print("moe", sizes, sparse, act, kind, flush=True)
        c = Case(7 * n + sizes[0], *sizes, sparse=sparse, act=act, kind=kind, res=res, extra=16 * n)
        c.check(c.run())


@pytest.mark.parametrize("sizes", [(1, 4, 2, 37, 41), (9, 7, 3, 131, 65), (19, 3, 2, 65, 129), (1, 2, 1, 1, 1), (4, 2, 2, 16, 300)])
def test_odd_sizes(sizes):
    print("moe odd", sizes, flush=True)
    c = Case(3, *sizes, kind=torch.float32)
    c.check(c.run())


@pytest.mark.parametrize("t", [65, 128, 200])
def test_more_tokens_than_a_pass(t):
    c = Case(t, t, 6, 2, 64, 32)
    c.check(c.run())


def test_ids_that_name_no_expert_and_the_same_twice():
    t, e, top = 34, 5, 4
    rng = np.random.default_rng(1)
    ids = rng.integers(-1, e, (t, top))
    ids[0] = -1                                                   # a token without an expert
    ids[1] = [2, 2, 2, 2]
    ids[2] = [0, 3, 0, 3]
    ids[3] = [e, 1 << 30, -(1 << 31), 1]
    ids[4:30] = 3                                                 # a crowd: over one item
    for kind in (torch.float32, torch.bfloat16):
        for sparse in (False, True):
            c = Case(2, t, e, top, 96, 64, sparse=sparse, kind=kind, ids=ids)
            got = c.run()
            c.check(got)
            assert np.array_equal(got[0], c.res[0])
    c = Case(2, 3, e, 2, 96, 64, ids=np.full((3, 2), -1), res=False)
    assert (c.run() == 0).all()


def test_no_hidden_units():
    c = Case(5, 3, 4, 2, 64, 0, kind=torch.float32)
    got = c.run()
    assert np.array_equal(got, c.res.astype(np.float64))


def test_residual_in_place():
    for kind in (torch.float32, torch.bfloat16):
        c = Case(6, 9, 4, 2, 72, 48, kind=kind)
        assert np.array_equal(c.run(), c.run(into_residual=True))


def test_rows_that_are_not_finite_stay_alone():
    """A token whose scale is NaN or infinite has an output of that kind; the others keep their bits."""
    c = Case(8, 6, 3, 2, 64, 48, kind=torch.float32)
    want = c.run()
    c.xs[2], c.xs[4] = np.nan, np.inf
    got = c.run()
    for r in range(6):
        if r in (2, 4):
            assert not np.isfinite(got[r]).any()
        else:
            assert np.array_equal(got[r], want[r])


def test_is_the_composition_of_its_products():
    """Each expert alone, weight 1, no residual: nm_glu_i8, nm_quant_i8, nm_spmm_i8 in bits, where no
    reduction is cut in parts that are scaled apart (a single wave's: few steps)."""
    for sparse in (False, True):
        t, e, h, i = 11, 3, 192, 64
        c = Case(9, t, e, 1, h, i, sparse=sparse, kind=torch.float32, res=False)
        c.w[:] = 1
        got = c.run()
        for k in range(e):
            rows = np.nonzero(c.ids[:, 0] == k)[0]
            x, xs = c.xd[dev(rows)].contiguous(), dev(c.xs[rows])
            hid = torch.empty(len(rows), i, dtype=torch.bfloat16, device="cuda")
            S.nm_glu_i8(x, xs, c.gate[0][k], c.gate[1][k], c.up[0][k], c.up[1][k], hid,
                        gate_meta=None if c.gate[2] is None else c.gate[2][k].contiguous(),
                        up_meta=None if c.up[2] is None else c.up[2][k].contiguous(), k=h)
            q, s = torch.zeros(len(rows), up(i, 16), dtype=torch.int8, device="cuda"), torch.zeros(len(rows), device="cuda")
            S.nm_quant_i8(hid, q, s)
            y = torch.empty(len(rows), h, device="cuda")
            S.nm_spmm_i8(q, s, c.down[0][k], c.down[1][k].contiguous(), y,
                         None if c.down[2] is None else c.down[2][k].contiguous(), k=i)
            sync()
            assert np.array_equal(got[rows], y.double().cpu().numpy()), (sparse, k)


def test_repeated_calls_give_the_same_bits():
    c = Case(10, 48, 12, 4, 512, 384)
    want = c.run()
    for _ in range(10):
        assert np.array_equal(c.run(), want)


def test_offsets_past_32_bits():
    """Experts whose weights start more than 2^32 bytes in."""
    e, h, i = 70, 64, 64
    c = Case(11, 5, e, 3, h, i, kind=torch.float32, ids=np.random.default_rng(3).integers(65, e, (5, 3)))
    ld = 1 << 20
    for w, rows, k in ((c.gate, i, h), (c.up, i, h)):
        far = torch.empty(e, rows, ld, dtype=torch.int8, device="cuda")
        far[:, :, :k] = w[0][:, :, :k]
        c.__dict__["gate" if w is c.gate else "up"] = (far,) + w[1:]
    far = torch.empty(e, h, ld, dtype=torch.int8, device="cuda")
    far[:, :, :i] = c.down[0][:, :, :i]
    c.down = (far,) + c.down[1:]
    c.check(c.run())


def test_captured_streams_and_a_shared_workspace():
    """Two captured layers with one workspace, replayed in turn with eager work between, and the layer on
    a stream of its own."""
    cases = [Case(20 + n, 6, 8, 2, 128, 96, sparse=bool(n)) for n in range(2)]
    t, e, top, h, i = cases[0].sizes
    ws = torch.empty(S.nm_moe_i8_workspace_size(t, e, top, h, i), dtype=torch.uint8, device="cuda")
    want = [c.run(ws=ws) for c in cases]
    graphs, outs = [], []
    for c in cases:
        args = [c.xd, dev(c.xs), dev(c.ids), dev(c.w), c.gate[0], c.gate[1], c.up[0], c.up[1], c.down[0], c.down[1]]
        y, r = torch.zeros(t, h, dtype=c.kind, device="cuda"), dev(c.res).to(c.kind)
        kw = dict(gate_meta=c.gate[2], up_meta=c.up[2], down_meta=c.down[2], residual=r, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            S.nm_moe_i8(*args, y, **kw)
        graphs.append((g, args, kw))
        outs.append(y)
    for n in (0, 1, 1, 0, 1, 0):
        outs[n].fill_(float("nan"))
        graphs[n][0].replay()
        sync()
        assert np.array_equal(outs[n].double().cpu().numpy(), want[n])
        torch.randn(100, 100, device="cuda").sum().item()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = torch.zeros(t, h, dtype=cases[0].kind, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    S.nm_moe_i8(*graphs[0][1], y, stream=side, **graphs[0][2])
    side.synchronize()
    assert np.array_equal(y.double().cpu().numpy(), want[0])


def test_route_then_layer():
    """The router's ids and weights as they come, rows without an expert among them."""
    rng = np.random.default_rng(30)
    t, e, top = 23, 12, 3
    logits = rng.standard_normal((t, e)).astype(np.float32)
    logits[5] = -np.inf
    logits[6, 1:] = -np.inf
    ids, w = torch.zeros(t, top, dtype=torch.int32, device="cuda"), torch.zeros(t, top, device="cuda")
    S.nm_moe_route(dev(logits), ids, w)
    sync()
    c = Case(31, t, e, top, 80, 56, kind=torch.float32, ids=ids.cpu().numpy())
    c.w = w.cpu().numpy()
    got = c.run()
    c.check(got)
    assert np.array_equal(got[5], c.res[5].astype(np.float64))
