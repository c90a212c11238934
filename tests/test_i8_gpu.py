"""The int8 layers on the GPU against the oracle's 64-bit definitions: codes, scales, blocked
positions bit for bit; products within the roundings their formula counts, and the same bits
on every route."""
import ctypes

import numpy as np
import pytest

import oracle as O
import synth
from nm_testutil import dev, empty, host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import semi_structured_sparse_amd as S  # noqa: E402

U = 2.0 ** -24            # half a step of fp32, relative
UB = 2.0 ** -8            # half a step of bf16, relative
ROUTES = {"auto": 0, "stream": S.route_bits("few_stream"), "split": S.route_bits("few_tile"),
          "tile": S.route_bits("tile_lds")}


def sync():
    torch.cuda.synchronize()


def up(v, m):
    return -(-v // m) * m


# -------------------------------------------------------------------------------- quant ---

def run_quant(x, n=0, m=0, ns=2, ldx=None, extra=16):
    """Codes and scales of bf16 rows x, checked: the zero padding, and the bytes beyond it and
    the row after the last one left as they were."""
    rows, k = x.shape
    kq = O.lowered_k(k, ns) if ns > 2 else k
    ldq = up(kq, 16) + extra
    q = torch.full((rows + 1, ldq), 77, dtype=torch.int8, device="cuda")
    s = torch.full((rows + 1,), -3.0, device="cuda")
    ldx = up(k, 8) if ldx is None else ldx
    xd = torch.full((rows, max(ldx, 8)), 0x7FC0, dtype=torch.int16, device="cuda")   # NaN past the row
    xd[:, :k] = dev(x)
    S.nm_quant_i8(xd, q, s, n, m, ns, rows=rows, k=k, ldx=ldx)
    sync()
    q, s = q.cpu().numpy(), s.cpu().numpy()
    assert (q[rows] == 77).all() and s[rows] == -3.0
    assert (q[:rows, up(kq, 16):] == 77).all()
    assert (q[:rows, kq:up(kq, 16)] == 0).all()
    return q[:rows, :kq], s[:rows]


def check_quant(x, n=0, m=0, ns=2, **kw):
    q, s = run_quant(x, n, m, ns, **kw)
    rq, rs = O.quantize_rows_i8(x, n, m, ns)
    assert (q == rq).all(), f"{(q != rq).sum()} codes differ"
    assert (s.view(np.uint32) == rs.view(np.uint32))[~np.isnan(rs)].all()
    assert np.isnan(s[np.isnan(rs)]).all()


@pytest.mark.parametrize("k", [0, 1, 7, 8, 9, 16, 17, 100, 513, 2048, 2056, 4096, 8192, 8200, 14336, 16400, 32768, 65536])
def test_quant_lengths(k):
    print("quant", k, flush=True)
    rng = np.random.default_rng(k)
    check_quant(synth.student_t_bf16(rng, (5 if k > 3000 else 11, k), 4.0, 0.5))
    check_quant(synth.student_t_bf16(rng, (1, k), 4.0, 0.5), extra=0 if k else 16, ldx=up(k, 8) + 8)


@pytest.mark.parametrize("m", [4, 8, 16, 32])
def test_quant_selected(m):
    rng = np.random.default_rng(m)
    for k in (m, 5 * m, 2048 - m, 2048 + m, 8192, 8192 + m, 14336, 32768 + m, 65536):
        print("quant", m, k, flush=True)
        x = synth.student_t_bf16(rng, (3, k), 4.0, 0.5)
        x[0, : k // 2] = x[0, 0]                                 # ties: the lower index
        for n in {1, m // 2, m - 1, m}:
            check_quant(x, n, m)


@pytest.mark.parametrize("ns", [3, 4, 5, 6, 7, 8])
def test_quant_lifted(ns):
    rng = np.random.default_rng(ns)
    for groups in (1, 3, 100, 256, 1025, 65536 // (2 * ns)):
        print("quant lift", ns, groups, flush=True)
        check_quant(synth.student_t_bf16(rng, (3, 2 * ns * groups), 4.0, 0.5), ns=ns)


def test_quant_borders_and_ranges():
    """Exact ties, every exponent of the largest value, and rows whose largest is subnormal."""
    a = np.arange(128, dtype=np.uint16) + 0x3F80
    rows = []
    for b in range(128):
        row = np.concatenate([a, a - 0x80, a - 0x100, a - 0x380])
        row = np.minimum(row, 0x3F80 + b).astype(np.uint16)
        row[::3] |= 0x8000
        row[0] = 0x3F80 + b
        rows.append(row)
    x = np.stack(rows)
    check_quant(x)
    for e in (1, 40, 86, 87, 88, 126, 128, 166, 167, 168, 253, 254):   # exponent fields of the largest
        y = (x.astype(np.int64) & 0x7FFF) + (e - 127) * 128
        y = np.where(y > 0, y, x & 0x7F) | (x & 0x8000)
        check_quant(y.astype(np.uint16))
    sub = np.arange(128, dtype=np.uint16)[None, :].repeat(6, 0)
    sub = np.minimum(sub, np.array([[1], [2], [3], [64], [126], [127]], np.uint16))
    check_quant(sub | np.where(np.arange(128) % 2, 0x8000, 0).astype(np.uint16))


def test_quant_more_rows_than_one_launch_takes():
    k, distinct, rows = 8, 61, (1 << 22) + 5
    x = synth.normal_bf16(np.random.default_rng(k), (distinct, k))
    rq, rs = O.quantize_rows_i8(x)
    pick = torch.arange(rows, device="cuda") % distinct
    xd = dev(x)[pick]
    q = torch.full((rows, up(k, 16)), 77, dtype=torch.int8, device="cuda")
    s = torch.zeros(rows, device="cuda")
    S.nm_quant_i8(xd, q, s, k=k)
    sync()
    wq = torch.zeros(distinct, up(k, 16), dtype=torch.int8, device="cuda")
    wq[:, :k] = torch.from_numpy(rq).cuda()
    assert torch.equal(q, wq[pick]) and torch.equal(s, dev(rs)[pick])


def test_quant_zero_and_nonfinite_rows():
    rng = np.random.default_rng(3)
    for k in (64, 4096, 16384):
        x = synth.normal_bf16(rng, (6, k))
        x[0] = 0
        x[1] = 0x8000
        x[2, k - 1] = 0x7F80
        x[3, 5] = 0xFFC1
        x[4, 7], x[4, 9] = 0xFF80, 0x7FC0
        check_quant(x)
        check_quant(x, 2, 4)
        check_quant(x, ns=4)
        check_quant(x[:, :60], ns=3)


# ------------------------------------------------------------------------------ products ---

def random_codes(rng, rows, k, ld, pad_zero):
    c = rng.integers(-128, 128, (rows, ld)).astype(np.int8)
    if pad_zero:
        c[:, k:up(k, 16)] = 0
    return c


def make_weight(rng, o, k, sparse, ld_extra=0):
    """(device codes, device blocked positions or None, scales, dense int values [o][k])."""
    s = (rng.random(o) * 0.01 + 1e-4).astype(np.float32)
    if not sparse:
        c = random_codes(rng, o, k, up(k, 16) + ld_extra, False)
        return torch.from_numpy(c).cuda(), None, s, c[:, :k]
    idx = np.sort(rng.random((o, k // 4, 4)).argsort(2)[:, :, :2], axis=2).reshape(o, k // 2).astype(np.uint8)
    c = random_codes(rng, o, k // 2, up(k // 2, 16) + ld_extra, False)
    meta = O.pack_meta_2bit(idx)
    blk = torch.empty(max(S.nm_meta_block_bytes(o, k), 16), dtype=torch.uint8, device="cuda")
    S.nm_meta_block(dev(meta), o, k, blk)
    return torch.from_numpy(c).cuda(), blk, s, O.expand_24(c[:, :k // 2], idx, k)


class Guarded:
    """An output [t][o] inside a larger buffer whose other elements must not change."""

    def __init__(self, t, o, ldy, bf16=False):
        self.t, self.o = t, o
        self.buf = torch.full((t + 3, ldy), 7.25, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
        self.y = self.buf[:t]

    def get(self):
        sync()
        b = self.buf.float().cpu().numpy().astype(np.float64)
        assert (b[self.t:] == 7.25).all() and (b[:, self.o:] == 7.25).all(), "written outside the output"
        return b[:self.t, :self.o]


def ws_for(t, o, k, sparse, glu, route=0):
    n = S.nm_i8_workspace_size(t, o, k, sparse, glu, route)
    return torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")


def check_product(rng, t, o, k, sparse, routes=("auto",), bf16=False, shift=0, accumulate=0, ldy=None, ld_extra=0):
    print("product", t, o, k, "sparse" if sparse else "dense", flush=True)
    x = random_codes(rng, t, k, up(k, 16) + ld_extra, True)
    xs = (rng.random(t) * 0.1 + 1e-3).astype(np.float32)
    wd, meta, sc, wv = make_weight(rng, o, k, sparse, ld_extra)
    xd, xsd, scd = torch.from_numpy(x).cuda(), dev(xs), dev(sc)
    cs = rng.standard_normal(o).astype(np.float32) if shift else None
    rb = rng.standard_normal(t).astype(np.float32) if shift == 2 else None
    v = O.scaled_i8(O.sums_i8(x[:, :k], wv), xs, sc)
    term = (np.ones((t, 1)) if rb is None else rb[:, None].astype(np.float64)) * (0 if cs is None else cs[None, :])
    want = v + term + (7.25 if accumulate else 0.0)
    # the sum to fp32, two products; the shift's product and sum; the accumulation
    tol = 3.01 * U * np.abs(v) + (U * np.abs(term) + 1.01 * U * np.abs(v + term) if shift else 0)
    if accumulate:
        tol = tol + 1.01 * U * np.abs(want)
    if bf16:
        tol = tol + 1.01 * UB * np.abs(want)
    got = {}
    for r in routes:
        for ws in (ws_for(t, o, k, sparse, False, ROUTES[r]), None):
            g = Guarded(t, o, ldy or o, bf16)
            taken = ctypes.c_uint32(0)
            S.nm_spmm_i8(xd, xsd, wd, scd, g.y, meta, None if rb is None else dev(rb), None if cs is None else dev(cs),
                         accumulate, ws, t=t, o=o, k=k, route=ROUTES[r], taken=taken)
            y = g.get()
            names = S.taken_names(taken.value)
            assert ("sparse_mma" in names) == bool(sparse)
            assert (np.abs(y - want) <= tol).all(), (r, np.abs(y - want).max())
            got[r, ws is None] = y
    first = next(iter(got.values()))
    for key, y in got.items():
        assert np.array_equal(y, first), key
    return names


@pytest.mark.parametrize("sparse", [False, True])
def test_product_small_shapes(sparse):
    rng = np.random.default_rng(20 + sparse)
    for t, o, k in [(1, 1, 4), (1, 16, 64), (3, 17, 128), (16, 33, 100), (17, 5, 132), (33, 64, 60), (64, 16, 256),
                    (65, 129, 260), (130, 260, 516), (1, 1000, 2048), (2, 48, 8192)]:
        check_product(rng, t, o, k, sparse, routes=tuple(ROUTES), ldy=o + (t % 3))


@pytest.mark.parametrize("k", [1, 2, 15, 16, 17, 63, 65, 127, 129, 1999])
def test_dense_odd_reductions(k):
    rng = np.random.default_rng(k)
    for t, o in [(1, 7), (20, 40), (70, 130), (300, 257)]:
        check_product(rng, t, o, k, False, routes=tuple(ROUTES), ld_extra=16 * (k % 3))


@pytest.mark.parametrize("sparse", [False, True])
def test_product_forms(sparse):
    rng = np.random.default_rng(30 + sparse)
    for t, o, k in [(5, 100, 512), (40, 72, 384), (200, 300, 640)]:
        for bf16, shift, acc in [(True, 0, 0), (True, 1, 0), (False, 2, 0), (False, 0, 1), (False, 2, 1), (True, 2, 0)]:
            check_product(rng, t, o, k, sparse, routes=tuple(ROUTES), bf16=bf16, shift=shift, accumulate=acc, ldy=o + 5 * acc)
            check_product(rng, t, o, k, sparse, bf16=bf16, shift=shift, accumulate=acc, ldy=up(o, 8) + 8)


@pytest.mark.parametrize("sparse", [False, True])
def test_product_larger_shapes(sparse):
    rng = np.random.default_rng(40 + sparse)
    for t, o, k in [(1, 4096, 4096), (16, 1024, 14336), (61, 1030, 4096), (256, 512, 4096), (333, 1025, 2048),
                    (700, 1024, 1536), (1100, 2100, 640)]:
        check_product(rng, t, o, k, sparse)
        check_product(rng, t, o, k, sparse, bf16=True, ldy=up(o, 8))
        check_product(rng, t, o, k, sparse, bf16=True, shift=1, ldy=o + 1 - o % 2)
        check_product(rng, t, o, k, sparse, accumulate=1, ldy=o + 1 - o % 2)


SPLIT_SHAPES = [(1, 65, 32768), (8, 501, 32768), (16, 512, 14336), (40, 258, 14336), (61, 1030, 8192), (130, 300, 9000),
                (200, 1001, 6144)]


@pytest.mark.parametrize("sparse", [False, True])
def test_split_reductions(sparse):
    """Shapes whose reduction is cut across workgroups, with every epilogue of the summing kernel."""
    rng = np.random.default_rng(44 + sparse)
    for t, o, k in SPLIT_SHAPES:
        assert S.nm_i8_workspace_size(t, o, k, sparse, False) > 0, (t, o, k)
        check_product(rng, t, o, k, sparse, routes=("auto", "stream", "split"))
        check_product(rng, t, o, k, sparse, bf16=True, shift=1, ldy=up(o, 8))
        check_product(rng, t, o, k, sparse, shift=2, accumulate=1, ldy=o + 3)
        check_product(rng, t, o, k, sparse, shift=2, ldy=up(o, 4), routes=("auto", "tile"))


@pytest.mark.parametrize("sparse", [False, True])
def test_tiles_give_the_same_bits_every_time(sparse):
    """Smaller and 256 x 256 tiles, several workgroups a CU and long reductions, call after call."""
    rng = np.random.default_rng(46 + sparse)
    for t, o, k in [(700, 1024, 4096), (500, 1536, 4096), (700, 2048, 2048), (1024, 3000, 1024)]:
        x = torch.from_numpy(random_codes(rng, t, k, k, True)).cuda()
        wd, meta, _, _ = make_weight(rng, o, k, sparse)
        ones_t, ones_o = torch.ones(t, device="cuda"), torch.ones(o, device="cuda")
        want, y = (torch.empty(t, o + 1, device="cuda") for _ in range(2))
        S.nm_spmm_i8(x, ones_t, wd, ones_o, want, meta, k=k, route=ROUTES["stream"])
        for i in range(90):
            y.fill_(float("nan"))
            S.nm_spmm_i8(x, ones_t, wd, ones_o, y, meta, k=k, route=ROUTES["split" if i % 3 else "tile"])
            sync()
            assert torch.equal(y[:, :o], want[:, :o]), (t, o, k, i)


def test_longest_reduction_stays_inside_32_bits():
    """All codes -128: the sum is 128 * 128 * k, the largest that can occur."""
    k = S.NM_I8_MAX_K
    for t in (1, 40, 200):
        x = torch.zeros(t, up(k, 16), dtype=torch.int8, device="cuda")
        x[:, :k] = -128
        w = torch.full((20, up(k, 16)), -128, dtype=torch.int8, device="cuda")
        one = torch.ones(200, device="cuda")
        for r in ROUTES.values():
            g = Guarded(t, 20, 20)
            S.nm_spmm_i8(x, one, w, one, g.y, k=k, route=r, workspace=ws_for(t, 20, k, False, False, r))
            assert (g.get() == float(np.float32(16384 * k))).all()


def test_zero_reduction():
    one = torch.ones(40, device="cuda")
    cs = torch.arange(40, device="cuda").float()
    g = Guarded(3, 40, 40)
    S.nm_spmm_i8(None, one, None, one, g.y, col_shift=cs, t=3, o=40, k=0, ldx=0, ldw=0)
    assert (g.get() == np.arange(40)).all()
    g = Guarded(3, 40, 40, True)
    S.nm_glu_i8(None, one, None, one, None, one, g.y, t=3, inter=40, k=0, ldx=0, ldw=0)
    assert (g.get() == 0).all()


def test_nonfinite_rows_give_nan_and_no_other_row_changes():
    rng = np.random.default_rng(50)
    k, o = 256, 70
    for t in (4, 70, 300):
        xb = synth.normal_bf16(rng, (t, k))
        clean = xb.copy()
        xb[1, 3], xb[t - 1, 200] = 0x7F80, 0x7FC0
        wd, meta, sc, _ = make_weight(rng, o, k, True)
        ys = []
        for b in (xb, clean):
            q = torch.empty(t, k, dtype=torch.int8, device="cuda")
            s = torch.empty(t, device="cuda")
            S.nm_quant_i8(dev(b), q, s)
            g = Guarded(t, o, o)
            S.nm_spmm_i8(q, s, wd, dev(sc), g.y, meta, k=k)
            ys.append(g.get())
        bad = np.zeros(t, bool)
        bad[[1, t - 1]] = True
        assert np.isnan(ys[0][bad]).all() and np.array_equal(ys[0][~bad], ys[1][~bad])


# ----------------------------------------------------------------------------------- glu ---

def check_glu(rng, t, o, k, sparse, act, routes=("auto",), bf16=False, ldy=None, big=1.0):
    print("glu", t, o, k, sparse, act, flush=True)
    x = random_codes(rng, t, k, up(k, 16), True)
    xs = (rng.random(t) * 0.1 + 1e-3).astype(np.float32)
    w0, m0, s0, v0 = make_weight(rng, o, k, sparse)
    w1, m1, s1, v1 = make_weight(rng, o, k, sparse)
    s0 = (s0 * big / np.sqrt(k)).astype(np.float32)
    xd = torch.from_numpy(x).cuda()
    g = O.scaled_i8(O.sums_i8(x[:, :k], v0), xs, s0)
    u = O.scaled_i8(O.sums_i8(x[:, :k], v1), xs, s1)
    want = O.glu_gate(g, act) * u
    # g and u are 3 U off.  The gate is g / (1 + e^-z): a relative error e of g gives at most
    # (1 + |g z'|) e, |g z'| <= 3 |z|; z itself is formed with 4 roundings and its exponential
    # with one more of |z| U and two steps (4 U); then the sum (U), the reciprocal (one ulp:
    # 2 U), its product with g and the product with u (U each).
    z = g if act == "silu" else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    rel = (3 * (1 + 3 * np.abs(z)) + 5 * np.abs(z) + 3 + 4 + 5) * 1.01 * U
    tol = rel * np.abs(want) + 2.0 ** -120 * (1 + np.abs(u))     # e^-z past the fp32 range: 0
    if bf16:
        tol = tol + 1.01 * UB * np.abs(want)
    got = []
    for r in routes:
        for ws in (ws_for(t, o, k, sparse, True, ROUTES[r]), None):
            gd = Guarded(t, o, ldy or o, bf16)
            S.nm_glu_i8(xd, dev(xs), w0, dev(s0), w1, dev(s1), gd.y,
                        S.NM_GLU_SILU if act == "silu" else S.NM_GLU_GELU_TANH, m0, m1, ws, t=t, inter=o, k=k,
                        route=ROUTES[r])
            y = gd.get()
            assert (np.abs(y - want) <= tol).all(), (r, (np.abs(y - want) / np.maximum(tol, 1e-300)).max())
            got.append(y)
    for y in got[1:]:
        assert np.array_equal(y, got[0])


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("sparse", [False, True])
def test_glu(sparse, act):
    rng = np.random.default_rng(60 + sparse)
    for t, o, k in [(1, 1, 4), (1, 40, 64), (8, 100, 516), (17, 129, 256), (64, 72, 128), (70, 130, 1024), (300, 200, 260)]:
        for big in (1.0, 40.0):
            check_glu(rng, t, o, k, sparse, act, routes=tuple(ROUTES), big=big, ldy=o + t % 2)
        check_glu(rng, t, o, k, sparse, act, routes=tuple(ROUTES), bf16=True, ldy=up(o, 8))
        check_glu(rng, t, o, k, sparse, act, routes=tuple(ROUTES), bf16=True, ldy=o + 1 - o % 2)
    for t, o, k in [(1, 2048, 4096), (8, 14336, 256), (600, 1030, 1024), (1100, 1100, 640)]:
        check_glu(rng, t, o, k, sparse, act)
        check_glu(rng, t, o, k, sparse, act, bf16=True)


@pytest.mark.parametrize("sparse", [False, True])
def test_glu_split_reductions(sparse):
    rng = np.random.default_rng(64 + sparse)
    for t, o, k in SPLIT_SHAPES[:-2] + [(130, 300, 9000)]:
        assert S.nm_i8_workspace_size(t, o, k, sparse, True) > 0, (t, o, k)
        check_glu(rng, t, o, k, sparse, "silu", routes=("auto", "stream", "split"))
        check_glu(rng, t, o, k, sparse, "gelu", bf16=True, ldy=up(o, 4))


def test_glu_far_gates():
    """Gates where the exponential overflows, and infinite and NaN ones."""
    one = torch.ones(16, device="cuda")
    x = torch.zeros(4, 16, dtype=torch.int8, device="cuda")
    x[:, 0] = 1
    wg = torch.zeros(16, 16, dtype=torch.int8, device="cuda")
    wg[0::2, 0], wg[1::2, 0] = 1, -1
    xs = torch.tensor([1.0, 1e4, 3e38, float("nan")], device="cuda")
    gs = torch.full((16,), 100.0, device="cuda")
    for act in (S.NM_GLU_SILU, S.NM_GLU_GELU_TANH):
        g = Guarded(4, 16, 16)
        S.nm_glu_i8(x, xs, wg, gs, wg, 1e-30 * one, g.y, act)
        y = g.get()
        assert np.isnan(y[3]).all()
        assert (np.abs(y[:3, 1::2]) <= 1e-30).all()              # far negative gates vanish
        assert (y[2, 0::2] == np.inf).all() or (y[2, 0::2] > 1e30).all()
        assert np.allclose(y[:2, 0::2], np.array([[1e-28], [1e6 * 1e-26]]), rtol=1e-5)


# ------------------------------------------------------------------- positions, the run ---

def test_meta_block():
    rng = np.random.default_rng(70)
    for o, kc in [(1, 4), (3, 8), (7, 60), (5, 128), (33, 132), (64, 1024), (9, 2052), (300, 4096)]:
        meta = rng.integers(0, 256, (o, -(-kc // 8))).astype(np.uint8)
        n = S.nm_meta_block_bytes(o, kc)
        out = torch.full((n + 32,), 0xEE, dtype=torch.uint8, device="cuda")
        S.nm_meta_block(dev(meta), o, kc, out)
        sync()
        got = out.cpu().numpy()
        assert (got[n:] == 0xEE).all()
        assert (got[:n].reshape(-1, o, 16) == O.block_meta(meta, kc)).all(), (o, kc)


def mlp(x, lowered, t, hid, inter, bufs):
    """One GLU MLP as a served layer runs it: quantize, gate and up, quantize (8:16 or the 6:8
    lift), down."""
    w = bufs["w"]
    S.nm_quant_i8(x, bufs["q1"], bufs["s1"])
    S.nm_glu_i8(bufs["q1"], bufs["s1"], w["g"], w["gs"], w["u"], w["us"], bufs["h"], S.NM_GLU_SILU, w["gm"], w["um"],
                bufs["ws"], k=hid)
    if lowered:
        S.nm_quant_i8(bufs["h"], bufs["q2"], bufs["s2"], ns=4)
        S.nm_spmm_i8(bufs["q2"], bufs["s2"], w["d"], w["ds"], bufs["y"], w["dm"], workspace=bufs["ws"], k=inter * 3 // 2)
    else:
        S.nm_quant_i8(bufs["h"], bufs["q2"], bufs["s2"], 8, 16)
        S.nm_spmm_i8(bufs["q2"], bufs["s2"], w["d"], w["ds"], bufs["y"], workspace=bufs["ws"], k=inter)


def pack_24(w_bits):
    """bf16 weights -> (codes, scales, blocked positions) with the library's own packing."""
    o, k = w_bits.shape
    v, meta = empty((o, k // 2), np.uint16), empty((o, -(-k // 8)), np.uint8)
    S.nm_compress(dev(w_bits), 2, 4, v, meta, S.NM_META_2BIT)
    return pack_values(v, meta, o, k)


def pack_values(v, meta, o, kc):
    q = torch.zeros(o, up(kc // 2, 16), dtype=torch.int8, device="cuda")
    s = torch.empty(o, device="cuda")
    S.nm_quant_i8(v, q, s, k=kc // 2)
    blk = torch.empty(S.nm_meta_block_bytes(o, kc), dtype=torch.uint8, device="cuda")
    S.nm_meta_block(meta, o, kc, blk)
    return q, s, blk


def pack_slide(w_bits, ns):
    o, k = w_bits.shape
    n, m = 2 * ns - 2, 2 * ns
    v, idx = empty((o, k // m * n), np.uint16), empty((o, k // m * n), np.uint8)
    S.nm_compress(dev(w_bits), n, m, v, idx, S.NM_META_U8)
    kc = S.lowered_k(k, ns)
    lv, lm = empty((o, kc // 2), np.uint16), empty((o, -(-kc // 8)), np.uint8)
    S.nm_lower_slide(v, idx, o, k, ns, lv, lm)
    return pack_values(lv, lm, o, kc)


def build_mlp(rng, t, hid, inter, lowered):
    wg, wu, wd = (synth.normal_bf16(rng, s, 0.05) for s in ((inter, hid), (inter, hid), (hid, inter)))
    g, gs, gm = pack_24(wg)
    u, us, um = pack_24(wu)
    if lowered:
        d, ds, dm = pack_slide(wd, 4)
    else:
        d, ds, dm = torch.zeros(hid, inter, dtype=torch.int8, device="cuda"), torch.empty(hid, device="cuda"), None
        S.nm_quant_i8(dev(wd), d, ds)
    k2 = inter * 3 // 2 if lowered else inter
    n = max(S.nm_i8_workspace_size(t, inter, hid, True, True), S.nm_i8_workspace_size(t, hid, k2, lowered, False), 16)
    bufs = {"w": dict(g=g, gs=gs, gm=gm, u=u, us=us, um=um, d=d, ds=ds, dm=dm),
            "q1": torch.empty(t, hid, dtype=torch.int8, device="cuda"), "s1": torch.empty(t, device="cuda"),
            "q2": torch.empty(t, k2, dtype=torch.int8, device="cuda"), "s2": torch.empty(t, device="cuda"),
            "h": torch.empty(t, inter, dtype=torch.bfloat16, device="cuda"), "y": torch.empty(t, hid, device="cuda"),
            "ws": torch.empty(n, dtype=torch.uint8, device="cuda")}
    return bufs, (wg, wu, wd)


def check_mlp(bufs, x_bits, weights, lowered):
    """Each step against its definition from what the step before gave, and the whole against
    the unquantized MLP of the pruned weights (two 8-bit roundings of operands, about 1% each)."""
    wg, wu, wd = weights
    q1, s1 = O.quantize_rows_i8(x_bits)
    assert (bufs["q1"].cpu().numpy() == q1).all() and (host(bufs["s1"], np.float32) == s1).all()
    vals = {}
    for name, w in (("g", wg), ("u", wu)):
        v, idx = O.compress(w, 2, 4)
        c, s = O.quantize_rows_i8(v)
        vals[name] = O.scaled_i8(O.sums_i8(q1, O.expand_24(c, idx, w.shape[1])), s1, s)
    want = O.glu_gate(vals["g"], "silu") * vals["u"]
    h = bufs["h"].float().cpu().numpy().astype(np.float64)
    # as in check_glu: (15 + 14 |g|) U from the gate, and the bf16 rounding
    tol = ((16 + 14 * np.abs(vals["g"])) * U + UB) * 1.02 * np.abs(want) + 2.0 ** -120
    assert (np.abs(h - want) <= tol).all()
    hb = bufs["h"].view(torch.int16).cpu().numpy().view(np.uint16)
    if lowered:
        q2, s2 = O.quantize_rows_i8(hb, ns=4)
        v, idx = O.compress(wd, 6, 8)
        vp, ip = O.slide_lower(v, idx, wd.shape[1], 4)
        c, s = O.quantize_rows_i8(vp)
        wv = O.expand_24(c, ip, q2.shape[1])
        pruned, _ = O.sparsify(wd, 6, 8)
        act = O.bf16_to_f64(hb)
    else:
        q2, s2 = O.quantize_rows_i8(hb, 8, 16)
        wv, s = O.quantize_rows_i8(wd)
        pruned = wd
        act = O.bf16_to_f64(O.sparsify(hb, 8, 16)[0])
    assert (bufs["q2"].cpu().numpy() == q2).all() and (host(bufs["s2"], np.float32) == s2).all()
    y = host(bufs["y"], np.float32).astype(np.float64)
    ref = O.scaled_i8(O.sums_i8(q2, wv), s2, s)
    assert (np.abs(y - ref) <= 3.01 * U * np.abs(ref)).all()
    # codes are off by at most half a step: |q s - v| <= amax / 254 in both operands of down
    dense = O.bf16_to_f64(pruned)
    e_h = np.abs(O.bf16_to_f64(hb)).max(1) / 254
    e_w = np.abs(dense).max(1) / 254
    full = act @ dense.T
    n_h = (np.abs(act).sum(1))[:, None] * e_w[None, :] + e_h[:, None] * np.abs(dense).sum(1)[None, :] \
        + e_h[:, None] * e_w[None, :] * dense.shape[1]
    assert (np.abs(y - full) <= 1.01 * n_h + 1e-6).all()


@pytest.mark.parametrize("lowered", [False, True])
@pytest.mark.parametrize("t", [1, 13, 90, 300])
def test_mlp_run(t, lowered):
    rng = np.random.default_rng(80 + t)
    hid, inter = 256, 768
    x = synth.normal_bf16(rng, (t, hid))
    bufs, weights = build_mlp(rng, t, hid, inter, lowered)
    mlp(dev(x), lowered, t, hid, inter, bufs)
    sync()
    check_mlp(bufs, x, weights, lowered)


def test_mlp_captured_and_replayed():
    """The whole run in one graph, replayed with new inputs, eager work in between."""
    rng = np.random.default_rng(90)
    t, hid, inter = 5, 256, 8192
    bufs, weights = build_mlp(rng, t, hid, inter, False)
    xd = torch.empty(t, hid, dtype=torch.int16, device="cuda")
    xs = [synth.normal_bf16(rng, (t, hid)) for _ in range(4)]
    xd.copy_(dev(xs[0]))
    mlp(xd, False, t, hid, inter, bufs)      # eager once
    sync()
    eager = []
    for x in xs:
        xd.copy_(dev(x))
        mlp(xd, False, t, hid, inter, bufs)
        eager.append(bufs["y"].clone())
    sync()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mlp(xd, False, t, hid, inter, bufs)
    for i in (0, 1, 2, 3, 1, 0):
        xd.copy_(dev(xs[i]))
        bufs["y"].fill_(float("nan"))
        g.replay()
        sync()
        assert torch.equal(bufs["y"], eager[i])
        torch.randn(100, 100, device="cuda").sum().item()
    check_mlp(bufs, xs[0], weights, False)


def test_two_streams_at_once():
    """Two streams, each with its own buffers and workspace, give what one after the other gives."""
    rng = np.random.default_rng(91)
    t, hid, inter = 24, 256, 4096
    sets = [build_mlp(rng, t, hid, inter, False) for _ in range(2)]
    xs = [dev(synth.normal_bf16(rng, (t, hid))) for _ in range(2)]
    want = []
    for (b, _), x in zip(sets, xs):
        mlp(x, False, t, hid, inter, b)
        sync()
        want.append(b["y"].clone())
        b["y"].zero_()
    sync()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for (b, _), x, s in zip(sets, xs, streams):
            with torch.cuda.stream(s):
                mlp(x, False, t, hid, inter, b)
    sync()
    for (b, _), w in zip(sets, want):
        assert torch.equal(b["y"], w)


def test_same_buffers_twice():
    """Gate and up may be one weight, and a call may be repeated: the same bits."""
    rng = np.random.default_rng(92)
    x = torch.from_numpy(random_codes(rng, 40, 256, 256, True)).cuda()
    wd, _, sc, _ = make_weight(rng, 100, 256, False)
    xs, scd = torch.ones(40, device="cuda"), dev(sc)
    ys = []
    for _ in range(3):
        g = Guarded(40, 100, 100)
        S.nm_glu_i8(x, xs, wd, scd, wd, scd, g.y)
        ys.append(g.get())
    assert np.array_equal(ys[0], ys[1]) and np.array_equal(ys[0], ys[2])


def test_binding_refuses_what_does_not_fit():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    q, s = torch.zeros(4, 64, dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda")
    y = torch.zeros(4, 4, device="cuda")
    for bad in (lambda: S.nm_quant_i8(x.half(), q, s), lambda: S.nm_spmm_i8(q, s, q, s, y.half()),
                lambda: S.nm_quant_i8(x.float(), q, s), lambda: S.nm_quant_i8(x, x, s), lambda: S.nm_quant_i8(x.t(), q, s),
                lambda: S.nm_quant_i8(x, q, s[:3]), lambda: S.nm_quant_i8(x, q, s.double()),
                lambda: S.nm_quant_i8(x, q.cpu(), s), lambda: S.nm_spmm_i8(q, s[:3], q, s, y),
                lambda: S.nm_spmm_i8(q, s, q, s[::2], y), lambda: S.nm_spmm_i8(x, s, q, s, y),
                lambda: S.nm_spmm_i8(q, s, q, s, y.to(torch.int8)), lambda: S.nm_spmm_i8(q, s, q, s, y.double()),
                lambda: S.nm_spmm_i8(q, s, q, s, y[:3]), lambda: S.nm_spmm_i8(q, s, q, s, y[:, :3]),
                lambda: S.nm_glu_i8(q, s, q, s, q, s, y[:3]), lambda: S.nm_glu_i8(q, s, q, s, q[:3], s, y),
                lambda: S.nm_quant_i8(x, q[:3], s), lambda: S.nm_spmm_i8(q, s, q, s, y, q[:, :15], k=64), lambda: S.nm_spmm_i8(q, s, q, s, y.cpu()), lambda: S.nm_spmm_i8(q, s, q, s, y, col_shift=s[:2]),
                lambda: S.nm_spmm_i8(q, s, q, s, y, workspace=q.cpu()), lambda: S.nm_glu_i8(q, s, q, s, q.t(), s, y),
                lambda: S.nm_glu_i8(q, s, q, s, torch.zeros(4, 128, dtype=torch.int8, device="cuda"), s, y)):
        with pytest.raises(ValueError):
            bad()


def far_rows(rows, ld, dtype, cols, host_rows):
    """rows x ld with the first columns set, the rest as the allocator left them."""
    a = torch.empty(rows, ld, dtype=dtype, device="cuda")
    a[:, :cols] = torch.from_numpy(host_rows).cuda().to(dtype)
    return a


@pytest.mark.parametrize("sparse", [False, True])
def test_offsets_past_32_bits(sparse):
    """Rows of X, W and y that start more than 2^32 bytes into their tensors, on every route, and
    an X whose leading dimension only the streaming kernel takes."""
    rng = np.random.default_rng(93 + sparse)
    k = 128
    for t, o, ldx, ldw, ldy, routes in [(4200, 300, 1 << 20, 256, 304, ("auto", "stream", "split", "tile")),
                                        (4200, 300, 256, 256, 1 << 18, ("auto", "stream", "split", "tile")),
                                        (40, 4200, 256, 1 << 20, 4200, ("auto", "stream", "split", "tile")),
                                        (520, 70, 1 << 23, 256, 70, ("auto",))]:
        print("far", t, o, ldx, ldw, ldy, flush=True)
        xc = random_codes(rng, t, k, k, True)
        _, meta, sc, wv = make_weight(rng, o, k, sparse)
        wk = k // 2 if sparse else k
        wc = rng.integers(-128, 128, (o, wk)).astype(np.int8)
        if sparse:
            idx = np.sort(rng.random((o, k // 4, 4)).argsort(2)[:, :, :2], axis=2).reshape(o, k // 2).astype(np.uint8)
            S.nm_meta_block(dev(O.pack_meta_2bit(idx)), o, k, meta)
            wv = O.expand_24(wc, idx, k)
        else:
            wv = wc
        want = O.sums_i8(xc, wv).astype(np.float64)      # exact in fp32: |sum| <= 2^21
        x, w = far_rows(t, ldx, torch.int8, k, xc), far_rows(o, ldw, torch.int8, wk, wc)
        y = torch.empty(t, ldy, device="cuda")
        one_t, one_o = torch.ones(t, device="cuda"), torch.ones(o, device="cuda")
        for r in routes:
            y[:, :o] = float("nan")
            S.nm_spmm_i8(x, one_t, w, one_o, y, meta, t=t, o=o, k=k, route=ROUTES[r],
                         workspace=ws_for(t, o, k, sparse, False, ROUTES[r]))
            sync()
            assert np.array_equal(y[:, :o].cpu().numpy().astype(np.float64), want), r
        del x, w, y
        torch.cuda.empty_cache()


def test_quant_offsets_past_32_bits():
    k, rows, ld = 100, 4200, 1 << 20
    xb = synth.normal_bf16(np.random.default_rng(95), (rows, k))
    x = torch.empty(rows, ld, dtype=torch.int16, device="cuda")
    x[:, :k] = dev(xb)
    q = torch.empty(rows, ld, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, device="cuda")
    S.nm_quant_i8(x, q, s, k=k)
    sync()
    rq, rs = O.quantize_rows_i8(xb)
    assert np.array_equal(q[:, :112].cpu().numpy(), np.pad(rq, ((0, 0), (0, 12)))) and np.array_equal(s.cpu().numpy(), rs)


def test_more_token_blocks_than_a_grid_dimension():
    t, o, k = 65535 * 64 + 70, 3, 16
    g = torch.Generator(device="cuda").manual_seed(96)
    x = torch.randint(-128, 128, (t, k), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (o, k), generator=g, device="cuda", dtype=torch.int8)
    y = torch.full((t + 1, 4), 7.25, device="cuda")
    for r in ROUTES:
        y[:t, :o] = float("nan")
        S.nm_spmm_i8(x, torch.ones(t, device="cuda"), w, torch.ones(o, device="cuda"), y, t=t, o=o, k=k, route=ROUTES[r])
        sync()
        want = torch.stack([(x.to(torch.int32) * w[i].to(torch.int32)).sum(1).float() for i in range(o)], 1)
        assert torch.equal(y[:t, :o], want), r
        assert (y[t] == 7.25).all() and (y[:, o:] == 7.25).all()


def test_two_graphs_share_a_workspace():
    """Two captured products with split reductions and one workspace, replayed in turn."""
    rng = np.random.default_rng(97)
    t, o, k = 20, 256, 16384
    assert S.nm_i8_workspace_size(t, o, k, False, False, 0) > 0
    ws = ws_for(t, o, k, False, False)
    calls = []
    for _ in range(2):
        x = torch.from_numpy(random_codes(rng, t, k, k, True)).cuda()
        wd, _, sc, _ = make_weight(rng, o, k, False)
        calls.append((x, torch.ones(t, device="cuda"), wd, dev(sc), torch.empty(t, o, device="cuda")))
    want, graphs = [], []
    for c in calls:
        S.nm_spmm_i8(*c, workspace=ws)
        sync()
        want.append(c[4].clone())
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            S.nm_spmm_i8(*c, workspace=ws)
        graphs.append(g)
    for i in (0, 1, 1, 0, 1, 0):
        calls[i][4].fill_(float("nan"))
        graphs[i].replay()
        sync()
        assert torch.equal(calls[i][4], want[i])
        torch.randn(100, device="cuda").sum().item()
