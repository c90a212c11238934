"""The norm to int8 codes and the routing of experts on the GPU against the oracle's 64-bit
definitions: codes, sums of the stream and ids bit for bit, the rest within the roundings that the
formulas count."""
import numpy as np
import pytest

import oracle as O
import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import semi_structured_sparse_amd as S  # noqa: E402

U = 2.0 ** -24            # half a step of fp32, relative
UB = 2.0 ** -8            # half a step of bf16, relative
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def sync():
    torch.cuda.synchronize()


def up(v, m):
    return -(-v // m) * m


def heavy(rng, rows, k):
    return O.f32_from_bf16(synth.student_t_bf16(rng, (rows, k), 4.0, 0.5))


def rows_on(v, ld, kind, fill=float("nan")):
    """fp32 values as rows of a type, NaN behind each row."""
    t = torch.full((v.shape[0], ld), fill, dtype=TYPES[kind], device="cuda")
    t[:, :v.shape[1]] = torch.from_numpy(v).cuda().to(TYPES[kind])
    return t


def run_norm(x, xt="bf16", r=None, rt="bf16", w=None, eps=1e-6, n=0, m=0, ns=2, extra=16, y=True, inplace=None):
    """Codes, scales, s and y, checked: zero codes up to 16, nothing else past the rows written."""
    rows, k = x.shape
    kq = O.lowered_k(k, ns) if ns > 2 else k
    q = torch.full((rows + 1, up(kq, 16) + extra), 77, dtype=torch.int8, device="cuda")
    scale = torch.full((rows + 1,), -3.0, device="cuda")
    ld = up(k, 8) + 8
    xd = rows_on(x, ld, xt)
    rd = None if r is None else rows_on(r, ld + 8, rt)
    sd = None if r is None else torch.full((rows + 1, ld + 16), 5.5, dtype=TYPES[rt], device="cuda")
    if inplace == "x":
        sd = xd
    elif inplace == "r":
        sd = rd
    yd = torch.full((rows + 1, ld), 5.5, dtype=torch.bfloat16, device="cuda") if y else None
    S.nm_rmsnorm_i8(xd, None if w is None else torch.from_numpy(w).cuda(), q, scale, rd, sd, yd, eps, n, m, ns, rows=rows,
                    k=k)
    sync()
    assert (q[rows] == 77).all() and scale[rows] == -3.0
    assert (q[:rows, up(kq, 16):] == 77).all() and (q[:rows, kq:up(kq, 16)] == 0).all()
    if sd is not None and inplace is None:
        assert (sd[rows] == 5.5).all() and (sd[:, k:] == 5.5).all()
    if inplace is not None:
        assert sd[:, k:].isnan().all()
    if y:
        assert (yd[rows] == 5.5).all() and (yd[:, k:] == 5.5).all()
    return (q[:rows, :kq].cpu().numpy(), scale[:rows].cpu().numpy().astype(np.float64),
            None if sd is None else sd[:rows, :k].float().cpu().numpy(),
            yd[:rows, :k].double().cpu().numpy() if y else None)


def check_norm(x, xt="bf16", r=None, rt="bf16", w=None, eps=1e-6, n=0, m=0, ns=2, **kw):
    q, scale, s, y = run_norm(x, xt, r, rt, w, eps, n, m, ns, **kw)
    rq, rscale, rs, ry = O.rmsnorm_i8(x, r, rt, w, eps, n, m, ns)
    assert (q == rq).all(), f"{(q != rq).sum()} codes differ"
    bad = ~np.isfinite(rscale)
    assert np.array_equal(scale[bad], rscale[bad], equal_nan=True)
    # rounded once from fp64 (whose own sums are off by 2^-40 at most)
    assert (np.abs(scale[~bad] - rscale[~bad]) <= U * (1 + 2.0 ** -10) * rscale[~bad] + 2.0 ** -150).all()
    if s is not None:
        assert np.array_equal(s.view(np.uint32)[~np.isnan(rs)], rs.view(np.uint32)[~np.isnan(rs)])
        assert np.isnan(s[np.isnan(rs)]).all()
    if y is not None:
        # the factor's and the product's roundings in fp32, then bf16's; 2^-134: half its least step
        good = np.isfinite(ry)
        assert (np.abs(y[good] - ry[good]) <= (UB + 4 * U) * np.abs(ry[good]) + 2.0 ** -134).all()


@pytest.mark.parametrize("k", [1, 7, 8, 9, 17, 100, 513, 2048, 2056, 4096, 4104, 8192, 14336, 16400, 32768])
def test_norm_lengths(k):
    rng = np.random.default_rng(k)
    for rows in (1, 7):
        print("norm", rows, k, flush=True)
        x, r = heavy(rng, rows, k), heavy(rng, rows, k)
        w = (1 + 0.3 * rng.standard_normal(k)).astype(np.float32)
        check_norm(x, "bf16", r, "bf16", w)
        check_norm(x, "bf16", None, "bf16", w, y=False, extra=0)
        check_norm(rng.standard_normal((rows, k)).astype(np.float32), "f32",
                   rng.standard_normal((rows, k)).astype(np.float32), "f32", w)


@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("rt", ["bf16", "f32"])
def test_norm_types_and_places(xt, rt):
    rng = np.random.default_rng(5)
    for k in (40, 3001, 5000):
        x, r = heavy(rng, 6, k), heavy(rng, 6, k)
        print("norm", xt, rt, k, flush=True)
        check_norm(x, xt, r, rt)
        check_norm(x, xt, r, rt, inplace="r")
        if xt == rt:
            check_norm(x, xt, r, rt, inplace="x")


@pytest.mark.parametrize("m", [4, 8, 16, 32])
def test_norm_selected(m):
    rng = np.random.default_rng(m)
    for k in (m, 5 * m, 2048 - m, 2048 + m, 8192, 8192 + m, 32768):
        print("norm", m, k, flush=True)
        x, r = heavy(rng, 3, k), heavy(rng, 3, k)
        x[0, :], r[0, :] = x[0, 0], r[0, 0]                       # ties: the lower index
        w = (1 + 0.3 * rng.standard_normal(k)).astype(np.float32)
        for n in {1, m // 2, m - 1, m}:
            check_norm(x, "bf16", r, "bf16", None, n=n, m=m)
            check_norm(x, "f32", r, "f32", w, n=n, m=m)


@pytest.mark.parametrize("m", [4, 8, 16, 32])
def test_norm_selected_ties(m):
    """Groups of a few values only, so that the border of what is kept falls between equal ones, which
    several lanes may hold; every n, rows of a wave's and of a workgroup's length."""
    rng = np.random.default_rng(50 + m)
    for k in (32 * 13, 32 * 90, 32 * 200):
        print("norm ties", m, k, flush=True)
        for n in range(1, m + 1):
            x = rng.integers(-3, 4, (4, k)).astype(np.float32)    # exact in either type; zeros too
            x[1] = np.abs(x[1]) + 1
            x[2] *= rng.random(k) < 0.2
            check_norm(x, "bf16", n=n, m=m, y=False)


@pytest.mark.parametrize("ns", [3, 4, 5, 6, 7, 8])
def test_norm_lifted(ns):
    rng = np.random.default_rng(ns)
    for groups in (1, 3, 100, 256, 513, 32768 // (2 * ns)):
        print("norm lift", ns, groups, flush=True)
        x = heavy(rng, 5, 2 * ns * groups)
        check_norm(x, "bf16", heavy(rng, *x.shape), "bf16", (1 + 0.3 * rng.standard_normal(x.shape[1])).astype(np.float32), ns=ns)


def test_norm_borders():
    """Values on, and one or two steps of fp32 beside, every half of a code, for largest values of
    many significant bits and every size."""
    rng = np.random.default_rng(8)
    rows = []
    for e in (-140, -126, -120, -60, -42, -40, -39, 0, 40, 100, 120):
        for _ in range(6):
            top = np.float32(np.ldexp(1 + rng.integers(0, 1 << 23) * 2.0 ** -23, e))
            halves = (np.arange(-127, 127) + 0.5) / 127.0
            v = (halves * np.float64(top)).astype(np.float32)
            more = [v]
            for way in (np.inf, -np.inf):
                u = v
                for _ in range(2):
                    u = np.nextafter(u, np.float32(way), dtype=np.float32)
                    more.append(u)
            rows.append(np.concatenate([[top, -top], *more]).astype(np.float32))
    x = np.stack(rows)
    check_norm(x, "f32")
    # ties that are exact: 127 p / 254 = p / 2 and powers of two of it
    t = np.concatenate([[254.0], np.arange(-253, 254, dtype=np.float64)]).astype(np.float32)
    check_norm(np.stack([np.ldexp(t, e) for e in (-140, -40, -8, 0, 90)]).astype(np.float32), "f32")


def test_norm_codes_next_to_a_half():
    """Quotients 1/2 +- 1 / (256 M), M a 24-bit number: as near a half as codes come without being one
    (127 (128 n -+ 1) = 128 (127 n -+ 1) +- 1), at every size."""
    for e in (-148, -60, 0, 90):
        for first in (66054, 99000, 131000):
            n = first + np.arange(0, 60, 3, dtype=np.int64)
            for side in (-1, 1):
                if (128 * n + side).max() >= 1 << 24:
                    continue
                p, top = 128 * n + side, 256 * (127 * n + side)
                assert ((127 * p - 128 * (127 * n + side)) == -side).all()
                x = np.stack([top, p, -p], axis=1).astype(np.float64) * 2.0 ** e
                x = np.pad(x.astype(np.float32), ((0, 0), (0, 37)))
                assert (x[:, 1].astype(np.float64) == p * 2.0 ** e).all()
                check_norm(x, "f32")
                q = run_norm(x, "f32")[0]
                assert (q[:, 0] == 127).all() and (q[:, 1] == (side < 0)).all() and (q[:, 2] == -(side < 0)).all()


def test_norm_rows_without_a_value():
    k = 200
    x = heavy(np.random.default_rng(1), 8, k)
    x[0] = 0
    x[1, 7] = np.inf
    x[2, 3] = np.nan
    x[3] = 1e-40                                                  # subnormal in fp32, not in the sum
    x[4] *= np.float32(1e30)                                      # its squares pass fp32
    x[5, 5], x[5, 9] = np.inf, -np.inf
    for xt in ("f32", "bf16"):
        check_norm(O.bf16_round(x) if xt == "bf16" else x, xt)
        check_norm(O.bf16_round(x) if xt == "bf16" else x, xt, n=2, m=4)
    r = np.zeros_like(x)
    r[0, 3], x[6, 2], r[6, 2] = 0, 3e38, 3e38                     # a sum past the type
    check_norm(O.bf16_round(x), "f32", O.bf16_round(r), "bf16")
    check_norm(x, "f32", r, "f32")
    w = np.ones(k, np.float32)
    w[7] = 0                                                      # 0 * inf
    check_norm(x, "f32", None, "f32", w)


def test_norm_no_columns_and_no_rows():
    q, s = torch.full((3, 16), 77, dtype=torch.int8, device="cuda"), torch.zeros(3, device="cuda")
    S.nm_rmsnorm_i8(torch.zeros(3, 0, device="cuda"), None, q, s)
    sync()
    assert (q == 77).all() and (s == 1).all()
    S.nm_rmsnorm_i8(torch.zeros(0, 8, device="cuda"), None, q, s)


def test_norm_more_rows_than_one_launch_takes():
    k, distinct, rows = 8, 61, (1 << 22) + 5
    x = heavy(np.random.default_rng(9), distinct, k)
    rq, rs, _, _ = O.rmsnorm_i8(x, x, "bf16")
    pick = torch.arange(rows, device="cuda") % distinct
    xd = torch.from_numpy(x).cuda().bfloat16()[pick]
    q, s = torch.zeros(rows, 16, dtype=torch.int8, device="cuda"), torch.zeros(rows, device="cuda")
    S.nm_rmsnorm_i8(xd, None, q, s, xd)
    sync()
    want = torch.zeros(distinct, 16, dtype=torch.int8, device="cuda")
    want[:, :k] = torch.from_numpy(rq).cuda()
    assert torch.equal(q, want[pick])
    assert ((s - torch.from_numpy(rs).cuda()[pick]).abs() <= 2 * U * s).all()


def test_norm_offsets_past_32_bits():
    rng = np.random.default_rng(12)
    k, rows, ld = 100, 2100, 1 << 20
    x, r = heavy(rng, rows, k), heavy(rng, rows, k)
    t = torch.empty(rows, ld, device="cuda")
    t[:, :k] = torch.from_numpy(x).cuda()
    rd = torch.from_numpy(np.pad(r, ((0, 0), (0, 4)))).cuda()
    q = torch.empty(rows, 2 * ld, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, device="cuda")
    S.nm_rmsnorm_i8(t, None, q, s, rd, t, k=k)
    sync()
    rq, _, rs, _ = O.rmsnorm_i8(x, r, "f32")
    assert np.array_equal(q[:, :k].cpu().numpy(), rq) and np.array_equal(t[:, :k].cpu().numpy(), rs)


def test_norm_is_the_quantizer_of_an_unweighted_row():
    """Without a weight the codes are nm_quant_i8's of the stored sum."""
    rng = np.random.default_rng(13)
    x, r = heavy(rng, 50, 4096), heavy(rng, 50, 4096)
    xd, rd = torch.from_numpy(x).cuda().bfloat16(), torch.from_numpy(r).cuda().bfloat16()
    q, q2 = torch.zeros(50, 4096, dtype=torch.int8, device="cuda"), torch.zeros(50, 4096, dtype=torch.int8, device="cuda")
    s, total = torch.zeros(50, device="cuda"), torch.empty_like(xd)
    for n, m in ((0, 0), (2, 4), (3, 8), (8, 16), (16, 32)):
        S.nm_rmsnorm_i8(xd, None, q, s, rd, total, n=n, m=m)
        S.nm_quant_i8(total, q2, s, n, m)
        sync()
        assert torch.equal(q, q2)


# --------------------------------------------------------------------------------- routing ---

def check_route(logits, top, kind=S.NM_ROUTER_SOFTMAX, bias=None, renormalize=True, scale=1.0, ld=None):
    t, e = logits.shape
    ld = e if ld is None else ld
    l = torch.full((t, ld), 1e9, device="cuda")
    l[:, :e] = torch.from_numpy(logits).cuda()
    ids = torch.full((t + 1, top), 99, dtype=torch.int32, device="cuda")
    w = torch.full((t + 1, top), -3.0, device="cuda")
    S.nm_moe_route(l, ids, w, kind, None if bias is None else torch.from_numpy(bias).cuda(), renormalize, scale, t=t,
                   experts=e)
    sync()
    assert (ids[t] == 99).all() and (w[t] == -3.0).all()
    rid, rw = O.moe_route(logits, top, kind == S.NM_ROUTER_SIGMOID, bias, renormalize, scale)
    assert np.array_equal(ids[:t].cpu().numpy(), rid)
    got = w[:t].cpu().numpy().astype(np.float64)
    # e^x within 2 ulp of the rounded difference (|x| U relative, |x| <= 104 where it is not 0), 1 + e^x
    # and the quotients round once each, the sum of up to 1024 terms in a tree of 16 + 6 additions
    assert (np.abs(got - rw) <= (2 * 104 + 40) * U * np.abs(rw) + 2.0 ** -126).all()
    assert (got[rid < 0] == 0).all()


@pytest.mark.parametrize("e", [1, 2, 4, 31, 60, 64, 65, 128, 200, 256, 500, 512, 1000, 1024])
def test_route_sizes(e):
    rng = np.random.default_rng(e)
    for t in (1, 5, 33):
        for top in sorted({1, min(e, 2), min(e, 8), min(e, 32)}):
            print("route", t, e, top, flush=True)
            l = (2 * rng.standard_normal((t, e))).astype(np.float32)
            check_route(l, top, ld=e + 3)
            check_route(l, top, renormalize=False, scale=2.5)
            check_route(l, top, S.NM_ROUTER_SIGMOID, renormalize=False)
            check_route(l, top, S.NM_ROUTER_SIGMOID, (0.3 * rng.standard_normal(e)).astype(np.float32), scale=0.5)


def test_route_ties_and_rows_without_an_expert():
    inf = np.inf
    rng = np.random.default_rng(2)
    l = rng.integers(-2, 3, (40, 96)).astype(np.float32)          # ties: the lower index
    l[:, 40] = -0.0
    l[1] = -inf
    l[2] = np.nan
    l[3, 1:] = -inf
    l[4, :] = -inf
    l[4, 95] = -88.0
    l[5, 7], l[5, 90] = inf, inf
    l[6, :60] = np.nan
    l[7] = -1e30
    l[8] = 3e38
    for kind in (S.NM_ROUTER_SOFTMAX, S.NM_ROUTER_SIGMOID):
        for renormalize in (True, False):
            check_route(l, 8, kind, None, renormalize)
    check_route(l, 8, S.NM_ROUTER_SIGMOID, rng.integers(0, 2, 96).astype(np.float32))


def test_route_many_tokens():
    rng = np.random.default_rng(4)
    l = rng.standard_normal((3001, 200)).astype(np.float32)
    check_route(l, 6)


def test_captured_and_replayed():
    """Routing and norm in one graph, replayed on new inputs with eager work between."""
    rng = np.random.default_rng(14)
    t, k, e = 9, 520, 48
    xs = [torch.from_numpy(heavy(rng, t, k)).cuda().bfloat16() for _ in range(3)]
    ls = [torch.randn(t, e, device="cuda") for _ in range(3)]
    x, l, r = xs[0].clone(), ls[0].clone(), xs[1].clone()
    q, s = torch.zeros(t, up(k, 16), dtype=torch.int8, device="cuda"), torch.zeros(t, device="cuda")
    ids, w = torch.zeros(t, 4, dtype=torch.int32, device="cuda"), torch.zeros(t, 4, device="cuda")
    out = torch.empty_like(x)

    def step():
        S.nm_rmsnorm_i8(x, None, q, s, r, out)
        S.nm_moe_route(l, ids, w)

    eager = []
    for a, b in zip(xs, ls):
        x.copy_(a), l.copy_(b)
        step()
        sync()
        eager.append([v.clone() for v in (q, s, ids, w, out)])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in (0, 2, 1, 1, 0):
        x.copy_(xs[i]), l.copy_(ls[i])
        for v in (q, s, ids, w, out):
            v.zero_()
        g.replay()
        sync()
        assert all(torch.equal(a, b) for a, b in zip((q, s, ids, w, out), eager[i]))
        torch.randn(100, 100, device="cuda").sum().item()


def test_streams_and_other_devices():
    rng = np.random.default_rng(15)
    x = torch.from_numpy(heavy(rng, 4, 64)).cuda()
    q, s = torch.zeros(4, 64, dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda")
    ids, w = torch.zeros(4, 4, dtype=torch.int32, device="cuda"), torch.zeros(4, 4, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    S.nm_rmsnorm_i8(x, None, q, s, stream=side)
    with torch.cuda.stream(side):
        S.nm_moe_route(x, ids, w)
    side.synchronize()
    rq, _, _, _ = O.rmsnorm_i8(x.cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(ids.cpu().numpy(), O.moe_route(x.cpu().numpy(), 4)[0])
    for bad in (lambda: S.nm_rmsnorm_i8(x.cpu(), None, q, s), lambda: S.nm_rmsnorm_i8(x, None, q.cpu(), s),
                lambda: S.nm_moe_route(x, ids.cpu(), w), lambda: S.nm_moe_route(x.cpu(), ids, w, stream=side)):
        with pytest.raises(ValueError):
            bad()


def test_route_scores_next_to_each_other():
    """Biased scores that fp32 cannot tell apart, or takes for equal: the order is that of 64 bits."""
    rng = np.random.default_rng(16)
    t, e = 300, 64
    l = (2 * rng.standard_normal((t, e))).astype(np.float32)
    # biases that bring many experts' scores of the first token to within a few 2^-25 of one value
    bias = (1.0 - 1.0 / (1.0 + np.exp(-l[0].astype(np.float64)))).astype(np.float32)
    for r in range(1, t):
        # tokens near the first one: their scores spread by fractions of a step, and ties among them
        l[r] = np.nextafter(l[0], np.float32(rng.choice([-9, 9])), dtype=np.float32) if r % 3 else l[0]
        pick = rng.random(e) < 0.2
        l[r, pick] = rng.standard_normal(int(pick.sum())).astype(np.float32)
    for top in (1, 8, 32):
        check_route(l, top, S.NM_ROUTER_SIGMOID, bias)
    check_route(l, 8, S.NM_ROUTER_SIGMOID, np.zeros(e, np.float32))
    check_route(l, 8, S.NM_ROUTER_SIGMOID, (bias * 1000).astype(np.float32))
    check_route(np.tile(l[:1], (1, 2)), 20, S.NM_ROUTER_SIGMOID, np.tile(bias, 2))


def test_route_sigmoid_weights_far_below_zero():
    """Chosen logits whose sigmoid passes the least fp32 value (below -88.7) keep their shares: those of
    64 bits, where it is 0 from -709.78 down."""
    rng = np.random.default_rng(17)
    l = np.full((64, 40), -np.inf, np.float32)
    l[0, :3] = -88.0, -89.0, -90.0
    l[1, 5] = -120.0
    l[2, 10:20] = -500.0
    l[3, :8] = -705.0, -705.5, -709.0, -709.75, -709.8, -712.0, -745.0, -1e30
    l[4, :8] = -710.0 - np.arange(8)                              # every weight is 0
    l[5, :6] = -0.5, 3.0, -89.0, -104.0, -300.0, -720.0           # one that counts, others that do not
    l[6, :6] = -1.0, -2.0, -80.0, -87.0, -88.5, -89.0
    for r in range(7, 64):
        far = np.float32(-80.0 - 620.0 * rng.random())            # neighbours within some units of a far place
        l[r] = far - (10.0 * rng.random(40)).astype(np.float32)
    for top in (1, 3, 8, 32):
        for bias in (None, np.zeros(40, np.float32), rng.standard_normal(40).astype(np.float32)):
            print("route far", top, bias is None, flush=True)
            check_route(l, top, S.NM_ROUTER_SIGMOID, bias)
            check_route(l, top, S.NM_ROUTER_SIGMOID, bias, scale=2.5)
            check_route(l, top, S.NM_ROUTER_SIGMOID, bias, renormalize=False)
    ids, w = torch.empty(1, 3, dtype=torch.int32, device="cuda"), torch.empty(1, 3, device="cuda")
    S.nm_moe_route(torch.from_numpy(l[:1, :4]).cuda().contiguous(), ids, w, S.NM_ROUTER_SIGMOID)
    e = np.exp(-np.arange(3.0))
    e = e / e.sum()
    assert (np.abs(w[0].double().cpu().numpy() - e) <= (2 * 104 + 40) * U * e).all()   # as in check_route
