"""Every kernel of the int8 layers with every epilogue, on the GPU: bits of the documented
roundings, tile shapes and splits that the sizes of test_i8_gpu.py do not reach, and runs whose
reductions are split across workgroups, captured and on two streams."""
import numpy as np
import pytest

import oracle as O
import synth
from nm_testutil import dev
from test_i8_gpu import (ROUTES, Guarded, build_mlp, check_glu, check_mlp, check_product, make_weight, mlp,
                         random_codes, sync, up, ws_for)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import semi_structured_sparse_amd as S  # noqa: E402


# ------------------------------------------------------------------------------ roundings ---

def few_bits(rng, n):
    """fp32 values of 8 significant bits in [0.5, 4), either sign: products of two have 16."""
    v = rng.integers(128, 256, n) * 2.0 ** rng.integers(-8, -5, n)
    return (v * rng.choice([-1.0, 1.0], n)).astype(np.float32)


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("ldy_extra", [0, 1, 4])
def test_outputs_have_the_documented_roundings(sparse, ldy_extra):
    """fp32(sum) * x_scale * w_scale, each rounded; the shift's product and sum rounded once together;
    the accumulation once more: the same bits on every route.  With factors of 8 bits numpy gives
    them: the shift's product and its sum with v are exact in 64 bits.  The product is below 2^4 and a
    multiple of 2^-16; v is a multiple of 2^-43 where it is below 2^4, and of 2^-19 from there to
    2^18, so the sum has at most 48 bits."""
    rng = np.random.default_rng(110 + sparse + 2 * ldy_extra)
    for t, o, k in [(7, 300, 512), (24, 512, 16384), (40, 256, 14336), (90, 520, 640), (300, 260, 1024)]:
        x = random_codes(rng, t, k, k, True)
        wd, meta, _, wv = make_weight(rng, o, k, sparse)
        xs, sc = np.abs(few_bits(rng, t)) / 256, np.abs(few_bits(rng, o)) / 1024
        rb, cs = few_bits(rng, t), few_bits(rng, o)
        v = (O.sums_i8(x, wv).astype(np.float32) * xs[:, None]) * sc[None, :]
        assert v.dtype == np.float32 and np.abs(v).max() < 2 ** 18
        term = rb.astype(np.float64)[:, None] * cs.astype(np.float64)[None, :]
        shifted = (v.astype(np.float64) + term).astype(np.float32)
        for shift, acc in [(0, 0), (0, 1), (1, 0), (1, 1)]:
            want = shifted if shift else v
            if acc:
                want = want + np.float32(7.25)
            for name, r in ROUTES.items():
                g = Guarded(t, o, o + ldy_extra)
                S.nm_spmm_i8(torch.from_numpy(x).cuda(), dev(xs.astype(np.float32)), wd, dev(sc.astype(np.float32)), g.y, meta,
                             dev(rb) if shift else None, dev(cs) if shift else None, acc, ws_for(t, o, k, sparse, False, r),
                             t=t, o=o, k=k, route=r)
                assert np.array_equal(g.get(), want.astype(np.float64)), (t, o, k, shift, acc, name)


# ---------------------------------------------------------------- tile shapes and splits ---
# Sizes by the rule of the smaller tiles: the largest of 128 x 128, 128 x 64, 64 x 64, 64 x 32 (weight
# rows x tokens; a GLU tile has half as many outputs) that gives 192 workgroups.

@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("sparse", [False, True])
def test_glu_on_128_by_128_tiles(sparse, act):
    rng = np.random.default_rng(120 + sparse)
    for t, o, k in [(128, 12992, 256), (250, 6530, 132), (190, 7001, 644)]:
        check_glu(rng, t, o, k, sparse, act, routes=("auto", "split"))
        check_glu(rng, t, o, k, sparse, act, routes=("split",), bf16=True, ldy=up(o, 8))
        check_glu(rng, t, o, k, sparse, act, routes=("split",), bf16=True, ldy=o + 1 - o % 2)
    check_glu(rng, 128, 12403, 128, sparse, act, routes=("split",), ldy=12403)


@pytest.mark.parametrize("sparse", [False, True])
def test_products_on_128_by_128_and_128_by_64_tiles(sparse):
    rng = np.random.default_rng(124 + sparse)
    for t, o, k in [(300, 8300, 260), (1000, 3202, 644), (90, 13001, 388), (64, 25001, 128)]:
        for bf16, shift, acc in [(True, 0, 0), (True, 1, 0), (False, 2, 0), (False, 0, 1), (False, 2, 1)]:
            check_product(rng, t, o, k, sparse, routes=("split",), bf16=bf16, shift=shift, accumulate=acc, ldy=o + 1 - o % 2)
            check_product(rng, t, o, k, sparse, routes=("split",), bf16=bf16, shift=shift, accumulate=acc, ldy=up(o, 8))


def in_two(t, o, k, sparse, glu):
    """The call's reduction is cut in two ranges (two partial sums of every output)."""
    return S.nm_i8_workspace_size(t, o, k, sparse, glu) == 2 * (2 if glu else 1) * t * up(o, 4) * 4


@pytest.mark.parametrize("sparse", [False, True])
def test_products_of_long_reductions_in_two_ranges(sparse):
    """64 x 64 tiles twice where 64 x 32 tiles would have over 64 steps."""
    rng = np.random.default_rng(128 + sparse)
    for t, o, k in [(100, 4100, 8320), (70, 4221, 8324), (40, 6300, 8448)]:
        assert in_two(t, o, k, sparse, False)
        check_product(rng, t, o, k, sparse, routes=("auto", "stream", "tile"))
        check_product(rng, t, o, k, sparse, bf16=True, shift=1, ldy=up(o, 8))
        check_product(rng, t, o, k, sparse, bf16=True, shift=2, ldy=o + 1 - o % 2)
        check_product(rng, t, o, k, sparse, shift=2, accumulate=1, ldy=up(o, 4))


@pytest.mark.parametrize("sparse", [False, True])
def test_glu_of_long_reductions_in_two_ranges(sparse):
    rng = np.random.default_rng(132 + sparse)
    for t, o, k in [(100, 2100, 8320), (70, 2221, 8324)]:
        assert in_two(t, o, k, sparse, True)
        check_glu(rng, t, o, k, sparse, "silu", routes=("auto", "stream", "tile"))
        check_glu(rng, t, o, k, sparse, "gelu", bf16=True, ldy=up(o, 8))
        check_glu(rng, t, o, k, sparse, "gelu", bf16=True, ldy=o + 1 - o % 2)


@pytest.mark.parametrize("sparse", [False, True])
def test_more_tiles_give_the_same_bits_every_time(sparse):
    """128 x 64 tiles, GLU tiles of each size, and reductions in ranges, call after call."""
    rng = np.random.default_rng(136 + sparse)
    for t, o, k, glu in [(500, 3300, 2048, False), (100, 4100, 8320, False), (61, 1024, 8192, False), (250, 6530, 1024, True),
                         (500, 1700, 2048, True), (100, 3300, 2048, True), (100, 2100, 8320, True)]:
        x = torch.from_numpy(random_codes(rng, t, k, k, True)).cuda()
        w0, m0, s0, _ = make_weight(rng, o, k, sparse)
        w1, m1, s1, _ = make_weight(rng, o, k, sparse)
        xs, s0, s1 = torch.full((t,), 1 / 4096, device="cuda"), dev(s0), dev(s1)
        want, y = (torch.empty(t, o + 1, device="cuda") for _ in range(2))

        def run(out, route):
            ws = ws_for(t, o, k, sparse, glu, route)
            if glu:
                S.nm_glu_i8(x, xs, w0, s0, w1, s1, out, S.NM_GLU_SILU, m0, m1, ws, k=k, inter=o, route=route)
            else:
                S.nm_spmm_i8(x, xs, w0, s0, out, m0, workspace=ws, k=k, o=o, route=route)

        run(want, ROUTES["stream"])
        for i in range(60):
            y.fill_(float("nan"))
            run(y, ROUTES["split" if i % 4 else "tile"])
            sync()
            assert torch.equal(y[:, :o], want[:, :o]), (t, o, k, glu, i)


# ------------------------------------------------------------- split runs in a served MLP ---

def both_split(t, hid, inter):
    return [S.nm_i8_workspace_size(t, inter, hid, True, True) > 0, S.nm_i8_workspace_size(t, hid, inter, False, False) > 0]


# the down product in eight ranges, the gate and up products in four, the down product in two
SPLIT_MLPS = [(24, 256, 16384, [False, True]), (24, 8192, 256, [True, False]), (100, 4112, 8448, [False, True])]


@pytest.mark.parametrize("t,hid,inter,split", SPLIT_MLPS)
def test_split_mlp_captured_and_replayed(t, hid, inter, split):
    """The whole run with its partial sums and their second kernel in one graph, replayed with new
    inputs, eager work in between."""
    assert both_split(t, hid, inter) == split
    rng = np.random.default_rng(140)
    bufs, weights = build_mlp(rng, t, hid, inter, False)
    xs = [dev(synth.normal_bf16(rng, (t, hid))) for _ in range(3)]
    xd = xs[0].clone()
    eager = []
    for x in xs:
        xd.copy_(x)
        mlp(xd, False, t, hid, inter, bufs)
        eager.append(bufs["y"].clone())
    sync()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mlp(xd, False, t, hid, inter, bufs)
    for i in (0, 1, 2, 1, 0):
        xd.copy_(xs[i])
        bufs["y"].fill_(float("nan"))
        bufs["ws"].fill_(0x55)
        g.replay()
        sync()
        assert torch.equal(bufs["y"], eager[i])
        torch.randn(100, 100, device="cuda").sum().item()
    if inter * hid < 1 << 23:
        check_mlp(bufs, xs[0].cpu().numpy().view(np.uint16), weights, False)


@pytest.mark.parametrize("t,hid,inter,split", SPLIT_MLPS)
def test_split_mlps_on_two_streams_at_once(t, hid, inter, split):
    """Two streams, each with its own buffers and partial sums, give what one after the other gives."""
    assert both_split(t, hid, inter) == split
    rng = np.random.default_rng(144)
    sets = [build_mlp(rng, t, hid, inter, False)[0] for _ in range(2)]
    xs = [dev(synth.normal_bf16(rng, (t, hid))) for _ in range(2)]
    want = []
    for b, x in zip(sets, xs):
        mlp(x, False, t, hid, inter, b)
        sync()
        want.append(b["y"].clone())
        b["y"].zero_()
    assert not torch.equal(want[0], want[1])
    sync()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for b, x, s in zip(sets, xs, streams):
            with torch.cuda.stream(s):
                mlp(x, False, t, hid, inter, b)
    sync()
    for b, w in zip(sets, want):
        assert torch.equal(b["y"], w)
