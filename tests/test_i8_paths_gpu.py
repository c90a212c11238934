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
