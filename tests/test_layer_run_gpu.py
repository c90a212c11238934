"""The operators around the products together, as a decoder layer uses them: the output projection onto
the residual stream (nm_linear), the norm to int8 codes and a bf16 row (nm_rmsnorm_i8), the router's
logits (nm_linear, fp32), the experts of each token (nm_moe_route), their MLPs back onto the stream
(nm_moe_i8).  Each step is held against the oracle on what the step before it gave."""
import numpy as np
import pytest

import oracle as O
import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import semi_structured_sparse_amd as S  # noqa: E402
from test_moe_gpu import expert_weights  # noqa: E402

U, UB = 2.0 ** -24, 2.0 ** -8


def sync():
    torch.cuda.synchronize()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Layer:
    def __init__(self, seed, t, hidden, inter, experts, top, sparse):
        rng = np.random.default_rng(seed)
        self.n = (t, hidden, inter, experts, top)
        bf = lambda *s, scale=1.0: O.f32_from_bf16(synth.normal_bf16(rng, s, scale))  # noqa: E731
        self.attn, self.stream = bf(t, hidden), bf(t, hidden)
        self.proj, self.router = bf(hidden, hidden, scale=0.05), bf(experts, hidden, scale=0.05)
        self.norm = (1 + 0.2 * rng.standard_normal(hidden)).astype(np.float32)
        self.gate, self.up, self.down = (expert_weights(rng, experts, r, k, sparse)
                                         for r, k in ((inter, hidden), (inter, hidden), (hidden, inter)))
        b = self.b = {}
        b["attn"], b["stream"] = dev(self.attn).bfloat16(), dev(self.stream).bfloat16()
        b["proj"], b["router"], b["norm"] = dev(self.proj).bfloat16(), dev(self.router).bfloat16(), dev(self.norm)
        b["mid"] = torch.empty(t, hidden, dtype=torch.bfloat16, device="cuda")
        b["q"] = torch.zeros(t, hidden + -hidden % 16, dtype=torch.int8, device="cuda")
        b["s"], b["row"] = torch.empty(t, device="cuda"), torch.empty(t, hidden, dtype=torch.bfloat16, device="cuda")
        b["logits"] = torch.empty(t, experts, device="cuda")
        b["ids"], b["w"] = torch.empty(t, top, dtype=torch.int32, device="cuda"), torch.empty(t, top, device="cuda")
        b["out"] = torch.empty(t, hidden, dtype=torch.bfloat16, device="cuda")
        size = max(S.nm_linear_workspace_size(t, hidden, hidden), S.nm_linear_workspace_size(t, experts, hidden),
                   S.nm_moe_i8_workspace_size(t, experts, top, hidden, inter, sparse), 16)
        b["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")

    def run(self):
        b = self.b
        t, hidden, inter, experts, top = self.n
        S.nm_linear(b["attn"], b["proj"], b["mid"], residual=b["stream"], workspace=b["ws"])
        S.nm_rmsnorm_i8(b["mid"], b["norm"], b["q"], b["s"], y=b["row"])
        S.nm_linear(b["row"], b["router"], b["logits"], workspace=b["ws"])
        S.nm_moe_route(b["logits"], b["ids"], b["w"])
        S.nm_moe_i8(b["q"], b["s"], b["ids"], b["w"], self.gate[0], self.gate[1], self.up[0], self.up[1], self.down[0],
                    self.down[1], b["out"], gate_meta=self.gate[2], up_meta=self.up[2], down_meta=self.down[2],
                    residual=b["mid"], workspace=b["ws"], hidden=hidden)

    def check(self):
        b = {k: v.double().cpu().numpy() if v.is_floating_point() else v.cpu().numpy() for k, v in self.b.items() if k != "ws"}
        t, hidden, inter, experts, top = self.n
        y, size = O.linear(b["attn"], self.proj, None, "none", b["stream"])
        err = 2 * U * (hidden + 1) * size + 4 * U * np.abs(y)
        assert (np.abs(b["mid"] - y) <= err + UB * (np.abs(y) + err)).all()
        q, scale, _, row = O.rmsnorm_i8(b["mid"].astype(np.float32), None, "bf16", self.norm, 1e-6)
        assert np.array_equal(b["q"][:, :hidden], q) and (np.abs(b["s"] - scale) <= 2 * U * scale).all()
        assert (np.abs(b["row"] - row) <= (UB + 4 * U) * np.abs(row)).all()
        y, size = O.linear(b["row"], self.router)
        assert (np.abs(b["logits"] - y) <= 2 * U * (hidden + 1) * size).all()
        ids, w = O.moe_route(b["logits"].astype(np.float32), top)
        assert np.array_equal(b["ids"], ids) and (np.abs(b["w"] - w) <= 256 * U * w).all()
        y, far, size = O.moe_i8(b["q"][:, :hidden], b["s"], ids, b["w"], self.gate[3:], self.up[3:], self.down[3:], "silu",
                                b["mid"])
        err = far + size * U * (top + 40)
        assert (np.abs(b["out"] - y) <= err + UB * (np.abs(y) + err)).all()


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("n", [(1, 256, 128, 8, 2), (7, 512, 96, 24, 4), (40, 320, 64, 6, 2), (64, 128, 260, 70, 6)])
def test_eager_then_captured(n, sparse):
    print("layer", n, sparse, flush=True)
    layer = Layer(sum(n), *n, sparse)
    layer.run()
    sync()
    layer.check()
    first = {k: v.clone() for k, v in layer.b.items() if k != "ws"}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.run()
    other = torch.randn_like(layer.b["attn"])
    for again in (False, True, True, False, False):
        layer.b["attn"].copy_(other if again else first["attn"])
        for k in ("mid", "row", "logits", "w", "out", "s"):
            layer.b[k].fill_(float("nan"))
        g.replay()
        sync()
        if again:
            layer.check()
        else:
            assert all(torch.equal(layer.b[k], first[k]) for k in ("mid", "q", "s", "row", "logits", "ids", "w", "out"))
        torch.randn(64, 64, device="cuda").sum().item()
