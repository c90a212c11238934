"""The int8 operators of the sparse linear layers, as cases that can be measured.

Four operators, each in its plain form (elementary torch operations) and, with `own`, as the
library's call:

  quant   rows of bf16 -> int8 codes and one scale per row, after an n:m selection or followed
          by the lift of the (2N-2):2N weights (nm_quant_i8)
  dense   y = (codes . weight codes^T) * token scale * channel scale (+ bias) (nm_spmm_i8)
  sp24    the same with 2:4 weights, values and step-blocked 2-bit positions (nm_spmm_i8)
  glu     act(gate product) * up product, dense or 2:4 weights (nm_glu_i8)

The product's operands are what a serving program holds: codes and scales of the activations,
and the packed weights.  Code rows are padded with zeros to a multiple of 16 bytes.
"""
import math

import torch

own = False

DEV = "cuda"


def up(v, m):
    return -(-v // m) * m


# ------------------------------------------------------------------------------ the cases ---

def listed():
    return [
        # one decoded token's activations before the q, k, v or gate, up products
        {"name": "quant 1x4096", "op": "quant", "t": 1, "k": 4096, "n": 0, "m": 0, "ns": 2},
        # activation sparsity 8:16 on the input of the down projection, a prefill of 2048 tokens
        {"name": "quant 8:16 2048x14336", "op": "quant", "t": 2048, "k": 14336, "n": 8, "m": 16, "ns": 2},
        # 6:8 weights: codes written lifted, a ragged prefill
        {"name": "quant 6:8 8191x4096", "op": "quant", "t": 8191, "k": 4096, "n": 0, "m": 0, "ns": 4},
        # decode, one sequence: the output or query projection
        {"name": "dense 1x4096x4096", "op": "dense", "t": 1, "o": 4096, "k": 4096, "y": "f32", "bias": False},
        # decode, 61 sequences: down projection with a bias, bf16 out
        {"name": "dense 61x4096x14336", "op": "dense", "t": 61, "o": 4096, "k": 14336, "y": "bf16", "bias": True},
        # a chunk of prefill on an odd reduction length and odd sizes
        {"name": "dense 777x1025x1999", "op": "dense", "t": 777, "o": 1025, "k": 1999, "y": "f32", "bias": True},
        # a large prefill through an up projection
        {"name": "dense 8192x14336x4096", "op": "dense", "t": 8192, "o": 14336, "k": 4096, "y": "bf16", "bias": False},
        # decode, 16 sequences, 2:4 weights
        {"name": "sp24 16x14336x4096", "op": "sp24", "t": 16, "o": 14336, "k": 4096, "y": "bf16", "bias": False},
        # 6:8 weights lowered to 2:4 (4096 -> 6144), a short prefill
        {"name": "sp24 333x4096x6144", "op": "sp24", "t": 333, "o": 4096, "k": 6144, "y": "f32", "bias": False},
        # a large prefill through a 2:4 down projection, fp32 out
        {"name": "sp24 8192x4096x14336", "op": "sp24", "t": 8192, "o": 4096, "k": 14336, "y": "f32", "bias": False},
        # decode, 8 sequences: gate and up of one layer
        {"name": "glu 8x14336x4096", "op": "glu", "t": 8, "o": 14336, "k": 4096, "y": "bf16", "act": "silu", "sparse": False},
        # prefill: 2:4 gate and up
        {"name": "glu 24 4096x14336x4096", "op": "glu", "t": 4096, "o": 14336, "k": 4096, "y": "bf16", "act": "gelu",
         "sparse": True},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["quant", "dense", "sp24", "glu"])
    t = spread(1, 8192)
    if op == "quant":
        form = rng.choice(["plain", "select", "lift"])
        n, m, ns = 0, 0, 2
        unit = 1
        if form == "select":
            m = unit = rng.choice([4, 8, 16, 32])
            n = rng.randint(1, m)
        elif form == "lift":
            ns = rng.randint(3, 8)
            unit = 2 * ns
        k = max(unit, spread(64, 14336) // unit * unit)
        return {"op": op, "t": t, "k": k, "n": n, "m": m, "ns": ns}
    o, k = spread(16, 14336), spread(64, 14336)
    sparse = op == "sp24" or (op == "glu" and rng.random() < 0.5)
    if sparse:
        k = max(4, k // 4 * 4)
    # at most the work of the largest listed case
    most = 8192 * 14336 * 4096 // (2 if op == "glu" else 1)
    t = max(1, min(t, most // (o * k)))
    case = {"op": op, "t": t, "o": o, "k": k, "y": rng.choice(["f32", "bf16"])}
    if op == "glu":
        return {**case, "act": rng.choice(["silu", "gelu"]), "sparse": sparse}
    return {**case, "bias": rng.random() < 0.3}


# ----------------------------------------------------------------------------- the inputs ---

def _activations(t, k, g):
    """Student-t(4) * 0.5 in bf16: heavy-tailed, as the input of a down projection."""
    z = torch.randn(t, k, generator=g, device=DEV)
    c = torch.zeros(t, k, device=DEV)
    for _ in range(4):
        c += torch.randn(t, k, generator=g, device=DEV).square_()
    return (0.5 * z / (c / 4).sqrt_()).to(torch.bfloat16)


def _codes(v):
    """int8 codes (rows padded with zeros to 16 bytes) and scales of fp32 rows."""
    rows, k = v.shape
    amax = v.abs().amax(1, keepdim=True)
    q = torch.zeros(rows, up(k, 16), dtype=torch.int8, device=DEV)
    q[:, :k] = (v * (127.0 / amax)).round_().clamp_(-127, 127).to(torch.int8)
    return q, (amax / 127.0)[:, 0].contiguous()


def _dense_weight(o, k, g):
    q, s = _codes(torch.randn(o, k, generator=g, device=DEV) * 0.02)
    return {"w": q, "s": s}


def _sparse_weight(o, k, g):
    """2:4 weights: the two largest of four, values as int8 codes [o][k/2 padded to 16], 2-bit
    positions in step blocks [ceil(k/128)][o][16]."""
    w = (torch.randn(o, k, generator=g, device=DEV) * 0.02).view(o, k // 4, 4)
    pos = w.abs().argsort(dim=2, descending=True, stable=True)[:, :, :2].sort(dim=2).values
    q, s = _codes(w.gather(2, pos).reshape(o, k // 2))
    pairs = pos[:, :, 0] | (pos[:, :, 1] << 2)                    # 4 bits for a group of four
    steps = -(-k // 128)
    full = torch.full((o, steps * 32), 4, dtype=torch.int64, device=DEV)   # padding: positions 0, 1
    full[:, :k // 4] = pairs
    by = (full[:, 0::2] | (full[:, 1::2] << 4)).to(torch.uint8)
    return {"w": q, "s": s, "meta": by.view(o, steps, 16).transpose(0, 1).contiguous()}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 13)
    t, k = case["t"], case["k"]
    x = _activations(t, k, g)
    if case["op"] == "quant":
        return {"case": case, "x": torch.nn.functional.pad(x, (0, up(k, 8) - k))}
    q, s = _codes(x.float())
    st = {"case": case, "q": q, "s": s}
    o = case["o"]
    make = _sparse_weight if case["op"] == "sp24" or case.get("sparse") else _dense_weight
    st["a"] = make(o, k, g)
    if case["op"] == "glu":
        st["b"] = make(o, k, g)
    st["bias"] = torch.randn(o, generator=g, device=DEV) if case.get("bias") else None
    return st


# ------------------------------------------------------------------------- the plain forms ---

def _lift_index(k, ns):
    """Lifted position -> position: window w of group p covers positions 2 ns p + 2 w + [0, 4)."""
    p = torch.arange(k // (2 * ns), device=DEV).view(-1, 1, 1) * 2 * ns
    w = torch.arange(ns - 1, device=DEV).view(1, -1, 1) * 2
    return (p + w + torch.arange(4, device=DEV).view(1, 1, -1)).reshape(-1)


def _plain_quant(st):
    c = st["case"]
    k, m = c["k"], c["m"]
    x = st["x"][:, :k]
    v = x.double()                                                # codes next to a border
    amax = v.abs().amax(1, keepdim=True)
    scale = torch.where(amax > 0, amax / 127, torch.ones_like(amax))
    q = torch.where(amax > 0, 127 * v / amax, torch.zeros_like(v)).round()
    if m:
        # magnitude bits, then the lower index first: distinct keys
        bits = x.contiguous().view(torch.int16).to(torch.int32) & 0x7FFF
        key = bits.view(c["t"], k // m, m) * 64 + (63 - torch.arange(m, device=DEV, dtype=torch.int32))
        rank = (key[:, :, None, :] > key[:, :, :, None]).sum(3)
        q = torch.where((rank < c["n"]).view(c["t"], k), q, torch.zeros_like(q))
    if c["ns"] > 2:
        q = q[:, _lift_index(k, c["ns"])]
    return [q.to(torch.int8), scale[:, 0].float()]


def _dense_of(p, k):
    """fp32 [o][k] weights (codes as values) of a dense or 2:4 weight."""
    if "meta" not in p:
        return p["w"][:, :k].float()
    o = p["w"].shape[0]
    by = p["meta"].transpose(0, 1).reshape(o, -1).int()
    slots = torch.stack([by & 3, (by >> 2) & 3, (by >> 4) & 3, by >> 6], dim=2).view(o, -1)[:, :k // 2]
    at = slots.view(o, k // 4, 2).long()
    w = torch.zeros(o, k // 4, 4, device=DEV)
    w.scatter_(2, at, p["w"][:, :k // 2].float().view(o, k // 4, 2))
    return w.view(o, k)


def _plain_product(st, p):
    k = st["case"]["k"]
    return (st["q"][:, :k].float() @ _dense_of(p, k).t()) * st["s"][:, None] * p["s"]


def _act(v, kind):
    if kind == "silu":
        return v / (1 + torch.exp(-v))
    return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))


def _type(case):
    return torch.float32 if case["y"] == "f32" else torch.bfloat16


# ------------------------------------------------------------------- the library's operators ---

def _own_run(st):
    import semi_structured_sparse_amd as S

    c = st["case"]
    t, k = c["t"], c["k"]
    if c["op"] == "quant":
        kq = 4 * (c["ns"] - 1) * (k // (2 * c["ns"])) if c["ns"] > 2 else k
        q = torch.empty(t, up(kq, 16), dtype=torch.int8, device=DEV)
        s = torch.empty(t, dtype=torch.float32, device=DEV)
        S.nm_quant_i8(st["x"], q, s, c["n"], c["m"], c["ns"], k=k)
        return [q[:, :kq], s]
    y = torch.empty(t, c["o"], dtype=_type(c), device=DEV)
    a = st["a"]
    if "ws" not in st:                 # a serving program keeps one workspace for its calls
        n = S.nm_i8_workspace_size(t, c["o"], k, sparse="meta" in a, glu=c["op"] == "glu")
        st["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    if c["op"] == "glu":
        b = st["b"]
        S.nm_glu_i8(st["q"], st["s"], a["w"], a["s"], b["w"], b["s"], y,
                    S.NM_GLU_SILU if c["act"] == "silu" else S.NM_GLU_GELU_TANH,
                    gate_meta=a.get("meta"), up_meta=b.get("meta"), workspace=st["ws"], k=k)
    else:
        S.nm_spmm_i8(st["q"], st["s"], a["w"], a["s"], y, w_meta=a.get("meta"), col_shift=st["bias"],
                     workspace=st["ws"], k=k)
    return [y]


def run(state):
    if own:
        return _own_run(state)
    c = state["case"]
    if c["op"] == "quant":
        return _plain_quant(state)
    y = _plain_product(state, state["a"])
    if c["op"] == "glu":
        y = _act(y, c["act"]) * _plain_product(state, state["b"])
    elif state["bias"] is not None:
        y = y + state["bias"]
    return [y.to(_type(c))]


# --------------------------------------------------------------------------------- the work ---

def work(case):
    t, k = case["t"], case["k"]
    if case["op"] == "quant":
        kq = 4 * (case["ns"] - 1) * (k // (2 * case["ns"])) if case["ns"] > 2 else k
        return {"bytes": 2 * t * k + t * kq + 4 * t, "flops": 0}
    o = case["o"]
    sparse = case["op"] == "sp24" or bool(case.get("sparse"))
    mats = 2 if case["op"] == "glu" else 1
    wbytes = o * k // 2 + o * (-(-k // 8)) if sparse else o * k
    out = t * o * (4 if case["y"] == "f32" else 2)
    bias = 4 * o if case.get("bias") else 0
    return {"bytes": t * k + 4 * t + mats * (wbytes + 4 * o) + out + bias,
            "flops": mats * t * o * k * (1 if sparse else 2)}


# ------------------------------------------------------------------------- the definition ---

def _exact_quant(st):
    c = st["case"]
    t, k, m, n, ns = c["t"], c["k"], c["m"], c["n"], c["ns"]
    x = st["x"][:, :k].to(torch.float64)
    mag = x.abs()
    top = mag.max(dim=1).values
    some = top > 0
    q = torch.round(x * 127.0 / torch.where(some, top, torch.ones_like(top)).unsqueeze(1))
    if m:
        order = torch.sort(mag.reshape(t, -1, m), dim=-1, descending=True, stable=True).indices[..., :n]
        keep = torch.zeros(t, k // m, m, dtype=torch.bool, device=DEV).scatter_(-1, order, True)
        q = q * keep.reshape(t, k)
    if ns > 2:
        groups = q.reshape(t, k // (2 * ns), 2 * ns)
        q = groups.unfold(2, 4, 2).reshape(t, -1)
    return [q.to(torch.int64).to(torch.int8), torch.where(some, top / 127.0, torch.ones_like(top))]


def _exact_weight(p, k):
    if "meta" not in p:
        return p["w"][:, :k].to(torch.float64)
    w = p["w"][:, :k // 2].to(torch.float64)
    o = w.shape[0]
    dense = torch.zeros(o, k, dtype=torch.float64, device=DEV)
    slot = torch.arange(k // 2, device=DEV)                       # slot j: byte j / 4 of its row
    byte = slot // 4
    at = p["meta"][byte // 16, :, byte % 16].t().long()           # [o][k / 2]
    at = (at >> (2 * (slot % 4))) % 4
    # a later slot never falls on an earlier one's place: positions of a group ascend
    return dense.scatter_add_(1, at + 4 * (slot // 2), w)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quant":
        return _exact_quant(st)
    k = case["k"]
    x = st["q"][:, :k].to(torch.float64) * st["s"].to(torch.float64).unsqueeze(1)

    def product(p):
        return torch.matmul(x, _exact_weight(p, k).t().contiguous()) * p["s"].to(torch.float64)

    y = product(st["a"])
    if case["op"] == "glu":
        gated = torch.sigmoid(y) * y if case["act"] == "silu" else \
            y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
        return [gated * product(st["b"])]
    return [y if st["bias"] is None else y + st["bias"].to(torch.float64)]
