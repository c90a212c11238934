"""What the int8 entry points of the binding accept of their tensors, without a GPU: the library is
replaced by a recorder and the tensors live on the CPU (the binding takes -1, their device, for
the current one).  A call whose memory the tensors do not hold must be refused before the
library is reached; the calls that the layouts allow must reach it with the right arguments."""
import sys

import pytest

import semi_structured_sparse_amd as S

torch = pytest.importorskip("torch")


class Recorder:
    """Stands for the loaded library: every entry point notes its arguments and succeeds."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def calls(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(S, "lib", lambda: rec)
    monkeypatch.setattr(S, "_current_device", lambda: -1)
    monkeypatch.setattr(S, "_current_raw_stream", lambda dev: 0)
    S._bind_types(torch)
    return rec.calls


def refused(calls, f, *args, **kw):
    before = len(calls)
    with pytest.raises(ValueError):
        f(*args, **kw)
    assert len(calls) == before, "the library was reached"


def taken(calls, f, *args, **kw):
    """Arguments that the library received."""
    before = len(calls)
    assert f(*args, **kw) == 0
    assert len(calls) == before + 1
    return calls[-1][1]


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def i8(*shape):
    return torch.zeros(*shape, dtype=torch.int8)


# ------------------------------------------------------------------------------- nm_quant_i8 ---

def test_quant_refuses_codes_narrower_than_their_rows(calls):
    x, s = bf16(4, 64), torch.zeros(4)
    refused(calls, S.nm_quant_i8, x, i8(4, 256)[:, 192:256], s, ns=4)      # 96 codes a row
    refused(calls, S.nm_quant_i8, x, i8(4, 256)[:, :48], s)
    refused(calls, S.nm_quant_i8, x, i8(4, 256)[:, :64], s, ns=4)
    refused(calls, S.nm_quant_i8, x, i8(4, 64), s, ldq=80)                  # the last row ends past the tensor
    flat = i8(4 * 64 - 14)                                                 # rows of 50 codes: the last one's pad is cut off
    refused(calls, S.nm_quant_i8, x, flat.as_strided((4, 50), (64, 1)), s, k=50)
    refused(calls, S.nm_quant_i8, x, i8(3, 64), s)
    a = taken(calls, S.nm_quant_i8, x, i8(4, 256)[:, 128:224], s, ns=4)
    assert a[8] == 256
    q = i8(4 * 64)
    a = taken(calls, S.nm_quant_i8, x, q.as_strided((4, 50), (64, 1)), s, k=50)   # its pad is there
    assert a[7] == q.data_ptr() and a[8] == 64
    a = taken(calls, S.nm_quant_i8, x, i8(8, 64), s, ldq=128)                   # every second row
    assert a[8] == 128
    taken(calls, S.nm_quant_i8, x, 1 << 20, s, ldq=64)                      # a raw pointer is the caller's
    taken(calls, S.nm_quant_i8, x[:0], i8(0, 64), s)


def test_quant_refuses_values_that_x_does_not_hold(calls):
    q, s = i8(64, 256), torch.zeros(64)
    refused(calls, S.nm_quant_i8, bf16(4, 64), q, s, rows=64)
    refused(calls, S.nm_quant_i8, bf16(4, 64), q, s, k=72)
    refused(calls, S.nm_quant_i8, bf16(4, 256)[:, :64], q, s, k=72)
    refused(calls, S.nm_quant_i8, bf16(4, 64), q, s, ldx=72)                # the last row ends past the tensor
    flat = bf16(3 * 56 + 50)                                               # pieces of 8: the last row needs 56 values
    refused(calls, S.nm_quant_i8, flat.as_strided((4, 50), (56, 1)), q, s)
    flat = bf16(4 * 56)
    a = taken(calls, S.nm_quant_i8, flat.as_strided((4, 50), (56, 1)), q, s)
    assert a[:4] == (flat.data_ptr(), 4, 50, 56)
    a = taken(calls, S.nm_quant_i8, bf16(4, 56), q, s, k=50)                # padded rows
    assert a[1:4] == (4, 50, 56)
    a = taken(calls, S.nm_quant_i8, bf16(8, 64), q, s, rows=4, ldx=128)     # every second row
    assert a[1:4] == (4, 64, 128)
    taken(calls, S.nm_quant_i8, 1 << 20, q, s, rows=64, k=64, ldx=64)       # a raw pointer is the caller's


# ----------------------------------------------------------------------------- nm_meta_block ---

def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def test_meta_block_refuses_positions_that_do_not_fit(calls):
    meta, out = u8(5, 17), u8(2 * 5 * 16)                                   # kc = 132: two step blocks
    refused(calls, S.nm_meta_block, meta, 5, 132, out[:-16])
    refused(calls, S.nm_meta_block, meta, 5, 132, u8(2, 5, 17)[:, :, :16])  # blocks with gaps
    refused(calls, S.nm_meta_block, meta[:4], 5, 132, out)
    refused(calls, S.nm_meta_block, u8(5, 16), 5, 132, out)
    refused(calls, S.nm_meta_block, u8(5, 32)[:, :17], 5, 132, out)         # rows of meta lie 17 bytes apart
    a = taken(calls, S.nm_meta_block, meta, 5, 132, out)
    assert a[:4] == (meta.data_ptr(), 5, 132, out.data_ptr())
    taken(calls, S.nm_meta_block, torch.zeros(5, 9, dtype=torch.int16), 5, 132, torch.zeros(40, dtype=torch.int32))
    taken(calls, S.nm_meta_block, 1 << 20, 5, 132, 1 << 24)
    taken(calls, S.nm_meta_block, u8(0, 17), 0, 132, u8(0))


# -------------------------------------------------------------------------------- products ---

def product(x, w, y, w_meta=None, **kw):
    return S.nm_spmm_i8(x, torch.ones(64), w, torch.ones(64), y, w_meta, **kw)


def gated(x, w, y, w_meta=None, up=None, **kw):
    if "o" in kw:
        kw["inter"] = kw.pop("o")
    return S.nm_glu_i8(x, torch.ones(64), w, torch.ones(64), w if up is None else up, torch.ones(64), y,
                       gate_meta=w_meta, up_meta=w_meta, **kw)


@pytest.mark.parametrize("call", [product, gated])
def test_products_refuse_operands_that_are_not_there(calls, call):
    y = torch.zeros(64, 64)
    x, w, meta = i8(4, 64), i8(8, 64), u8(8 * 16)
    refused(calls, call, x, w, y, t=64)
    refused(calls, call, x, w, y, o=64)
    refused(calls, call, x, i8(8, 128), y, k=128)
    refused(calls, call, i8(4, 128), w, y)                                  # x's width is the reduction
    refused(calls, call, x, i8(8, 32), y)                                   # dense weights of half the length
    refused(calls, call, x, i8(8, 16), y, meta)                             # 2:4: 32 values a row
    refused(calls, call, x, w, y, ldx=80)                                   # last rows past the tensors' ends
    refused(calls, call, x, w, y, ldw=80)
    refused(calls, call, i8(4 * 64 - 14).as_strided((4, 50), (64, 1)), w, y)
    refused(calls, call, x, i8(8 * 64 - 14).as_strided((8, 50), (64, 1)), y, k=50)
    flat = i8(4 * 64)
    a = taken(calls, call, flat.as_strided((4, 50), (64, 1)), w, y)         # its pad is there
    assert a[:4] == (flat.data_ptr(), 4, 50, 64)
    a = taken(calls, call, i8(4, 112), i8(8, 112)[:, :100], y)              # W's pad counts: X is zero there
    assert a[1:4] == (4, 112, 112)
    taken(calls, call, x, w, y, meta)                                       # wider than its 32 values
    taken(calls, call, x, i8(8, 32), y, meta)
    a = taken(calls, call, i8(8, 64), i8(16, 64), y, t=4, o=8, ldx=128, ldw=128)   # every second row
    assert a[1:4] == (4, 64, 128)
    taken(calls, call, 1 << 20, w, y, t=64, k=64, ldx=64)                   # a raw pointer is the caller's


def test_gated_products_check_both_weights(calls):
    y, x, w = torch.zeros(64, 64), i8(4, 64), i8(8, 64)
    refused(calls, gated, x, w, y, up=i8(8, 64)[:7], o=8)
    refused(calls, gated, x, w, y, up=i8(8 * 64 - 1).as_strided((8, 63), (64, 1)))
    refused(calls, gated, x, w, y, up=i8(8, 32), ldw=64)
    taken(calls, gated, x, w, y, up=i8(9, 64), o=8)


@pytest.mark.parametrize("call", [product, gated])
def test_products_refuse_outputs_written_past_their_end(calls, call):
    x, w = i8(4, 64), i8(8, 64)
    y = torch.zeros(4, 8)
    refused(calls, call, x, w, y, ldy=9)
    refused(calls, call, x, w, y.bfloat16(), y_dtype=S.NM_Y_F32)             # twice its bytes
    refused(calls, call, x, w, y, y_dtype=S.NM_Y_BF16)
    refused(calls, call, x, w, torch.zeros(16, 8)[:4], t=8)
    refused(calls, call, x, w, torch.zeros(4, 7), y_dtype=S.NM_Y_F32)
    for dt in (torch.float32, torch.bfloat16, torch.int16):
        out = torch.zeros(8, 8, dtype=dt)
        a = taken(calls, call, x, w, out, ldy=16)                            # every second row
        at = a.index(out.data_ptr())
        assert a[at + 1:at + 3] == (16, S.NM_Y_F32 if dt is torch.float32 else S.NM_Y_BF16)
        taken(calls, call, x, w, out[:4], y_dtype=S.NM_Y_F32 if dt is torch.float32 else S.NM_Y_BF16)
    a = taken(calls, call, x, w, 1 << 20, o=8, ldy=8, y_dtype=S.NM_Y_BF16)   # a raw pointer is the caller's
    at = a.index(1 << 20)
    assert a[at + 1:at + 3] == (8, S.NM_Y_BF16)


@pytest.mark.parametrize("call", [product, gated])
def test_products_refuse_workspaces_they_would_write_past(calls, call):
    x, w, y, ws = i8(4, 64), i8(8, 64), torch.zeros(4, 8), u8(256)
    refused(calls, call, x, w, y, workspace=u8(512)[::2])                    # every second byte is someone else's
    refused(calls, call, x, w, y, workspace=u8(16, 32)[:, :16])
    refused(calls, call, x, w, y, workspace=ws, workspace_bytes=257)
    for kw, size in (({}, 256), ({"workspace_bytes": 64}, 64), ({"workspace": torch.zeros(64)}, 256),
                     ({"workspace": 1 << 20, "workspace_bytes": 512}, 512), ({"workspace": 1 << 20}, 0),
                     ({"workspace": None}, 0)):
        kw = {"workspace": ws, **kw}
        a = taken(calls, call, x, w, y, **kw)
        p = kw["workspace"]
        assert a[-5:-3] == (p.data_ptr() if torch.is_tensor(p) else p, size)


# ------------------------------------------------------------------- raw pointers and tensors ---

def test_tensors_beside_raw_pointers_on_a_named_stream(calls, monkeypatch):
    """With the stream given, tensors count wherever they stand among raw pointers."""
    class OnGpu(torch.Tensor):
        def get_device(self):
            return 0

    monkeypatch.setattr(S, "_current_device", lambda: 0)
    gpu = lambda t: t.as_subclass(OnGpu)  # noqa: E731
    one, p = gpu(torch.ones(64)), 1 << 20
    taken(calls, S.nm_spmm_i8, p, one, p, p, p, stream=0, t=4, o=8, k=64, ldx=64, ldw=64, ldy=8)
    taken(calls, S.nm_spmm_i8, p, p, p, p, p, p, None, one, stream=0, t=4, o=8, k=64, ldx=64, ldw=64, ldy=8)
    taken(calls, S.nm_spmm_i8, p, p, p, p, p, gpu(u8(128)), stream=0, t=4, o=8, k=64, ldx=64, ldw=64, ldy=8)
    taken(calls, S.nm_spmm_i8, p, p, p, p, p, workspace=gpu(u8(64)), stream=0, t=4, o=8, k=64, ldx=64, ldw=64, ldy=8)
    taken(calls, S.nm_glu_i8, p, p, p, p, p, one, p, stream=0, t=4, inter=8, k=64, ldx=64, ldw=64, ldy=8)
    taken(calls, S.nm_glu_i8, p, p, p, p, gpu(i8(8, 64)), p, p, stream=0, t=4, inter=8, k=64, ldx=64, ldw=64, ldy=8)
    refused(calls, S.nm_spmm_i8, p, torch.ones(64), p, p, p, stream=0, t=4, o=8, k=64, ldx=64, ldw=64, ldy=8)   # on the CPU
    refused(calls, S.nm_spmm_i8, p, one, p, torch.ones(64), p, stream=0, t=4, o=8, k=64, ldx=64, ldw=64, ldy=8)


# ----------------------------------------------------------------------------- empty rows ---

def test_rows_of_no_values(calls):
    """torch gives a matrix of no columns the leading dimension 1, which no alignment rule takes."""
    a = taken(calls, S.nm_quant_i8, bf16(4, 0), i8(4, 0), torch.zeros(4))
    assert a[1:4] == (4, 0, 0) and a[8] == 0
    a = taken(calls, S.nm_quant_i8, bf16(4, 64), i8(4, 64), torch.zeros(4), k=0)
    assert a[1:4] == (4, 0, 0) and a[8] == 0
    for call in (product, gated):
        a = taken(calls, call, i8(4, 0), i8(8, 0), torch.zeros(4, 8))
        assert a[1:4] == (4, 0, 0) and 1 not in a[:14]
        a = taken(calls, call, i8(4, 64), i8(8, 64), torch.zeros(4, 8), k=0)
        assert a[1:4] == (4, 0, 0)


def test_rows_of_no_values_are_valid():
    """The library itself (nothing to launch: no rows)."""
    assert S.lib().nm_quant_i8(None, 0, 0, 0, 0, 0, 2, None, 0, None, None) == S.NM_OK
    assert S.lib().nm_quant_i8(None, 0, 0, 1, 0, 0, 2, None, 0, None, None) == S.NM_EALIGN


# --------------------------------------------------------------------------- element types ---

def test_one_byte_floats_are_no_codes(calls):
    """fp8 weights and activations are other operators' operands: their bytes are not integers."""
    x, q, s, y = bf16(4, 64), i8(4, 64), torch.zeros(64), torch.zeros(4, 8)
    w = i8(8, 64)
    for dt in (torch.float8_e4m3fn, torch.float8_e5m2, torch.bool):
        refused(calls, S.nm_quant_i8, x, q.to(dt), s)
        for call in (product, gated):
            refused(calls, call, q.to(dt), w, y)
            refused(calls, call, q, w.to(dt), y)
        refused(calls, gated, q, w, y, up=w.to(dt))
    refused(calls, S.nm_quant_i8, x.half(), q, s)
    for dt in (torch.int8, torch.uint8):                                    # the codes' bits
        taken(calls, S.nm_quant_i8, x, q.to(dt), s)
        for call in (product, gated):
            taken(calls, call, q.to(dt), w.to(dt), y)
    for dt in (torch.int16, torch.uint16):                                  # bf16 bits
        taken(calls, S.nm_quant_i8, x.view(dt), q, s)


# ----------------------------------------------------------------------------- first calls ---

@pytest.mark.parametrize("raw", [True, False])
def test_first_calls_of_two_threads(monkeypatch, raw):
    """At no point of the first call's binding may another thread find part of it: the stream
    lookup, which tells that the rest is there, comes last."""
    for name in ("_current_raw_stream", "_current_device", "_int8s", "_bf16s", "_half"):
        monkeypatch.setattr(S, name, None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: None)
    if raw:
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    else:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    seen = []

    def step(frame, event, arg):
        frame.f_trace_opcodes = True
        seen.append(S._current_raw_stream is None or None not in (S._current_device, S._int8s, S._bf16s, S._half))
        return step

    before = sys.gettrace()
    sys.settrace(step)
    try:
        S._bind_torch()
    finally:
        sys.settrace(before)
    assert len(seen) > 20 and all(seen) and S._current_raw_stream is not None
