"""What the Python calls of the balance loss and of the MX matrices look at in their tensors before the library gets
an address (no GPU: a context of the CPU's number, -1, with a library that only takes notes)."""
import ctypes

import pytest
import torch

from bit_expert_ffn_router_b200 import moe as M


class Notes:
    """A library whose calls succeed and are counted."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or M.OK


class Stream:
    cuda_stream = 77


def context():
    c = object.__new__(M.Context)
    c.lib, c.h, c.device = Notes(), ctypes.c_void_p(), -1
    c._bind_torch()
    return c


class Elsewhere(torch.Tensor):
    def get_device(self):
        return 1


def elsewhere(t):
    return t.as_subclass(Elsewhere)


def strided(t):
    """The same values with a gap after each."""
    return torch.stack((t, t), -1)[..., 0]


def misfits(t):
    """t in ways that the library would misread: another type, too short, with gaps, no tensor."""
    yield "wide", t.to(torch.int64 if t.dtype != torch.float32 else torch.float64)
    yield "half", t.to(torch.float16)
    yield "short", t.reshape(-1)[:-1]
    yield "strided", strided(t)
    yield "numpy", t.numpy()
    if t.dim() == 2:
        yield "transposed", t.t().contiguous().t()
        yield "one row for all", t[:1].expand(t.shape)


T, E, k = 6, 16, 3


def loss_args(mask=True):
    return dict(logits=torch.randn(T, E), idx=torch.zeros(T, k, dtype=torch.int32),
                mask=torch.ones(T, dtype=torch.uint8) if mask else None, T=T, stats=torch.zeros(4),
                counts=torch.zeros(E, dtype=torch.int32), prob=torch.zeros(E), ws=torch.zeros(4096, dtype=torch.uint8))


def grad_args(gates=True, mask=True):
    a = loss_args(mask)
    return dict(logits=a["logits"], idx=a["idx"], gate=torch.rand(T, k) if gates else None, mask=a["mask"], T=T,
                stats=a["stats"], counts=a["counts"], d_loss=torch.ones(2), d_gate=torch.rand(T, k) if gates else None,
                d_logits=torch.zeros(T, E))


CFG = M.LayerCfg(d=256, f=128, E=E, k=k)
CALLS = {"balance_loss": loss_args, "balance_loss_backward": grad_args}


@pytest.mark.parametrize("call", CALLS)
def test_balance_calls_take_what_fits(call):
    c = context()
    for kw in ({}, {"mask": False}):
        a = CALLS[call](**kw)
        getattr(c, call)(CFG, **a, stream=Stream)
        args = c.lib.calls.pop()[1]
        for n, t in a.items():
            if isinstance(t, torch.Tensor):
                assert t.data_ptr() in args, n
        assert 77 in args and (None in args) == bool(kw)
    a = CALLS[call]()
    # longer than needed, of any shape; a mask of any single-byte type
    for n in set(a) - {"T"}:
        a[n] = torch.cat((a[n].reshape(-1), a[n].reshape(-1)))
    for t in (torch.bool, torch.int8):
        a["mask"] = a["mask"].to(t)
        getattr(c, call)(CFG, **a, stream=Stream)
    # no tokens: tensors without elements
    a = CALLS[call]()
    a["T"] = 0
    for n in ("logits", "idx", "mask", "gate", "d_gate", "d_logits"):
        if n in a:
            a[n] = a[n][:0]
    getattr(c, call)(CFG, **a, stream=Stream)
    assert len(c.lib.calls) == 3


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in CALLS[c]() if n not in ("T", "ws")])
def test_balance_calls_refuse_what_does_not(call, name):
    c = context()
    good = CALLS[call]()
    for what, t in misfits(good[name]):
        with pytest.raises(M.MoeError) as e:
            getattr(c, call)(CFG, **{**good, name: t}, stream=Stream)
        assert e.value.status == M.EINVAL, what
    if name not in ("mask", "gate", "d_gate"):
        with pytest.raises(M.MoeError):
            getattr(c, call)(CFG, **{**good, name: None}, stream=Stream)
    assert not c.lib.calls


def test_balance_workspace_and_gates():
    c = context()
    a = loss_args()
    for ws in (strided(a["ws"]), None):
        with pytest.raises(M.MoeError):
            c.balance_loss(CFG, **{**a, "ws": ws}, stream=Stream)
    with pytest.raises(M.MoeError):  # gates are needed for their gradient
        c.balance_loss_backward(CFG, **{**grad_args(), "gate": None}, stream=Stream)
    assert not c.lib.calls
    c.balance_loss_backward(CFG, **grad_args(gates=False), stream=Stream)
    c.balance_loss_backward(CFG, **{**grad_args(), "d_gate": None}, stream=Stream)
    assert len(c.lib.calls) == 2


@pytest.mark.parametrize("call", CALLS)
def test_logits_of_another_device_are_refused(call):
    c, a = context(), CALLS[call]()
    a["logits"] = elsewhere(a["logits"])
    with pytest.raises(M.MoeError):
        getattr(c, call)(CFG, **a, stream=Stream)
    c.device = 0  # the others' are then the CPU's
    with pytest.raises(M.MoeError):
        getattr(c, call)(CFG, **CALLS[call](), stream=Stream)
    assert not c.lib.calls


def test_indices_as_torch_gives_them_are_refused():
    c = context()
    a = loss_args()
    a["idx"] = a["logits"].topk(k, 1)[1]
    assert a["idx"].dtype == torch.int64
    assert c.balance_loss_status(CFG, **a, stream=Stream) == M.EINVAL
    a["idx"] = a["idx"].to(torch.int32)
    assert c.balance_loss_status(CFG, **a, stream=Stream) == M.OK


def mx(rows, cols):
    codes, scales = M.mx4_buffers(rows, cols, device="cpu")
    return codes.zero_(), scales.zero_()


def test_mx_rows_of_another_device_are_refused():
    c = context()
    x, out = torch.randn(5, 64), torch.zeros(5, 32)
    w, q = M.Mx4Matrix(*mx(32, 64), 64), mx(5, 64)
    calls = [lambda e: c.mx4_quantize(e(x), *q, stream=Stream), lambda e: c.mx4_dequantize(*q, e(x), stream=Stream),
             lambda e: c.mx4_product(*q, w, e(out), stream=Stream)]
    for f in calls:
        f(lambda t: t)
        with pytest.raises(M.MoeError):
            f(elsewhere)
    there = M.Mx4Matrix(*map(elsewhere, mx(32, 64)), 64)
    assert there.device == 1 and w.device == -1
    with pytest.raises(M.MoeError):
        c.mx4_product(*q, there, out, stream=Stream)
    codes, scales = mx(32, 64)
    with pytest.raises(M.MoeError):
        M.Mx4Matrix(codes, elsewhere(scales), 64)
    assert [n for n, _ in c.lib.calls] == ["moe_mx4_quantize", "moe_mx4_dequantize", "moe_mx4_product"]


@pytest.mark.parametrize("n_shared", [0, 1])
def test_ffn_rows_that_combine_would_misread_are_refused(n_shared):
    c = context()
    T, k, d, f, slots = 4, 2, 256, 128, 3
    cfg = M.LayerCfg(d=d, f=f, E=8, k=k, n_shared=n_shared)
    g = M.Grouping()
    g.T, g.k, g.E, g.n_pairs = T, k, 8, T * k
    n = T * (k + n_shared)

    def pool(rows, cols):
        q, s = mx(slots * rows, cols)
        return M.Mx4Matrix(q.view(slots, rows, -1), s.view(slots, rows, -1), cols)

    up, down, bufs = pool(2 * f, d), pool(d, f), M.mx4_ffn_buffers(cfg, T, device="cpu")
    x, shared = torch.randn(T, d), 2 if n_shared else -1
    call = lambda z: c.expert_ffn_mx4(cfg, x, g, up, down, shared, bufs, z, stream=Stream)  # noqa: E731
    call(torch.zeros(n, d))
    assert [name for name, _ in c.lib.calls] == ["moe_mx4_quantize", "moe_mx4_product"] * 2
    del c.lib.calls[:]
    z = torch.zeros(n, d)
    for bad in (z.bfloat16(), z.half(), z.double(), z[:n - 1], torch.zeros(n, d + 8)[:, :d], torch.zeros(2 * n, d)[::2]):
        with pytest.raises(M.MoeError):
            call(bad)
    assert not c.lib.calls  # refused before anything ran
