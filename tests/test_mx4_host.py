"""Host-side checks of the MX and balance-loss calls (no GPU): sizes, and every
refusal, which each call makes before it touches the device."""
import ctypes

import pytest

from bit_expert_ffn_router_b200 import build as B
from bit_expert_ffn_router_b200 import moe as M


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


# A zeroed block in the place of a context: a refused call never looks into it.
CTX = ctypes.create_string_buffer(4096)
A = 1 << 20  # an aligned address that no refused call reads


def test_scale_pitch():
    for cols, want in ((32, 16), (512, 16), (544, 32), (768, 32), (2048, 64), (65536, 2048), (0, 0), (-32, 0), (48, 0),
                       (65568, 0)):
        assert M.mx4_scale_pitch(cols) == want, cols


def test_balance_workspace():
    n = M.load_library().moe_balance_workspace_bytes
    assert 0 < n(ctypes.byref(M.TINY.c())) < n(ctypes.byref(M.FULL.c()))
    assert n(ctypes.byref(M.TINY.replace(k=17).c())) == 0
    assert n(None) == 0


def _balance(cfg=M.TINY, T=4, ws_bytes=1 << 30, ctx=CTX, **kw):
    a = dict(logits=A, idx=A, mask=None, stats=A, counts=A, prob=A, ws=A)
    a.update(kw)
    return M.load_library().moe_balance_loss(ctx, ctypes.byref(cfg.c()), a["logits"], a["idx"], a["mask"], T, a["stats"],
                                             a["counts"], a["prob"], a["ws"], ws_bytes, None)


def test_balance_loss_refusals():
    assert _balance(ctx=None) == M.EINVAL
    assert _balance(T=-1) == M.EINVAL
    for name in ("logits", "idx", "stats", "counts", "prob", "ws"):
        assert _balance(**{name: None}) == M.EINVAL, name
    for name in ("logits", "idx", "stats", "counts", "prob"):
        assert _balance(**{name: A + 2}) == M.EINVAL, name
    assert _balance(ws=A + 16) == M.EINVAL
    assert _balance(ws_bytes=1000) == M.ENOSPACE
    assert _balance(cfg=M.TINY.replace(k=17)) == M.EINVAL
    assert _balance(cfg=M.TINY.replace(E=2048)) == M.EUNSUPPORTED
    assert _balance(cfg=M.TINY.replace(skip_from=1)) == M.EUNSUPPORTED


def _backward(cfg=M.TINY, T=4, ctx=CTX, **kw):
    a = dict(logits=A, idx=A, gate=A, mask=None, stats=A, counts=A, d_loss=A, d_gate=A, d_logits=A)
    a.update(kw)
    return M.load_library().moe_balance_loss_backward(ctx, ctypes.byref(cfg.c()), a["logits"], a["idx"], a["gate"],
                                                      a["mask"], T, a["stats"], a["counts"], a["d_loss"], a["d_gate"],
                                                      a["d_logits"], None)


def test_balance_backward_refusals():
    assert _backward(ctx=None) == M.EINVAL
    assert _backward(T=-1) == M.EINVAL
    for name in ("logits", "idx", "gate", "stats", "counts", "d_loss", "d_logits"):
        assert _backward(**{name: None}) == M.EINVAL, name
        assert _backward(**{name: A + 1}) == M.EINVAL, name
    assert _backward(T=0) == M.OK  # nothing to write
    assert _backward(T=0, logits=None) == M.OK


def _quant(fn, ctx=CTX, x=A, t=M.TYPE_BF16, rows=4, cols=64, ld=64, codes=A, scales=A):
    lib = M.load_library()
    if fn == "q":
        return lib.moe_mx4_quantize(ctx, x, t, rows, cols, ld, codes, scales, None)
    return lib.moe_mx4_dequantize(ctx, codes, scales, rows, cols, x, t, ld, None)


@pytest.mark.parametrize("fn", ["q", "d"])
def test_conversion_refusals(fn):
    assert _quant(fn, ctx=None) == M.EINVAL
    assert _quant(fn, x=None) == M.EINVAL
    assert _quant(fn, x=A + 1) == M.EINVAL
    assert _quant(fn, x=A + 2, t=M.TYPE_FP32) == M.EINVAL
    assert _quant(fn, codes=None) == M.EINVAL
    assert _quant(fn, codes=A + 8) == M.EINVAL
    assert _quant(fn, scales=None) == M.EINVAL
    assert _quant(fn, scales=A + 4) == M.EINVAL
    assert _quant(fn, rows=-1) == M.EINVAL
    assert _quant(fn, cols=0) == M.EINVAL
    assert _quant(fn, cols=48) == M.EUNSUPPORTED
    assert _quant(fn, cols=65568, ld=65568) == M.EUNSUPPORTED
    assert _quant(fn, rows=2 ** 31 - 1, cols=65536, ld=65536) == M.EUNSUPPORTED
    assert _quant(fn, t=3) == M.EUNSUPPORTED
    assert _quant(fn, t=-1) == M.EUNSUPPORTED
    assert _quant(fn, ld=63) == M.EINVAL
    assert _quant(fn, rows=0, x=None) == M.OK


def _grouping(T=4, k=2, E=16, **kw):
    g = M.Grouping()
    g.T, g.k, g.E, g.n_pairs, g.n_rows = T, k, E, T * k, T * k + T
    for n in ("pair_token", "pair_gate", "uniq_slot", "uniq_offset", "n_uniq"):
        setattr(g, n, A)
    for n, v in kw.items():
        setattr(g, n, v)
    return g


def _product(ctx=CTX, xc=A, xs=A, x_rows=4, wc=A, ws=A, cstride=64 * 32, sstride=64 * 16, n_slots=17, rows=64, cols=64,
             g=None, shared=-1, flags=0, out=A, t=M.TYPE_BF16, ld=64, w=True):
    m = M._Mx4(wc, ws, cstride, sstride, n_slots, rows, cols)
    return M.load_library().moe_mx4_product(ctx, xc, xs, x_rows, ctypes.byref(m) if w else None,
                                            None if g is None else ctypes.byref(g), shared, flags, out, t, ld, None)


def test_product_refusals():
    assert _product(ctx=None) == M.EINVAL
    assert _product(w=False) == M.EINVAL
    for name in ("xc", "xs", "wc", "ws"):
        assert _product(**{name: None}) == M.EINVAL, name
        assert _product(**{name: A + 8}) == M.EINVAL, name
    assert _product(out=None) == M.EINVAL
    assert _product(out=A + 1) == M.EINVAL
    assert _product(out=A + 2, t=M.TYPE_FP32) == M.EINVAL
    assert _product(t=7) == M.EUNSUPPORTED
    assert _product(rows=0) == M.EINVAL
    assert _product(rows=72) == M.EUNSUPPORTED
    assert _product(cols=80) == M.EUNSUPPORTED
    assert _product(n_slots=0) == M.EINVAL
    assert _product(cstride=64 * 32 - 16) == M.EINVAL
    assert _product(cstride=64 * 32 + 8) == M.EINVAL
    assert _product(sstride=64 * 16 - 16) == M.EINVAL
    assert _product(ld=63) == M.EINVAL
    assert _product(ld=31, flags=M.MX4_SWIGLU) == M.EINVAL
    assert _product(x_rows=-1) == M.EINVAL
    assert _product(flags=8) == M.EINVAL
    assert _product(x_rows=0, xc=None) == M.OK
    # one group takes no grouping's options
    assert _product(shared=0) == M.EINVAL
    assert _product(flags=M.MX4_GATHER) == M.EINVAL
    assert _product(flags=M.MX4_GATE) == M.EINVAL


def test_grouped_product_refusals():
    assert _product(g=_grouping(), x_rows=5, flags=M.MX4_GATHER) == M.EINVAL   # one row per token
    assert _product(g=_grouping(), x_rows=7) == M.EINVAL                       # one row per pair
    assert _product(g=_grouping(), x_rows=8, shared=3) == M.EINVAL             # and the shared expert's
    assert _product(g=_grouping(), x_rows=12, shared=17) == M.EINVAL           # past the pool
    assert _product(g=_grouping(), x_rows=12, shared=-2) == M.EINVAL
    assert _product(g=_grouping(n_pairs=9), x_rows=12) == M.EINVAL
    assert _product(g=_grouping(T=-1), x_rows=12) == M.EINVAL
    assert _product(g=_grouping(k=40), x_rows=200) == M.EINVAL
    assert _product(g=_grouping(E=4096), x_rows=12) == M.EINVAL
    for name in ("pair_token", "pair_gate", "uniq_slot", "uniq_offset", "n_uniq"):
        assert _product(g=_grouping(**{name: None}), x_rows=12) == M.EINVAL, name
    assert _product(g=_grouping(T=0), x_rows=0) == M.OK


def test_grouped_product_sizes_past_32_bits():
    # T * k that wraps around to n_pairs; output rows that no int numbers
    t = (1 << 28) + 1
    assert _product(g=_grouping(T=t, k=16, n_pairs=16, n_rows=16 + t), x_rows=t, flags=M.MX4_GATHER) == M.EINVAL
    t = 1 << 30
    assert _product(g=_grouping(T=t, k=1), x_rows=t, shared=3, flags=M.MX4_GATHER) == M.EUNSUPPORTED
    assert _product(x_rows=t + 1) == M.EUNSUPPORTED


def test_matrix_and_buffer_checks():
    import torch
    with pytest.raises(M.MoeError):
        M.mx4_buffers(4, 40, device="cpu")
    with pytest.raises(M.MoeError):
        M.mx4_buffers(-1, 64, device="cpu")
    codes, scales = M.mx4_buffers(6, 768, device="cpu")
    assert codes.shape == (6, 384) and scales.shape == (6, 32)
    with pytest.raises(M.MoeError):
        M.Mx4Matrix(codes, scales[:, :24], 768)
    with pytest.raises(M.MoeError):
        M.Mx4Matrix(codes[:, :300], scales, 768)
    pool = torch.zeros(3, 1 << 14, dtype=torch.uint8)
    w = M.Mx4Matrix(pool[:, :16 * 384].view(3, 16, 384), pool[:, 8192:8192 + 512].view(3, 16, 32), 768)
    assert (w.n_slots, w.rows, w.c().code_stride, w.c().scale_stride) == (3, 16, 1 << 14, 1 << 14)
    with pytest.raises(M.MoeError):
        M._rows(torch.zeros(4, 8).t())


def test_balance_token_limit():
    """2^24 tokens: their number, and the detail t * k + j of a bad choice, stay exact."""
    t = 1 << 24
    for n in (t + 1, 2 ** 31 - 1):
        assert _balance(T=n) == M.EUNSUPPORTED
        assert _backward(T=n) == M.EUNSUPPORTED
    # at the limit the next check speaks
    assert _balance(T=t, ws_bytes=0) == M.ENOSPACE
    assert _backward(T=t, d_logits=None) == M.EINVAL
