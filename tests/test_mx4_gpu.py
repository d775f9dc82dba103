"""4-bit MX matrices on the GPU against the fp64 oracle: quantisation and back
bit for bit, products within their roundings.

Tolerance of a product: the products of two levels times their scales are exact
in fp32; of the sum of K terms every addition is off by at most one step (2^-23)
of the running magnitude (the tensor cores may truncate), so K 2^-23 sum |x w|
bounds the sum's error. A store rounds once: half a step of the output type.
SwiGLU of gate g and up u with errors dg and du: silu' is at most 1.1, the
exponential, division and product add 8 steps of fp32 (|g| below 87).
"""
import numpy as np
import pytest
import torch

from bit_expert_ffn_router_b200 import moe as M
from oracle import train_oracle as O
from tests import harness as H

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}  # half the smallest subnormal, fp16
TYPES = list(HALF)


def values(rows, cols, seed, t=torch.float32):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, cols)) * np.exp(rng.normal(size=(rows, 1)))
    x.reshape(rows, cols // 32, 32)[rng.random((rows, cols // 32)) < 0.05] = 0
    return torch.from_numpy(x.astype(np.float32)).cuda().to(t)


def quantize(x):
    codes, scales = M.mx4_buffers(*x.shape)
    codes.fill_(0xEE), scales.fill_(0xEE)
    H.ctx().mx4_quantize(x, codes, scales)
    return codes, scales


def npy(t):
    return t.cpu().numpy()


# ------------------------------------------------------------------ conversions

@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 32), (1, 64), (5, 96), (1, 2048), (7, 768), (33, 544), (260, 160),
                                       (2, 65536), (1030, 32)])
def test_quantize_bit_for_bit(rows, cols, t):
    x = values(rows, cols, rows + cols, t)
    codes, scales = quantize(x)
    want = O.mx4_quantize(npy(x.float()))
    assert np.array_equal(npy(codes), want[0]) and np.array_equal(npy(scales), want[1])
    out = torch.empty_like(x)
    H.ctx().mx4_dequantize(codes, scales, out)
    v = torch.from_numpy(O.mx4_values(*want)).to(t)
    assert torch.equal(out.cpu(), v)


def test_every_border_and_its_neighbours():
    """All fp32 values next to the borders between levels, at several scales, and every bf16 in a block of its own."""
    mids = np.array([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 6.5, 7, 7.99], np.float32)
    near = np.concatenate([mids, np.nextafter(mids, np.float32(9)), np.nextafter(mids, np.float32(-9))])
    near = np.concatenate([near, -near])
    rows = []
    for e in (-126, -120, -30, 0, 40, 125):
        for i in range(0, near.size, 31):
            blk = np.zeros(32, np.float32)
            blk[:near[i:i + 31].size] = near[i:i + 31]
            blk[31] = 4  # the block's scale is 2^e
            rows.append(np.ldexp(blk, e))
    x = torch.from_numpy(np.stack(rows)).cuda()
    codes, scales = quantize(x)
    want = O.mx4_quantize(npy(x))
    assert np.array_equal(npy(codes), want[0]) and np.array_equal(npy(scales), want[1])
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = torch.zeros(65536, 32, dtype=torch.bfloat16)
    x[:, 7] = bits
    x[:, 20] = bits / 2
    codes, scales = quantize(x.cuda())
    want = O.mx4_quantize(npy(x.float()))
    assert np.array_equal(npy(codes), want[0]) and np.array_equal(npy(scales), want[1])


def test_extreme_blocks():
    x = torch.zeros(1, 32 * 12)
    b = x.view(12, 32)
    b[0, 3] = float("nan")
    b[1, 4] = float("inf")
    b[2, 5] = float("-inf")
    b[3, :] = torch.finfo(torch.float32).max
    b[4, :] = -torch.finfo(torch.float32).max
    b[5, 0] = 1e-45
    b[6, :] = 2.0 ** -126
    b[7, 1], b[7, 2] = 2.0 ** -125, 2.0 ** -149
    b[8, :] = -0.0
    b[9, 0], b[9, 1] = 3e38, 1e-30
    x = x.cuda()
    codes, scales = quantize(x)
    want = O.mx4_quantize(npy(x))
    assert np.array_equal(npy(codes), want[0]) and np.array_equal(npy(scales), want[1])
    for t in TYPES:
        out = torch.empty(x.shape, dtype=t, device="cuda")
        H.ctx().mx4_dequantize(codes, scales, out)
        v = torch.from_numpy(O.mx4_values(*want)).to(t)
        assert torch.equal(out.cpu().isnan(), v.isnan())
        assert torch.equal(out.cpu().nan_to_num(nan=0.0), v.nan_to_num(nan=0.0))


def test_every_code_at_every_scale():
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 16)[:, :16 * 16].contiguous()
    scales = torch.zeros(256, M.mx4_scale_pitch(512), dtype=torch.uint8)
    scales[:] = torch.arange(256, dtype=torch.uint8)[:, None]
    want = O.mx4_values(npy(codes), npy(scales))
    for t in TYPES:
        out = torch.empty(256, 512, dtype=t, device="cuda")
        H.ctx().mx4_dequantize(codes.cuda(), scales.cuda(), out)
        v = torch.from_numpy(want).to(t)
        assert torch.equal(out.cpu().isnan(), v.isnan())
        assert torch.equal(out.cpu().nan_to_num(nan=0.0), v.nan_to_num(nan=0.0))


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("gap,shift", [(1, 0), (8, 0), (3, 1), (16, 8)])
def test_strides_and_alignment(t, gap, shift):
    rows, cols = 9, 160
    buf = torch.full((rows * (cols + gap) + shift,), 3.0, dtype=t, device="cuda")
    x = buf[shift:].view(rows, cols + gap)[:, :cols]
    x.copy_(values(rows, cols, 4, t))
    codes, scales = quantize(x)
    want = O.mx4_quantize(npy(x.float()))
    assert np.array_equal(npy(codes), want[0]) and np.array_equal(npy(scales), want[1])
    H.ctx().mx4_dequantize(codes, scales, x)
    assert torch.equal(x.cpu(), torch.from_numpy(O.mx4_values(*want)).to(t))
    assert (buf[shift:].view(rows, cols + gap)[:, cols:] == 3).all()  # the gaps are left alone


def test_no_rows():
    codes, scales = M.mx4_buffers(0, 64)
    H.ctx().mx4_quantize(torch.empty(0, 64, device="cuda"), codes, scales)
    H.ctx().mx4_dequantize(codes, scales, torch.empty(0, 64, device="cuda"))


# ------------------------------------------------------------------ products

def assert_product(out, x, w, half, swiglu=False, gate=None, tiny=0.0):
    """out against x [r, K] w [n, K]^T in fp64, with the bound of the module's docstring."""
    K = x.shape[1]
    s, a = x @ w.T, np.abs(x) @ np.abs(w).T * (K * 2.0 ** -23)
    if swiglu:
        g, u, dg, du = s[:, 0::2], s[:, 1::2], a[:, 0::2], a[:, 1::2]
        silu = g / (1 + np.exp(-np.minimum(np.maximum(g, -700), 700)))
        s = silu * u
        a = 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du + np.abs(s) * (8 + 2.4 * np.abs(g)) * 2.0 ** -23
    if gate is not None:
        s, a = s * gate[:, None], a * gate[:, None] + np.abs(s * gate[:, None]) * 2.0 ** -24
    o = npy(out.float()).astype(np.float64)
    bad = np.isnan(s)
    assert np.array_equal(np.isnan(o), bad)
    tol = a + (np.abs(s) + a) * half + tiny
    err = np.where(bad, 0, np.abs(o - s))
    i = np.unravel_index(np.argmax(np.where(bad, -1, err - tol)), err.shape)
    assert np.all(bad | (err <= tol)), f"{i}: {o[i]} for {s[i]}, bound {tol[i]}"


def matrix(n_slots, rows, cols, seed, gap=0):
    """Random weights as a pool, some blocks of large and of tiny scale."""
    rng = np.random.default_rng(seed)
    pitch = M.mx4_scale_pitch(cols)
    codes = rng.integers(0, 256, size=(n_slots, rows, cols // 2), dtype=np.uint8)
    scales = np.zeros((n_slots, rows, pitch), np.uint8)
    scales[:, :, :cols // 32] = rng.integers(118, 125, size=(n_slots, rows, cols // 32))
    scales[:, :, cols // 32:] = 255  # the padding is not read as scales
    cbytes, sbytes = rows * cols // 2, rows * pitch
    pool = torch.full((n_slots, (cbytes + sbytes + gap) // 16 * 16), 0xEE, dtype=torch.uint8, device="cuda")
    pool[:, :cbytes] = torch.from_numpy(codes.reshape(n_slots, -1)).cuda()
    pool[:, cbytes:cbytes + sbytes] = torch.from_numpy(scales.reshape(n_slots, -1)).cuda()
    w = M.Mx4Matrix(pool[:, :cbytes].view(n_slots, rows, cols // 2), pool[:, cbytes:cbytes + sbytes].view(n_slots, rows, pitch),
                    cols)
    return w, [O.mx4_values(codes[s], scales[s]) for s in range(n_slots)]


DENSE = [(1, 16, 32), (1, 128, 256), (2, 144, 64), (7, 16, 2048), (15, 256, 288), (16, 1536, 768), (17, 48, 544),
         (33, 272, 96), (100, 128, 512), (129, 400, 1024), (192, 128, 256), (193, 144, 224), (300, 2048, 160),
         (385, 256, 1056), (1000, 96, 352), (3, 32, 8192)]


@pytest.mark.parametrize("swiglu", [False, True], ids=["plain", "swiglu"])
@pytest.mark.parametrize("rows,n,cols", DENSE)
def test_one_matrix(rows, n, cols, swiglu):
    w, wv = matrix(1, n, cols, rows + n)
    x = values(rows, cols, 1, torch.bfloat16)
    codes, scales = quantize(x)
    xv = O.mx4_values(npy(codes), npy(scales))
    for t in TYPES:
        out = torch.empty(rows, n // 2 if swiglu else n, dtype=t, device="cuda")
        H.ctx().mx4_product(codes, scales, w, out, swiglu=swiglu)
        assert_product(out, xv, wv[0], HALF[t], swiglu, tiny=TINY[t])
    assert H.ctx().check_device_status() == M.OK


def test_nan_and_zero_scales():
    rows, n, cols = 40, 128, 512
    w, wv = matrix(1, n, cols, 3)
    x = values(rows, cols, 2)
    x[3, 100] = float("nan")
    x[11, 300] = float("inf")
    x[20] = 0
    codes, scales = quantize(x)
    xv = O.mx4_values(npy(codes), npy(scales))
    assert np.isnan(xv[3]).any() and np.isnan(xv[11]).any()
    w.scales[0, 50, 2] = 255
    wv[0][50, 64:96] = np.nan
    out = torch.empty(rows, n, device="cuda")
    H.ctx().mx4_product(codes, scales, w, out)
    assert_product(out, xv, wv[0], HALF[torch.float32])


def test_far_scales():
    """Products whose scales are near both ends of the format's range."""
    rows, n, cols = 5, 16, 64
    w, wv = matrix(1, n, cols, 4)
    w.scales[0, :, 0] = torch.arange(16, device="cuda") + 20
    w.scales[0, :, 1] = torch.arange(16, device="cuda") + 15
    codes, scales = quantize(values(rows, cols, 3))
    scales[:, 0] = 250
    scales[:, 1] = 245
    wv = O.mx4_values(npy(w.codes[0]), npy(w.scales[0]))
    out = torch.empty(rows, n, device="cuda")
    H.ctx().mx4_product(codes, scales, w, out)
    assert_product(out, O.mx4_values(npy(codes), npy(scales)), wv, HALF[torch.float32])


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("gap,shift", [(1, 0), (8, 0), (3, 1), (2, 2)])
@pytest.mark.parametrize("swiglu", [False, True], ids=["plain", "swiglu"])
def test_output_strides(t, gap, shift, swiglu):
    rows, n, cols = 21, 144, 96
    w, wv = matrix(1, n, cols, 5)
    codes, scales = quantize(values(rows, cols, 6))
    nc = n // 2 if swiglu else n
    buf = torch.full((rows * (nc + gap) + shift + 8,), 3.0, dtype=t, device="cuda")
    out = buf[shift:shift + rows * (nc + gap)].view(rows, nc + gap)[:, :nc]
    H.ctx().mx4_product(codes, scales, w, out, swiglu=swiglu)
    assert_product(out, O.mx4_values(npy(codes), npy(scales)), wv[0], HALF[t], swiglu, tiny=TINY[t])
    assert (buf[:shift] == 3).all() and (buf[shift + rows * (nc + gap):] == 3).all()
    assert (buf[shift:shift + rows * (nc + gap)].view(rows, nc + gap)[:, nc:] == 3).all()


class Grouped:
    """T tokens routed to k of E experts in a pool of E + 1 + spare slots, with a shared expert."""

    def __init__(self, T, E, k, seed, hot=None, absent=()):
        rng = np.random.default_rng(seed)
        self.T, self.E, self.k = T, E, k
        self.n_slots = E + 3
        s = rng.normal(size=(T, E))
        if hot is not None:
            s[:, hot] += 3
        self.idx = np.argsort(-s, axis=1, kind="stable")[:, :k].astype(np.int32)
        self.gate = rng.random((T, k)).astype(np.float32) + 0.1
        perm = rng.permutation(self.n_slots)
        self.slot_of = perm[:E].astype(np.int32)
        self.slot_of[list(absent)] = -1
        self.shared = int(perm[E])
        self.cfg = M.LayerCfg(d=256, f=128, E=E, k=k)
        self.ws = M.workspace(self.cfg, T)
        self.dev = [torch.from_numpy(a).cuda() for a in (self.idx, self.gate, self.slot_of)]
        self.g = H.ctx().group_tokens(self.cfg, self.dev[0], self.dev[1], T, self.dev[2], self.n_slots, self.ws)
        # sorted pairs, from the choices alone
        pairs = [(e, t, j) for t in range(T) for j, e in enumerate(self.idx[t]) if self.slot_of[e] >= 0]
        self.pairs = sorted(pairs)

    def rows(self, shared=True):
        return self.T * self.k + (self.T if shared else 0)

    def parts(self, shared=True):
        """(output rows, tokens, slot, gates) of every group."""
        out = []
        for e in range(self.E):
            p = [i for i, q in enumerate(self.pairs) if q[0] == e]
            if p:
                out.append((p, [self.pairs[i][1] for i in p], self.slot_of[e],
                            np.array([self.gate[self.pairs[i][1], self.pairs[i][2]] for i in p], np.float64)))
        if shared:
            out.append(([self.T * self.k + t for t in range(self.T)], list(range(self.T)), self.shared, np.ones(self.T)))
        return out


GROUPED = [(1, 16, 2, None), (2, 64, 10, None), (8, 512, 10, None), (5, 8, 8, None), (64, 16, 2, 3), (200, 8, 2, 1),
           (333, 40, 3, None), (450, 4, 1, 0), (130, 600, 4, None)]


@pytest.mark.parametrize("T,E,k,hot", GROUPED)
def test_grouped_gate_up(T, E, k, hot):
    G = Grouped(T, E, k, T + E, hot)
    f, d = 48, 288
    w, wv = matrix(G.n_slots, 2 * f, d, 7, gap=48)
    codes, scales = quantize(values(T, d, 8, torch.bfloat16))
    xv = O.mx4_values(npy(codes), npy(scales))
    out = torch.full((G.rows(), f), 7.0, dtype=torch.bfloat16, device="cuda")
    H.ctx().mx4_product(codes, scales, w, out, grouping=G.g, shared_slot=G.shared, gather=True, swiglu=True)
    for rows, tokens, slot, _ in G.parts():
        assert_product(out[rows], xv[tokens], wv[slot], HALF[torch.bfloat16], swiglu=True)
    assert H.ctx().check_device_status() == M.OK


@pytest.mark.parametrize("T,E,k,hot", GROUPED)
def test_grouped_down(T, E, k, hot):
    G = Grouped(T, E, k, T + E + 1, hot)
    f, d = 96, 144
    w, wv = matrix(G.n_slots, d, f, 9)
    codes, scales = quantize(values(G.rows(), f, 10, torch.float16))
    xv = O.mx4_values(npy(codes), npy(scales))
    out = torch.full((G.rows(), d), 7.0, device="cuda")
    H.ctx().mx4_product(codes, scales, w, out, grouping=G.g, shared_slot=G.shared, gate=True)
    for rows, _, slot, gate in G.parts():
        assert_product(out[rows], xv[rows], wv[slot], HALF[torch.float32], gate=gate)
    # without the shared expert its rows are left as they were
    out.fill_(7.0)
    H.ctx().mx4_product(codes, scales, w, out, grouping=G.g, gate=True)
    assert (out[G.T * G.k:] == 7).all() and not (out[:G.T * G.k] == 7).all()
    assert H.ctx().check_device_status() == M.OK


def test_absent_experts_leave_their_rows():
    G = Grouped(40, 8, 2, 3, absent=(1, 4, 7))
    w, wv = matrix(G.n_slots, 32, 64, 11)
    codes, scales = quantize(values(40, 64, 12))
    xv = O.mx4_values(npy(codes), npy(scales))
    out = torch.full((G.rows(), 32), 7.0, device="cuda")
    H.ctx().mx4_product(codes, scales, w, out, grouping=G.g, shared_slot=G.shared, gather=True)
    used = 0
    for rows, tokens, slot, _ in G.parts():
        assert_product(out[rows], xv[tokens], wv[slot], HALF[torch.float32])
        used += len(rows)
    assert used < G.rows()
    assert (out[len(G.pairs):G.T * G.k] == 7).all()
    # a device that holds none of the chosen experts, without the shared one, writes nothing
    G = Grouped(10, 4, 2, 3, absent=(0, 1, 2, 3))
    out.fill_(7.0)
    H.ctx().mx4_product(*quantize(values(10, 64, 1)), w, out, grouping=G.g, gather=True)
    assert (out == 7).all()
    assert H.ctx().check_device_status() == M.OK


def test_a_slot_past_the_pool_is_reported_and_not_read():
    G = Grouped(12, 6, 2, 5)
    w, wv = matrix(G.n_slots, 32, 64, 13)
    worst = int(G.slot_of.max())
    small = M.Mx4Matrix(w.codes[:worst], w.scales[:worst], 64)
    codes, scales = quantize(values(12, 64, 14))
    xv = O.mx4_values(npy(codes), npy(scales))
    out = torch.full((G.rows(), 32), 7.0, device="cuda")
    H.ctx().mx4_product(codes, scales, small, out, grouping=G.g, gather=True)
    for rows, tokens, slot, _ in G.parts(shared=False):
        if slot < worst:
            assert_product(out[rows], xv[tokens], wv[slot], HALF[torch.float32])
        else:
            assert (out[rows] == 7).all()
    assert H.ctx().check_device_status() == M.EDEVICE


def test_a_token_past_x_is_reported():
    G = Grouped(12, 6, 2, 6)
    w, wv = matrix(G.n_slots, 32, 64, 13)
    codes, scales = quantize(values(12, 64, 14))
    xv = O.mx4_values(npy(codes), npy(scales))
    view = H.ctx().layer_routing(G.cfg, G.T, G.ws)["pair_token"]
    view[3], view[7] = 12, -1
    out = torch.full((G.rows(), 32), 7.0, device="cuda")
    H.ctx().mx4_product(codes, scales, w, out, grouping=G.g, shared_slot=G.shared, gather=True)
    for rows, tokens, slot, _ in G.parts():
        keep = [i for i, r in enumerate(rows) if r not in (3, 7)]
        if keep:
            assert_product(out[[rows[i] for i in keep]], xv[[tokens[i] for i in keep]], wv[slot], HALF[torch.float32])
    assert H.ctx().check_device_status() == M.EDEVICE
    assert H.ctx().last_device_error_detail() in (3, 7)


def test_an_expert_named_twice_has_more_rows_than_tokens():
    """40 tokens that name expert 1 three times each: 120 rows of one group."""
    T = 40
    cfg = M.LayerCfg(d=256, f=128, E=4, k=3)
    idx = torch.ones(T, 3, dtype=torch.int32, device="cuda")
    gate = torch.rand(T, 3, device="cuda")
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    ws = M.workspace(cfg, T)
    g = H.ctx().group_tokens(cfg, idx, gate, T, slots, 4, ws)
    w, wv = matrix(4, 48, 96, 3)
    codes, scales = quantize(values(T, 96, 4))
    xv = O.mx4_values(npy(codes), npy(scales))
    out = torch.empty(T * 3, 48, device="cuda")
    H.ctx().mx4_product(codes, scales, w, out, grouping=g, gather=True, gate=True)
    tok = npy(H.ctx().layer_routing(cfg, T, ws)["pair_token"])
    pg = npy(H.ctx().layer_routing(cfg, T, ws)["pair_gate"]).astype(np.float64)
    assert_product(out, xv[tok], wv[1], HALF[torch.float32], gate=pg)


def test_more_items_than_a_block_lists():
    """1024 groups of one row by 96 weight tiles: about 660 items per SM."""
    T, k, E, n = 64, 16, 1024, 18416
    cfg = M.LayerCfg(d=256, f=128, E=E, k=k)
    idx = torch.arange(T * k, dtype=torch.int32, device="cuda").view(T, k)
    gate = torch.rand(T, k, device="cuda")
    slots = torch.randperm(E, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    ws = M.workspace(cfg, T)
    g = H.ctx().group_tokens(cfg, idx, gate, T, slots, E, ws)
    codes, scales = quantize(values(T, 32, 5))
    wc = torch.randint(0, 256, (E, n, 16), dtype=torch.uint8, device="cuda")
    wsc = torch.randint(118, 125, (E, n, 16), dtype=torch.uint8, device="cuda")
    out = torch.empty(T * k, n, device="cuda")
    H.ctx().mx4_product(codes, scales, M.Mx4Matrix(wc, wsc, 32), out, grouping=g, gather=True)
    xv = O.mx4_values(npy(codes), npy(scales))
    for e in (0, 1, 511, 700, 1023):
        s = int(slots[e])
        assert_product(out[e:e + 1], xv[e // k:e // k + 1], O.mx4_values(npy(wc[s]), npy(wsc[s])), HALF[torch.float32])
    # every row against its neighbours' arithmetic: the same x row and matrix through the one-matrix call
    for e in range(0, E, 41):
        one = torch.empty(1, n, device="cuda")
        s = int(slots[e])
        t = e // k
        H.ctx().mx4_product(codes[t:t + 1], scales[t:t + 1], M.Mx4Matrix(wc[s], wsc[s], 32), one)
        assert torch.equal(one[0], out[e])
    assert H.ctx().check_device_status() == M.OK


def test_the_longest_rows():
    w, wv = matrix(1, 16, 65536, 21)
    codes, scales = quantize(values(2, 65536, 22))
    out = torch.empty(2, 16, device="cuda")
    H.ctx().mx4_product(codes, scales, w, out)
    assert_product(out, O.mx4_values(npy(codes), npy(scales)), wv[0], HALF[torch.float32])


def test_two_captured_products_replayed_at_once():
    runs = []
    for i in range(2):
        G = Grouped(90 + 60 * i, 8, 2, 60 + i)
        w, _ = matrix(G.n_slots, 256, 512, 25 + i)
        codes, scales = quantize(values(G.T, 512, 26 + i))
        out = torch.empty(G.rows(), 128, dtype=torch.bfloat16, device="cuda")
        call = lambda s=None, a=(codes, scales, w, out, G): H.ctx().mx4_product(  # noqa: E731
            *a[:4], grouping=a[4].g, shared_slot=a[4].shared, gather=True, swiglu=True, stream=s)
        call()
        torch.cuda.synchronize()
        want = out.clone()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                for _ in range(4):
                    call(s)
        runs.append((graph, s, out, want, G))
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, s, out, *_ in runs:
            with torch.cuda.stream(s):
                out.zero_()
                graph.replay()
    torch.cuda.synchronize()
    for _, _, out, want, _ in runs:
        assert torch.equal(out, want)


def test_python_refusals():
    G = Grouped(4, 6, 2, 5)
    w, _ = matrix(G.n_slots, 32, 64, 13)
    codes, scales = quantize(values(4, 64, 14))
    out = torch.empty(G.rows(), 32, device="cuda")
    ctx = H.ctx()
    ctx.mx4_product(codes, scales, w, out, grouping=G.g, shared_slot=G.shared, gather=True)
    bad = [dict(out=out[:5]), dict(out=out[:, :16]), dict(out=out.double()), dict(codes=codes[:3]), dict(scales=scales[:, :8]),
           dict(gather=False), dict(shared_slot=G.n_slots), dict(out=out.to(torch.int32))]
    for kw in bad:
        a = dict(codes=codes, scales=scales, out=out, shared_slot=G.shared, gather=True)
        a.update(kw)
        with pytest.raises(M.MoeError):
            ctx.mx4_product(a["codes"], a["scales"], w, a["out"], grouping=G.g, shared_slot=a["shared_slot"],
                            gather=a["gather"])
    with pytest.raises(M.MoeError):
        ctx.mx4_quantize(values(4, 64, 1).double(), codes, scales)
    with pytest.raises(M.MoeError):
        ctx.mx4_quantize(values(5, 64, 1), codes, scales)
    with pytest.raises(M.MoeError):
        ctx.mx4_quantize(values(64, 64, 1).t(), *M.mx4_buffers(64, 64))


def test_ffn_refusals():
    G = Grouped(4, 6, 2, 5)
    cfg = G.cfg
    up, _ = matrix(G.n_slots, 2 * cfg.f, cfg.d, 13)
    down, _ = matrix(G.n_slots, cfg.d, cfg.f, 13)
    x, z = values(4, cfg.d, 1, torch.bfloat16), torch.empty(G.rows(), cfg.d, device="cuda")
    bufs = M.mx4_ffn_buffers(cfg, 4)
    for a in ((up, down, -1), (down, down, G.shared), (up, up, G.shared)):
        with pytest.raises(M.MoeError):
            H.ctx().expert_ffn_mx4(cfg, x, G.g, *a, bufs, z)


# ------------------------------------------------------------------ together

def ffn(G, x, up, down, f, d, y, stream=None, bufs=None):
    """A whole expert step on 4-bit weights: quantise, gate/up, quantise, down, join."""
    c, cfg = H.ctx(), G.cfg.replace(d=d, f=f)
    xq, h, hq, z = bufs
    c.expert_ffn_mx4(cfg, x, G.g, up, down, G.shared, (xq, h, hq), z, stream=stream)
    c.combine(cfg, G.g, z, x, G.T, y, stream=stream)


def ffn_buffers(G, f, d):
    return (*M.mx4_ffn_buffers(G.cfg.replace(d=d, f=f), G.T), torch.empty(G.rows(), d, device="cuda"))


@pytest.mark.parametrize("T", [1, 3, 8, 77, 400])
def test_the_whole_step_eager_and_captured(T):
    E, k, d, f = 16, 2, 256, 128
    G = Grouped(T, E, k, 21 + T)
    up, upv = matrix(G.n_slots, 2 * f, d, 15)
    down, downv = matrix(G.n_slots, d, f, 16)
    x = values(T, d, 17, torch.bfloat16)
    y = torch.empty(T, d, device="cuda")
    bufs = ffn_buffers(G, f, d)
    ffn(G, x, up, down, f, d, y, bufs=bufs)
    torch.cuda.synchronize()
    (xc, xs), h, (hc, hs), z = bufs
    xv = O.mx4_values(npy(xc), npy(xs))
    assert np.array_equal(xv, O.mx4_values(*O.mx4_quantize(npy(x.float()))))
    # each step against the oracle on the inputs that it was given
    assert np.array_equal(O.mx4_values(npy(hc), npy(hs)), O.mx4_values(*O.mx4_quantize(npy(h.float()))))
    hv = O.mx4_values(npy(hc), npy(hs))
    want = np.zeros((T, d))
    for rows, tokens, slot, gate in G.parts():
        assert_product(h[rows], xv[tokens], upv[slot], HALF[torch.bfloat16], swiglu=True)
        assert_product(z[rows], hv[rows], downv[slot], HALF[torch.float32], gate=gate)
        np.add.at(want, tokens, npy(z[rows]).astype(np.float64))
    # k + 1 terms, each addition half a step of the sum of magnitudes
    size = np.zeros((T, d))
    for rows, tokens, _, _ in G.parts():
        np.add.at(size, tokens, np.abs(npy(z[rows]).astype(np.float64)))
    assert np.all(np.abs(npy(y) - want) <= (k + 1) * 2.0 ** -24 * size)
    first = y.clone()
    # captured, on a side stream, replayed with other tokens in between
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            ffn(G, x, up, down, f, d, y, stream=s, bufs=bufs)
        keep = x.clone()
        x.copy_(values(T, d, 99, torch.bfloat16))
        graph.replay()
        s.synchronize()
        assert not torch.equal(y, first)
        x.copy_(keep)
        graph.replay()
        s.synchronize()
    assert torch.equal(y, first)
    assert H.ctx().check_device_status() == M.OK


def test_two_streams_at_once():
    runs = []
    for i in range(2):
        G = Grouped(150 + i, 16, 2, 40 + i)
        up, _ = matrix(G.n_slots, 256, 256, 15 + i)
        down, _ = matrix(G.n_slots, 256, 128, 16 + i)
        x = values(G.T, 256, 50 + i, torch.bfloat16)
        bufs, y = ffn_buffers(G, 128, 256), torch.empty(G.T, 256, device="cuda")
        ffn(G, x, up, down, 128, 256, y, bufs=bufs)
        runs.append((G, x, up, down, bufs, y, y.clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for G, x, up, down, bufs, y, _, s in runs:
            with torch.cuda.stream(s):
                ffn(G, x, up, down, 128, 256, y, stream=s, bufs=bufs)
    torch.cuda.synchronize()
    for *_, y, want, s in runs:
        assert torch.equal(y, want)


@pytest.mark.parametrize("T,absent,n_shared", [(5, (0, 3, 5), 1), (90, (0, 3, 5), 1), (7, (), 0), (300, (1,), 0),
                                               (4, tuple(range(8)), 0), (6, tuple(range(8)), 1), (0, (), 1), (0, (), 0)])
def test_the_whole_step_with_experts_or_tokens_left_out(T, absent, n_shared):
    """What the buffers held before shows nowhere, rows of absent experts included."""
    E, k, d, f = 8, 2, 256, 128
    G = Grouped(max(T, 1), E, k, 60 + T, absent=absent)
    up, upv = matrix(G.n_slots, 2 * f, d, 15)
    down, downv = matrix(G.n_slots, d, f, 16)
    cfg = G.cfg.replace(d=d, f=f, n_shared=n_shared)
    shared = G.shared if n_shared else -1
    ws = M.workspace(cfg, max(T, 1))  # the grouping lives in it
    g = H.ctx().group_tokens(cfg, G.dev[0][:T], G.dev[1][:T], T, G.dev[2], G.n_slots, ws)
    x = values(max(T, 1), d, 17, torch.bfloat16)[:T]
    (xc, xs), h, (hc, hs) = M.mx4_ffn_buffers(cfg, T)
    for b in (xc, xs, hc, hs):
        b.fill_(0xFF)
    z = torch.full((T * (k + n_shared), d), float("nan"), device="cuda")
    h.fill_(float("nan"))
    y = torch.full((T, d), 7.0, device="cuda")
    H.ctx().expert_ffn_mx4(cfg, x, g, up, down, shared, ((xc, xs), h, (hc, hs)), z)
    H.ctx().combine(cfg, g, z, x, T, y)
    assert H.ctx().check_device_status() == M.OK
    if T == 0:
        return
    xv, hv = O.mx4_values(npy(xc), npy(xs)), O.mx4_values(npy(hc), npy(hs))
    want, size = np.zeros((T, d)), np.zeros((T, d))
    seen = np.zeros(len(z), bool)
    for rows, tokens, slot, gate in G.parts(shared=bool(n_shared)):
        assert_product(h[rows], xv[tokens], upv[slot], HALF[torch.bfloat16], swiglu=True)
        assert_product(z[rows], hv[rows], downv[slot], HALF[torch.float32], gate=gate)
        seen[rows] = True
        np.add.at(want, tokens, npy(z[rows]).astype(np.float64))
        np.add.at(size, tokens, np.abs(npy(z[rows]).astype(np.float64)))
    assert np.isnan(npy(z)[~seen]).all()
    assert np.all(np.abs(npy(y) - want) <= (k + 1) * 2.0 ** -24 * size)
