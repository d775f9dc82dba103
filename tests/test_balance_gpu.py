"""The router's balance loss and its gradient against the fp64 oracle.

Tolerances, with u = 2^-24 (half a step of fp32). The kernels take exp(x), x = l
- max <= 0, as 2^y with y = l log2(e) - max log2(e): the second product's
rounding is the same for the whole row (it cancels in p and is worth |max| u in
lse), y rounds by u |y|, which is u |x| of the result, the constant by half
that, and 2^y by two steps: (4 + 1.5 |x|) u relative. Taken here as (4 + 2.4
|x|) u, which covers the documented error of the fast exponential too; the row's
sum of E terms adds E u at most, the division u. P(x) below is that sum: the
relative error of one p. |x| up to 87: beyond, exp(x) is below 2^-125 and the
absolute floor covers it.
* prob: the mean of the p over the tokens; each p is off by P u p, the sum of T
  terms by T u of itself.
* stats: the balance loss is a weighted mean of prob with exact weights; lse =
  max + log(sum) is off by 4 u |lse| + the sum's relative error, squared twice
  that.
* d_logits: every factor is a few roundings of terms of known magnitude
  (`size`, from the oracle), with P from p and from the weighted sum: 3 P + 16,
  and k more for the gates' sum.
"""
import numpy as np
import pytest
import torch

from bit_expert_ffn_router_b200 import moe as M
from oracle import train_oracle as O
from tests import harness as H

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def make(T, E, k, seed, renorm=True, mask=False, drop=False, scale=1.5):
    rng = np.random.default_rng(seed)
    l = (rng.normal(size=(T, E)) * scale + rng.normal(size=E)).astype(np.float32)
    if drop:
        l[:, rng.random(E) < 0.15] = -np.inf
        l[rng.random(T) < 0.1] = -np.inf
    idx = np.argsort(-l, axis=1, kind="stable")[:, :k].astype(np.int32)
    ex = np.exp(l.astype(np.float64) - np.maximum(l.max(1, keepdims=True), -1e30))
    g = np.take_along_axis(ex, idx, 1)
    gate = (g / np.maximum(g.sum(1, keepdims=True) if renorm else ex.sum(1, keepdims=True), 1e-300)).astype(np.float32)
    m = (rng.random(T) < 0.7).astype(np.uint8) if mask else None
    d_gate = (rng.normal(size=(T, k)) / max(T, 1)).astype(np.float32)
    return dict(l=l, idx=idx, gate=gate, mask=m, d_gate=d_gate, d_loss=np.array([0.7, -0.3], np.float32), renorm=renorm)


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Run:
    def __init__(self, c, logits=None, d_gate=True, d_logits=None):
        self.T, self.E = c["l"].shape
        self.k = c["idx"].shape[1]
        self.cfg = M.LayerCfg(d=256, f=128, E=self.E, k=self.k, renorm=int(c["renorm"]))
        self.l = dev(c["l"]) if logits is None else logits
        self.idx, self.gate, self.mask, self.d_loss = (dev(c[n]) for n in ("idx", "gate", "mask", "d_loss"))
        self.d_gate = dev(c["d_gate"]) if d_gate else None
        self.ws = M.balance_workspace(self.cfg).fill_(0xA5)
        self.stats = torch.full((4,), 7.0, device="cuda")
        self.counts = torch.full((self.E,), 7, dtype=torch.int32, device="cuda")
        self.prob = torch.full((self.E,), 7.0, device="cuda")
        self.d = torch.full((self.T, self.E), 7.0, device="cuda") if d_logits is None else d_logits

    def __call__(self, stream=None):
        H.ctx().balance_loss(self.cfg, self.l, self.idx, self.mask, self.T, self.stats, self.counts, self.prob, self.ws,
                             stream=stream)
        H.ctx().balance_loss_backward(self.cfg, self.l, self.idx, self.gate, self.mask, self.T, self.stats, self.counts,
                                      self.d_loss, self.d_gate, self.d, stream=stream)
        return self

    def out(self):
        torch.cuda.synchronize()
        return tuple(t.cpu().numpy() for t in (self.stats, self.counts, self.prob, self.d))


def check(c, got, d_gate=True):
    stats, counts, prob, d = (np.asarray(a) for a in got)
    T, E = c["l"].shape
    k = c["idx"].shape[1]
    w_stats, w_counts, w_prob = O.balance(c["l"], c["idx"], c["mask"])
    assert np.array_equal(counts, w_counts)
    keep = O.counted(c["l"], c["mask"])
    if not keep.any():
        assert not stats.any() and not prob.any() and not d.any()
        return
    lk = c["l"][keep].astype(np.float64)
    x = np.minimum(lk.max(1, keepdims=True) - lk, 87.0)
    P = np.zeros((T, E))
    P[keep] = 4 + 2.4 * x + E + 2
    worst = P.max()
    assert np.all(np.abs(prob - w_prob) <= (worst + T) * U * w_prob + 1e-37)
    lse = np.abs(np.log(np.exp(lk - lk.max(1, keepdims=True)).sum(1)) + lk.max(1))
    assert abs(stats[0] - w_stats[0]) <= (worst + T + 4) * U * w_stats[0]
    assert abs(stats[1] - w_stats[1]) <= (2 * (lse * (4 * lse + np.abs(lk.max(1)) + worst)).mean() + 4 * w_stats[1]) * U
    assert stats[2] == w_stats[2]
    assert abs(stats[3] - w_stats[3]) <= 2 * U * w_stats[3]
    want, size = O.balance_grad(c["l"], c["idx"], c["gate"], c["mask"], c["d_loss"], c["d_gate"] if d_gate else None,
                                c["renorm"])
    # lse enters with its own error: (4 |lse| + |max| + worst) u of the z factor
    z = np.zeros(T)
    z[keep] = abs(c["d_loss"][1]) * 2 / keep.sum() * (np.abs(lk.max(1)) + worst)
    pz = np.zeros((T, E))
    pz[keep] = np.exp(-x) / np.exp(-x).sum(1, keepdims=True) * z[keep][:, None]
    assert np.all(np.abs(d - want) <= ((3 * P + 16 + k) * size + pz) * U + 1e-37)
    assert not d[~keep].any()


SHAPES = [(1, 1, 1), (1, 8, 2), (3, 7, 7), (37, 16, 2), (64, 17, 4), (65, 32, 3), (129, 33, 5), (200, 64, 8), (31, 100, 9),
          (300, 128, 8), (77, 130, 10), (257, 256, 6), (8, 512, 10), (64, 512, 10), (65, 512, 10), (1000, 512, 10),
          (130, 513, 32), (70, 1023, 11), (90, 1024, 32), (1900, 768, 8), (1901, 767, 5), (1800, 1000, 12)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("renorm", [True, False], ids=["renorm", "full"])
def test_against_the_oracle(T, E, k, renorm):
    c = make(T, E, k, seed=T + E, renorm=renorm, mask=(T + E) % 2 == 0, drop=E > 30 and k < 8)
    check(c, Run(c)().out())
    assert H.ctx().check_device_status() == M.OK


# enough rows that up to 256 experts share a warp: 8 and 16 lanes a row, choices fewer and more than that
@pytest.mark.parametrize("T,E,k", [(3600, 65, 32), (4001, 100, 3), (5000, 128, 8), (3700, 130, 20), (4100, 255, 2),
                                   (3999, 256, 9)])
@pytest.mark.parametrize("renorm", [True, False], ids=["renorm", "full"])
def test_many_tokens_of_few_experts(T, E, k, renorm):
    c = make(T, E, k, seed=T, renorm=renorm, mask=T % 2 == 0, drop=k < 4)
    c["idx"][5:400:7, 1] = c["idx"][5:400:7, 0]  # named twice
    c["l"][11] = -1e30
    c["d_loss"][1] = 0
    stats, counts, prob, d = Run(c)().out()
    counted = c["mask"] is None or c["mask"][11] != 0
    assert np.isinf(stats[1]) == counted
    if counted:
        stats = stats.astype(np.float64)
        stats[1] = O.balance(c["l"], c["idx"], c["mask"])[0][1]
    check(c, (stats, counts, prob, d))
    assert H.ctx().check_device_status() == M.OK


@pytest.mark.parametrize("T,E", [(37, 16), (1500, 60), (700, 512)])
def test_losses_alone(T, E):
    c = make(T, E, 2, seed=5, mask=True)
    r = Run(c, d_gate=False)
    r.gate = None
    check(c, r().out(), d_gate=False)


@pytest.mark.parametrize("T,E", [(40, 16), (900, 512)])
def test_no_token_counts(T, E):
    c = make(T, E, 2, seed=6, mask=True)
    c["mask"][:] = 0
    c["l"][:] = np.nan  # what a masked row holds is not looked at
    check(c, Run(c)().out())
    c = make(T, E, 2, seed=6)
    c["l"][:] = -np.inf
    check(c, Run(c)().out())


@pytest.mark.parametrize("T,E", [(40, 16), (900, 512)])
def test_masked_rows_with_nan_infinities_and_bad_choices(T, E):
    c = make(T, E, 2, seed=7)
    c["mask"] = np.ones(T, np.uint8)
    for i, bad in enumerate((np.nan, np.inf, -np.inf)):
        c["mask"][i] = 0
        c["l"][i] = bad
        c["gate"][i] = np.nan
        c["idx"][i] = -5 - i
    c["mask"][9] = 200  # any byte but 0 counts
    check(c, Run(c)().out())
    assert H.ctx().check_device_status() == M.OK


def test_masks_of_the_lowest_value_and_wide_logits():
    c = make(50, 64, 4, seed=8, scale=30.0)
    c["l"][:, 5:9] = np.finfo(np.float32).min
    c["idx"] = np.argsort(-c["l"], axis=1, kind="stable")[:, :4].astype(np.int32)
    check(c, Run(c)().out())
    # every logit the lowest value: an even row whose lse^2 is past fp32; without a z loss the gradient stays finite
    c = make(3, 8, 2, seed=9)
    c["l"][1] = np.finfo(np.float32).min
    c["d_loss"][1] = 0
    stats, _, prob, d = Run(c)().out()
    assert np.isinf(stats[1]) and np.isfinite(stats[0]) and np.isfinite(d).all()


@pytest.mark.parametrize("T,E,k", [(40, 16, 2), (900, 16, 2), (64, 61, 3), (300, 256, 4), (900, 512, 10), (50, 1024, 32)])
@pytest.mark.parametrize("renorm", [True, False], ids=["renorm", "full"])
def test_rows_far_from_zero(T, E, k, renorm):
    """A row's maximum times log2(e) has a rounding that leaves fp32's exponents from about 1e10 on; the sums must
    not depend on it. Whole rows at such values (a mask added to every logit), and single logits far above the rest."""
    c = make(T, E, k, seed=12, renorm=renorm)
    l = c["l"]
    for i, far in enumerate((3e4, -7e4, 2e6, 1e10, -1e10, 2e10, 4e12, -1e18)):
        l[i] += np.float32(far)
    l[8, 3], l[9, 5], l[10, 1], l[11, 2] = 1e9, 2e10, 1e15, 7e17
    l[12, :5], l[12, 5:] = 1e12, -1e12
    check(c, Run(c)().out())
    # the z loss of these is past fp32; everything else is not
    l[13], l[14], l[15, 1] = -1e30, 1e30, 1e30
    l[16, :5], l[16, 5:] = 3e38, -3e38
    l[17, :] = np.finfo(np.float32).max
    c["d_loss"][1] = 0
    stats, counts, prob, d = Run(c)().out()
    assert np.isinf(stats[1])
    stats = stats.astype(np.float64)
    stats[1] = O.balance(l, c["idx"], c["mask"])[0][1]
    check(c, (stats, counts, prob, d))


def test_nan_logits_show():
    c = make(30, 16, 2, seed=10)
    c["l"][4, 3] = np.nan
    stats, counts, prob, d = Run(c)().out()
    assert np.isnan(stats[:2]).all() and np.isnan(prob).all() and np.isnan(d[4]).all()
    assert counts.sum() == 60 and stats[2] == 30


@pytest.mark.parametrize("E", [16, 512])
def test_bad_choice_is_reported_and_counts_nowhere(E):
    c = make(20, E, 2, seed=11)
    c["idx"][3, 1] = E
    c["idx"][8, 0] = -1
    check(c, Run(c)().out())
    assert H.ctx().check_device_status() == M.EDEVICE
    assert H.ctx().last_device_error_detail() in (7, 16)


@pytest.mark.parametrize("T,E,k", [(40, 16, 2), (40, 16, 11), (300, 61, 20), (3900, 100, 20), (3700, 256, 17), (90, 512, 10),
                                   (60, 1024, 32)])
@pytest.mark.parametrize("renorm", [True, False], ids=["renorm", "full"])
def test_a_bad_choice_takes_no_part_in_the_gradient(T, E, k, renorm):
    """Its gate and d_gate are not looked at, and the row's other choices and experts go on without it."""
    c = make(T, E, k, seed=16, renorm=renorm)
    rng = np.random.default_rng(17)
    for bad, g, dg in ((E, 0.5, 1.0), (-1, np.nan, 1.0), (2 ** 31 - 1, 0.25, np.inf), (-2 ** 31, np.inf, np.nan)):
        for t in rng.integers(0, T, size=9):
            j = int(rng.integers(0, k))
            c["idx"][t, j], c["gate"][t, j], c["d_gate"][t, j] = bad, g, dg
    c["idx"][3], c["gate"][3], c["d_gate"][3] = -1, np.nan, np.nan  # a row without a choice
    check(c, Run(c)().out())
    assert H.ctx().check_device_status() == M.EDEVICE


@pytest.mark.parametrize("E,k", [(16, 4), (512, 10)])
def test_an_expert_named_twice_takes_both_parts(E, k):
    c = make(33, E, k, seed=12)
    c["idx"][:, 1] = c["idx"][:, 0]
    c["idx"][5:, k - 1] = c["idx"][5:, 0]
    check(c, Run(c)().out())


@pytest.mark.parametrize("shift", [1, 2, 3])
def test_unaligned_arrays(shift):
    c = make(70, 512, 3, seed=13)
    big = torch.zeros(70 * 512 + 8, device="cuda")
    l = big[shift:shift + 70 * 512].view(70, 512)
    l.copy_(dev(c["l"]))
    out = torch.full((70 * 512 + 8,), 7.0, device="cuda")
    r = Run(c, logits=l, d_logits=out[shift:shift + 70 * 512].view(70, 512))
    check(c, r().out())
    assert (out[:shift] == 7).all() and (out[shift + 70 * 512:] == 7).all()


def test_no_tokens():
    c = make(1, 16, 2, seed=14)
    r = Run(c)
    r.T = 0
    stats, counts, prob, d = r().out()
    assert not stats.any() and not counts.any() and not prob.any() and (d == 7).all()


@pytest.mark.parametrize("E,k", [(16, 2), (13, 3), (512, 10), (1024, 32)])
@pytest.mark.parametrize("mask", [False, True])
def test_empty_tensors(E, k, mask):
    """A batch without tokens: tensors of no elements have the null address."""
    c = make(0, E, k, seed=E, mask=mask)
    r = Run(c)
    assert r.T == 0 and r.l.data_ptr() == 0 and r.idx.data_ptr() == 0
    assert not any(a.any() for a in r().out())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            r(stream=s)
        for t in (r.stats, r.counts, r.prob):
            t.fill_(7)
        g.replay()
        s.synchronize()
    assert not any(a.any() for a in r.out())
    assert H.ctx().check_device_status() == M.OK


def test_long_batch_equal_bits_and_captured_replays():
    c = make(9001, 512, 10, seed=15, mask=True)
    r = Run(c)
    a = [x.copy() for x in r().out()]
    check(c, a)
    r.ws.fill_(0x3C)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            r(stream=s)
        for _ in range(3):
            r.stats.zero_(), r.counts.zero_(), r.prob.zero_(), r.d.zero_()
            g.replay()
            assert all(np.array_equal(x, y) for x, y in zip(a, r.out()))


def test_two_streams_with_their_own_workspaces():
    cs = [make(2000 + i, 512, 10, seed=20 + i) for i in range(2)]
    runs = [Run(c) for c in cs]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(5):
        for r, s in zip(runs, streams):
            with torch.cuda.stream(s):
                r(stream=s)
    for c, r in zip(cs, runs):
        check(c, r.out())


@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(renorm):
    """The kernel's gradient against central differences of the oracle's scalar in fp64 (step 1e-4: the
    differences' own error is about 1e-8 of the third derivative and 1e-16 / 1e-4 of the value)."""
    c = make(6, 24, 3, seed=30, renorm=renorm, mask=True)
    d = Run(c)().out()[3]
    h = 1e-4
    l0 = c["l"].astype(np.float64)
    for t in range(6):
        for e in range(24):
            lp, lm = l0.copy(), l0.copy()
            lp[t, e] += h
            lm[t, e] -= h
            f = [O.balance_total(l, c["idx"], c["mask"], c["d_loss"], c["d_gate"], renorm) for l in (lp, lm)]
            assert abs((f[0] - f[1]) / (2 * h) - d[t, e]) <= 1e-6


def test_after_the_router():
    """Router, top-k, losses and gradient as a training step runs them, on one stream without a wait between."""
    cfg = M.FULL
    T = 300
    L = H.Layer(M.TINY.replace(E=16), 1)  # builds the context
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.normal(size=(T, cfg.d)).astype(np.float32)).cuda().to(torch.bfloat16)
    wr = torch.from_numpy((rng.normal(size=(cfg.E, cfg.d)) * cfg.d ** -0.5).astype(np.float32)).cuda()
    logits = torch.empty(T, cfg.E, device="cuda")
    idx = torch.empty(T, cfg.k, dtype=torch.int32, device="cuda")
    gate = torch.empty(T, cfg.k, device="cuda")
    c = make(T, cfg.E, cfg.k, seed=31)
    r = Run(c, logits=logits)
    r.idx, r.gate = idx, gate
    H.ctx().router_topk(cfg, x, wr, None, T, logits, idx, gate)
    r()
    got = r.out()
    c.update(l=logits.cpu().numpy(), idx=idx.cpu().numpy(), gate=gate.cpu().numpy())
    check(c, got)
    assert L.T == 1
