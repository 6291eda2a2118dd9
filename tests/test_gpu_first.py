"""Attention with a sliding window and first tokens that stay visible
(prefill, prefill_lse and backward with first > 0), against the definition in 64 bits.

Tolerances, from the roundings (bf16 2^-8): the output's P is rounded once and the
output once, |err| <= 2^-8 (sum_j w_j |v_j| + |o|); every gradient element is a sum
of products with one rounded factor (P in dV, dS in dQ and dK), rounded once, and dS
carries the rounding of the saved output through delta = sum_d dO O:
|err| <= 2^-8 (A + |ref| + E), A the sum of its terms' absolute values, E the terms
with sum_d |dO O| in the place of dP - delta.  The fp32 sums (at most 2^-16 of the
absolute sums) are counted as 2^-14 of A and E, and of the output's terms.
"""
import math

import pytest
import torch

from sliding_window_gqa_tfa_b200 import binding as tb

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -8 + 2.0 ** -14


def _make(B, Hq, Hkv, L, S, D, seed, sharp=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(B, h, n, D, generator=g, device="cuda").mul(m).bfloat16()
            for h, n, m in ((Hq, L, 1), (Hkv, S, sharp), (Hkv, S, 1), (Hq, L, 1))]


def visible(L, S, W, F, key_mask=None):
    p = S - L + torch.arange(L, device="cuda")[:, None]
    j = torch.arange(S, device="cuda")
    see = (j <= p) & ((j > p - W) | (j < F))
    return see if key_mask is None else see & (key_mask > 0.5)


def reference(q, k, v, W, F, key_mask=None, softcap=0.0, sinks=None, do=None):
    """Outputs and bounds: (o, bound, lse) or, with do, ((dq, dk, dv), bounds)."""
    B, Hq, L, D = q.shape
    Hkv, S = k.shape[1], k.shape[2]
    c = D ** -0.5
    o, bo = torch.zeros(2, *q.shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(q.shape[:3], dtype=torch.float64, device="cuda")
    grads = [torch.zeros(2, *t.shape, dtype=torch.float64, device="cuda") for t in (q, k, v)]
    for b in range(B):
        see = visible(L, S, W, F, None if key_mask is None else key_mask[b])
        for h in range(Hq):
            g = h // (Hq // Hkv)
            x, y, z = q[b, h].double(), k[b, g].double(), v[b, g].double()
            t = x @ y.T * c
            if softcap > 0:
                t = softcap * torch.tanh(t / softcap)
            t = t.masked_fill(~see, -math.inf)
            m = t.amax(1, keepdim=True).clamp(min=-1e30)
            w = torch.exp(t - m)
            den = w.sum(1, keepdim=True)
            if sinks is not None:
                den = den + torch.where(see.any(1, keepdim=True), torch.exp(sinks[h].double() - m), 0.0)
            lse[b, h] = torch.where(den > 0, (m + den.log()) / math.log(2), torch.full_like(m, math.inf))[:, 0]
            w = torch.where(den > 0, w / den, torch.zeros_like(w))
            o[b, h] = w @ z
            bo[b, h] = EPS * (w @ z.abs() + o[b, h].abs())
            if do is not None:
                e = do[b, h].double()
                dp = e @ z.T
                ds = w * (dp - (w * dp).sum(1, keepdim=True))
                size = (e * o[b, h]).abs().sum(1, keepdim=True)
                a = ds.abs() + w * size
                (dq, aq), (dk, ak), (dv, av) = grads
                dq[b, h] = c * ds @ y
                aq[b, h] = c * a @ y.abs()
                dk[b, g] += c * ds.T @ x
                ak[b, g] += c * a.T @ x.abs()
                dv[b, g] += w.T @ e
                av[b, g] += w.T @ e.abs()
    if do is None:
        return o, bo, lse
    return tuple(x[0] for x in grads), tuple(EPS * (x[1] + x[0].abs()) + 1e-6 for x in grads)


CASES = [
    # name, B, Hq, Hkv, L, S, D, W, F
    ("one", 1, 1, 1, 1, 1, 128, 1, 1),
    ("decode", 2, 14, 2, 1, 3000, 128, 100, 4),
    ("decode_l8", 1, 8, 2, 8, 1000, 64, 64, 130),
    ("rows37", 2, 8, 2, 37, 1029, 128, 256, 64),
    ("no_prefix", 1, 4, 4, 300, 300, 128, 17, 3),
    ("tile_pairs", 1, 3, 1, 700, 2000, 128, 300, 4),
    ("head_pairs", 1, 4, 2, 700, 2000, 128, 300, 4),
    ("first_two_tiles", 1, 4, 2, 300, 1500, 128, 129, 200),
    ("first_meets_window", 1, 4, 2, 200, 700, 64, 128, 400),
    ("first_past_all", 1, 2, 1, 150, 400, 128, 33, 10 ** 6),
    ("window1", 1, 2, 2, 200, 500, 128, 1, 1),
    ("window_past_all", 1, 2, 1, 100, 300, 64, 2 ** 30, 5),
    ("first128_window128", 1, 4, 1, 256, 1024, 128, 128, 128),
    ("cut_ranges", 1, 1, 1, 260, 20000, 128, 9000, 70),
    ("cut_items", 1, 80, 20, 256, 9000, 64, 8000, 70),
    ("many_items", 3, 16, 4, 513, 900, 64, 200, 9),
    ("cut_key_tiles", 2, 4, 2, 1500, 1500, 128, 100, 4),
    ("two_cut_tiles_prefix", 1, 3, 1, 1200, 4000, 64, 128, 200),
    ("uncut_tiles", 1, 2, 1, 900, 900, 128, 100, 600),
    ("window_int_max", 1, 4, 2, 300, 700, 128, 2 ** 31 - 1, 2 ** 31 - 1),
    ("few_key_tiles_g7", 1, 7, 1, 1236, 1692, 128, 727, 85),
    ("few_key_tiles_b2", 2, 4, 1, 700, 700, 64, 300, 3),
    ("few_key_tiles_first_past_all", 1, 6, 2, 520, 600, 128, 200, 600),
    ("most_parts", 1, 1, 1, 9000, 9000, 64, 1, 1),
]
IDS = [c[0] for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("masked", [False, True])
def test_forward(case, masked):
    _, B, Hq, Hkv, L, S, D, W, F = case
    q, k, v, _ = _make(B, Hq, Hkv, L, S, D, 1, 2.0)
    km = None
    if masked:
        km = (torch.rand(B, S, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda") < 0.6).float()
        km[0, :F] = 0  # rows that see nothing where the window is hidden too
        km[0, -W - 3:] = 0
    got = tb.prefill(q, k, v, window=W, first=F, key_mask=km)
    o2, lse = tb.prefill_lse(q, k, v, window=W, first=F, key_mask=km)
    tb.check_status()
    ref, bound, rlse = reference(q, k, v, W, F, km)
    assert ((got.double() - ref).abs() <= bound).all()
    assert torch.equal(got, o2)
    assert torch.equal(lse.isinf(), rlse.isinf())
    fin = rlse.isfinite()
    assert ((lse.double() - rlse)[fin].abs() <= 2 ** -14 * (1 + rlse[fin].abs())).all()


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("masked", [False, True])
def test_backward(case, masked):
    _, B, Hq, Hkv, L, S, D, W, F = case
    q, k, v, do = _make(B, Hq, Hkv, L, S, D, 3)
    km = None
    if masked:
        km = (torch.rand(B, S, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda") < 0.6).float()
        km[0, :F] = 0
    saved = tb.prefill_lse(q, k, v, window=W, first=F, key_mask=km)
    got = tb.backward(q, k, v, do, window=W, first=F, key_mask=km, saved=saved)
    tb.check_status()
    ref, bound = reference(q, k, v, W, F, km, do=do)
    for name, a, r, lim in zip(("dq", "dk", "dv"), got, ref, bound):
        assert a.isfinite().all(), name
        assert ((a.double() - r).abs() <= lim).all(), name
    again = tb.backward(q, k, v, do, window=W, first=F, key_mask=km, saved=saved)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_gradient_against_differences():
    """Along a random direction, against central differences of the definition in
    64 bits; only the bf16 roundings of the gradients and of what enters them count."""
    B, Hq, Hkv, L, S, D, W, F = 1, 4, 2, 140, 400, 128, 100, 5
    q, k, v, do = _make(B, Hq, Hkv, L, S, D, 5)
    got = tb.backward(q, k, v, do, window=W, first=F, saved=tb.prefill_lse(q, k, v, window=W, first=F))
    _, bound = reference(q, k, v, W, F, do=do)
    gen = torch.Generator(device="cuda").manual_seed(6)
    for i, x in enumerate((q, k, v)):
        d = torch.randn(x.shape, generator=gen, device="cuda", dtype=torch.float64)

        def loss(t):
            a = [q.double(), k.double(), v.double()]
            a[i] = a[i] + t * d
            return (reference(*a, W, F)[0] * do.double()).sum()

        want = (loss(1e-4) - loss(-1e-4)) / 2e-4
        lim = (bound[i] * d.abs()).sum()
        assert ((got[i].double() * d).sum() - want).abs() <= lim + 1e-5 * want.abs()


@pytest.mark.parametrize("L", [5, 100, 300])
def test_score_variants(L):
    q, k, v, _ = _make(2, 8, 2, L, 900, 128, 7, 4.0)
    sinks = 2 * torch.randn(8, generator=torch.Generator(device="cuda").manual_seed(8), device="cuda")
    for softcap, s in ((30.0, None), (0.0, sinks), (20.0, sinks)):
        got = tb.prefill(q, k, v, window=200, first=4, softcap=softcap, sinks=s)
        ref, bound, _ = reference(q, k, v, 200, 4, softcap=softcap, sinks=s)
        # the softcap's approximate exponential and reciprocal: 2^-20 of the cap, twice in the weights
        assert ((got.double() - ref).abs() <= bound + 2 ** -18 * max(softcap, 1) * v.abs().max().double()).all()


def test_first_zero_is_the_window_and_all_first_is_causal():
    q, k, v, do = _make(1, 8, 2, 200, 600, 128, 9)
    assert torch.equal(tb.prefill(q, k, v, window=100, first=0), tb.prefill(q, k, v, window=100))
    a, b = tb.prefill(q, k, v, window=100, first=600), tb.prefill(q, k, v)
    ref, bound, _ = reference(q, k, v, 600, 0)
    assert ((a.double() - ref).abs() <= bound).all() and ((b.double() - ref).abs() <= bound).all()


def test_keys_that_no_row_sees_are_not_read_into_the_result():
    """NaN and infinities in the tiles between the first tokens and the window."""
    q, k, v, do = _make(1, 4, 2, 200, 2000, 128, 10)
    W, F = 256, 4
    want = tb.prefill(q, k, v, window=W, first=F)
    saved = tb.prefill_lse(q, k, v, window=W, first=F)
    grads = tb.backward(q, k, v, do, window=W, first=F, saved=saved)
    lo = (2000 - 200 - W + 1) // 128 * 128  # the window's first tile
    for bad in (float("nan"), float("inf")):
        k2, v2 = k.clone(), v.clone()
        k2[:, :, 128:lo], v2[:, :, 128:lo] = bad, bad
        assert torch.equal(tb.prefill(q, k2, v2, window=W, first=F), want)
        g2 = tb.backward(q, k2, v2, do, window=W, first=F, saved=saved)
        assert torch.equal(g2[0], grads[0])
        assert (grads[1][:, :, 128:lo] == 0).all() and (grads[2][:, :, 128:lo] == 0).all()


def test_captured_training_step():
    q, k, v, do = _make(1, 8, 2, 300, 700, 128, 11)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o, lse = tb.prefill_lse(q, k, v, window=200, first=4)
        want = tb.backward(q, k, v, do, window=200, first=4, saved=(o, lse))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        o2, lse2 = tb.prefill_lse(q, k, v, window=200, first=4)
        got = tb.backward(q, k, v, do, window=200, first=4, saved=(o2, lse2))
    for _ in range(2):
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("L2,S2,W2", [(300, 700, 200), (900, 1300, 200)])  # as many rows, more rows
def test_a_captured_step_outlives_a_larger_workspace(L2, S2, W2):
    """A training step captured on a stream, then steps on the same stream that need
    more workspace: the graph's replay writes neither into freed memory (which the
    canaries take) nor anything else than before."""
    q, k, v, do = _make(1, 8, 2, 300, 4000, 128, 12)
    others = _make(1, 8, 2, L2, S2, 128, 13)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step(x, W):
        saved = tb.prefill_lse(*x[:3], window=W, first=4)
        return tb.backward(*x, window=W, first=4, saved=saved)

    with torch.cuda.stream(s):
        want = step((q, k, v, do), 40)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = step((q, k, v, do), 40)
    with torch.cuda.stream(s):
        want2 = step(others, W2)
    torch.cuda.synchronize()
    canaries = [torch.full((1 << n,), 7, dtype=torch.uint8, device="cuda") for n in range(12, 28) for _ in range(4)]
    for _ in range(3):
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all((c == 7).all() for c in canaries)
    with torch.cuda.stream(s):
        again = step(others, W2)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, want2))


def test_unseen_keys_reach_neither_gradient_of_keys_and_values():
    """NaN and infinities in K and V between the first tokens and the window: the
    gradients are those of clean inputs, zero where no row looks."""
    for D, G in ((128, 2), (64, 1)):
        q, k, v, do = _make(1, 2 * G, 2, 200, 2000, D, 14)
        W, F = 256, 4
        saved = tb.prefill_lse(q, k, v, window=W, first=F)
        want = tb.backward(q, k, v, do, window=W, first=F, saved=saved)
        lo = (2000 - 200 - W + 1) // 128 * 128
        for bad in (float("nan"), float("inf")):
            k2, v2 = k.clone(), v.clone()
            k2[:, :, 128:lo], v2[:, :, 128:lo] = bad, bad
            got = tb.backward(q, k2, v2, do, window=W, first=F, saved=saved)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            assert (got[1][:, :, 128:lo] == 0).all() and (got[2][:, :, 128:lo] == 0).all()
