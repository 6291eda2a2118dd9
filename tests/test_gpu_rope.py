"""Norms of queries and keys for each head with the rotary position (qk_norm_rope)
and their gradient, against the definition in 64 bits.

Tolerances, from the roundings: outputs are computed in fp32 (a few dozen
roundings of 2^-24 each, on values of at most |y_a| + |y_b|) and rounded once to
bf16 (2^-8 relative).  A pair's rotation can cancel, so the fp32 part is counted
on the pair's length: |err| <= 2^-8 |ref| + 2^-18 (pair length, or |ref|).  The
gradient's fp32 part is counted on r (|w g|_max + |h|_max |w g|_max |h|_max), the
size of the terms that cancel.  The angle's error, 2^-24 half turns of pi plus the
sine's 2 ulp, is inside the 2^-18.
"""
import math

import pytest
import torch

from sliding_window_gqa_tfa_b200 import binding as tb

pytestmark = pytest.mark.gpu


def _rotate(x, ang, rot, inter, m, back=False):
    """x [B,L,H,D] fp64, ang [B,L,1,rot/2]; (rotated, each channel's pair length)."""
    c, s = ang.cos() * m, ang.sin() * m * (-1 if back else 1)
    y, size = x.clone(), x.abs()
    if rot:
        ia = torch.arange(0, rot, 2, device=x.device) if inter else torch.arange(rot // 2, device=x.device)
        ib = ia + (1 if inter else rot // 2)
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        ln = (a.abs() + b.abs()) * abs(m)
        size[..., ia], size[..., ib] = ln, ln
    return y, size


def _reference(x, w, pos, f, rot, inter, m, eps):
    x = x.double()
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    return _rotate(x, pos.double()[:, :, None, None] * f, rot, inter, m)


def _make(B, L, Hq, Hkv, D, rot, seed, start=0, base=1e4):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(B, L, Hq + 2 * Hkv, D, generator=g, device="cuda").bfloat16()
    w = (1 + 0.2 * torch.randn(2, D, generator=g, device="cuda")).bfloat16()
    f, _ = tb.rope_inv_freq(rot, base)
    pos = start + torch.randint(0, 50, (B,), generator=g, device="cuda", dtype=torch.int32)
    return qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], w[0], w[1], f, pos


CASES = [
    # B, L, Hq, Hkv, D, rot, norm, interleaved, start
    (1, 1, 1, 1, 128, 128, True, False, 0),
    (16, 1, 16, 8, 128, 128, True, False, 8191),
    (2, 37, 7, 1, 128, 64, True, True, 5),
    (3, 5, 56, 8, 128, 128, False, True, 1_000_000),
    (1, 700, 16, 8, 128, 96, True, False, 12),
    (2, 300, 3, 3, 64, 64, True, False, 100_000),
    (1, 9, 33, 31, 64, 16, False, False, 0),
    (1, 601, 12, 4, 64, 32, True, True, 2_000_000_000),
    (2, 3, 4, 2, 128, 0, True, False, 0),
    (40, 50, 1, 1, 64, 64, True, False, 3),  # many tokens and sequences in a round
    (1000, 1, 3, 1, 128, 32, True, True, 77),
    (7, 131, 20, 5, 128, 112, True, False, 9),
]
IDS = ["-".join(map(str, c)) for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    B, L, Hq, Hkv, D, rot, norm, inter, start = case
    q, k, wq, wk, f, pos = _make(B, L, Hq, Hkv, D, rot, 1, start)
    if not norm:
        wq = wk = None
    qo, ko = tb.qk_norm_rope(q, k, pos, f, q_weight=wq, k_weight=wk, eps=1e-6, interleaved=inter, mscale=1.25)
    rows = pos[:, None] + torch.arange(L, device="cuda")
    for x, w, got in ((q, wq, qo), (k, wk, ko)):
        ref, size = _reference(x, w, rows, f, rot, inter, 1.25, 1e-6)
        err = (got.transpose(1, 2).double() - ref).abs()
        assert (err <= 2 ** -8 * ref.abs() + 2 ** -18 * size).all()


def _reference_backward(dy, x, w, pos, f, rot, inter, m, eps):
    g, size = _rotate(dy.transpose(1, 2).double(), pos.double()[:, :, None, None] * f, rot, inter, m, back=True)
    if w is None:
        return g, size, None, None
    x, w = x.double(), w.double()
    r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    h = x * r
    dw, dw_size = (g * h).sum((0, 1, 2)), (size * h.abs()).sum((0, 1, 2))
    u = g * w
    dx = r * (u - h * (u * h).mean(-1, keepdim=True))
    us = (size * w.abs()).amax(-1, keepdim=True)
    return dx, r * us * (1 + h.abs().amax(-1, keepdim=True) ** 2), dw, dw_size


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case):
    B, L, Hq, Hkv, D, rot, norm, inter, start = case
    q, k, wq, wk, f, pos = _make(B, L, Hq, Hkv, D, rot, 2, start)
    if not norm:
        wq = wk = None
    gen = torch.Generator(device="cuda").manual_seed(3)
    dqo = torch.randn(B, Hq, L, D, generator=gen, device="cuda").bfloat16()
    dko = torch.randn(B, Hkv, L, D, generator=gen, device="cuda").bfloat16()
    dq, dk, dwq, dwk = tb.qk_norm_rope_backward(dqo, dko, q, k, pos, f, q_weight=wq, k_weight=wk, eps=1e-6,
                                                interleaved=inter, mscale=0.75)
    rows = pos[:, None] + torch.arange(L, device="cuda")
    for dy, x, w, got, dw in ((dqo, q, wq, dq, dwq), (dko, k, wk, dk, dwk)):
        ref, size, rdw, dw_size = _reference_backward(dy, x, w, rows, f, rot, inter, 0.75, 1e-6)
        assert ((got.double() - ref).abs() <= 2 ** -8 * ref.abs() + 2 ** -18 * size).all()
        if w is None:
            assert dw is None
        else:
            assert ((dw.double() - rdw).abs() <= 2 ** -18 * dw_size).all()


def test_gradient_against_differences():
    """The gradient's inner product with a direction, against the definition's own
    central differences in 64 bits along it: |step^2 terms| ~ 1e-8 of the sum's
    size, so only the gradient's bf16 roundings (2^-8 of each product) are counted."""
    B, L, Hq, Hkv, D, rot = 2, 11, 6, 2, 128, 64
    q, k, wq, wk, f, pos = _make(B, L, Hq, Hkv, D, rot, 4)
    gen = torch.Generator(device="cuda").manual_seed(5)
    dqo = torch.randn(B, Hq, L, D, generator=gen, device="cuda").bfloat16()
    dko = torch.randn(B, Hkv, L, D, generator=gen, device="cuda").bfloat16()
    dq, dk, dwq, dwk = tb.qk_norm_rope_backward(dqo, dko, q, k, pos, f, q_weight=wq, k_weight=wk, interleaved=True)
    rows = pos[:, None] + torch.arange(L, device="cuda")
    for dy, x, w, dx, dw in ((dqo, q, wq, dq, dwq), (dko, k, wk, dk, dwk)):
        vx = torch.randn(x.shape, generator=gen, device="cuda", dtype=torch.float64)
        vw = torch.randn(w.shape, generator=gen, device="cuda", dtype=torch.float64)

        def loss(t):
            y, _ = _reference(x.double() + t * vx, w.double() + t * vw, rows, f, rot, True, 1.0, 1e-6)
            return (y.transpose(1, 2) * dy.double()).sum()

        t = 1e-4
        want = (loss(t) - loss(-t)) / (2 * t)
        got = (dx.double() * vx).sum() + (dw.double() * vw).sum()
        bound = 2 ** -8 * (dx.double() * vx).abs().sum() + 1e-6 * (dw.double() * vw).abs().sum()
        assert (got - want).abs() <= bound + 1e-5 * want.abs()


def test_positions_per_row_and_as_int():
    q, k, wq, wk, f, _ = _make(2, 6, 4, 2, 128, 128, 6)
    pos = torch.tensor([[0, 5, 3, 70000, -4, 9], [1, 1, 1, 2, 2, 2]], dtype=torch.int32, device="cuda")
    qo, ko = tb.qk_norm_rope(q, k, pos, f, q_weight=wq, k_weight=wk)
    for x, w, got in ((q, wq, qo), (k, wk, ko)):
        ref, size = _reference(x, w, pos, f, 128, False, 1.0, 1e-6)
        assert ((got.transpose(1, 2).double() - ref).abs() <= 2 ** -8 * ref.abs() + 2 ** -18 * size).all()
    a = tb.qk_norm_rope(q, k, 17, f)
    b = tb.qk_norm_rope(q, k, torch.full((2,), 17, dtype=torch.int32, device="cuda"), f)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_writes_a_caches_rows_and_in_place():
    """k_out as rows [P, P + L) of a cache: those rows and no others; the pass over
    its own inputs gives the same numbers."""
    q, k, wq, wk, f, pos = _make(2, 5, 4, 2, 128, 64, 7)
    qo, ko = tb.qk_norm_rope(q, k, pos, f, q_weight=wq, k_weight=wk)
    cache = torch.full((2, 2, 20, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    tb.qk_norm_rope(q, k, pos, f, q_weight=wq, k_weight=wk, k_out=cache[:, :, 8:13])
    assert torch.equal(cache[:, :, 8:13], ko)
    assert (cache[:, :, :8] == 7).all() and (cache[:, :, 13:] == 7).all()
    q2, k2 = q.clone(), k.clone()
    tb.qk_norm_rope(q2, k2, pos, f, q_weight=wq, k_weight=wk, q_out=q2.transpose(1, 2), k_out=k2.transpose(1, 2))
    assert torch.equal(q2.transpose(1, 2), qo) and torch.equal(k2.transpose(1, 2), ko)


def test_rotation_and_its_gradient_undo_each_other_and_repeat():
    """Rotating the gradient back is the transposed rotation, its inverse for
    mscale 1 (two bf16 roundings, each on the pair's length); two passes agree bit for bit."""
    q, k, wq, wk, f, pos = _make(2, 40, 8, 4, 128, 128, 8)
    qo, ko = tb.qk_norm_rope(q, k, pos, f, interleaved=True)
    dq, dk, _, _ = tb.qk_norm_rope_backward(qo, ko, q, k, pos, f, interleaved=True)
    _, size = _rotate(q.double(), torch.zeros(2, 40, 1, 64, dtype=torch.float64, device="cuda"), 128, True, 1.0)
    assert ((dq.double() - q.double()).abs() <= 2 ** -6.9 * size).all()
    a = tb.qk_norm_rope_backward(qo, ko, q, k, pos, f, q_weight=wq, k_weight=wk)
    b = tb.qk_norm_rope_backward(qo, ko, q, k, pos, f, q_weight=wq, k_weight=wk)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_other_stream_and_graph():
    q, k, wq, wk, f, pos = _make(1, 64, 8, 4, 128, 128, 9)
    want = tb.qk_norm_rope(q, k, pos, f, q_weight=wq, k_weight=wk)
    wantb = tb.qk_norm_rope_backward(*want, q, k, pos, f, q_weight=wq, k_weight=wk)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = tb.qk_norm_rope(q, k, pos, f, q_weight=wq, k_weight=wk, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fwd = tb.qk_norm_rope(q, k, pos, f, q_weight=wq, k_weight=wk)
        bwd = tb.qk_norm_rope_backward(*fwd, q, k, pos, f, q_weight=wq, k_weight=wk)
    for _ in range(2):
        for t in (*fwd, *bwd):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(fwd[0], want[0]) and all(torch.equal(x, y) for x, y in zip(bwd, wantb))


def test_scaled_frequencies():
    f, m = tb.rope_inv_freq(128, 1e6)
    assert m == 1.0 and f.shape == (64,) and abs(f[1].item() - 1e6 ** (-2 / 128)) < 1e-15
    g, m = tb.rope_inv_freq(128, 1e6, scaling="yarn", factor=4.0, original=8192)
    assert m == pytest.approx(0.1 * math.log(4) + 1)
    assert g[0] == f[0] and torch.allclose(g[-1], f[-1] / 4, rtol=1e-14, atol=0)
    assert ((g <= f) & (g >= f / 4 - 1e-20)).all()
    g, m = tb.rope_inv_freq(128, 1e6, scaling="linear", factor=8.0)
    assert m == 1.0 and torch.allclose(g, f / 8, rtol=1e-14, atol=0)


@pytest.mark.parametrize("as_int", [True, False])
def test_positions_past_31_bits(as_int):
    """Rows behind a first position near 2^31: the angle goes on, it does not wrap."""
    start = 2 ** 31 - 3
    q, k, wq, wk, f, _ = _make(2, 9, 4, 2, 128, 128, 10)
    first = start if as_int else torch.full((2,), start, dtype=torch.int32, device="cuda")
    rows = start + torch.arange(9, device="cuda").expand(2, 9)
    qo, ko = tb.qk_norm_rope(q, k, first, f, q_weight=wq, k_weight=wk)
    for x, w, got in ((q, wq, qo), (k, wk, ko)):
        ref, size = _reference(x, w, rows, f, 128, False, 1.0, 1e-6)
        assert ((got.transpose(1, 2).double() - ref).abs() <= 2 ** -8 * ref.abs() + 2 ** -18 * size).all()
    back = tb.qk_norm_rope_backward(qo, ko, q, k, first, f, q_weight=wq, k_weight=wk)
    for dy, x, w, got in ((qo, q, wq, back[0]), (ko, k, wk, back[1])):
        ref, size, _, _ = _reference_backward(dy, x, w, rows, f, 128, False, 1.0, 1e-6)
        assert ((got.double() - ref).abs() <= 2 ** -8 * ref.abs() + 2 ** -18 * size).all()
