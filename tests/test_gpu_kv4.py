"""The 4-bit key/value cache (kv4_append, kv4_read) and attention over it
(kv4_decode), against the definitions in 64 bits.

Tolerances, from the roundings.  Writing is exact: steps, minima and codes are
those of the definition.  Reading rounds c s + m once in fp32 and once to bf16.
Decoding rounds p s to fp16 (less than 2^-8 of each term of sum_j w_j s c_j; the dense
kernel that longer chunks take rounds p and the values to bf16, 2^-8) and the output
to bf16 (2^-8); the sum of a group's q is held in two bf16 (2^-17 of the minimum's
part of the score: inside delta); the scores' fp32 sums are of at most 143 s sum|q| a group, in fewer
than 64 additions of 2^-24 each (2^-18 of that), which moves the weights by twice
the scores' error delta: |err| <= 2^-8 (sum_j w_j s c_j + |o|) + 2 delta sum_j w_j |v_j - o|,
the last sum at most max|v| + |o|.
"""
import math

import pytest
import torch

from sliding_window_gqa_tfa_b200 import binding as tb

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def quantise(x):
    """(codes uint8 [..., D/2], meta bf16 [..., D/32, 2]) of bf16 rows, from the definition."""
    g = x.double().unflatten(-1, (-1, 32))
    mn, mx = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    s = ((mx - mn) / 15).bfloat16()
    c = torch.where(s > 0, torch.round((g - mn) / s.double()), torch.zeros_like(g)).clamp(0, 15)
    c = c.flatten(-2).to(torch.uint8).unflatten(-1, (-1, 2))
    return c[..., 0] + 16 * c[..., 1], torch.cat([s, mn.bfloat16()], -1)


def parts(codes, meta):
    """(s c, m) fp64 of every channel."""
    c = torch.stack([codes % 16, codes // 16], -1).flatten(-2).double().unflatten(-1, (-1, 32))
    m = meta.double()
    return (c * m[..., :1]).flatten(-2), (m[..., 1:] + 0 * c).flatten(-2)


def cache_of(k, v, cap, fill=None):
    """A cache whose first rows hold k and v, the others random bytes and NaN steps."""
    B, H, S, D = k.shape
    out = []
    for i, x in enumerate((k, v)):
        codes = torch.randint(0, 256, (B, H, cap, D // 2), generator=_gen(90 + i), device="cuda", dtype=torch.uint8)
        meta = torch.full((B, H, cap, D // 32, 2), float("nan"), dtype=torch.bfloat16, device="cuda")
        codes[:, :, :S], meta[:, :, :S] = quantise(x)
        out += [codes, meta]
    return out


# ------------------------------------------------------------ append and read
@pytest.mark.parametrize("B,H,L,D,cap,start", [
    (1, 1, 1, 128, 1, [0]), (1, 8, 1, 128, 40, [39]), (3, 2, 37, 64, 100, [0, 63, 11]), (2, 8, 300, 128, 311, [4, 11]),
    (64, 8, 1, 128, 50, [i % 50 for i in range(64)]), (2, 3, 5, 64, 9, [2, -1]), (1, 1, 129, 64, 200, [70]),
])
def test_append_and_read(B, H, L, D, cap, start):
    gen = _gen(1)
    kv = _randn(gen, B, L, 2 * H, D) * torch.exp(2 * _randn(gen, B, L, 2 * H, 1))
    kv[0, 0, 0, :32] = 0.75  # a group without a range
    kv[-1, -1, -1, -32:] = 1e-39  # (rounds to a subnormal)
    kv = kv.bfloat16()
    k, v = kv[:, :, :H].transpose(1, 2), kv[:, :, H:].transpose(1, 2)
    cache = [torch.randint(0, 256, (B, H, cap, D // 2), generator=gen, device="cuda", dtype=torch.uint8),
             _randn(gen, B, H, cap, D // 32, 2).bfloat16()]
    cache += [t.clone() for t in cache]
    want = [t.clone() for t in cache]
    st = torch.tensor(start, dtype=torch.int32, device="cuda")
    tb.kv4_append(k, v, *cache, start=st)
    tb.check_status()
    rows = tb.kv4_read(*cache, start=st, rows=L)
    tb.check_status()
    for i, x in enumerate((k, v)):
        codes, meta = quantise(x)
        for b in range(B):
            if start[b] >= 0:
                want[2 * i][b, :, start[b]:start[b] + L] = codes[b]
                want[2 * i + 1][b, :, start[b]:start[b] + L] = meta[b]
        sc, m = parts(codes, meta)
        ref = sc + m
        for b in range(B):
            if start[b] < 0:
                assert (rows[i][b] == 0).all()
            else:  # 2^-24 of c s + m before the rounding to bf16
                err = (rows[i][b].double() - ref[b]).abs()
                assert (err <= 2 ** -8 * ref[b].abs() + 2 ** -23 * (sc[b].abs() + m[b].abs()) + 1e-40).all()
                # and every value is within half a step (and the step's own rounding) of what went in
                s = meta[b][..., :1].double().expand(-1, -1, -1, 32).flatten(-2)
                assert ((ref[b] - x[b].double()).abs() <= s * (0.5 + 15 * 2 ** -8) + 1e-40).all()
    for got, w in zip(cache, want):  # the rows written, and nothing else
        assert torch.equal(got.view(torch.uint8), w.view(torch.uint8))


def test_append_with_an_int_start_and_contiguous_rows():
    gen = _gen(2)
    k, v = (_randn(gen, 2, 4, 6, 128).bfloat16() for _ in range(2))
    cache = tb.kv4_cache(2, 4, 16, 128)
    tb.kv4_append(k, v, *cache, start=10)
    a, b = tb.kv4_read(*cache, start=10), tb.kv4_read(*cache)
    assert a[0].shape == (2, 4, 6, 128) and b[0].shape == (2, 4, 16, 128)
    assert torch.equal(b[0][:, :, 10:], a[0]) and (b[1][:, :, :10] == 0).all()
    with pytest.raises(tb.TfaError) as e:
        tb.kv4_append(k, v, *cache, start=11)
    assert e.value.code == tb.TFA_ERR_CACHE


def test_rows_past_the_capacity_are_refused_on_the_device():
    gen = _gen(3)
    k, v = (_randn(gen, 2, 2, 4, 64).bfloat16() for _ in range(2))
    cache = tb.kv4_cache(2, 2, 8, 64)
    start = torch.tensor([6, 2 ** 31 - 2], dtype=torch.int32, device="cuda")
    tb.kv4_append(k, v, *cache, start=start)
    with pytest.raises(tb.TfaError) as e:
        tb.check_status()
    assert e.value.code == tb.TFA_ERR_SEQLENS
    codes, meta = quantise(k)
    assert torch.equal(cache[0][0, :, 6:8], codes[0, :, :2]) and (cache[0][0, :, :6] == 0).all()
    assert (cache[0][1] == 0).all()
    r = tb.kv4_read(*cache, start=start, rows=4)
    with pytest.raises(tb.TfaError):
        tb.check_status()
    assert (r[0][0, :, 2:] == 0).all() and (r[0][1] == 0).all()
    tb.check_status()


def test_values_that_are_not_finite_poison_their_group_only():
    k = torch.ones(1, 1, 4, 128, device="cuda")
    k[0, 0, 0, 5], k[0, 0, 1, 40], k[0, 0, 2, 70] = float("nan"), float("inf"), float("-inf")
    k[0, 0, 3, 100], k[0, 0, 3, 101] = 3.3e38, -3.3e38
    k = k.bfloat16()
    cache = tb.kv4_cache(1, 1, 4, 128)
    tb.kv4_append(k, k, *cache, start=0)
    for r in tb.kv4_read(*cache):
        bad = r.isnan().view(4, 4, 32)
        for row in range(4):
            for gr in range(4):
                assert bad[row, gr].all() if row == gr else not bad[row, gr].any()


# ------------------------------------------------------------------ attention
def reference(q, cache, lens, scale, window=0, first=0, softcap=0.0, sinks=None):
    """(o, bound) fp64, sequence by sequence."""
    B, Hq, L, D = q.shape
    Hkv = cache[0].shape[1]
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(o)
    for b in range(B):
        n = int(lens[b])
        if n <= 0:
            continue
        pos = n - L + torch.arange(L, device="cuda")[:, None]
        j = torch.arange(n, device="cuda")
        see = j <= pos
        if window > 0:
            see = see & ((j > pos - window) | (j < first))
        for h in range(Hq):
            g = h // (Hq // Hkv)
            kc, km = parts(cache[0][b, g, :n], cache[1][b, g, :n])
            vc, vm = parts(cache[2][b, g, :n], cache[3][b, g, :n])
            x = q[b, h].double()
            t = x @ (kc + km).T * scale
            steps = cache[1][b, g, :n, :, 0].double()
            delta = abs(scale) * 2 ** -18 * (x.abs().unflatten(-1, (-1, 32)).sum(-1) @ (143 * steps.T))
            delta = torch.where(see, delta, torch.zeros_like(delta)).nan_to_num().amax(1, keepdim=True)
            if softcap > 0:
                t = softcap * torch.tanh(t / softcap)
            t = t.masked_fill(~see, -math.inf)
            m = t.amax(1, keepdim=True).clamp(min=-1e30)
            w = torch.exp(t - m)
            den = w.sum(1, keepdim=True)
            if sinks is not None:
                den = den + torch.where(see.any(1, keepdim=True), torch.exp(sinks[h].double() - m), 0.0)
            w = torch.where(den > 0, w / den, torch.zeros_like(w))
            clean = torch.where(see.any(0)[:, None], vc + vm, torch.zeros_like(vc))  # nothing of what no row sees
            o[b, h] = torch.where(see, w, torch.zeros_like(w)) @ clean
            vcs = torch.where(see.any(0)[:, None], vc, torch.zeros_like(vc))
            bound[b, h] = 2 ** -8 * (w @ vcs + o[b, h].abs()) + 2 * delta * (clean.abs().amax() + o[b, h].abs())
    return o, bound


CASES = [
    # B, Hq, Hkv, L, D, cap, lens, window, first
    ("one_key", 1, 1, 1, 1, 128, 1, [1], 0, 0),
    ("g7", 1, 56, 8, 1, 128, 700, [700], 0, 0),
    ("ragged_g2", 5, 16, 8, 1, 128, 300, [300, 1, 0, 33, 64], 0, 0),
    ("d64_g4_l2", 3, 8, 2, 2, 64, 1000, [1000, 2, 31], 0, 0),
    ("l8_g7_chunks", 2, 14, 2, 8, 128, 500, [500, 8], 0, 0),
    ("l5_g1", 2, 3, 3, 5, 128, 97, [97, 3], 0, 0),  # fewer positions than rows: rows that see none
    ("g16_l1", 2, 32, 2, 1, 64, 260, [260, 129], 0, 0),
    ("g40", 1, 40, 1, 1, 128, 200, [200], 0, 0),
    ("long_split", 1, 8, 8, 1, 128, 20000, [20000], 0, 0),
    ("many", 70, 4, 2, 1, 64, 64, [(7 * i) % 65 for i in range(70)], 0, 0),
    ("window1", 2, 4, 2, 1, 128, 200, [200, 1], 1, 0),
    ("window1_first1", 2, 4, 2, 3, 128, 200, [200, 3], 1, 1),
    ("stream", 4, 8, 2, 1, 64, 5000, [5000, 1027, 1028, 1029], 1024, 4),
    ("stream_l4", 3, 14, 2, 4, 128, 3000, [3000, 1100, 90], 100, 64),
    ("first_past_window", 2, 4, 2, 2, 128, 400, [400, 150], 33, 300),
    ("window_past_all", 1, 4, 2, 2, 128, 100, [100], 2 ** 31 - 1, 7),
    ("first33", 1, 7, 1, 8, 64, 900, [900], 128, 33),
    # one to four rows of a KV head: copies in the products' columns
    ("rows1", 2, 3, 3, 1, 128, 700, [700, 40], 0, 0),
    ("rows2_window", 3, 4, 2, 1, 128, 900, [900, 33, 5], 70, 3),
    ("rows2_l2", 1, 2, 2, 2, 128, 300, [300], 0, 0),
    ("rows3", 2, 6, 2, 1, 128, 500, [500, 100], 0, 0),
    ("rows4_l4", 2, 2, 2, 4, 128, 400, [400, 3], 50, 7),
    ("rows1_d64", 1, 2, 2, 1, 64, 400, [399], 0, 0),
    ("rows3_l3_d64", 2, 2, 2, 3, 64, 400, [399, 2], 20, 1),
]


@pytest.mark.parametrize("c", CASES, ids=[c[0] for c in CASES])
@pytest.mark.parametrize("sharp", [1.0, 6.0])
def test_decode(c, sharp):
    _, B, Hq, Hkv, L, D, cap, lens, window, first = c
    gen = _gen(10)
    k, v = (_randn(gen, B, Hkv, cap, D) for _ in range(2))
    cache = cache_of((k * sharp).bfloat16(), v.bfloat16(), cap)
    for b, n in enumerate(lens):  # what lies behind a sequence is not read
        cache[1][b, :, n:], cache[3][b, :, n:] = float("nan"), float("nan")
    q = _randn(gen, B, Hq, L, D).bfloat16()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = tb.kv4_decode(q, *cache, n, window=window, first=first)
    tb.check_status()
    ref, bound = reference(q, cache, lens, D ** -0.5, window, first)
    assert got.isfinite().all()
    assert ((got.double() - ref).abs() <= bound).all()
    assert torch.equal(got, tb.kv4_decode(q, *cache, n, window=window, first=first))  # the same bits again


@pytest.mark.parametrize("softcap,use_sinks", [(30.0, False), (0.0, True), (5.0, True)])
def test_decode_score_variants(softcap, use_sinks):
    """A softcap's tanh has slope at most 1 and errs by a few 2^-24: inside delta."""
    B, Hq, Hkv, L, D, cap = 2, 12, 4, 3, 128, 700
    gen = _gen(11)
    cache = cache_of((4 * _randn(gen, B, Hkv, cap, D)).bfloat16(), _randn(gen, B, Hkv, cap, D).bfloat16(), cap)
    q = _randn(gen, B, Hq, L, D).bfloat16()
    sinks = 2 * _randn(gen, Hq) if use_sinks else None
    lens = [700, 2]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = tb.kv4_decode(q, *cache, n, window=64, first=5, softcap=softcap, sinks=sinks)
    ref, bound = reference(q, cache, lens, D ** -0.5, 64, 5, softcap, sinks)
    assert ((got.double() - ref).abs() <= bound).all()


def test_what_is_hidden_does_not_reach_the_output():
    """NaN in cached rows: between the first tokens and the window of every row, no
    effect; inside one row's window only, that row alone."""
    B, Hq, Hkv, L, D, cap, W, F = 1, 4, 2, 4, 128, 400, 50, 6
    gen = _gen(12)
    cache = cache_of(_randn(gen, B, Hkv, cap, D).bfloat16(), _randn(gen, B, Hkv, cap, D).bfloat16(), cap)
    q = _randn(gen, B, Hq, L, D).bfloat16()
    n = torch.tensor([cap], dtype=torch.int32, device="cuda")
    clean = tb.kv4_decode(q, *cache, n, window=W, first=F)
    for which in (1, 3):
        bad = [t.clone() for t in cache]
        bad[which][:, :, F:cap - L - W + 1] = float("nan")  # seen by no row
        assert torch.equal(tb.kv4_decode(q, *bad, n, window=W, first=F), clean)
        bad[which][:, :, cap - L - W + 1] = float("nan")  # the first row's oldest position
        got = tb.kv4_decode(q, *bad, n, window=W, first=F)
        assert got[:, :, 0].isnan().any() and torch.equal(got[:, :, 1:], clean[:, :, 1:])
        bad[which][:, :, cap - L - W + 1] = float("inf")
        got = tb.kv4_decode(q, *bad, n, window=W, first=F)
        assert torch.equal(got[:, :, 1:], clean[:, :, 1:])


def test_a_large_step_that_no_row_sees_takes_no_bits():
    """V's steps bound the fp16 products' range; one of 2^60 just outside the window, in
    a step of 32 positions that the window begins in, is none of them."""
    B, Hq, Hkv, D, cap, W, F = 1, 4, 2, 128, 400, 50, 6
    gen = _gen(12)
    cache = cache_of(_randn(gen, B, Hkv, cap, D).bfloat16(), _randn(gen, B, Hkv, cap, D).bfloat16(), cap)
    n = torch.tensor([cap], dtype=torch.int32, device="cuda")
    for L in (1, 3, 8):
        q = _randn(gen, B, Hq, L, D).bfloat16()
        clean = tb.kv4_decode(q, *cache, n, window=W, first=F)
        bad = [t.clone() for t in cache]
        bad[3][:, :, F:cap - L - W + 1, :, 0] = 2.0 ** 60
        assert torch.equal(tb.kv4_decode(q, *bad, n, window=W, first=F), clean)


def test_lengths_out_of_range_are_reported_and_give_zeros():
    gen = _gen(13)
    cache = cache_of(_randn(gen, 3, 2, 64, 64).bfloat16(), _randn(gen, 3, 2, 64, 64).bfloat16(), 64)
    q = _randn(gen, 3, 4, 1, 64).bfloat16()
    got = tb.kv4_decode(q, *cache, torch.tensor([65, 64, -3], dtype=torch.int32, device="cuda"))
    with pytest.raises(tb.TfaError) as e:
        tb.check_status()
    assert e.value.code == tb.TFA_ERR_SEQLENS
    assert (got[0] == 0).all() and (got[2] == 0).all()
    ref, bound = reference(q, cache, [0, 64, 0], 0.125)
    assert ((got.double() - ref).abs() <= bound).all()


def test_offsets_past_32_bits():
    """A cache of 2^31 code bytes and more a tensor: the last head's rows."""
    B, Hkv, cap, D = 1, 9, 4_000_000, 128
    cache = [torch.zeros(B, Hkv, cap, D // 2, dtype=torch.uint8, device="cuda"),
             torch.zeros(B, Hkv, cap, D // 32, 2, dtype=torch.bfloat16, device="cuda")]
    cache += [t.clone() for t in cache]
    assert cache[0].numel() > 2 ** 31
    gen = _gen(14)
    k, v = (_randn(gen, B, Hkv, 70, D).bfloat16() for _ in range(2))
    tb.kv4_append(k, v, *cache, start=cap - 70)
    r = tb.kv4_read(*cache, start=cap - 70)
    codes, meta = quantise(v)
    assert torch.equal(cache[2][:, :, cap - 70:], codes) and torch.equal(r[1][0, -1], sum(parts(codes[0, -1], meta[0, -1])).bfloat16())
    q = _randn(gen, B, 2 * Hkv, 1, D).bfloat16()
    n = torch.tensor([cap], dtype=torch.int32, device="cuda")
    got = tb.kv4_decode(q, *cache, n, window=70, first=0)
    small = [t[:, :, cap - 70:].contiguous() for t in cache]
    ref, bound = reference(q, small, [70], D ** -0.5)
    assert ((got.double() - ref).abs() <= bound).all()
    # everything: the zeros before weigh 1 each
    got = tb.kv4_decode(q, *cache, n)
    x = (q.double()[0, :, 0].view(Hkv, 2, D) @ sum(parts(small[0], small[1]))[0].transpose(1, 2)) * D ** -0.5
    w = torch.exp(x)
    ref = (w @ sum(parts(small[2], small[3]))[0]) / (w.sum(-1, keepdim=True) + cap - 70)
    assert ((got.double().view(Hkv, 2, D) - ref).abs() <= 2 ** -6 * ref.abs() + 1e-6).all()


def test_step_captured_and_replayed():
    """A serving step as it is used: norms and rotation, append, attention; captured
    once and replayed while the lengths on the device move."""
    B, Hq, Hkv, D, cap = 3, 8, 2, 128, 200
    gen = _gen(15)
    f, _ = tb.rope_inv_freq(D, 1e6)
    lens0 = [0, 57, 190]
    cache = cache_of(_randn(gen, B, Hkv, cap, D).bfloat16(), _randn(gen, B, Hkv, cap, D).bfloat16(), cap)
    other = [t.clone() for t in cache]
    w = (1 + 0.1 * _randn(gen, D)).bfloat16()
    qkv = torch.zeros(B, 1, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor(lens0, dtype=torch.int32, device="cuda")

    def step(cache, at):
        q, k = tb.qk_norm_rope(qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], at, f, q_weight=w, k_weight=w)
        tb.kv4_append(k, qkv[:, :, Hq + Hkv:].transpose(1, 2), *cache, start=at)
        at += 1
        return tb.kv4_decode(q, *cache, at, window=64, first=4)

    graph = torch.cuda.CUDAGraph()
    mine = at.clone()
    tb.check_status()
    with torch.cuda.graph(graph):
        out = step(cache, at)
    for i in range(5):
        qkv.copy_(_randn(gen, B, 1, Hq + 2 * Hkv, D))
        graph.replay()
        want = step(other, mine)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        # and against the definition, from the cache as it now is
        q, _ = tb.qk_norm_rope(qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], mine - 1, f, q_weight=w, k_weight=w)
        ref, bound = reference(q, cache, mine.tolist(), D ** -0.5, 64, 4)
        assert ((out.double() - ref).abs() <= bound).all()
    tb.check_status()


def test_two_streams_at_once():
    gen = _gen(16)
    cache = cache_of(_randn(gen, 2, 4, 3000, 128).bfloat16(), _randn(gen, 2, 4, 3000, 128).bfloat16(), 3000)
    n = torch.tensor([3000, 1234], dtype=torch.int32, device="cuda")
    qs = [_randn(gen, 2, 8, 1, 128).bfloat16() for _ in range(2)]
    want = [tb.kv4_decode(q, *cache, n) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(tb.kv4_decode(qs[i], *cache, n, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


PREFILL = [
    # B, Hq, Hkv, L, S, D, cap, window, first
    (1, 4, 2, 1, 1, 128, 1, 0, 0),
    (2, 14, 2, 9, 300, 128, 333, 0, 0),
    (1, 8, 8, 129, 129, 64, 140, 0, 0),
    (2, 4, 2, 200, 1000, 128, 1000, 100, 0),
    (2, 4, 2, 200, 1000, 128, 1001, 100, 4),
    (1, 6, 2, 70, 900, 64, 1000, 65, 300),
    (1, 4, 1, 300, 700, 128, 700, 128, 600),
    (3, 4, 4, 5, 2000, 128, 2048, 1024, 64),
    (1, 2, 1, 40, 500, 64, 500, 2 ** 31 - 1, 9),
    (40, 2, 2, 3, 70, 64, 77, 0, 0),
    (40, 8, 2, 130, 200, 64, 210, 50, 4),
    # many rows and heads: the dense kernel
    (2, 32, 2, 200, 1000, 128, 1000, 0, 0),
    (2, 32, 2, 260, 1000, 128, 1001, 100, 4),
    (4, 32, 4, 300, 700, 64, 720, 128, 600),
]


@pytest.mark.parametrize("c", PREFILL, ids=["-".join(map(str, c)) for c in PREFILL])
def test_prefill(c):
    """K and V are rounded to bf16 once more (2^-8 of each value), and P and the
    output once: the scores move by delta = scale 2^-8 sum_d |q_d k_jd|, at random
    signs; the bound takes half of the largest delta of a row, |err| <= 2^-8 (2 sum w |v| + |o|)
    + 2 delta' sum_j w_j |v_j - o|."""
    B, Hq, Hkv, L, S, D, cap, window, first = c
    gen = _gen(20)
    cache = cache_of(_randn(gen, B, Hkv, S, D).bfloat16(), _randn(gen, B, Hkv, S, D).bfloat16(), cap)
    q = _randn(gen, B, Hq, L, D).bfloat16()
    got = tb.kv4_prefill(q, *cache, S=S, window=window, first=first)
    tb.check_status()
    ref, _ = reference(q, cache, [S] * B, D ** -0.5, window, first)
    for b in range(B):
        for h in range(Hq):
            g = h // (Hq // Hkv)
            k, v = (sum(parts(cache[i][b, g, :S], cache[i + 1][b, g, :S])) for i in (0, 2))
            x = q[b, h].double()
            pos = S - L + torch.arange(L, device="cuda")[:, None]
            j = torch.arange(S, device="cuda")
            see = (j <= pos) & ((j > pos - window) | (j < first)) if window > 0 else j <= pos
            w = torch.softmax((x @ k.T * D ** -0.5).masked_fill(~see, -math.inf), 1)
            delta = D ** -0.5 * 2 ** -8 * (x.abs() @ k.abs().T).masked_fill(~see, 0).amax(1, keepdim=True)
            spread = w @ v.abs() + ref[b, h].abs()
            bound = 2 ** -8 * (2 * (w @ v.abs()) + ref[b, h].abs()) + delta * spread
            assert ((got[b, h].double() - ref[b, h]).abs() <= bound).all()


def test_prefill_is_the_dense_attention_of_the_values_read_back():
    gen = _gen(21)
    cache = cache_of(_randn(gen, 2, 2, 600, 128).bfloat16(), _randn(gen, 2, 2, 600, 128).bfloat16(), 640)
    q = _randn(gen, 2, 32, 260, 128).bfloat16()
    k, v = tb.kv4_read(*cache, rows=600)
    sinks = _randn(gen, 32)
    a = dict(softcap=20.0, sinks=sinks)
    assert torch.equal(tb.kv4_prefill(q, *cache, S=600), tb.prefill(q, k, v))
    assert torch.equal(tb.kv4_prefill(q, *cache, S=600, **a), tb.prefill(q, k, v, **a))
    # without the positions that no row sees, the tiles fall elsewhere: two outputs' roundings apart
    x = tb.kv4_prefill(q, *cache, S=600, window=70, first=5, **a).double()
    y = tb.prefill(q, k, v, window=70, first=5, **a).double()
    assert ((x - y).abs() <= 2 ** -7 * (y.abs() + v.abs().max().double())).all()


def test_a_chunk_then_decoding():
    """A prompt chunk written and attended to, then tokens one by one, against the
    whole sequence at once."""
    B, Hq, Hkv, D, cap, n = 2, 8, 2, 128, 100, 90
    gen = _gen(22)
    k, v = (_randn(gen, B, Hkv, n, D).bfloat16() for _ in range(2))
    q = _randn(gen, B, Hq, n, D).bfloat16()
    cache = tb.kv4_cache(B, Hkv, cap, D)
    tb.kv4_append(k[:, :, :80], v[:, :, :80], *cache, start=0)
    outs = [tb.kv4_prefill(q[:, :, :80].contiguous(), *cache, S=80, window=40, first=4)]
    for i in range(80, n):
        lens = torch.full((B,), i, dtype=torch.int32, device="cuda")
        tb.kv4_append(k[:, :, i:i + 1], v[:, :, i:i + 1], *cache, start=lens)
        outs.append(tb.kv4_decode(q[:, :, i:i + 1].contiguous(), *cache, lens + 1, window=40, first=4))
    whole = tb.kv4_prefill(q, *cache, S=n, window=40, first=4)
    ref, bound = reference(q, cache, [n] * B, D ** -0.5, 40, 4)
    got = torch.cat(outs, 2)
    assert ((got[:, :, 80:].double() - ref[:, :, 80:]).abs() <= bound[:, :, 80:]).all()
    assert ((got.double() - whole.double()).abs() <= 2 ** -5 * (1 + whole.double().abs())).all()


def test_prefill_workspace_is_used_within_its_size():
    gen = _gen(23)
    cache = cache_of(_randn(gen, 1, 2, 400, 64).bfloat16(), _randn(gen, 1, 2, 400, 64).bfloat16(), 400)
    for L in (20, 200):  # few rows, and many
        q = _randn(gen, 1, 64, L, 64).bfloat16()
        need = tb.lib().tfa_kv4_prefill_workspace(1, 64, 2, L, 400, 64, 30, 4)
        ws = torch.full((need + 64,), 77, dtype=torch.uint8, device="cuda")
        got = tb.kv4_prefill(q, *cache, S=400, window=30, first=4, workspace=ws)
        assert torch.equal(got, tb.kv4_prefill(q, *cache, S=400, window=30, first=4)) and (ws[need:] == 77).all()
    with pytest.raises(ValueError):
        tb.kv4_prefill(q, *cache, S=400, workspace=ws)


def test_few_rows_and_many_agree():
    """Chunks on both sides of the border between the two kernels: the same rows."""
    gen = _gen(24)
    cache = cache_of(_randn(gen, 1, 2, 900, 128).bfloat16(), _randn(gen, 1, 2, 900, 128).bfloat16(), 900)
    q = _randn(gen, 1, 64, 200, 128).bfloat16()
    whole = tb.kv4_prefill(q, *cache, S=900, window=300, first=3)
    n = torch.tensor([900], dtype=torch.int32, device="cuda")
    for L in (1, 8, 33, 127):
        part = tb.kv4_prefill(q[:, :, -L:].contiguous(), *cache, S=900, window=300, first=3)
        ref, bound = reference(q[:, :, -L:], cache, [900], 128 ** -0.5, 300, 3)
        assert ((part.double() - ref).abs() <= bound).all()
        assert ((part.double() - whole[:, :, -L:].double()).abs() <= 2 ** -5 * (1 + ref.abs())).all()
        if L <= 8:
            assert torch.equal(part, tb.kv4_decode(q[:, :, -L:].contiguous(), *cache, n, window=300, first=3))


SCALES = [
    # B, Hq, Hkv, L, D, cap, lens, window, first, softcap
    (2, 14, 2, 1, 128, 700, [700, 65], 0, 0, 0.0),
    (2, 4, 2, 3, 128, 300, [300, 2], 50, 4, 0.0),
    (1, 32, 2, 2, 64, 500, [500], 0, 0, 0.0),
    (3, 3, 3, 1, 64, 400, [400, 1, 0], 33, 1, 0.0),
    (2, 14, 2, 8, 128, 300, [300, 9], 0, 0, 12.0),
]


@pytest.mark.parametrize("scale", [-0.11, -1.0, 0.0, 0.5])
@pytest.mark.parametrize("c", SCALES, ids=["-".join(map(str, c[:6])) for c in SCALES])
def test_decode_scales(c, scale):
    """Scales of either sign and 0 (the mean of what a row sees), against the definition."""
    B, Hq, Hkv, L, D, cap, lens, window, first, softcap = c
    if scale == 0 and softcap > 0:
        pytest.skip("refused")
    gen = _gen(30)
    cache = cache_of(_randn(gen, B, Hkv, cap, D).bfloat16(), _randn(gen, B, Hkv, cap, D).bfloat16(), cap)
    q = _randn(gen, B, Hq, L, D).bfloat16()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = tb.kv4_decode(q, *cache, n, scale=scale, window=window, first=first, softcap=softcap)
    tb.check_status()
    ref, bound = reference(q, cache, lens, scale, window, first, softcap)
    assert ((got.double() - ref).abs() <= bound).all()


def _lost(cache, lens, L, window):
    """What the fp16 range takes at most: a product p s is rounded to no less than 2^-25
    in units where the sum of the weights is at least 2^(7 - es), 2^es at most twice the
    largest step of V; a code is at most 15, so 15 2^-31 of that step a position."""
    out = torch.zeros(len(lens), cache[0].shape[1], dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        if n:
            lo = max(0, n - L - window + 1) if window else 0
            out[b] = (n - lo) * 15 * 2.0 ** -31 * cache[3][b, :, lo:n, :, 0].double().amax((1, 2))
    return out


@pytest.mark.parametrize("along", ["grow", "shrink", "mixed"])
@pytest.mark.parametrize("c", [
    # B, Hq, Hkv, L, D, lens, window
    (1, 2, 2, 1, 128, [3000], 0), (1, 4, 2, 3, 128, [2000], 0), (1, 7, 1, 1, 64, [4000], 0), (1, 14, 1, 2, 128, [1500], 0),
    (40, 4, 2, 1, 64, [61 + 40 * i for i in range(40)], 0), (3, 8, 8, 2, 64, [2000, 90, 1000], 700),
], ids=lambda c: "-".join(map(str, c[:5])))
def test_decode_with_steps_of_many_sizes(along, c):
    """V whose steps differ by 2^12 along the sequence and by 2^8 between groups, in one
    piece and in many: the weights' reference follows them, and pieces with references
    of their own are joined.  Single positions are 2^6 above the others."""
    B, Hq, Hkv, L, D, lens, window = c
    cap = max(lens)
    gen = _gen(31)
    x = torch.linspace(0, 12, cap, device="cuda")
    e = {"grow": x, "shrink": x.flip(0), "mixed": 12 * torch.rand(cap, generator=gen, device="cuda")}[along]
    e = e + 6 * (torch.rand(cap, generator=gen, device="cuda") < 0.01)
    groups = 2.0 ** (-8.0 * torch.rand(B, Hkv, cap, D // 32, 1, generator=gen, device="cuda"))
    v = (_randn(gen, B, Hkv, cap, D // 32, 32) * groups).flatten(-2) * torch.exp2(e)[:, None]
    cache = cache_of((2 * _randn(gen, B, Hkv, cap, D)).bfloat16(), v.bfloat16(), cap)
    q = _randn(gen, B, Hq, L, D).bfloat16()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = tb.kv4_decode(q, *cache, n, window=window)
    tb.check_status()
    ref, bound = reference(q, cache, lens, D ** -0.5, window)
    lost = _lost(cache, lens, L, window).repeat_interleave(Hq // Hkv, 1)[:, :, None, None]
    assert ((got.double() - ref).abs() <= bound + lost).all()
    assert torch.equal(got, tb.kv4_decode(q, *cache, n, window=window))


@pytest.mark.parametrize("D,L", [(128, 1), (64, 1), (128, 5)])
def test_decode_with_a_few_large_key_channels(D, L):
    """Two channels of K 30 times the others and of one sign, as rotary keys often have:
    their groups' steps are large, and the scores are as exact as ever."""
    gen = _gen(32)
    B, Hq, Hkv, cap, lens = 2, 8, 2, 900, [900, 333]
    k = _randn(gen, B, Hkv, cap, D)
    k[..., 5] += 30
    k[..., D - 7] -= 30
    cache = cache_of(k.bfloat16(), _randn(gen, B, Hkv, cap, D).bfloat16(), cap)
    q = _randn(gen, B, Hq, L, D).bfloat16()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for window, first in ((0, 0), (100, 4)):
        got = tb.kv4_decode(q, *cache, n, window=window, first=first)
        ref, bound = reference(q, cache, lens, D ** -0.5, window, first)
        assert ((got.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("c", [
    # B, Hq, Hkv, L, S, D, window, first, large key channels
    (2, 32, 2, 200, 1000, 128, 0, 0, False), (2, 32, 2, 260, 1000, 128, 100, 4, True), (4, 32, 4, 300, 700, 64, 128, 600, False),
    (16, 32, 8, 40, 700, 128, 0, 0, True), (1, 56, 8, 513, 1025, 128, 0, 0, False), (2, 28, 4, 333, 1500, 64, 500, 70, True),
], ids=lambda c: "-".join(map(str, c)))
def test_long_chunks_against_the_values_read_back(c):
    """The dense kernel's chunks against the definition over the values that kv4_read
    gives (K and V rounded to bf16 once; the read back is tested by itself), so that only
    the weights' and the output's roundings are left: 2^-8 (sum w |v| + |o|), the fp32
    sums (2^-16 of the absolute ones) as 2^-14."""
    B, Hq, Hkv, L, S, D, window, first, large = c
    gen = _gen(33)
    k = _randn(gen, B, Hkv, S, D)
    if large:
        k[..., 3] += 20
    cache = cache_of(k.bfloat16(), _randn(gen, B, Hkv, S, D).bfloat16(), S + 5)
    assert tb.lib().tfa_kv4_prefill_workspace(B, Hq, Hkv, L, S, D, window, first) != tb.lib().tfa_kv4_decode_workspace(Hq, Hkv, L, D)
    q = _randn(gen, B, Hq, L, D).bfloat16()
    got = tb.kv4_prefill(q, *cache, S=S, window=window, first=first)
    tb.check_status()
    ks, vs = (t.double() for t in tb.kv4_read(*cache, rows=S))
    pos, j = S - L + torch.arange(L, device="cuda")[:, None], torch.arange(S, device="cuda")
    see = (j <= pos) & ((j > pos - window) | (j < first)) if window > 0 else j <= pos
    for b in range(B):
        for h in range(Hq):
            g = h // (Hq // Hkv)
            w = torch.softmax((q[b, h].double() @ ks[b, g].T * D ** -0.5).masked_fill(~see, -math.inf), 1)
            ref = w @ vs[b, g]
            bound = (2 ** -8 + 2 ** -14) * (w @ vs[b, g].abs() + ref.abs())
            assert ((got[b, h].double() - ref).abs() <= bound).all()
