"""The long-context operators of this library as measurable cases.

Four operators that a serving or training step uses one after another:

  rope     norms of queries and keys for each head with the rotary position in
           the same pass, forward and backward
  append   quantising new keys and values into a 4-bit cache, and reading them back
  kv4      attention over that 4-bit cache: decoding (1..8 rows) and prompt chunks
  first    attention with a sliding window and a few first tokens that stay
           visible: forward (any length) and the training step's gradients

`run` computes each in its plain form (elementary torch operations in 32 bits,
rounded once at the end), or, with `own` set, through the library's entry points.

The 4-bit cache: per position and KV head, D channels in groups of 32; a group
holds its minimum m and step s = (max - min) / 15, both bf16, and 4-bit codes
c = round((x - m) / s) clamped to 0..15; the value is c s + m.  Byte i of a row
holds channel 2i in its low and 2i + 1 in its high half.
"""
import math
import random

import torch

own = False

GROUP = 32  # channels that share a step and a minimum


def _api():
    from sliding_window_gqa_tfa_b200 import binding

    return binding


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decoding step of 16 Qwen3-shaped sequences some 8K tokens in: norms and rotation
        dict(name="rope_decode_b16", op="rope", back=False, B=16, L=1, Hq=16, Hkv=8, D=128, rot=128, norm=True,
             inter=False, base=1e6, stretch=1.0, start=8191),
        # a 2048-token chunk of the 56-head geometry over a 6144-token prefix, rotation only
        # (pairs of neighbours), stretched four times for a long context
        dict(name="rope_chunk_llama_2048", op="rope", back=False, B=1, L=2048, Hq=56, Hkv=8, D=128, rot=128,
             norm=False, inter=True, base=5e5, stretch=4.0, start=6144),
        # the same pass's gradients in a training step of four Qwen3-shaped sequences, half
        # of each head rotated, a ragged length
        dict(name="rope_backward_b4_2047", op="rope", back=True, B=4, L=2047, Hq=16, Hkv=8, D=128, rot=64, norm=True,
             inter=False, base=1e6, stretch=1.0, start=0),
        # one decoding step of 64 sequences: a new row for each, at its own place
        dict(name="append_decode_b64", op="append", B=64, L=1, Hkv=8, D=128, cap=1088, start=1000),
        # a prompt chunk of four sequences of a ragged length, written over a prefix
        dict(name="append_chunk_b4_2047", op="append", B=4, L=2047, Hkv=8, D=128, cap=4096, start=1025),
        # batched decoding, 16 ragged sequences of at most 8192 tokens
        dict(name="kv4_decode_b16_8192", op="kv4", B=16, Hq=16, Hkv=8, L=1, S=8192, cap=8192, D=128, window=0, first=0,
             ragged=True),
        # one sequence 32K tokens in: all of the machine on eight KV heads
        dict(name="kv4_decode_1x32768", op="kv4", B=1, Hq=56, Hkv=8, L=1, S=32768, cap=32768, D=128, window=0, first=0,
             ragged=False),
        # streaming: 64 ragged sequences of at most 8192 tokens that keep 4 first tokens and a 1024-token window
        dict(name="kv4_stream_b64_w1024", op="kv4", B=64, Hq=32, Hkv=8, L=1, S=8192, cap=8192, D=64, window=1024,
             first=4, ragged=True),
        # a 2048-token prompt chunk over 8192 cached tokens
        dict(name="kv4_chunk_2048x8192", op="kv4", B=1, Hq=56, Hkv=8, L=2048, S=8192, cap=8192, D=128, window=0,
             first=0, ragged=False),
        # a short ragged chunk (e.g. the verification of drafts) far into a streaming context
        dict(name="first_chunk_37x8229", op="first", back=False, B=4, Hq=32, Hkv=8, L=37, S=8229, D=128, window=1024,
             first=64),
        # a 2048-token prompt chunk, 1024-token window, 4 first tokens
        dict(name="first_chunk_2048x8192", op="first", back=False, B=1, Hq=32, Hkv=8, L=2048, S=8192, D=128,
             window=1024, first=4),
        # a training step of the same layer: forward and gradients of one 4096-token sequence
        dict(name="first_train_4096", op="first", back=True, B=1, Hq=32, Hkv=8, L=4096, S=4096, D=128, window=1024,
             first=4),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_back", "append", "kv4", "kv4_chunk", "first", "first_back"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 7])
    if op in ("rope", "rope_back"):
        B = rng.choice([1, 2, 4, 16])
        L = _spread(rng, 1, 8192 // B)
        return dict(op="rope", back=op == "rope_back", B=B, L=L, Hq=G * Hkv, Hkv=Hkv, D=D,
                    rot=rng.choice([D, D // 2, 16]), norm=rng.random() < 0.6, inter=rng.random() < 0.5,
                    base=rng.choice([1e4, 5e5, 1e6]), stretch=rng.choice([1.0, 4.0, 32.0]),
                    start=_spread(rng, 1, 1_000_000) - 1)
    if op == "append":
        B = rng.choice([1, 3, 16, 64])
        L = _spread(rng, 1, 8192 // B)
        start = _spread(rng, 1, 2048) - 1
        return dict(op="append", B=B, L=L, Hkv=Hkv, D=D, cap=start + L + B + rng.randrange(64), start=start)
    if op == "kv4":
        B = rng.choice([1, 3, 16, 64])
        L = rng.choice([1, 1, 1, 2, 4, 8])
        S = _spread(rng, max(L, 16), 131072 // B)
        W = rng.choice([0, 0, 128, 1024])
        return dict(op="kv4", B=B, Hq=G * Hkv, Hkv=Hkv, L=L, S=S, cap=S + rng.randrange(100), D=D, window=W,
                    first=rng.choice([1, 4, 100]) if W else 0, ragged=rng.random() < 0.7)
    if op == "kv4_chunk":
        L = _spread(rng, 9, 2048)
        S = L + rng.randrange(6144)
        W = rng.choice([0, 1024])
        return dict(op="kv4", B=1, Hq=G * Hkv, Hkv=Hkv, L=L, S=S, cap=S + rng.randrange(100), D=D, window=W,
                    first=rng.choice([1, 4, 100]) if W else 0, ragged=False)
    if op == "first":
        B = rng.choice([1, 2, 4])
        L = _spread(rng, 1, 2048 // B)
        return dict(op="first", back=False, B=B, Hq=G * Hkv, Hkv=Hkv, L=L, S=L + rng.randrange(8192 // B), D=D,
                    window=_spread(rng, 1, 2048), first=_spread(rng, 1, 256))
    L = _spread(rng, 1, 2048)
    return dict(op="first", back=True, B=1, Hq=G * Hkv, Hkv=Hkv, L=L, S=L + rng.randrange(2048), D=D,
                window=_spread(rng, 1, 2048), first=_spread(rng, 1, 256))


def _lens(case):
    """Cached tokens of each sequence, the new ones among them."""
    B, L, S = case["B"], case["L"], case["S"]
    if not case["ragged"]:
        return [S] * B
    r = random.Random(1000003 * S + B)
    return [S] + [r.randint(max(L, S // 4), S) for _ in range(B - 1)]


def _inv_freq(case):
    """Radians a position for each rotated pair, and the factor on cos and sin: the
    YaRN rule for contexts `stretch` times the first 8192 tokens (fast pairs as they
    are, slow ones stretched, a ramp between), plain where stretch is 1."""
    rot, base, s = case["rot"], case["base"], case["stretch"]
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if s == 1.0:
        return f, 1.0
    lo, hi = 1.0, 32.0  # turns over the first context: slower than lo is stretched whole, faster than hi not at all
    out = []
    for x in f:
        turns = 8192 * x / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - lo) / (hi - lo)))
        out.append(x * keep + x / s * (1 - keep))
    return out, 0.1 * math.log(s) + 1.0


# ------------------------------------------------------------------- the data
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _quantise(x):
    """(codes, steps and minima, values) of fp32 rows of bf16 numbers [..., D]."""
    g = x.unflatten(-1, (-1, GROUP))
    mn = g.amin(-1, keepdim=True)
    fifteen = torch.full((), 15.0, device=x.device)
    step = ((g.amax(-1, keepdim=True) - mn) / fifteen).bfloat16().float()
    code = torch.where(step > 0, torch.round((g - mn) / step).clamp(0, 15), torch.zeros_like(g))
    value = (code * step + mn).flatten(-2)
    code = code.flatten(-2).to(torch.uint8).unflatten(-1, (-1, 2))
    return code[..., 0] | (code[..., 1] << 4), torch.cat([mn * 0 + step, mn], -1).bfloat16(), value


def _values(codes, meta):
    """fp32 values of a cache's rows."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    return (c * meta[..., :1].float() + meta[..., 1:].float()).flatten(-2)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    st = {"case": case}
    if case["op"] == "rope":
        B, L, Hq, Hkv, D = (case[k] for k in ("B", "L", "Hq", "Hkv", "D"))
        # the projections' output, token by token: queries, keys and values of a token side by side
        qkv = _randn(gen, B, L, Hq + 2 * Hkv, D).bfloat16()
        st["q"], st["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv]
        f, st["mscale"] = _inv_freq(case)
        st["inv_freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        # every sequence at its own position
        st["pos"] = case["start"] + torch.randint(0, 8, (B,), generator=gen, device="cuda", dtype=torch.int32)
        st["wq"] = (1 + 0.1 * _randn(gen, D)).bfloat16() if case["norm"] else None
        st["wk"] = (1 + 0.1 * _randn(gen, D)).bfloat16() if case["norm"] else None
        if case["back"]:
            st["dq"] = _randn(gen, B, Hq, L, D).bfloat16()
            st["dk"] = _randn(gen, B, Hkv, L, D).bfloat16()
        return st
    if case["op"] == "append":
        B, L, Hkv, D, cap = (case[k] for k in ("B", "L", "Hkv", "D", "cap"))
        # keys and values as the projections leave them, token by token
        kv = _randn(gen, B, L, 2 * Hkv, D).bfloat16()
        st["k"], st["v"] = kv[:, :, :Hkv].transpose(1, 2), kv[:, :, Hkv:].transpose(1, 2)
        st["start"] = case["start"] + torch.arange(B, device="cuda", dtype=torch.int32)
        for n in ("k", "v"):
            st[n + "c"] = torch.zeros(B, Hkv, cap, D // 2, dtype=torch.uint8, device="cuda")
            st[n + "m"] = torch.zeros(B, Hkv, cap, D // GROUP, 2, dtype=torch.bfloat16, device="cuda")
        st["at"] = (st["start"].long()[:, None] + torch.arange(L, device="cuda"))[:, None]  # [B, 1, L]
        st["b"] = torch.arange(B, device="cuda")[:, None, None]
        st["h"] = torch.arange(Hkv, device="cuda")[None, :, None]
        return st
    B, Hq, Hkv, L, S, D = (case[k] for k in ("B", "Hq", "Hkv", "L", "S", "D"))
    st["q"] = _randn(gen, B, Hq, L, D).bfloat16()
    if case["op"] == "kv4":
        for n in ("k", "v"):
            st[n + "c"], st[n + "m"], _ = _quantise(_randn(gen, B, Hkv, case["cap"], D).bfloat16().float())
        st["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
        return st
    st["k"], st["v"] = _randn(gen, B, Hkv, S, D).bfloat16(), _randn(gen, B, Hkv, S, D).bfloat16()
    if case["back"]:
        st["do"] = _randn(gen, B, Hq, L, D).bfloat16()
    return st


# ------------------------------------------------------------ the plain forms
def _angles(st):
    """cos and sin of every token's angles, fp32 [B, L, 1, rot / 2]: the angle in 64 bits."""
    c = st["case"]
    pos = st["pos"].double()[:, None] + torch.arange(c["L"], device="cuda")
    a = pos[:, :, None, None] * st["inv_freq"]
    return a.cos().float() * st["mscale"], a.sin().float() * st["mscale"]


def _rotate(x, cos, sin, rot, inter):
    """x [..., D] with its first `rot` channels rotated pair by pair."""
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., :rot // 2], r[..., rot // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([u, v], -1).flatten(-2) if inter else torch.cat([u, v], -1)
    return torch.cat([r, rest], -1)


EPS = 1e-6


def _norm_rope(x, w, cos, sin, c):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    return _rotate(x, cos, sin, c["rot"], c["inter"]).transpose(1, 2).contiguous().bfloat16()


def _norm_rope_back(dy, x, w, cos, sin, c):
    g = _rotate(dy.transpose(1, 2).float(), cos, -sin, c["rot"], c["inter"])
    if w is None:
        return g.bfloat16(), None
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    h = x * r
    dw = (g * h).sum((0, 1, 2))
    g = g * w.float()
    return (r * (g - h * (g * h).mean(-1, keepdim=True))).bfloat16(), dw


def _visible(c, lens=None):
    """Whether row i of a sequence sees key j: [B or 1, 1, 1, L, S]."""
    L, S, W, F = c["L"], c["S"], c["window"], c["first"]
    n = torch.tensor([S], device="cuda") if lens is None else lens
    p = n[:, None, None] - L + torch.arange(L, device="cuda")[:, None]
    j = torch.arange(S, device="cuda")
    see = j <= p
    if W > 0:
        see = see & ((j > p - W) | (j < F))
    return see[:, None, None]


def _weights(q, k, c, lens=None):
    """Softmax weights fp32 [B, Hkv, G, L, S] of fp32 q [B, Hq, L, D], k [B, Hkv, S, D]."""
    B, Hkv, S, D = k.shape
    s = torch.matmul(q.reshape(B, Hkv, -1, D), k.transpose(-1, -2)).view(B, Hkv, -1, c["L"], S) * (D ** -0.5)
    s = s.masked_fill(~_visible(c, lens), -math.inf)
    s = torch.exp(s - s.amax(-1, keepdim=True))
    return s / s.sum(-1, keepdim=True)


def _attend(p, v, shape):
    B, Hkv, S, D = v.shape
    return torch.matmul(p.view(B, Hkv, -1, S), v).view(shape)


def run(st):
    c = st["case"]
    if own:
        return _run_own(st, c)
    if c["op"] == "rope":
        cos, sin = _angles(st)
        if not c["back"]:
            return _norm_rope(st["q"], st["wq"], cos, sin, c), _norm_rope(st["k"], st["wk"], cos, sin, c)
        dq, dwq = _norm_rope_back(st["dq"], st["q"], st["wq"], cos, sin, c)
        dk, dwk = _norm_rope_back(st["dk"], st["k"], st["wk"], cos, sin, c)
        return (dq, dk) if dwq is None else (dq, dk, dwq, dwk)
    if c["op"] == "append":
        kc, km, kx = _quantise(st["k"].float())
        vc, vm, vx = _quantise(st["v"].float())
        at = (st["b"], st["h"], st["at"])
        st["kc"][at], st["km"][at], st["vc"][at], st["vm"][at] = kc, km, vc, vm
        return kx.bfloat16(), vx.bfloat16()
    if c["op"] == "kv4":
        S = c["S"]
        k, v = _values(st["kc"][:, :, :S], st["km"][:, :, :S]), _values(st["vc"][:, :, :S], st["vm"][:, :, :S])
        return _attend(_weights(st["q"].float(), k, c, st["lens"]), v, st["q"].shape).bfloat16()
    q, k, v = st["q"].float(), st["k"].float(), st["v"].float()
    p = _weights(q, k, c)
    o = _attend(p, v, q.shape)
    if not c["back"]:
        return o.bfloat16()
    B, Hkv, S, D = k.shape
    do = st["do"].float()
    p, q2, do2 = p.view(B, Hkv, -1, S), q.reshape(B, Hkv, -1, D), do.reshape(B, Hkv, -1, D)
    ds = torch.matmul(do2, v.transpose(-1, -2))
    ds = p * (ds - (do2 * o.reshape(B, Hkv, -1, D)).sum(-1, keepdim=True)) * (D ** -0.5)
    dq = torch.matmul(ds, k).view(q.shape)
    dk, dv = torch.matmul(ds.transpose(-1, -2), q2), torch.matmul(p.transpose(-1, -2), do2)
    return o.bfloat16(), dq.bfloat16(), dk.bfloat16(), dv.bfloat16()


# ------------------------------------------------------------ the library's calls
def _run_own(st, c):
    tb = _api()
    if c["op"] == "rope":
        a = dict(q_weight=st["wq"], k_weight=st["wk"], eps=EPS, interleaved=c["inter"], mscale=st["mscale"])
        if not c["back"]:
            return tb.qk_norm_rope(st["q"], st["k"], st["pos"], st["inv_freq"], **a)
        dq, dk, dwq, dwk = tb.qk_norm_rope_backward(st["dq"], st["dk"], st["q"], st["k"], st["pos"], st["inv_freq"], **a)
        return (dq, dk) if dwq is None else (dq, dk, dwq, dwk)
    if c["op"] == "append":
        cache = st["kc"], st["km"], st["vc"], st["vm"]
        tb.kv4_append(st["k"], st["v"], *cache, start=st["start"])
        return tb.kv4_read(*cache, start=st["start"], rows=c["L"])
    if c["op"] == "kv4":
        a = dict(window=c["window"], first=c["first"])
        if c["L"] <= 8:
            return tb.kv4_decode(st["q"], st["kc"], st["km"], st["vc"], st["vm"], st["lens"], **a)
        return tb.kv4_prefill(st["q"], st["kc"], st["km"], st["vc"], st["vm"], S=c["S"], **a)
    a = dict(causal=True, window=c["window"], first=c["first"])
    if not c["back"]:
        return tb.prefill(st["q"], st["k"], st["v"], **a)
    o, lse = tb.prefill_lse(st["q"], st["k"], st["v"], **a)
    dq, dk, dv = tb.backward(st["q"], st["k"], st["v"], st["do"], saved=(o, lse), **a)
    return o, dq, dk, dv


# ------------------------------------------------------------------- the work
def _keys_seen(p, c):
    """Keys that the row at position p sees."""
    if p < 0:
        return 0
    W = c["window"]
    return p + 1 if W <= 0 else min(W, p + 1) + min(c["first"], max(0, p + 1 - W))


def _keys_read(n, c):
    """Cached positions that some row of a sequence of n tokens sees."""
    W = c["window"]
    tail = n if W <= 0 else min(n, W + c["L"] - 1)
    return tail + min(c["first"], n - tail)


def work(case):
    c = case
    D, L, B, Hkv = c["D"], c["L"], c["B"], c["Hkv"]
    if c["op"] == "rope":
        n = B * L * (c["Hq"] + Hkv) * D
        per = 3 * c["rot"] / D + (8 if c["norm"] else 0)
        return {"bytes": (3 if c["back"] and c["norm"] else 2) * 2 * n, "flops": n * per * (2 if c["back"] else 1)}
    if c["op"] == "append":
        n = 2 * B * Hkv * L * D
        # bf16 rows in; codes, steps and minima out; and the values back from them
        return {"bytes": n * (2 + 2 * (0.5 + 4 / GROUP) + 2), "flops": 6 * n}
    if c["op"] == "kv4":
        lens = _lens(c)
        rows = sum(_keys_read(n, c) for n in lens) * Hkv
        pairs = sum(_keys_seen(n - L + i, c) for n in lens for i in range(L)) * c["Hq"]
        return {"bytes": rows * 2 * (D / 2 + 4 * D / GROUP) + 4 * B * c["Hq"] * L * D, "flops": 4 * D * pairs}
    S = c["S"]
    pairs = sum(_keys_seen(S - L + i, c) for i in range(L)) * B * c["Hq"]
    q, k = 2 * B * c["Hq"] * L * D, 2 * B * Hkv * _keys_read(S, c) * D
    if c["back"]:  # q, k, v, dO in; o, dq, dk, dv out (gradients of every key); 2 + 5 products
        return {"bytes": 4 * q + 2 * k + 4 * B * Hkv * S * D, "flops": 14 * D * pairs}
    return {"bytes": 2 * q + 2 * k, "flops": 4 * D * pairs}


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    """From the definitions in 64 bits, sequence by sequence and KV head by KV head."""
    st = prepare(case, seed)
    c = case
    if c["op"] == "rope":
        return _exact_rope(st, c)
    if c["op"] == "append":
        return tuple(_exact_quantised(st[n].double(), c["D"]) for n in ("k", "v"))
    B, Hq, Hkv, L, D = (c[k] for k in ("B", "Hq", "Hkv", "L", "D"))
    G = Hq // Hkv
    lens = _lens(c) if c["op"] == "kv4" else [c["S"]] * B
    o = torch.zeros(B, Hq, L, D, dtype=torch.float64, device="cuda")
    back = c.get("back", False)
    if back:
        dq = torch.zeros_like(o)
        dk = torch.zeros(B, Hkv, c["S"], D, dtype=torch.float64, device="cuda")
        dv = torch.zeros_like(dk)
    for b in range(B):
        n = lens[b]
        row = torch.arange(L, device="cuda").view(L, 1) + (n - L)
        col = torch.arange(n, device="cuda").view(1, n)
        hidden = col > row
        if c["window"] > 0:
            hidden |= (row - col >= c["window"]) & (col >= c["first"])
        for g in range(Hkv):
            if c["op"] == "kv4":
                k, v = (_exact_cache(st[a + "c"][b, g, :n], st[a + "m"][b, g, :n]) for a in ("k", "v"))
            else:
                k, v = st["k"][b, g].double(), st["v"][b, g].double()
            for h in range(g * G, (g + 1) * G):
                x = st["q"][b, h].double()
                t = (x @ k.T) / math.sqrt(D)
                t[hidden] = -math.inf
                w = torch.softmax(t, 1)
                y = w @ v
                o[b, h] = y
                if back:
                    e = st["do"][b, h].double()
                    dv[b, g] += w.T @ e
                    # the softmax's Jacobian: w (dw - sum w dw)
                    dt = e @ v.T
                    dt = w * (dt - (w * dt).sum(1, keepdim=True)) / math.sqrt(D)
                    dq[b, h] = dt @ k
                    dk[b, g] += dt.T @ x
    return (o, dq, dk, dv) if back else o


def _exact_cache(codes, meta):
    """Rows of one head: channel by channel from the bytes."""
    n, half = codes.shape
    x = torch.empty(n, 2 * half, dtype=torch.float64, device=codes.device)
    x[:, 0::2] = (codes % 16).double()
    x[:, 1::2] = torch.div(codes, 16, rounding_mode="floor").double()
    for i in range(2 * half // GROUP):
        x[:, i * GROUP:(i + 1) * GROUP] = x[:, i * GROUP:(i + 1) * GROUP] * meta[:, i, :1].double() + meta[:, i, 1:].double()
    return x


def _exact_quantised(x, D):
    out = torch.empty_like(x)
    for i in range(D // GROUP):
        g = x[..., i * GROUP:(i + 1) * GROUP]
        m = g.min(-1, keepdim=True).values
        s = ((g.max(-1, keepdim=True).values - m) / 15.0).bfloat16().double()
        q = torch.clamp(torch.round((g - m) / s), 0, 15)
        out[..., i * GROUP:(i + 1) * GROUP] = torch.where(s > 0, q * s, torch.zeros_like(g)) + m
    return out


def _exact_rope(st, c):
    L, rot, D = c["L"], c["rot"], c["D"]
    # a rotation of each pair as a complex factor of length mscale
    pos = (st["pos"].double()[:, None] + torch.arange(L, device="cuda").double()).unsqueeze(-1)
    z = torch.polar(torch.full_like(pos * st["inv_freq"], st["mscale"]), pos * st["inv_freq"]).unsqueeze(2)

    def turn(x, z):
        y = x.clone()
        if c["inter"]:
            w = torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * z
            y[..., :rot] = torch.view_as_real(w).flatten(-2)
        else:
            w = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * z
            y[..., :rot] = torch.cat([w.real, w.imag], -1)
        return y

    out, dws = [], []
    for n in ("q", "k"):
        x, w = st[n].double(), st["w" + n]
        size = (x * x).sum(-1, keepdim=True) / D + EPS
        if not c["back"]:
            y = x / size.sqrt() * w.double() if w is not None else x
            out.append(turn(y, z).transpose(1, 2))
            continue
        g = turn(st["d" + n].transpose(1, 2).double(), z.conj())
        if w is not None:
            dws.append((g * x / size.sqrt()).flatten(0, 2).sum(0))
            g = g * w.double()
            g = g / size.sqrt() - x * (g * x).sum(-1, keepdim=True) / (D * size ** 1.5)
        out.append(g)
    return tuple(out + dws)
