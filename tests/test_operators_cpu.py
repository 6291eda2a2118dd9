"""Refusals of the long-context operators, before any CUDA call: the pointers here
are never dereferenced."""
import ctypes
import random

import pytest

from sliding_window_gqa_tfa_b200 import binding as tb

A16 = ctypes.c_void_p(0x10000)
MIS = ctypes.c_void_p(0x10008)


def _strides(n, odd=None):
    import struct

    s = [1 << 20, 4096, 128] * (n // 3)
    if odd is not None:
        s[odd] += 4
    return struct.pack(f"{n}q", *s)


def _rope(back=False, **over):
    a = dict(B=2, L=5, Hq=8, Hkv=2, D=128, rot=64, inter=0, eps=1e-6, mscale=1.0, q=A16, k=A16, qo=A16, ko=A16, wq=A16,
             wk=A16, f=A16, pos=None, ws=A16, dw=A16, odd=None)
    a.update(over)
    dims = (a["B"], a["L"], a["Hq"], a["Hkv"], a["D"], a["rot"], a["inter"], a["eps"], a["mscale"])
    mid = (a["wq"], a["wk"], a["f"], a["pos"], 0, 0)
    if back:
        return tb.lib().tfa_qk_norm_rope_backward(a["qo"], a["ko"], a["q"], a["k"], A16, A16, a["dw"], a["dw"],
                                                  _strides(18, a["odd"]), *mid, *dims, a["ws"], None)
    return tb.lib().tfa_qk_norm_rope(a["q"], a["k"], a["qo"], a["ko"], _strides(12, a["odd"]), *mid, *dims, None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("over,code", [
    (dict(q=None), tb.TFA_ERR_NULL),
    (dict(ko=None), tb.TFA_ERR_NULL),
    (dict(f=None), tb.TFA_ERR_NULL),
    (dict(wk=None), tb.TFA_ERR_NULL),
    (dict(B=0), tb.TFA_ERR_SHAPE),
    (dict(L=0), tb.TFA_ERR_SHAPE),
    (dict(B=1 << 16, L=1 << 16), tb.TFA_ERR_SHAPE),
    (dict(Hq=0), tb.TFA_ERR_HEADS),
    (dict(Hkv=-1), tb.TFA_ERR_HEADS),
    (dict(D=96), tb.TFA_ERR_HEAD_DIM),
    (dict(rot=8), tb.TFA_ERR_ROPE),
    (dict(rot=144), tb.TFA_ERR_ROPE),
    (dict(rot=-16), tb.TFA_ERR_ROPE),
    (dict(eps=-1e-6), tb.TFA_ERR_ROPE),
    (dict(eps=float("nan")), tb.TFA_ERR_ROPE),
    (dict(mscale=float("inf")), tb.TFA_ERR_ROPE),
    (dict(k=MIS), tb.TFA_ERR_ALIGN),
    (dict(qo=MIS), tb.TFA_ERR_ALIGN),
    (dict(wq=MIS), tb.TFA_ERR_ALIGN),
    (dict(pos=ctypes.c_void_p(0x10002)), tb.TFA_ERR_ALIGN),
    (dict(odd=4), tb.TFA_ERR_ALIGN),
])
def test_rope_refusals(back, over, code):
    assert _rope(back, **over) == code


def test_rope_backward_needs_its_buffers_with_weights():
    assert _rope(True, ws=None) == tb.TFA_ERR_NULL
    assert _rope(True, dw=None) == tb.TFA_ERR_NULL
    assert tb.lib().tfa_qk_norm_rope_workspace(128) == 296 * 128 * 4


def test_rope_inv_freq_refusals():
    for a in (dict(rot=7), dict(rot=-2), dict(rot=16, scaling="other"), dict(rot=16, factor=0.0)):
        with pytest.raises(ValueError):
            tb.rope_inv_freq(device="cpu", **a)


# ------------------------------------------------------------- the 4-bit cache
def _append(**over):
    a = dict(k=A16, v=A16, kc=A16, km=A16, vc=A16, vm=A16, start=A16, first=0, B=2, Hkv=2, L=5, cap=64, D=128, odd=None)
    a.update(over)
    return tb.lib().tfa_kv4_append(a["k"], a["v"], _strides(6, a["odd"]), a["kc"], a["km"], a["vc"], a["vm"], a["start"],
                                   a["first"], a["B"], a["Hkv"], a["L"], a["cap"], a["D"], None)


def _read(**over):
    a = dict(k=A16, v=A16, kc=A16, km=A16, vc=A16, vm=A16, start=A16, first=0, B=2, Hkv=2, L=5, cap=64, D=128)
    a.update(over)
    return tb.lib().tfa_kv4_read(a["kc"], a["km"], a["vc"], a["vm"], a["k"], a["v"], a["start"], a["first"], a["B"],
                                 a["Hkv"], a["L"], a["cap"], a["D"], None)


@pytest.mark.parametrize("call", [_append, _read])
@pytest.mark.parametrize("over,code", [
    (dict(k=None), tb.TFA_ERR_NULL),
    (dict(vm=None), tb.TFA_ERR_NULL),
    (dict(kc=None), tb.TFA_ERR_NULL),
    (dict(Hkv=0), tb.TFA_ERR_HEADS),
    (dict(B=0), tb.TFA_ERR_SHAPE),
    (dict(L=0), tb.TFA_ERR_SHAPE),
    (dict(cap=0), tb.TFA_ERR_SHAPE),
    (dict(cap=(1 << 30) + 1), tb.TFA_ERR_SHAPE),
    (dict(B=1 << 20, Hkv=1 << 10, L=1 << 20, cap=1 << 10), tb.TFA_ERR_SHAPE),
    (dict(D=96), tb.TFA_ERR_HEAD_DIM),
    (dict(start=None, first=-1), tb.TFA_ERR_CACHE),
    (dict(start=None, first=60), tb.TFA_ERR_CACHE),
    (dict(start=None, first=2 ** 31 - 1), tb.TFA_ERR_CACHE),
    (dict(v=MIS), tb.TFA_ERR_ALIGN),
    (dict(km=MIS), tb.TFA_ERR_ALIGN),
    (dict(start=ctypes.c_void_p(0x10002)), tb.TFA_ERR_ALIGN),
])
def test_cache_refusals(call, over, code):
    assert call(**over) == code


def test_append_refuses_odd_strides():
    for i in range(6):
        assert _append(odd=i) == tb.TFA_ERR_ALIGN


def _decode(**over):
    a = dict(q=A16, kc=A16, km=A16, vc=A16, vm=A16, lens=A16, o=A16, B=2, Hq=8, Hkv=2, L=1, cap=64, D=128, scale=0.1,
             window=0, first=0, softcap=0.0, sinks=None, ws=A16)
    a.update(over)
    return tb.lib().tfa_kv4_decode(*a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(q=None), tb.TFA_ERR_NULL),
    (dict(lens=None), tb.TFA_ERR_NULL),
    (dict(ws=None), tb.TFA_ERR_NULL),
    (dict(vc=None), tb.TFA_ERR_NULL),
    (dict(Hq=7), tb.TFA_ERR_HEADS),
    (dict(Hq=0), tb.TFA_ERR_HEADS),
    (dict(L=0), tb.TFA_ERR_SHAPE),
    (dict(L=9), tb.TFA_ERR_SHAPE),
    (dict(B=1025), tb.TFA_ERR_SHAPE),
    (dict(D=32), tb.TFA_ERR_HEAD_DIM),
    (dict(first=-1, window=4), tb.TFA_ERR_WINDOW),
    (dict(first=4), tb.TFA_ERR_WINDOW),
    (dict(scale=float("nan")), tb.TFA_ERR_SCALE),
    (dict(softcap=-1.0), tb.TFA_ERR_SOFTCAP),
    (dict(softcap=1.0, scale=0.0), tb.TFA_ERR_SOFTCAP),
    (dict(o=MIS), tb.TFA_ERR_ALIGN),
    (dict(ws=MIS), tb.TFA_ERR_ALIGN),
    (dict(sinks=ctypes.c_void_p(0x10002)), tb.TFA_ERR_ALIGN),
])
def test_kv4_decode_refusals(over, code):
    assert _decode(**over) == code


# ------------------------------------------- a window with visible first tokens
def _first(back=False, **over):
    a = dict(q=A16, k=A16, v=A16, o=A16, lse=None, B=1, Hq=8, Hkv=2, L=33, S=47, D=128, scale=0.1, window=16, first=4,
             key_mask=None, softcap=0.0, sinks=None, do=A16, dk=A16)
    if back:
        a["lse"] = A16
    a.update(over)
    sizes = (a["B"], a["Hq"], a["Hkv"], a["L"], a["S"], a["D"], a["scale"], a["window"], a["first"], a["key_mask"])
    if back:
        return tb.lib().tfa_prefill_first_backward(a["q"], a["k"], a["v"], a["o"], a["lse"], a["do"], A16, a["dk"], A16,
                                                   *sizes, None)
    return tb.lib().tfa_prefill_first(a["q"], a["k"], a["v"], a["o"], a["lse"], *sizes, a["softcap"], a["sinks"], None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("over,code", [
    (dict(q=None), tb.TFA_ERR_NULL),
    (dict(Hq=7), tb.TFA_ERR_HEADS),
    (dict(S=32), tb.TFA_ERR_SHAPE),
    (dict(D=96), tb.TFA_ERR_HEAD_DIM),
    (dict(window=0), tb.TFA_ERR_WINDOW),
    (dict(window=-5), tb.TFA_ERR_WINDOW),
    (dict(first=-1), tb.TFA_ERR_WINDOW),
    (dict(v=MIS), tb.TFA_ERR_ALIGN),
    (dict(lse=ctypes.c_void_p(0x10002)), tb.TFA_ERR_ALIGN),
    (dict(key_mask=ctypes.c_void_p(0x10002)), tb.TFA_ERR_ALIGN),
    (dict(scale=float("inf")), tb.TFA_ERR_SCALE),
])
def test_first_refusals(back, over, code):
    assert _first(back, **over) == code


def test_first_refusals_of_one_direction():
    assert _first(softcap=-1.0) == tb.TFA_ERR_SOFTCAP
    assert _first(softcap=3.0, lse=A16) == tb.TFA_ERR_SOFTCAP
    assert _first(sinks=A16, lse=A16) == tb.TFA_ERR_SOFTCAP
    assert _first(sinks=ctypes.c_void_p(0x10002)) == tb.TFA_ERR_ALIGN
    assert _first(True, lse=None) == tb.TFA_ERR_NULL
    assert _first(True, o=None) == tb.TFA_ERR_NULL
    assert _first(True, dk=None) == tb.TFA_ERR_NULL
    assert _first(True, dk=MIS) == tb.TFA_ERR_ALIGN


def _chunk(**over):
    a = dict(q=A16, kc=A16, km=A16, vc=A16, vm=A16, o=A16, B=2, Hq=8, Hkv=2, L=20, S=60, cap=64, D=128, scale=0.1,
             window=0, first=0, softcap=0.0, sinks=None, ws=A16)
    a.update(over)
    return tb.lib().tfa_kv4_prefill(*a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(q=None), tb.TFA_ERR_NULL),
    (dict(km=None), tb.TFA_ERR_NULL),
    (dict(ws=None), tb.TFA_ERR_NULL),
    (dict(Hq=7), tb.TFA_ERR_HEADS),
    (dict(L=0), tb.TFA_ERR_SHAPE),
    (dict(L=61), tb.TFA_ERR_SHAPE),
    (dict(S=65), tb.TFA_ERR_CACHE),
    (dict(D=96), tb.TFA_ERR_HEAD_DIM),
    (dict(first=4), tb.TFA_ERR_WINDOW),
    (dict(first=-1, window=3), tb.TFA_ERR_WINDOW),
    (dict(scale=float("inf")), tb.TFA_ERR_SCALE),
    (dict(softcap=float("nan")), tb.TFA_ERR_SOFTCAP),
    (dict(q=MIS), tb.TFA_ERR_ALIGN),
    (dict(ws=MIS), tb.TFA_ERR_ALIGN),
    (dict(B=1 << 10, Hkv=1 << 10, Hq=1 << 10, L=200, S=1 << 20, cap=1 << 20), tb.TFA_ERR_SHAPE),
])
def test_kv4_prefill_refusals(over, code):
    assert _chunk(**over) == code


def test_kv4_workspaces():
    size, few = tb.lib().tfa_kv4_prefill_workspace, tb.lib().tfa_kv4_decode_workspace(8, 2, 1, 128)
    assert size(2, 16, 4, 200, 1000, 128, 0, 0) == 2 * 4 * 1000 * 128 * 4
    assert size(2, 64, 4, 200, 1000, 64, 20, 5) == 2 * 4 * (5 + 219) * 64 * 4
    assert size(1, 64, 1, 200, 1000, 64, 20, 781) == 1000 * 64 * 4  # the first tokens meet the window
    assert size(1, 64, 1, 200, 1000, 64, 2 ** 31 - 1, 2 ** 31 - 1) == 1000 * 64 * 4
    assert size(1, 1, 1, 10, 9, 64, 20, 0) == 0
    # few rows: the kernel of tfa_kv4_decode and its pieces
    assert size(64, 32, 8, 16, 5000, 128, 0, 0) == few
    assert size(1, 32, 8, 32, 5000, 128, 0, 0) == few
    assert size(1, 1, 1, 200, 12000, 128, 0, 0) == few  # one item, which the dense kernel would cut for all SMs
    assert size(2, 16, 4, 200, 1000, 64, 20, 5) == tb.lib().tfa_kv4_decode_workspace(8, 2, 1, 64)
    assert size(1, 56, 8, 2048, 8192, 128, 0, 0) == 8 * 8192 * 128 * 4
    assert size(16, 32, 8, 32, 5000, 128, 0, 0) == 16 * 8 * 5000 * 128 * 4
    assert size(2000, 8, 8, 1, 10, 128, 0, 0) == 2000 * 8 * 10 * 128 * 4  # more sequences than it takes
    assert tb.lib().tfa_kv4_decode_workspace(8, 2, 1, 128) == 4 * 640 * 8 * 130 * 4
    assert tb.lib().tfa_kv4_decode_workspace(8, 0, 1, 128) == 0


def test_one_workspace_for_chunks_of_several_sizes():
    """A smaller chunk may need more than a larger one; _most covers them all."""
    size, most = tb.lib().tfa_kv4_prefill_workspace, tb.lib().tfa_kv4_prefill_workspace_most
    assert size(1, 8, 1, 2048, 2048, 64, 0, 0) < size(1, 8, 1, 5, 2048, 64, 0, 0) <= most(1, 8, 1, 2048, 2048, 64, 0, 0)
    r = random.Random(1)
    for _ in range(3000):
        B, Hkv, G, D = r.choice([1, 2, 16, 1500]), r.choice([1, 2, 8]), r.choice([1, 2, 4, 7]), r.choice([64, 128])
        W = r.choice([0, 0, 1, 128, 1024, 2 ** 31 - 1])
        F = r.choice([0, 1, 4, 300, 2 ** 31 - 1]) if W else 0
        L = r.randint(1, r.choice([8, 130, 4000]))
        S = L + r.randint(0, r.choice([1, 1000, 20000]))
        bound = most(B, G * Hkv, Hkv, L, S, D, W, F)
        for _ in range(5):
            l = r.randint(1, L)
            s = r.randint(l, S)
            assert size(B, G * Hkv, Hkv, l, s, D, W, F) <= bound, (B, G, Hkv, L, S, l, s, D, W, F)
    assert most(1, 1, 1, 10, 9, 64, 20, 0) == 0


def _longest(B, Hkv, G, L, S, window, first, sms, tiles, parts):
    """Steps of the CTA that is dealt the most, item by item in the kernel's snake order."""
    items = []
    for kt in range((S + 127) // 128):
        rc, lo, hi = tb.tfa_plan_ktile(L, S, True, 0 if kt * 128 < first else window, kt)
        assert rc == tb.TFA_OK
        n, into = max(0, hi - lo + 1), parts if kt < tiles else 1
        for i in range(into):
            items += [(n * (i + 1) // into - n * i // into) * G] * (B * Hkv)
    load = [0] * sms
    for x, w in enumerate(items):
        load[x % sms if x // sms % 2 == 0 else sms - 1 - x % sms] += w
    return max(load)


def test_first_cut_shortens_the_longest_cta_and_is_bounded():
    r = random.Random(2)
    cut = 0
    for _ in range(400):
        B, Hkv, G = r.choice([1, 2, 4, 9, 16, 64]), r.choice([1, 2, 8]), r.choice([1, 2, 4, 7])
        L = r.randint(1, r.choice([300, 2000, 9000]))
        S = L + r.choice([0, 0, r.randint(0, 4000)])
        window, first, sms = r.choice([1, 100, 128, 727, 1024, 4000]), r.choice([1, 4, 130, 512, 5000]), r.choice([148, 132, 60])
        rc, tiles, parts = tb.tfa_plan_first_cut(B, G * Hkv, Hkv, L, S, window, first, sms)
        assert rc == tb.TFA_OK and (tiles > 0) == (parts > 1)
        assert B * Hkv * tiles * parts <= 4 * sms
        if tiles:
            cut += 1
            a, b = (_longest(B, Hkv, G, L, S, window, min(first, S), sms, *c) for c in ((0, 1), (tiles, parts)))
            assert b + 3 < a, (B, Hkv, G, L, S, window, first, sms)
    assert cut > 100


def test_first_cut_of_known_shapes():
    plan = tb.tfa_plan_first_cut
    assert plan(1, 32, 8, 4096, 4096, 1024, 4, 148) == (tb.TFA_OK, 1, 4)  # a training step of one sequence
    # enough items to even out: nothing to save, whatever the window
    for B, first in ((16, 4), (64, 4), (64, 512)):
        for L in (4096, 8192):
            assert plan(B, 32, 8, L, L, 128, first, 148) == (tb.TFA_OK, 0, 1)
    assert plan(1, 7, 1, 1236, 1692, 727, 85, 148)[1] == 14  # few key tiles: all of them
    assert plan(1, 8, 2, 300, 300, 100, 0, 148) == (tb.TFA_OK, 0, 1)
    assert plan(1, 8, 2, 300, 300, 0, 4, 148)[0] == tb.TFA_ERR_WINDOW
    assert plan(1, 8, 2, 300, 300, 9, -1, 148)[0] == tb.TFA_ERR_WINDOW
    assert plan(1, 8, 2, 300, 300, 9, 4, 0)[0] == tb.TFA_ERR_SHAPE
    assert plan(1, 8, 3, 300, 300, 9, 4, 148)[0] == tb.TFA_ERR_HEADS


@pytest.mark.parametrize("how", ["missing", "another torch"])
def test_the_library_loads_without_its_native_calls(how, monkeypatch):
    """Everything that does not need them works, and says what is not there."""
    import sys

    import sliding_window_gqa_tfa_b200 as package
    import torch

    tb.lib()
    assert tb._calls is not None
    monkeypatch.setattr(tb, "_lib", None)
    monkeypatch.setattr(tb, "_calls", None)
    if how == "missing":
        monkeypatch.delattr(package, "_calls")
        monkeypatch.setitem(sys.modules, package.__name__ + "._calls", None)
    else:
        monkeypatch.setattr(torch, "__version__", "1.0")
    with pytest.warns(RuntimeWarning, match="_calls.so"):
        tb.lib()
    assert tb._calls is None
    assert tb.tfa_plan_ktile(200, 300, True, 0, 0) == (tb.TFA_OK, 0, 1)
    assert tb.tfa_plan_first_cut(1, 32, 8, 4096, 4096, 1024, 4, 148) == (tb.TFA_OK, 1, 4)
    assert _chunk(L=0) == tb.TFA_ERR_SHAPE
    with pytest.raises(ValueError, match="CUDA"):
        tb.prefill(*[torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16)] * 3, window=4, first=1)


@pytest.mark.parametrize("rot,base,factor,original", [(128, 1e6, 4.0, 8192), (64, 1e4, 32.0, 4096), (128, 5e5, 8.0, 32768),
                                                      (16, 1e4, 2.5, 100)])
def test_scaled_frequencies_pair_by_pair(rot, base, factor, original):
    """yarn: a ramp over the pairs' indexes between the whole indexes around the pairs of
    32 turns and of 1 turn in the original positions; llama3: over the wavelengths."""
    import math

    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    lo, hi = (rot * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (32, 1))
    lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
    got, mscale = tb.rope_inv_freq(rot, base, scaling="yarn", factor=factor, original=original, device="cpu")
    assert mscale == pytest.approx(0.1 * math.log(factor) + 1)
    for i, x in enumerate(got.tolist()):
        ramp = min(max((i - lo) / (hi - lo), 0.0), 1.0)
        assert x == pytest.approx(f[i] / factor * ramp + f[i] * (1 - ramp), rel=1e-12)
    got, mscale = tb.rope_inv_freq(rot, base, scaling="llama3", factor=factor, original=original, device="cpu")
    assert mscale == 1.0
    for i, x in enumerate(got.tolist()):
        wave = 2 * math.pi / f[i]
        if wave < original / 4:
            want = f[i]
        elif wave > original:
            want = f[i] / factor
        else:
            smooth = (original / wave - 1) / 3
            want = (1 - smooth) * f[i] / factor + smooth * f[i]
        assert x == pytest.approx(want, rel=1e-12)


def test_yarn_needs_a_base_above_one():
    with pytest.raises(ValueError):
        tb.rope_inv_freq(16, 1.0, scaling="yarn", factor=2.0, device="cpu")
    assert tb.rope_inv_freq(0, 1e4, scaling="yarn", factor=2.0, device="cpu")[0].numel() == 0


@pytest.mark.parametrize("B,Hq,Hkv,L,S,D,few", [
    # measured on both kernels, us: few rows, dense
    (16, 28, 4, 30, 159, 128, False),  # 48, 16
    (4, 64, 4, 125, 230, 64, False),  # 69, 21
    (16, 64, 4, 11, 97, 64, False),  # many pieces of three steps
    (16, 64, 8, 8, 311, 128, False),
    (1, 32, 8, 32, 5000, 128, True),  # 28, 76
    (1, 1, 1, 200, 12000, 128, True),  # 18, 446
    (1, 32, 4, 32, 8000, 64, True),
    (16, 8, 8, 1, 60, 128, True),
    (16, 64, 8, 1, 60, 64, True),
])
def test_which_chunks_take_the_kernel_for_few_rows(B, Hq, Hkv, L, S, D, few):
    size = tb.lib().tfa_kv4_prefill_workspace(B, Hq, Hkv, L, S, D, 0, 0)
    assert size == (tb.lib().tfa_kv4_decode_workspace(Hq, Hkv, L, D) if few else B * Hkv * S * D * 4)


@pytest.mark.parametrize("back", [False, True])
def test_rope_refuses_outputs_whose_rows_share_a_place(back):
    import struct

    n, out = (18, 12) if back else (12, 6)
    for i in range(out, n):
        for size in (1, 2):
            s = [1 << 20, 4096, 128] * (n // 3)
            s[i] = 0
            dims = [2, 2, 2]
            dims[(i - out) % 3] = size
            args = [struct.pack(f"{n}q", *s), A16, A16, A16, ctypes.c_void_p(0x10002), 0, 0, *dims, dims[2], 128, 64, 0, 1e-6, 1.0]
            lib = tb.lib()
            rc = (lib.tfa_qk_norm_rope_backward(*[A16] * 8, *args, A16, None) if back
                  else lib.tfa_qk_norm_rope(*[A16] * 4, *args, None))
            assert rc == (tb.TFA_ERR_SHAPE if size == 2 else tb.TFA_ERR_ALIGN)  # (else the positions are refused)
