"""Refusals of the long-context operators, before any CUDA call: the pointers here
are never dereferenced."""
import ctypes

import pytest

from sliding_window_gqa_tfa_b200 import binding as tb

A16 = ctypes.c_void_p(0x10000)
MIS = ctypes.c_void_p(0x10008)


def _strides(n, odd=None):
    s = [1 << 20, 4096, 128] * (n // 3)
    if odd is not None:
        s[odd] += 4
    return (ctypes.c_longlong * n)(*s)


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
    assert tb.lib().tfa_qk_norm_rope_workspace(128) == 592 * 2 * 128 * 4


def test_rope_inv_freq_refusals():
    for a in (dict(rot=7), dict(rot=-2), dict(rot=16, scaling="other"), dict(rot=16, factor=0.0)):
        with pytest.raises(ValueError):
            tb.rope_inv_freq(device="cpu", **a)
