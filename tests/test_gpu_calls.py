"""The native calls (csrc/calls.cpp) against the wrappers' Python code, which makes the
same C calls: the same bits, the same refusals, and None where a call is not theirs."""
import pytest
import torch

from sliding_window_gqa_tfa_b200 import binding as tb

D, B, HQ, HKV, L, CAP = 64, 3, 4, 2, 2, 70


def _rows(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).bfloat16()


def _calls(device):
    """name -> (a wrapper's call, given what overrides its tensors)."""
    on = lambda t: t.to(device)
    q, k = on(_rows(0, B, L, HQ, D)), on(_rows(1, B, L, HKV, D))
    w = on(_rows(2, D))
    freq, _ = tb.rope_inv_freq(D, device=device)
    pos = on(torch.tensor([0, 5, 900], dtype=torch.int32))
    dq, dk = on(_rows(3, B, HQ, L, D)), on(_rows(4, B, HKV, L, D))
    ck, cv = on(_rows(5, B, HKV, CAP, D)), on(_rows(6, B, HKV, CAP, D))
    lens = on(torch.tensor([CAP, 0, 33], dtype=torch.int32))
    long, long2 = on(_rows(8, B, HQ, 40, D)), on(_rows(9, B, HQ, 40, D))
    sinks = on(torch.randn(HQ, generator=torch.Generator().manual_seed(7)))

    def cache():
        c = tb.kv4_cache(B, HKV, CAP, D, device=device)
        tb.kv4_append(ck, cv, *c, start=0)
        return c

    def append():
        c = tb.kv4_cache(B, HKV, CAP, D, device=device)
        tb.kv4_append(ck[:, :, :L], cv[:, :, :L], *c, start=pos.clamp(max=CAP - L))
        return c

    return {
        "rope": lambda: tb.qk_norm_rope(q, k, pos, freq, q_weight=w, k_weight=w),
        "rope_plain": lambda: tb.qk_norm_rope(q, k, 17, freq, interleaved=True, mscale=1.25),
        "rope_per_row": lambda: tb.qk_norm_rope(q, k, pos[:, None].expand(B, L).contiguous(), freq),
        "backward": lambda: tb.qk_norm_rope_backward(dq, dk, q, k, pos, freq, q_weight=w, k_weight=w),
        "append": append,
        "read": lambda: tb.kv4_read(*cache(), start=pos.clamp(max=40), rows=9),
        "read_rest": lambda: tb.kv4_read(*cache(), start=60),
        "decode": lambda: tb.kv4_decode(dq, *cache(), lens, window=20, first=3, sinks=sinks),
        "decode_scaled": lambda: tb.kv4_decode(dq, *cache(), lens, scale=-0.25, softcap=9),
        "prefill": lambda: tb.kv4_prefill(dq, *cache(), S=61, window=20, first=3, softcap=5.0),
        "prefill_long": lambda: tb.kv4_prefill(long, *cache(), S=CAP),
        "first_backward": lambda: tb.backward(long, ck, cv, long2, window=16, first=4,
                                              saved=tb.prefill_lse(long, ck, cv, window=16, first=4)),
        "first": lambda: tb.prefill(dq, ck, cv, window=16, first=4, sinks=sinks),
        "first_lse": lambda: tb.prefill_lse(dq, ck, cv, window=16, first=4),
    }


@pytest.mark.gpu
@pytest.mark.parametrize("name", sorted(_calls("cpu")))
def test_native_calls_give_the_python_codes_bits(name, monkeypatch):
    call = _calls("cuda")[name]
    tb.lib()
    taken, native = [], tb._calls

    class Recorded:
        def __getattr__(self, attr):
            def f(*a):
                r = getattr(native, attr)(*a)
                taken.append(r is not None)
                return r
            return f

    monkeypatch.setattr(tb, "_calls", Recorded())
    a = call()
    # kv4_read without its rows is the Python code's
    assert taken and (all(taken) or name == "read_rest")
    monkeypatch.setattr(tb, "_calls", None)
    b = call()
    a, b = (x if isinstance(x, tuple) else (x,) for x in (a, b))
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert x.dtype == y.dtype and x.shape == y.shape and x.stride() == y.stride()
        bits = torch.int32 if x.dtype == torch.float32 else torch.int16 if x.dtype == torch.bfloat16 else x.dtype
        assert torch.equal(x.view(bits), y.view(bits))


def test_native_calls_leave_host_tensors_and_wrong_arguments_alone():
    tb.lib()
    q = _rows(0, 1, 1, 1, D)
    assert tb._calls.rope(q, q, 0, q, None, None, 1e-6, False, 1.0, None, None) is None
    assert tb._calls.rope(*[None] * 11) is None
    assert tb._calls.rope_backward(*["x"] * 11) is None
    assert tb._calls.append(*[q] * 7) is None
    assert tb._calls.read(q, q, q, q, 0, 1) is None
    assert tb._calls.decode(*[q] * 13) is None
    assert tb._calls.prefill(*[q] * 13) is None
    assert tb._calls.prefill_first(*[q] * 12) is None
    assert tb._calls.backward_first(*[q] * 10) is None
    with pytest.raises(TypeError):
        tb._calls.rope(q)


@pytest.mark.gpu
def test_native_calls_pass_statuses_and_refusals_on():
    dev = "cuda"
    tb.lib()
    q, k = _rows(0, B, L, HQ, D).to(dev), _rows(1, B, L, HKV, D).to(dev)
    freq, _ = tb.rope_inv_freq(24, device=dev)  # 24 channels: no multiple of 16
    with pytest.raises(tb.TfaError) as e:
        tb.qk_norm_rope(q, k, 0, freq)
    assert e.value.code == tb.TFA_ERR_ROPE
    freq, _ = tb.rope_inv_freq(D, device=dev)
    with pytest.raises(tb.TfaError) as e:  # eps refused by the C call
        tb.qk_norm_rope_backward(q.transpose(1, 2), k.transpose(1, 2), q, k, 0, freq,
                                 q_weight=q[0, 0, 0], k_weight=k[0, 0, 0], eps=-1.0)
    assert e.value.code == tb.TFA_ERR_ROPE
    cache = tb.kv4_cache(B, HKV, CAP, D, device=dev)
    rows = k.transpose(1, 2)
    with pytest.raises(tb.TfaError):  # past the capacity
        tb.kv4_append(rows, rows, *cache, start=CAP - 1)
    with pytest.raises(tb.TfaError):
        tb.kv4_decode(q.transpose(1, 2).contiguous(), *cache, torch.zeros(B, dtype=torch.int32, device=dev), first=1)
    with pytest.raises(ValueError):  # the Python code's refusal
        tb.kv4_decode(q.transpose(1, 2).contiguous(), *cache, torch.zeros(B + 1, dtype=torch.int32, device=dev))
    with pytest.raises(tb.TfaError):
        tb.prefill(q.transpose(1, 2).contiguous(), rows.contiguous(), rows.contiguous(), window=0, first=2)


@pytest.mark.gpu
def test_integers_that_do_not_fit_are_refused():
    """A C call's int would drop their upper bits: start 2^32 would write row 0."""
    c = tb.kv4_cache(1, 1, 64, D, device="cuda")
    rows, freq = _rows(0, 1, 1, 2, D).cuda(), tb.rope_inv_freq(D, device="cuda")[0]
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    big = 2 ** 32 + 5
    for call in (lambda: tb.kv4_append(rows, rows, *c, start=big), lambda: tb.kv4_read(*c, start=big, rows=1),
                 lambda: tb.kv4_read(*c, rows=big), lambda: tb.kv4_decode(rows, *c, lens, window=big),
                 lambda: tb.kv4_decode(rows, *c, lens, window=9, first=big),
                 lambda: tb.kv4_prefill(rows, *c, S=big), lambda: tb.qk_norm_rope(rows, rows, -big, freq),
                 lambda: tb.prefill(rows, rows, rows, window=big, first=2),
                 lambda: tb.prefill_lse(rows, rows, rows, window=4, first=big)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_native_calls_on_a_stream_that_is_current():
    """The current stream is the one a call runs on, and the one its outputs belong to."""
    call = _calls("cuda")["decode"]
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call()
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    q, c = _rows(8, B, HQ, L, D).cuda(), tb.kv4_cache(B, HKV, CAP, D, device="cuda")
    lens = torch.full((B,), CAP, dtype=torch.int32, device="cuda")
    tb.kv4_decode(q, *c, lens)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = tb.kv4_decode(q, *c, lens)
    rows = _rows(9, B, HKV, CAP, D).cuda()
    tb.kv4_append(rows, rows, *c, start=0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, tb.kv4_decode(q, *c, lens))


def _step(q, k, v, w, freq, cache, lens, window, first):
    """A decoding step in one stream: its kernels start while the ones before them end."""
    qr, kr = tb.qk_norm_rope(q, k, lens, freq, q_weight=w, k_weight=w)
    tb.kv4_append(kr, v, *cache, start=lens)
    return tb.kv4_decode(qr, *cache, lens + 1, window=window, first=first)


@pytest.mark.gpu
def test_a_chain_of_calls_needs_no_synchronisation():
    """Steps whose lengths and rows are written just before them, by slow kernels, with
    and without a wait between any two calls: the same bits."""
    g = torch.Generator(device="cuda").manual_seed(5)
    n, hq, hkv, cap, d = 4, 8, 2, 3000, 128
    freq, _ = tb.rope_inv_freq(d, device="cuda")
    w = torch.randn(d, generator=g, device="cuda").bfloat16()
    slow = torch.randn(4096, 4096, generator=g, device="cuda")
    base = torch.tensor([2900, 1, 700, 1500], dtype=torch.int32, device="cuda")
    rows = torch.randn(12, n, 1, hq + 2 * hkv, d, generator=g, device="cuda").bfloat16()

    def run(wait):
        cache = tb.kv4_cache(n, hkv, cap, d, device="cuda")
        lens, outs = torch.zeros_like(base), []
        qkv = torch.empty_like(rows[0])
        for i in range(12):
            slow @ slow  # keeps the stream busy while the next calls are made
            qkv.copy_(rows[i])
            lens.copy_(base + i)
            q, k, v = qkv.split([hq, hkv, hkv], dim=2)
            v = v.transpose(1, 2)
            if wait:
                torch.cuda.synchronize()
                qr, kr = tb.qk_norm_rope(q, k, lens, freq, q_weight=w, k_weight=w)
                torch.cuda.synchronize()
                tb.kv4_append(kr, v, *cache, start=lens)
                torch.cuda.synchronize()
                outs.append(tb.kv4_decode(qr, *cache, lens + 1, window=1000, first=4))
                torch.cuda.synchronize()
            else:
                outs.append(_step(q, k, v, w, freq, cache, lens, 1000, 4))
        return torch.stack(outs)

    want = run(True)
    for _ in range(3):
        assert torch.equal(run(False), want)


@pytest.mark.gpu
def test_training_calls_back_to_back():
    """Norms, windowed attention with first tokens and all gradients, call after call."""
    g = torch.Generator(device="cuda").manual_seed(6)
    b, hq, hkv, n, d = 1, 4, 2, 500, 128
    freq, _ = tb.rope_inv_freq(d, device="cuda")
    q0, k0, do = (torch.randn(b, n, h, d, generator=g, device="cuda").bfloat16() for h in (hq, hkv, hq))
    v = torch.randn(b, hkv, n, d, generator=g, device="cuda").bfloat16()
    do = do.transpose(1, 2).contiguous()
    w = torch.randn(d, generator=g, device="cuda").bfloat16()

    def run(wait):
        pause = torch.cuda.synchronize if wait else lambda: None
        q, k = tb.qk_norm_rope(q0, k0, 0, freq, q_weight=w, k_weight=w)
        pause()
        saved = tb.prefill_lse(q, k, v, window=100, first=4)
        pause()
        dq, dk, dv = tb.backward(q, k, v, do, window=100, first=4, saved=saved)
        pause()
        return (*tb.qk_norm_rope_backward(dq, dk, q0, k0, 0, freq, q_weight=w, k_weight=w), dv, saved[0])

    want = run(True)
    for _ in range(5):
        for x, y in zip(run(False), want):
            assert torch.equal(x, y)


@pytest.mark.gpu
def test_calls_on_two_streams_captured_into_one_graph():
    """A captured fork and join: each call waits for what it needs, on either stream."""
    g = torch.Generator(device="cuda").manual_seed(7)
    d, cap, n = 64, 200, 3
    freq, _ = tb.rope_inv_freq(d, device="cuda")
    q, k, v = (torch.randn(n, 1, h, d, generator=g, device="cuda").bfloat16() for h in (4, 2, 2))
    w = torch.randn(d, generator=g, device="cuda").bfloat16()
    lens = torch.tensor([100, 0, 150], dtype=torch.int32, device="cuda")
    caches = [tb.kv4_cache(n, 2, cap, d, device="cuda") for _ in range(3)]
    want = _step(q, k, v.transpose(1, 2), w, freq, caches[2], lens, 50, 2)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        kept = [q.clone(), k.clone()]
        side.wait_stream(here)
        with torch.cuda.stream(side):
            a = _step(*kept, v.transpose(1, 2), w, freq, caches[0], lens, 50, 2)
        b = _step(*kept, v.transpose(1, 2), w, freq, caches[1], lens, 50, 2)
        here.wait_stream(side)
        both = torch.stack([a, b])
        last = tb.kv4_decode(both[0], *caches[1], lens + 1, window=50, first=2)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(both[0], want) and torch.equal(both[1], want)
        assert torch.equal(last, tb.kv4_decode(want, *caches[2], lens + 1, window=50, first=2))


@pytest.mark.gpu
def test_strides_of_single_rows_do_not_count():
    """A dimension of size 1 has a stride that no address uses."""
    freq, _ = tb.rope_inv_freq(D, device="cuda")
    q, k = _rows(0, 1, 1, 4, D).cuda(), _rows(1, 1, 1, 1, D).cuda()
    want = tb.qk_norm_rope(q, k, 3, freq)
    odd = lambda t: t.as_strided(t.shape, [3 if n == 1 else s for n, s in zip(t.shape, t.stride())])
    got = tb.qk_norm_rope(odd(q), odd(k), 3, freq, q_out=odd(torch.empty_like(want[0])), k_out=odd(torch.empty_like(want[1])))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    cache, other = (tb.kv4_cache(1, 1, 4, D, device="cuda") for _ in range(2))
    tb.kv4_append(k, k, *cache, start=1)
    tb.kv4_append(odd(k), odd(k), *other, start=1)
    assert all(torch.equal(a, b) for a, b in zip(cache, other))


@pytest.mark.gpu
def test_numbers_of_numpy_and_of_torch(monkeypatch):
    """Sizes, scales and flags as prefill takes them: numpy's numbers and one-element
    tensors beside Python's, on both ways into the library."""
    np = pytest.importorskip("numpy")
    q, k = _rows(0, 1, 40, 4, D).cuda(), _rows(1, 1, 40, 2, D).cuda()
    freq, _ = tb.rope_inv_freq(D, device="cuda")
    w = _rows(2, D).cuda()
    qh, kh = q.transpose(1, 2).contiguous(), k.transpose(1, 2).contiguous()
    one = tb.kv4_cache(1, 2, 64, D, device="cuda")
    lens = torch.full((1,), 40, dtype=torch.int32, device="cuda")

    def run(i, f, t):
        tb.kv4_append(kh, kh, *one, start=i(3))
        saved = tb.prefill_lse(qh, kh, kh, window=i(9), first=i(2), scale=f(0.25))
        return [*tb.qk_norm_rope(q, k, i(5), freq, q_weight=w, k_weight=w, eps=f(1e-5), interleaved=t(True), mscale=f(0.5)),
                *tb.qk_norm_rope_backward(qh, kh, q, k, i(5), freq, q_weight=w, k_weight=w, eps=f(1e-5), interleaved=t(True)),
                *tb.kv4_read(*one, start=i(3), rows=i(7)), *saved,
                tb.kv4_decode(qh[:, :, :2].contiguous(), *one, lens, window=i(9), first=i(2), scale=f(0.25), softcap=f(3.0)),
                tb.kv4_prefill(qh, *one, S=i(43), window=i(9), first=i(2), scale=f(0.25), softcap=f(3.0)),
                tb.prefill(qh, kh, kh, window=i(9), first=i(2), softcap=f(3.0)),
                *tb.backward(qh, kh, kh, qh, window=i(9), first=i(2), scale=f(0.25), saved=saved)]

    want = run(int, float, bool)
    tb.lib()
    for native in (tb._calls, None):
        monkeypatch.setattr(tb, "_calls", native)
        for i, f, t in ((np.int64, np.float32, np.bool_), (np.int32, np.float64, bool),
                        (int, lambda x: torch.tensor(x, dtype=torch.float64), bool)):
            for a, b in zip(want, run(i, f, t)):
                # (numpy's float32 rounds 1e-5 as the C call does)
                assert torch.equal(a, b)


@pytest.mark.gpu
def test_a_flag_without_a_truth_value_is_refused():
    q, k = _rows(0, 1, 2, 4, D).cuda(), _rows(1, 1, 2, 2, D).cuda()
    freq, _ = tb.rope_inv_freq(D, device="cuda")
    flag = torch.ones(2)  # bool() of it raises
    with pytest.raises(RuntimeError):
        tb.qk_norm_rope(q, k, 0, freq, interleaved=flag)
    with pytest.raises(RuntimeError):
        tb.qk_norm_rope_backward(q.transpose(1, 2), k.transpose(1, 2), q, k, 0, freq, q_weight=q[0, 0, 0],
                                 k_weight=k[0, 0, 0], interleaved=flag)


@pytest.mark.gpu
def test_read_refuses_before_it_allocates(monkeypatch):
    c = tb.kv4_cache(1, 1, 64, D, device="cuda")
    tb.lib()
    for native in (tb._calls, None):
        monkeypatch.setattr(tb, "_calls", native)
        for kw, code in ((dict(start=0, rows=2 ** 31 - 1), tb.TFA_ERR_CACHE), (dict(start=60, rows=5), tb.TFA_ERR_CACHE),
                         (dict(start=-1, rows=1), tb.TFA_ERR_CACHE), (dict(start=65), tb.TFA_ERR_SHAPE),
                         (dict(start=0, rows=0), tb.TFA_ERR_SHAPE), (dict(start=0, rows=-4), tb.TFA_ERR_SHAPE)):
            torch.cuda.reset_peak_memory_stats()
            before = torch.cuda.memory_allocated()
            with pytest.raises(tb.TfaError) as e:
                tb.kv4_read(*c, **kw)
            assert e.value.code == code and torch.cuda.max_memory_allocated() == before
