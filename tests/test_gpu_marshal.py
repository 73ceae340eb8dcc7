"""The binding's two ways of marshalling a call (the extension, and Python where
it is absent or declines): the same results, and the same refusals."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_mm_gb300 as mm
import mixture_experts_layer_mm_gb300._lib as binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(mmlib):
    if binding._fast is None:
        pytest.skip("the extension is not built")
    return mmlib


def _calls():
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(300, 24, generator=g, device="cuda")
    mask = torch.rand(300, generator=g, device="cuda") > 0.3
    dw = torch.randn(300, 3, generator=g, device="cuda")
    dl = torch.ones(1, device="cuda")
    ids, w, counts, _, _ = mm.mm_route_logits(x, 3, True)
    m2 = torch.randn(70, 96, generator=g, device="cuda")
    m3 = torch.randn(3, 70, 96, generator=g, device="cuda").to(torch.float16)
    q2, q3 = mm.mm_mxfp4_quantize(m2), mm.mm_mxfp4_quantize(m3)
    T, H, E, I, k = 9, 128, 24, 64, 3
    hid = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    gu = mm.mm_mxfp4_quantize(torch.randn(2 * E, I, H, generator=g, device="cuda"))
    dn = mm.mm_mxfp4_quantize(torch.randn(E, H, I, generator=g, device="cuda"))
    some = (ids[:T].contiguous(), w[:T].contiguous())
    ws = torch.empty(mm.mm_moe_experts_mxfp4_workspace_size(T, H, E, I, k), dtype=torch.uint8,
                     device="cuda")
    out = torch.empty_like(hid)
    return {
        "route": lambda: mm.mm_route_logits(x, 3, True),
        "route masked": lambda: mm.mm_route_logits(x.to(torch.bfloat16), 2, False, token_mask=mask),
        "backward": lambda: mm.mm_route_logits_backward(x, ids, counts, True, dw, dl),
        "backward masked": lambda: mm.mm_route_logits_backward(
            x.to(torch.bfloat16), ids, counts, False, d_loss=dl, token_mask=mask.to(torch.uint8)),
        "quantise": lambda: mm.mm_mxfp4_quantize(m2),
        "quantise batch": lambda: mm.mm_mxfp4_quantize(m3),
        "dequantise": lambda: mm.mm_mxfp4_dequantize(*q2, dtype=torch.float32),
        "dequantise batch": lambda: mm.mm_mxfp4_dequantize(*q3),
        "product": lambda: mm.mm_mxfp4_gemm(*q2, q3[0][1:2], q3[1][1:2]),
        "product fp32": lambda: mm.mm_mxfp4_gemm(*q2, *q2, out_dtype=torch.float32),
        "experts": lambda: mm.mm_moe_experts_mxfp4(hid, *some, *gu, *dn),
        "experts given": lambda: mm.mm_moe_experts_mxfp4(
            hid, *some, gu[0].view(E, 2 * I, H // 2), gu[1], *dn, out=out, workspace=ws).clone(),
        "no tokens": lambda: mm.mm_route_logits(x[:0], 3, True),
        "no rows": lambda: mm.mm_mxfp4_quantize(m2[:0]),
    }


NAMES = ["route", "route masked", "backward", "backward masked", "quantise", "quantise batch",
         "dequantise", "dequantise batch", "product", "product fp32", "experts", "experts given",
         "no tokens", "no rows"]


@pytest.mark.parametrize("name", NAMES)
def test_both_ways_agree(name, monkeypatch):
    call = _calls()[name]
    declined = []

    class Spy:  # the extension, with a note of the calls it declines
        def __getattr__(self, fn):
            def f(*a):
                r = getattr(binding_fast, fn)(*a)
                if r is None:
                    declined.append(fn)
                return r
            return f

    binding_fast = binding._fast
    monkeypatch.setattr(binding, "_fast", Spy())
    fast = call()
    assert not declined
    monkeypatch.setattr(binding, "_fast", None)
    slow = call()
    fast, slow = (r if isinstance(r, tuple) else (r,) for r in (fast, slow))
    assert len(fast) == len(slow)
    for a, b in zip(fast, slow):
        assert a.dtype == b.dtype and a.shape == b.shape and a.device == b.device
        assert torch.equal(a, b)


def test_declined_calls_raise_as_in_python(monkeypatch):
    x = torch.randn(8, 64, device="cuda")
    q = mm.mm_mxfp4_quantize(x)
    ids, w, counts, _, _ = mm.mm_route_logits(x, 2, True)
    bad = [
        lambda: mm.mm_route_logits(x, 65, True), lambda: mm.mm_route_logits(x, 0, True),
        lambda: mm.mm_route_logits(x.half(), 2, True), lambda: mm.mm_route_logits(x.cpu(), 2, True),
        lambda: mm.mm_route_logits(x.t(), 2, True), lambda: mm.mm_route_logits(3, 2, True),
        lambda: mm.mm_route_logits(x, 2, True, token_mask=torch.ones(7, device="cuda").bool()),
        lambda: mm.mm_route_logits(x, 2, True, token_mask=torch.ones(8, device="cuda")),
        lambda: mm.mm_route_logits(x, "2", True),
        lambda: mm.mm_route_logits_backward(x, ids.long(), counts, True),
        lambda: mm.mm_route_logits_backward(x, ids, counts[:5], True),
        lambda: mm.mm_route_logits_backward(x, ids, counts, True, d_topk_w=w[:, :1]),
        lambda: mm.mm_route_logits_backward(x, ids, counts, True, d_loss=torch.ones(2).cuda()),
        lambda: mm.mm_mxfp4_quantize(x[:, :40].contiguous()),
        lambda: mm.mm_mxfp4_quantize(x[:, ::2]), lambda: mm.mm_mxfp4_quantize(x.double()),
        lambda: mm.mm_mxfp4_quantize(x[0]),
        lambda: mm.mm_mxfp4_dequantize(q[0], q[1][:, :, :256]),
        lambda: mm.mm_mxfp4_dequantize(*q, dtype=torch.int32),
        lambda: mm.mm_mxfp4_gemm(*q, *mm.mm_mxfp4_quantize(x[:, :32].contiguous())),
        lambda: mm.mm_mxfp4_gemm(*q, *q, out_dtype=torch.float16),
        lambda: mm.mm_moe_experts_mxfp4(x, ids, w, *q, *q),
        lambda: mm.mm_moe_experts_mxfp4(x.bfloat16(), ids, w, q[0][None], q[1][None], q[0][None],
                                        q[1][None]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(Exception) as fast:
            call()
        with monkeypatch.context() as m:
            m.setattr(binding, "_fast", None)
            with pytest.raises(Exception) as slow:
                call()
        assert (type(fast.value), str(fast.value)) == (type(slow.value), str(slow.value)), i
    torch.cuda.synchronize()
    assert mm.mm_poll_device_status() == mm.MM_OK


def test_results_are_the_callers():
    # Results are ordinary tensors: they survive the inputs, and the current
    # stream of the moment is the one that is used.
    side = torch.cuda.Stream()
    x = torch.randn(64, 256, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        c, s = mm.mm_mxfp4_quantize(x)
        v = mm.mm_mxfp4_dequantize(c, s, torch.float32)
    side.synchronize()
    want = mm.mm_mxfp4_dequantize(*mm.mm_mxfp4_quantize(x), dtype=torch.float32)
    assert torch.equal(v, want)
    keep = [mm.mm_route_logits(torch.randn(5, 8, device="cuda"), 2, True) for _ in range(50)]
    assert all(int(r[2].sum()) == 10 for r in keep)
    assert np.isfinite([float(r[4]) for r in keep]).all()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 5, 3), (65, 70, 7), (300, 256, 8)])
def test_results_of_one_allocation_are_apart(T, E, k):
    x = torch.randn(T, E, device="cuda")
    got = mm.mm_route_logits(x, k, True)
    assert all(t.data_ptr() % 16 == 0 and t.is_contiguous() for t in got)
    for i, t in enumerate(got):
        before = [u.clone() for u in got]
        t.fill_(77)
        assert all(torch.equal(u, b) for j, (u, b) in enumerate(zip(got, before)) if j != i)
        t.copy_(before[i])
    # and each goes on living without the others, and as an input
    ids, w = got[0], got[1]
    counts, loss = got[2].clone(), got[4]
    del got
    g = mm.mm_route_logits_backward(x, ids, counts, True, w, loss)
    torch.cuda.synchronize()
    assert torch.isfinite(g).all() and w.shape == (T, k)


def _on_a_stream():
    """Calls that take stream=, by name, with inputs that stay."""
    g = torch.Generator(device="cuda").manual_seed(11)
    x = torch.randn(40000, 64, generator=g, device="cuda")
    dw = torch.randn(40000, 6, generator=g, device="cuda")
    ids, w, counts, _, _ = mm.mm_route_logits(x, 6, True)
    m = torch.randn(2048, 2048, generator=g, device="cuda")
    q = mm.mm_mxfp4_quantize(m)
    T, H, E, I, k = 700, 256, 16, 128, 4
    hid = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    gu = mm.mm_mxfp4_quantize(torch.randn(2 * E, I, H, generator=g, device="cuda"))
    dn = mm.mm_mxfp4_quantize(torch.randn(E, H, I, generator=g, device="cuda"))
    some = mm.mm_route_logits(x[:T, :E].contiguous(), k, True)[:2]
    return {
        "route": lambda s=None: mm.mm_route_logits(x, 6, True, stream=s),
        "backward": lambda s=None: mm.mm_route_logits_backward(x, ids, counts, True, dw, stream=s),
        "quantise": lambda s=None: mm.mm_mxfp4_quantize(m, stream=s),
        "dequantise": lambda s=None: mm.mm_mxfp4_dequantize(*q, stream=s),
        "product": lambda s=None: mm.mm_mxfp4_gemm(*q, *q, stream=s),
        "experts": lambda s=None: mm.mm_moe_experts_mxfp4(hid, *some, *gu, *dn, stream=s),
    }


STREAM_CALLS = ["route", "backward", "quantise", "dequantise", "product", "experts"]


def _tuple(r):
    return r if isinstance(r, tuple) else (r,)


@pytest.mark.parametrize("by_handle", [False, True])
@pytest.mark.parametrize("name", STREAM_CALLS)
def test_results_on_a_given_stream_share_no_memory_in_use(name, by_handle):
    # Memory that the current stream has freed, but still writes: a call on a
    # stream of its own does not wait for those writes, so it may not take it.
    call = _on_a_stream()[name]
    want = [t.clone() for t in _tuple(call())]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.empty(t.numel() * t.element_size(), dtype=torch.uint8, device="cuda")
              for t in want]
    torch.cuda._sleep(200_000_000)
    for b in blocks:
        b.fill_(0x5A)
    del blocks, b
    got = _tuple(call(side.cuda_stream if by_handle else side))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert mm.mm_poll_device_status() == mm.MM_OK


@pytest.mark.parametrize("name", STREAM_CALLS)
def test_results_of_a_given_stream_outlive_their_readers(name):
    # Freed while the current stream still reads them: the next call on the
    # given stream takes other memory.
    call = _on_a_stream()[name]
    want = [t.clone() for t in _tuple(call())]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    cur = torch.cuda.current_stream()
    got = _tuple(call(side))
    cur.wait_stream(side)
    torch.cuda._sleep(200_000_000)
    copies = [t.clone() for t in got]
    del got
    for _ in range(3):  # other values into whatever the side stream's memory is
        with torch.cuda.stream(side):
            for t in want:
                torch.empty(t.numel() * t.element_size(), dtype=torch.uint8,
                            device="cuda").fill_(0x5A)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want))


@pytest.mark.parametrize("name", STREAM_CALLS)
def test_a_given_stream_inside_a_capture(name):
    call = _on_a_stream()[name]
    want = [t.clone() for t in _tuple(call())]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cur = torch.cuda.current_stream()
        side.wait_stream(cur)
        got = _tuple(call(side))
        cur.wait_stream(side)
        out = [t.clone() for t in got]
        same = _tuple(call(cur))
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for r in (out, same):
        assert all(torch.equal(a, b) for a, b in zip(r, want))


@pytest.mark.parametrize("top_k", [9, 33, 1 << 20, 1 << 30, (1 << 31) - 1, 1 << 31, 1 << 70])
@pytest.mark.parametrize("fast", [True, False])
def test_too_many_slots_are_refused_before_any_memory_is_taken(top_k, fast, monkeypatch):
    if not fast:
        monkeypatch.setattr(binding, "_fast", None)
    for E, code in ((8, mm.MM_ERR_UNSUPPORTED), (300, mm.MM_ERR_UNSUPPORTED),
                    (0, mm.MM_ERR_INVALID_ARG)):
        x = torch.randn(1000, E, device="cuda")
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        with pytest.raises(mm.MMError) as e:
            mm.mm_route_logits(x, top_k, True)
        assert e.value.code == code
        assert torch.cuda.max_memory_allocated() == before


@pytest.mark.parametrize("T,E,k", [(0, 5, 2), (1, 1, 1), (65, 70, 7), (3000, 256, 8)])
def test_results_share_storage_whether_or_not_the_extension_is_built(T, E, k, monkeypatch):
    x = torch.randn(T, E, device="cuda")
    fast = mm.mm_route_logits(x, k, True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    given = mm.mm_route_logits(x, k, True, stream=side)
    monkeypatch.setattr(binding, "_fast", None)
    slow = mm.mm_route_logits(x, k, True)
    torch.cuda.synchronize()
    for got in (fast, given, slow):
        place = [(t.untyped_storage().data_ptr(), t.storage_offset() * t.element_size())
                 for t in got]
        assert [p[0] == q[0] for p in place for q in place] == \
            [p == q for p in "aabbb" for q in "aabbb"]
        assert [p[1] for p in place] == [p[1] for p in [
            (t.untyped_storage().data_ptr(), t.storage_offset() * t.element_size()) for t in fast]]
        assert not any(t._is_view() or t.requires_grad for t in got)
        assert all(torch.equal(a, b) and a.stride() == b.stride() for a, b in zip(got, fast))


def _layer_on_a_stream():
    """The layer's own calls that allocate results, with inputs that stay."""
    g = torch.Generator(device="cuda").manual_seed(12)
    T, H, E, I, k = 1500, 512, 16, 128, 4

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    x, rw, gu, dn, nw = rand(T, H), rand(E, H), rand(E, 2 * I, H), rand(E, H, I), rand(H)
    ids, _ = mm.mm_route(x, rw, k, True)
    part = mm.mm_moe_forward_partial(x, rw, gu, dn, k, True)
    return {
        "route": lambda s=None: mm.mm_route(x, rw, k, True, stream=s),
        "align": lambda s=None: mm.mm_align(ids, E, 16, stream=s)[1:],
        "forward": lambda s=None: mm.mm_moe_forward(x, rw, gu, dn, k, True, stream=s),
        "partial": lambda s=None: mm.mm_moe_forward_partial(x, rw, gu, dn, k, True, stream=s),
        "round": lambda s=None: mm.mm_round_bf16(part, stream=s),
        "dense": lambda s=None: mm.mm_gated_mlp(x, gu[0], dn[0], stream=s),
        "norm": lambda s=None: mm.mm_add_rmsnorm(x, nw, 1e-6, stream=s),
        "norm and layer": lambda s=None: mm.mm_moe_forward_add_norm(x, nw, 1e-6, rw, gu, dn, k,
                                                                    True, stream=s),
        "residual": lambda s=None: mm.mm_moe_forward_add_norm_residual(x, nw, 1e-6, rw, gu, dn, k,
                                                                       True, stream=s),
    }


@pytest.mark.parametrize("name", ["route", "align", "forward", "partial", "round", "dense", "norm",
                                  "norm and layer", "residual"])
def test_layer_results_on_a_given_stream_share_no_memory_in_use(name):
    # By address: the layer adds its slots up in no fixed order, so two calls may
    # differ in a rounding.
    call = _layer_on_a_stream()[name]
    side = torch.cuda.Stream()
    sizes = [t.numel() * t.element_size() for t in _tuple(call())]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda._sleep(200_000_000)
    in_use = []
    for b in blocks:
        b.fill_(0x5A)
        in_use.append((b.data_ptr(), b.data_ptr() + b.numel()))
    del blocks, b
    got = _tuple(call(side))
    for t, n in zip(got, sizes):
        assert all(t.data_ptr() + n <= lo or hi <= t.data_ptr() for lo, hi in in_use)
    torch.cuda.synchronize()
    assert mm.mm_poll_device_status() == mm.MM_OK


@pytest.mark.parametrize("name", STREAM_CALLS)
def test_other_threads_run_while_a_launch_waits(name):
    # Behind a kernel of about a second the launches fill the device's queue and
    # wait; a thread beside them goes on.
    import threading
    import time
    call = _on_a_stream()[name]
    keep = [call() for _ in range(3)]
    torch.cuda.synchronize()
    done, gaps = threading.Event(), []

    def beside():
        last = time.perf_counter()
        while not done.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now

    thread = threading.Thread(target=beside)
    thread.start()
    torch.cuda._sleep(2_000_000_000)
    begun = time.perf_counter()
    while time.perf_counter() - begun < 0.5:
        keep = keep[-10:] + [call()]
    torch.cuda.synchronize()
    done.set()
    thread.join()
    assert max(gaps) < 0.3, max(gaps)
