"""The experts trained: the operators one after another as a training step uses
them, with the router's, against float64."""
import pytest
import torch

import mixture_experts_layer_mm_gb300 as mm
import mixture_experts_layer_mm_gb300._lib as binding
import train_reference as ref
from mixture_experts_layer_mm_gb300 import run_layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(mmlib):
    return mmlib


def _inputs(T, H, E, I, k, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*s, std=1.0):
        return (std * torch.randn(*s, generator=g, device="cuda")).to(dtype)

    logits = torch.randn(T, E, generator=g, device="cuda")
    return dict(hidden=rand(T, H), logits=logits, gu=rand(E, 2 * I, H, std=H ** -0.5),
                dn=rand(E, H, I, std=I ** -0.5), d_out=rand(T, H), k=k)


def _off(got, want):
    return ((got.double().cpu() - want).norm() / want.norm()).item()


# Roundings between the stages, as shares of a norm: rows, z, act, y, da, dz, dx are
# rounded once each, at most 2^-8 (bf16; sums of roundings of both signs stay below
# that), and the stored pre-activations are off by at most half a step, 2^-7 of a block's
# largest value, in norm at most 2^-7 sqrt(32) = 0.045 of the block and, evenly spread over
# a step, 0.045 / sqrt(3) = 0.026. The slopes of the SwiGLU in g and u are below 1.1 of
# these; both enter a gradient.
FORWARD = 4 * 2.0 ** -8
BACKWARD = 7 * 2.0 ** -8 + 2 * 1.1 * 0.026


@pytest.mark.parametrize("T,H,E,I,k", [(1, 64, 4, 32, 2), (16, 128, 8, 64, 2), (37, 72, 5, 96, 3),
                                       (60, 264, 12, 160, 4)])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_step_against_float64(T, H, E, I, k, masked, dtype):
    d = _inputs(T, H, E, I, k, dtype)
    mask = None
    if masked:
        mask = torch.ones(T, dtype=torch.bool, device="cuda")
        mask[::3] = False
    ids, w, counts, _, _ = mm.mm_route_logits(d["logits"], k, True, token_mask=mask)
    hidden, d_out = d["hidden"].clone(), d["d_out"].clone()
    if masked:                                   # padding holds anything
        hidden[::3], d_out[::3] = float("nan"), float("inf")
    out, saved = mm.moe_experts_train(hidden, ids, w, d["gu"], d["dn"], token_mask=mask)
    grads = mm.moe_experts_train_backward(d_out, saved, d["gu"], d["dn"],
                                          weight_dtype=torch.float32)
    d_logits = mm.mm_route_logits_backward(d["logits"], ids, counts, True, grads.d_topk_w,
                                           token_mask=mask)
    assert mm.mm_poll_device_status() == mm.MM_OK
    leaves = [t.double().cpu().requires_grad_(True)
              for t in (d["hidden"], d["logits"], d["gu"], d["dn"])]
    p = torch.softmax(leaves[1], -1).gather(1, ids.cpu().long())
    weights = p / p.sum(-1, keepdim=True)
    cm = None if mask is None else mask.cpu()
    want = ref.experts(leaves[0], ids.cpu(), weights, leaves[2], leaves[3], mask=cm)
    go = d["d_out"].double().cpu()
    if masked:
        go[::3] = 0
        assert not out[::3].any() and not grads.d_hidden[::3].any()
        assert not grads.d_topk_w[::3].any() and not d_logits[::3].any()
    if T == 1 and masked:
        assert not grads.d_w_gate_up.any() and not grads.d_w_down.any()
        return
    wanted = torch.autograd.grad((want * go).sum(), leaves)
    assert _off(out, want.detach()) <= FORWARD
    # d_logits: sums of weights' gradients of both signs, which cancel to some extent;
    # their error is that of the gradients they are made of.
    scale = _topk_scale(weights.detach(), grads.d_topk_w.double().cpu(), wanted[1])
    for got, ref_grad, k_ in ((grads.d_hidden, wanted[0], 1.0), (grads.d_w_gate_up, wanted[2], 1.0),
                              (grads.d_w_down, wanted[3], 1.0), (d_logits, wanted[1], scale)):
        assert _off(got, ref_grad) <= BACKWARD * max(1.0, k_)


def _topk_scale(w, dw, d_logits):
    """How much larger the terms of the logits' gradient are than their sum."""
    n = d_logits.norm()
    return float(2 * (w * dw).norm() / n) if n > 0 else 1.0


def test_step_is_its_operators():
    """The composed call gives what the operators give one by one, bit for bit."""
    d = _inputs(300, 256, 16, 128, 4)
    ids, w, _, _, _ = mm.mm_route_logits(d["logits"], 4, True)
    out, s = mm.moe_experts_train(d["hidden"], ids, w, d["gu"], d["dn"])
    g = mm.moe_experts_train_backward(d["d_out"], s, d["gu"], d["dn"])
    places, off = mm.mm_group_slots(ids, 16)
    rows, row_w = mm.mm_dispatch_rows(d["hidden"], places, w=w)
    act, q, sc = mm.mm_swiglu_pack(mm.mm_grouped_product(rows, d["gu"], off), offsets=off)
    y = mm.mm_grouped_product(act, d["dn"], off)
    assert torch.equal(out, mm.mm_combine_rows(y, places, w=w))
    dr, _ = mm.mm_dispatch_rows(d["d_out"], places)
    da = mm.mm_grouped_product_dx(dr, d["dn"], off)
    dz, a, dw = mm.mm_swiglu_pack_backward(q, sc, da, row_w=row_w, offsets=off)
    assert torch.equal(g.d_w_down, mm.mm_grouped_product_dw(dr, a, off))
    assert torch.equal(g.d_w_gate_up, mm.mm_grouped_product_dw(dz, rows, off))
    dh, dtw = mm.mm_combine_rows(mm.mm_grouped_product_dx(dz, d["gu"], off), places, row_values=dw)
    assert torch.equal(g.d_hidden, dh) and torch.equal(g.d_topk_w, dtw)


def test_forward_is_the_layers():
    """Beside mm_moe_forward, whose activations are rounded once as here and whose sum
    keeps the expert outputs in fp32."""
    T, H, E, I, k = 64, 256, 16, 128, 4
    d = _inputs(T, H, E, I, k)
    router = (torch.randn(E, H, device="cuda") / 16).bfloat16()
    ids, w = mm.mm_route(d["hidden"], router, k, True)
    want = mm.mm_moe_forward(d["hidden"], router, d["gu"], d["dn"], k, True)
    out, _ = mm.moe_experts_train(d["hidden"], ids, w, d["gu"], d["dn"])
    assert _off(out, want.double().cpu()) <= 2 * FORWARD


def test_micro_batches_add_up():
    """Two micro-batches added into fp32 gradients give the sum of theirs."""
    a, b = (_inputs(80, 128, 8, 64, 2, seed=s) for s in range(2))
    gu, dn = a["gu"], a["dn"]
    total = [torch.zeros(gu.shape, device="cuda"), torch.zeros(dn.shape, device="cuda")]
    apart = []
    for d in (a, b):
        ids, w, _, _, _ = mm.mm_route_logits(d["logits"], 2, True)
        _, s = mm.moe_experts_train(d["hidden"], ids, w, gu, dn)
        apart.append(mm.moe_experts_train_backward(d["d_out"], s, gu, dn,
                                                   weight_dtype=torch.float32))
        g = mm.moe_experts_train_backward(d["d_out"], s, gu, dn, *total, accumulate=True)
        assert g.d_w_gate_up is total[0] and g.d_w_down is total[1]
    assert torch.equal(total[0], apart[0].d_w_gate_up + apart[1].d_w_gate_up)
    assert torch.equal(total[1], apart[0].d_w_down + apart[1].d_w_down)


def test_step_captured_and_replayed():
    """A whole step in a graph, replayed on other inputs, beside eager steps."""
    T, H, E, I, k = 200, 128, 8, 64, 2
    sets = [_inputs(T, H, E, I, k, seed=s) for s in range(2)]
    gu, dn = sets[0]["gu"], sets[0]["dn"]
    live = {n: sets[0][n].clone() for n in ("hidden", "logits", "d_out")}

    def step(d):
        ids, w, counts, _, _ = mm.mm_route_logits(d["logits"], k, True)
        out, s = mm.moe_experts_train(d["hidden"], ids, w, gu, dn)
        g = mm.moe_experts_train_backward(d["d_out"], s, gu, dn)
        return (out, *g, mm.mm_route_logits_backward(d["logits"], ids, counts, True, g.d_topk_w))

    want = [step(d) for d in sets]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(live)
    for i in (1, 0, 1):
        for n in live:
            live[n].copy_(sets[i][n])
        graph.replay()
        eager = step(sets[1 - i])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
        assert all(torch.equal(a, b) for a, b in zip(eager, want[1 - i]))


def test_step_on_a_given_stream_and_without_tokens():
    d = _inputs(100, 128, 8, 64, 2)
    ids, w, _, _, _ = mm.mm_route_logits(d["logits"], 2, True)
    out, s = mm.moe_experts_train(d["hidden"], ids, w, d["gu"], d["dn"])
    g = mm.moe_experts_train_backward(d["d_out"], s, d["gu"], d["dn"])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    o2, s2 = mm.moe_experts_train(d["hidden"], ids, w, d["gu"], d["dn"], stream=st)
    g2 = mm.moe_experts_train_backward(d["d_out"], s2, d["gu"], d["dn"], stream=st)
    st.synchronize()
    assert torch.equal(out, o2) and all(torch.equal(a, b) for a, b in zip(g, g2))
    out, s = mm.moe_experts_train(d["hidden"][:0], ids[:0], w[:0], d["gu"], d["dn"])
    g = mm.moe_experts_train_backward(d["d_out"][:0], s, d["gu"], d["dn"])
    assert out.shape == (0, 128) and g.d_topk_w.shape == (0, 2)
    assert not g.d_w_gate_up.any() and not g.d_w_down.any()


def test_run_layer_trains(capsys):
    assert run_layer.main(["--workload", "tiny", "--passes", "2", "--train"]) == 0
    assert "2 passes" in capsys.readouterr().out


def _calls():
    d = _inputs(40, 64, 6, 32, 3)
    ids, w, _, _, _ = mm.mm_route_logits(d["logits"], 3, True)
    mask = torch.rand(40, device="cuda") > 0.2
    places, off = mm.mm_group_slots(ids, 6)
    rows, row_w = mm.mm_dispatch_rows(d["hidden"], places, w=w)
    z = mm.mm_grouped_product(rows, d["gu"], off)
    act, q, s = mm.mm_swiglu_pack(z)
    big = torch.randn(8192, 64, device="cuda").bfloat16()
    one = torch.tensor([0, 8192], dtype=torch.int32, device="cuda")
    vals = torch.rand(120, device="cuda")
    return {
        "group": lambda: mm.mm_group_slots(ids, 6),
        "group masked": lambda: mm.mm_group_slots(ids.repeat(100, 1), 6,
                                                  token_mask=mask.repeat(100).to(torch.uint8)),
        "dispatch": lambda: mm.mm_dispatch_rows(d["hidden"], places),
        "dispatch weights": lambda: mm.mm_dispatch_rows(d["hidden"], places, w=w),
        "dispatch given": lambda: tuple(t.clone() for t in mm.mm_dispatch_rows(
            d["hidden"], places, w=w, rows=torch.zeros(200, 64, device="cuda").bfloat16(),
            row_w=torch.zeros(200, device="cuda"))),
        "combine": lambda: mm.mm_combine_rows(rows, places),
        "combine values": lambda: mm.mm_combine_rows(
            rows, places, w=w, row_values=vals, out=torch.empty(40, 64, device="cuda").bfloat16()),
        "product": lambda: mm.mm_grouped_product(rows, d["gu"], off),
        "dx": lambda: mm.mm_grouped_product_dx(z, d["gu"], off, out=torch.empty_like(rows)),
        "dw": lambda: mm.mm_grouped_product_dw(z, rows, off),
        "dw parts": lambda: mm.mm_grouped_product_dw(big, big, one, out_dtype=torch.float32),
        "dw added": lambda: mm.mm_grouped_product_dw(
            z, rows, off, out=torch.ones(6, 64, 64, device="cuda"), accumulate=True),
        "dw added, by a number": lambda: mm.mm_grouped_product_dw(
            z, rows, off, out=torch.ones(6, 64, 64, device="cuda"), accumulate=1),
        "pack": lambda: mm.mm_swiglu_pack(z),
        "pack rows": lambda: tuple(t[:60] for t in mm.mm_swiglu_pack(z, offsets=off // 2)),
        "backward": lambda: mm.mm_swiglu_pack_backward(q, s, act)[:2],
        "backward weighted": lambda: mm.mm_swiglu_pack_backward(q, s, act, row_w=row_w,
                                                                offsets=off),
        "dequantise": lambda: mm.mm_mxint8_dequantize(q, s, dtype=torch.float16),
        "no tokens": lambda: mm.mm_group_slots(ids[:0], 6),
    }


NAMES = ["group", "group masked", "dispatch", "dispatch weights", "dispatch given", "combine",
         "combine values", "product", "dx", "dw", "dw parts", "dw added",
         "dw added, by a number", "pack", "pack rows",
         "backward", "backward weighted", "dequantise", "no tokens"]


@pytest.mark.parametrize("name", NAMES)
def test_both_ways_of_marshalling_agree(name, monkeypatch):
    if binding._fast is None:
        pytest.skip("the extension is not built")
    call, declined, fast_ext = _calls()[name], [], binding._fast

    class Spy:  # the extension, with a note of the calls it declines
        def __getattr__(self, fn):
            def f(*a):
                r = getattr(fast_ext, fn)(*a)
                if r is None:
                    declined.append(fn)
                return r
            return f

    monkeypatch.setattr(binding, "_fast", Spy())
    fast = call()
    assert not declined
    monkeypatch.setattr(binding, "_fast", None)
    slow = call()
    fast, slow = (r if isinstance(r, tuple) else (r,) for r in (fast, slow))
    assert len(fast) == len(slow)
    for a, b in zip(fast, slow):
        assert (a is None) == (b is None)
        if a is not None:
            assert a.dtype == b.dtype and a.shape == b.shape and a.device == b.device
            assert torch.equal(a, b)
    assert _shared(fast) == _shared(slow)


def _shared(results):
    """Which results lie in one allocation with which."""
    at = [None if r is None else r.untyped_storage().data_ptr() for r in results]
    return [[a == b for b in at] for a in at]


@pytest.mark.parametrize("R,one", [(1, True), (100, True), (5000, False)])
def test_small_results_share_an_allocation_and_do_not_meet(R, one):
    z = torch.randn(R, 128, device="cuda").bfloat16()
    act, q, s = mm.mm_swiglu_pack(z)
    assert _shared((act, q, s))[0] == [True, one, one]
    da, w = torch.randn(R, 64, device="cuda").bfloat16(), torch.rand(R, device="cuda")
    dz, a, dw = mm.mm_swiglu_pack_backward(q, s, da, row_w=w)
    assert _shared((dz, a, dw))[0] == [True, one, one]
    ids = torch.randint(0, 9, (R * 20, 4), dtype=torch.int32, device="cuda")
    p, o = mm.mm_group_slots(ids, 9)
    assert _shared((p, o))[0] == [True, R < 5000 and R * 320 < (1 << 20) - 512]
    for group in ((act, q, s), (dz, a, dw), (p, o)):
        kept = [t.clone() for t in group]
        for i, t in enumerate(group):                        # writing one leaves the others
            t.fill_(1)
            assert all(torch.equal(x, y) for x, y in zip(group[i + 1:], kept[i + 1:]))
            assert t.data_ptr() % 256 == 0


def test_declined_calls_raise_as_in_python(monkeypatch):
    d = _inputs(8, 64, 4, 32, 2)
    ids, w, _, _, _ = mm.mm_route_logits(d["logits"], 2, True)
    places, off = mm.mm_group_slots(ids, 4)
    x, gu = d["hidden"], d["gu"]
    rows, _ = mm.mm_dispatch_rows(x, places)
    act, q, s = mm.mm_swiglu_pack(rows)
    n3 = torch.ones(3, device="cuda")
    bad = [
        lambda: mm.mm_group_slots(ids.long(), 4), lambda: mm.mm_group_slots(ids, 0),
        lambda: mm.mm_group_slots(ids, 300), lambda: mm.mm_group_slots(ids[0], 4),
        lambda: mm.mm_group_slots(ids, 4, token_mask=n3.bool()),
        lambda: mm.mm_group_slots(ids, 4, token_mask=n3), lambda: mm.mm_group_slots(ids.t(), 4),
        lambda: mm.mm_dispatch_rows(x.float(), places),
        lambda: mm.mm_dispatch_rows(x[:, :60].contiguous(), places),
        lambda: mm.mm_dispatch_rows(x[:5], places), lambda: mm.mm_dispatch_rows(x, places, w=w[:5]),
        lambda: mm.mm_dispatch_rows(x, places, row_w=n3),
        lambda: mm.mm_dispatch_rows(x, places, rows=rows.half()),
        lambda: mm.mm_dispatch_rows(x, places, w=w, rows=rows, row_w=n3),
        lambda: mm.mm_dispatch_rows(x[:, ::2], places),
        lambda: mm.mm_combine_rows(rows.float(), places),
        lambda: mm.mm_combine_rows(rows, places.long()),
        lambda: mm.mm_combine_rows(rows, places, row_values=n3),
        lambda: mm.mm_combine_rows(rows, places, out=x.half()),
        lambda: mm.mm_combine_rows(rows.cpu(), places),
        lambda: mm.mm_grouped_product(rows, gu.half(), off),
        lambda: mm.mm_grouped_product(rows, gu, off[:3]),
        lambda: mm.mm_grouped_product(rows, gu, off.long()),
        lambda: mm.mm_grouped_product(rows[:, :32].contiguous(), gu, off),
        lambda: mm.mm_grouped_product(rows, gu[:, :60].contiguous(), off),
        lambda: mm.mm_grouped_product(rows, gu, off, out=rows[:3]),
        lambda: mm.mm_grouped_product_dx(rows, gu[0], off),
        lambda: mm.mm_grouped_product_dw(rows, rows[:3], off),
        lambda: mm.mm_grouped_product_dw(rows, rows, off, accumulate=True),
        lambda: mm.mm_grouped_product_dw(rows, rows, off, out_dtype=torch.float16),
        lambda: mm.mm_grouped_product_dw(rows, rows, off, out_dtype=torch.int8),
        lambda: mm.mm_grouped_product_dw(rows, rows, off[:1]),
        lambda: mm.mm_grouped_product_dw(rows[:, :20].contiguous(), rows, off),
        lambda: mm.mm_swiglu_pack(rows[:, :32].contiguous()), lambda: mm.mm_swiglu_pack(n3),
        lambda: mm.mm_swiglu_pack(rows, offsets=off[:0]),
        lambda: mm.mm_swiglu_pack(rows, offsets=off.long()),
        lambda: mm.mm_swiglu_pack_backward(q, s[:, :1], act),
        lambda: mm.mm_swiglu_pack_backward(q.view(torch.uint8), s, act),
        lambda: mm.mm_swiglu_pack_backward(q, s, act, row_w=n3),
        lambda: mm.mm_mxint8_dequantize(q, s, dtype=torch.int32),
        lambda: mm.mm_mxint8_dequantize(q[:, :40].contiguous(), s),
        lambda: mm.mm_mxint8_dequantize(q, s[:3]),
    ]
    errors = []
    for ext in (binding._fast, None):
        monkeypatch.setattr(binding, "_fast", ext)
        got = []
        for i, f in enumerate(bad):
            with pytest.raises((TypeError, ValueError, mm.MMError)) as e:
                f()
            got.append((i, type(e.value), str(e.value)))
        errors.append(got)
    assert errors[0] == errors[1]
    assert mm.mm_poll_device_status() == mm.MM_OK


_FIRST = """
import torch, mixture_experts_layer_mm_gb300 as mm
g = torch.cuda.CUDAGraph()
ids = torch.randint(0, 8, (2000, 2), dtype=torch.int32, device="cuda")
w = torch.rand(2000, 2, device="cuda")
x = torch.randn(2000, 64, device="cuda").bfloat16()
gu, dn = (torch.randn(8, n, k, device="cuda").bfloat16() for n, k in ((64, 64), (64, 32)))
torch.cuda.synchronize()
with torch.cuda.graph(g):
    out, s = mm.moe_experts_train(x, ids, w, gu, dn)
    grads = mm.moe_experts_train_backward(x, s, gu, dn)
g.replay()
torch.cuda.synchronize()
out2, s = mm.moe_experts_train(x, ids, w, gu, dn)
again = mm.moe_experts_train_backward(x, s, gu, dn)
assert torch.equal(out, out2) and all(torch.equal(a, b) for a, b in zip(grads, again))
assert mm.mm_poll_device_status() == mm.MM_OK
"""


def test_the_first_calls_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(mm.__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_a_refused_backward_leaves_the_gradients():
    """Whichever argument is refused, the gradients are as before, and the call made right
    adds the micro-batch once."""
    d = _inputs(40, 64, 6, 32, 2)
    gu, dn, d_out = d["gu"], d["dn"], d["d_out"]
    ids, w, _, _, _ = mm.mm_route_logits(d["logits"], 2, True)
    _, s = mm.moe_experts_train(d["hidden"], ids, w, gu, dn)
    ones = lambda t, dtype=torch.float32: torch.ones(t.shape, dtype=dtype, device="cuda")
    d_gu, d_dn = ones(gu), ones(dn)
    odd = torch.ones(gu.numel() + 1, device="cuda")[1:].view(gu.shape)
    odd_gu = torch.zeros(gu.numel() + 1, device="cuda").bfloat16()[1:].view(gu.shape)
    bad = [dict(d_w_gate_up=None), dict(d_w_down=None), dict(d_w_gate_up=d_gu[:5]),
           dict(d_w_gate_up=d_gu.half()), dict(d_w_gate_up=d_gu.cpu()), dict(d_w_gate_up=odd),
           dict(d_w_gate_up=ones(gu.transpose(1, 2)).transpose(1, 2)), dict(d_w_down=d_dn[:, :8]),
           dict(gu=gu.half()), dict(gu=odd_gu), dict(gu=gu[:, :32]), dict(dn=dn[:3]), dict(dn=dn.float()),
           dict(d_out=d_out.half()), dict(d_out=d_out[:7])]
    for change in bad:
        a = dict(d_out=d_out, gu=gu, dn=dn, d_w_gate_up=d_gu, d_w_down=d_dn) | change
        with pytest.raises((TypeError, ValueError, mm.MMError)):
            mm.moe_experts_train_backward(a["d_out"], s, a["gu"], a["dn"], a["d_w_gate_up"],
                                          a["d_w_down"], accumulate=True)
        assert (d_gu == 1).all() and (d_dn == 1).all() and (odd == 1).all()
    want = mm.moe_experts_train_backward(d_out, s, gu, dn, weight_dtype=torch.float32)
    mm.moe_experts_train_backward(d_out, s, gu, dn, d_gu, d_dn, accumulate=True)
    assert torch.equal(d_gu, 1 + want.d_w_gate_up) and torch.equal(d_dn, 1 + want.d_w_down)
    assert mm.mm_poll_device_status() == mm.MM_OK


@pytest.mark.parametrize("T,H,E,I,k", [(16, 128, 8, 64, 2), (37, 72, 5, 96, 3),
                                       (60, 264, 12, 160, 4)])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_the_weights_gradient_against_float64(T, H, E, I, k, masked, dtype):
    """d_topk_w by itself, and d_logits against a scale that no result of the kernels enters.
    A weight's gradient is the product of a row of da with one of activations, both with
    the errors of the other gradients: over many slots its share is theirs."""
    d = _inputs(T, H, E, I, k, dtype, seed=3)
    mask = None
    if masked:
        mask = torch.arange(T, device="cuda") % 3 > 0
    ids, w, counts, _, _ = mm.mm_route_logits(d["logits"], k, True, token_mask=mask)
    _, saved = mm.moe_experts_train(d["hidden"], ids, w, d["gu"], d["dn"], token_mask=mask)
    got = mm.moe_experts_train_backward(d["d_out"], saved, d["gu"], d["dn"]).d_topk_w
    d_logits = mm.mm_route_logits_backward(d["logits"], ids, counts, True, got, token_mask=mask)
    leaf = w.double().cpu().requires_grad_(True)
    cm = None if mask is None else mask.cpu()
    out = ref.experts(d["hidden"].double().cpu(), ids.cpu(), leaf, d["gu"].double().cpu(),
                      d["dn"].double().cpu(), mask=cm)
    want, = torch.autograd.grad((out * d["d_out"].double().cpu()).sum(), leaf)
    assert _off(got, want) <= BACKWARD
    if masked:
        assert not got[~mask].any()
    logits = d["logits"].double().cpu().requires_grad_(True)
    p = torch.softmax(logits, -1).gather(1, ids.cpu().long())
    weights = p / p.sum(-1, keepdim=True)
    want_logits, = torch.autograd.grad((weights * want).sum(), logits)
    scale = _topk_scale(weights.detach(), want, want_logits)
    assert _off(d_logits, want_logits) <= BACKWARD * max(1.0, scale)
    assert mm.mm_poll_device_status() == mm.MM_OK
