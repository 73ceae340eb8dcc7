"""Routing from logits with the balance statistics, and its gradient, against
their float64 definitions."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_mm_gb300 as mm
import mx_reference as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24  # half a step of fp32


@pytest.fixture(scope="module", autouse=True)
def _lib(mmlib):
    return mmlib


def _case(seed, T, E, k, dtype=torch.float32, masked=0.0, std=1.5):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((T, E)) * std + 0.5 * rng.standard_normal((1, E)))
    x = torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()
    mask = None
    if masked:
        mask = torch.from_numpy(rng.random(T) >= masked).cuda()
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    return x, mask, dw


def _np64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def _spread(x):
    """max - min of each row's finite logits (0 for a row without any)."""
    fine = np.isfinite(x)
    top = np.where(fine, x, -np.inf).max(1)
    low = np.where(fine, x, np.inf).min(1)
    return np.where(fine.any(1), np.where(fine.any(1), top, 0) - np.where(fine.any(1), low, 0), 0)


def _p_rel(x):
    """Relative error of a kernel's p: l - m is rounded (|l - m| U as an
    absolute error of the exponent), expf is within 2 ulp (4 U), the sum of E
    terms goes through at most 8 + 5 additions (13 U, of terms with the error
    before), the reciprocal and the product 2 U."""
    return (2 * (_spread(x).max() if x.size else 0) + 4 * 2 + 13 + 3) * U


def _check(x, mask, k, renorm, got):
    x64 = _np64(x)
    want = ref.route(x64, k, renorm, None if mask is None else mask.cpu().numpy())
    ids, w, counts, sums, loss = got
    assert np.array_equal(ids.cpu().numpy(), want["ids"])
    assert np.array_equal(counts.cpu().numpy(), want["counts"])
    rel = _p_rel(x64)
    wrel = rel if not renorm else 2 * rel + (k + 3) * U
    assert (np.abs(_np64(w) - want["w"]) <= wrel * want["w"] + 2.0 ** -126).all()
    T = x64.shape[0]
    # prob_sums: T terms added in at most ceil(T / 16) + 16 + 320 steps
    steps = min(T, -(-T // 16) + 336)
    stol = (rel + steps * U) * want["prob_sums"]
    assert (np.abs(_np64(sums) - want["prob_sums"]) <= stol + 1e-37).all()
    assert abs(float(loss) - want["loss"]) <= (rel + (steps + 16) * U) * abs(want["loss"])
    return want


SHAPES = [(1, 1, 1), (1, 8, 2), (3, 256, 32), (16, 33, 5), (17, 60, 4), (64, 128, 8), (100, 31, 31),
          (513, 129, 8), (4096, 128, 8), (5003, 60, 4), (9000, 256, 8)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_forward(T, E, k, renorm, dtype):
    # bf16 logits are full of ties: the lower id wins.
    x, mask, _ = _case(T + E, T, E, k, dtype, masked=0.2 if T > 16 else 0.0)
    got = mm.mm_route_logits(x, k, renorm, token_mask=mask)
    _check(x, mask, k, renorm, got)
    again = mm.mm_route_logits(x, k, renorm, token_mask=mask)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert mm.mm_poll_device_status() == mm.MM_OK


def _grad_tol(x64, want, k, renorm, dw, dloss, counts):
    """Bound of |kernel - exact| for d_logits (before its own rounding):
    every term p (a - sum p a) is a product of p (relative error rel) and a
    difference whose two sides are each within rel + 20 U of sums of
    magnitudes."""
    rel = _p_rel(x64) * 3 + 40 * U
    T, E = x64.shape
    p = want["p"]
    n = counts.sum() / k
    c = np.abs(dloss) * E * counts / (n * k) / n if n > 0 else np.zeros(E)
    tol = p * (c + (p * c).sum(1, keepdims=True))
    if dw is not None:
        ch = np.take_along_axis(p, want["ids"], 1)
        a = np.abs(dw)
        tot = ch.sum(1, keepdims=True)
        s = np.where(tot > 0, tot, 1) if renorm else 1.0
        mean = (ch / s * a).sum(1, keepdims=True)
        sel = np.zeros((T, E))
        np.put_along_axis(sel, want["ids"], ch / s * (a + mean), 1)
        tol = tol + (sel if renorm else sel + p * mean)
        if renorm:
            # The reference's own rounding: off the selection it forms
            # p (0 - sum p dp), zero but for the float64 rounding of that sum
            # (terms of ch / s (a + mean), which add up to 2 mean; 2^-53 each
            # in the terms, the quotients and at most 32 additions: 2^-47).
            return rel * tol + 2.0 ** -47 * p * 2 * mean + 1e-37
    return rel * tol + 1e-37


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_backward(T, E, k, renorm, dtype):
    x, mask, dw = _case(T + 3 * E, T, E, k, dtype, masked=0.2 if T > 16 else 0.0)
    dloss = torch.tensor([0.7], device="cuda") * T  # both parts of the gradient visible
    ids, _, counts, _, _ = mm.mm_route_logits(x, k, renorm, token_mask=mask)
    x64, m = _np64(x), None if mask is None else mask.cpu().numpy()
    want = ref.route(x64, k, renorm, m)
    for use_w, use_l in ((True, True), (True, False), (False, True)):
        g = mm.mm_route_logits_backward(x, ids, counts, renorm, d_topk_w=dw if use_w else None,
                                        d_loss=dloss if use_l else None, token_mask=mask)
        d = _np64(dw) if use_w else None
        l = float(dloss) if use_l else 0.0
        exact = ref.route_grad(x64, k, renorm, d, l, m)
        tol = _grad_tol(x64, want, k, renorm, d, l, want["counts"])
        if dtype == torch.bfloat16:
            tol = tol + (np.abs(exact) + tol) * 2.0 ** -8
        off = np.abs(_np64(g) - exact)
        assert (off <= tol).all(), (use_w, use_l, (off / tol).max())
        if mask is not None:
            assert not g[~mask].any()
    assert mm.mm_poll_device_status() == mm.MM_OK


@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_is_the_slope_of_the_forward(renorm):
    # Differences of the float64 forward against the kernel's gradient, ids and
    # counts (step functions) unchanged by the step.
    T, E, k = 6, 12, 3
    x, _, dw = _case(1, T, E, k)
    ids, _, counts, _, _ = mm.mm_route_logits(x, k, renorm)
    dl = torch.tensor([2.0], device="cuda")
    g = _np64(mm.mm_route_logits_backward(x, ids, counts, renorm, d_topk_w=dw, d_loss=dl))
    x64, h = _np64(x), 1e-5

    def total(z):
        r = ref.route(z, k, renorm)
        assert np.array_equal(r["ids"], ids.cpu().numpy())
        return (r["w"] * _np64(dw)).sum() + 2.0 * r["loss"]

    num = np.zeros((T, E))
    for t in range(T):
        for e in range(E):
            d = np.zeros((T, E))
            d[t, e] = h
            num[t, e] = (total(x64 + d) - total(x64 - d)) / (2 * h)
    # central differences: h^2 |f'''| / 6 <= 1e-10 * 10, and 1e-16 * 20 / h = 2e-10
    assert np.abs(num - g).max() <= 1e-8 + 200 * U * np.abs(num).max()


def test_masked_rows_may_hold_anything():
    T, E, k = 70, 40, 4
    x, _, dw = _case(5, T, E, k)
    clean = torch.ones(T, dtype=torch.uint8, device="cuda")
    clean[[0, 7, 33, 69]] = 0
    want = mm.mm_route_logits(x, k, True, token_mask=clean)
    want_g = mm.mm_route_logits_backward(x, want[0], want[2], True, dw,
                                         torch.ones(1, device="cuda"), clean)
    y = x.clone()
    y[0], y[7], y[33] = float("nan"), float("inf"), -float("inf")
    y[69, ::2] = -torch.tensor(float("nan"), device="cuda")
    got = mm.mm_route_logits(y, k, True, token_mask=clean)
    rows = clean.bool()
    assert torch.equal(got[0][rows], want[0][rows])
    for a, b in zip(got[1:], want[1:]):
        assert torch.equal(a, b)
    ids = got[0][~rows].cpu().numpy()
    assert ((ids >= 0) & (ids < E)).all()
    assert all(len(set(r)) == k for r in ids) and (np.diff(ids) > 0).all()
    g = mm.mm_route_logits_backward(y, got[0], got[2], True, dw, torch.ones(1, device="cuda"),
                                    clean)
    assert torch.equal(g, want_g) and not g[~rows].any()


def test_unavailable_experts():
    T, E, k = 50, 20, 4
    x, _, dw = _case(6, T, E, k)
    x[:, 3] = -float("inf")
    x[10, 2:] = -float("inf")      # two experts left for four slots
    x[20] = -float("inf")          # none left: as a masked token
    for renorm in (False, True):
        got = mm.mm_route_logits(x, k, renorm)
        want = _check(x, None, k, renorm, got)
        assert not want["valid"][20] and got[1][20].eq(0).all()
        assert got[0][10].tolist() == [0, 1, 2, 3] and got[1][10, 2:].eq(0).all()
        assert got[0][20].tolist() == [0, 1, 2, 3]
        dl = torch.ones(1, device="cuda")
        g = _np64(mm.mm_route_logits_backward(x, got[0], got[2], renorm, dw, dl))
        exact = ref.route_grad(_np64(x), k, renorm, _np64(dw), 1.0)
        assert np.isfinite(g).all() and not g[20].any() and not g[:, 3].any()
        assert np.abs(g - exact).max() <= 300 * U * np.abs(dw.cpu().numpy()).max()


def test_all_tokens_masked_and_no_tokens():
    E, k = 24, 3
    for T in (0, 1, 40):
        x, _, dw = _case(7, T, E, k)
        mask = torch.zeros(T, dtype=torch.bool, device="cuda")
        ids, w, counts, sums, loss = mm.mm_route_logits(x, k, True, token_mask=mask)
        assert not w.any() and not counts.any() and not sums.any() and float(loss) == 0.0
        g = mm.mm_route_logits_backward(x, ids, counts, True, dw, torch.ones(1, device="cuda"),
                                        mask)
        assert g.shape == (T, E) and not g.any()
    assert mm.mm_poll_device_status() == mm.MM_OK


def test_extreme_logits():
    x = torch.tensor([[1e30, -1e30, 0.0, 1e30], [-1e38, -1e38, -1e38, -3e38],
                      [0.0, -0.0, 0.0, -0.0], [88.0, -88.0, 0.0, 1.0]], device="cuda")
    got = mm.mm_route_logits(x, 2, False)
    want = ref.route(_np64(x), 2, False)
    assert np.array_equal(got[0].cpu().numpy(), want["ids"])  # -0 and 0 tie: lower ids
    assert np.abs(_np64(got[1]) - want["w"]).max() <= 1e-6
    y = torch.zeros(2, 4, device="cuda")
    y[1, 2] = float("nan")
    ids, w, counts, sums, loss = mm.mm_route_logits(y, 2, True)
    assert torch.isnan(w[1]).all() and torch.isfinite(w[0]).all()
    assert torch.isnan(loss).all() and torch.isnan(sums).all()
    assert len(set(ids[1].tolist())) == 2 and int(counts.sum()) == 4


def test_replicas_share_their_counts():
    # Two halves of a batch, each differentiated with the summed counts, give
    # the gradient of the loss over the whole batch.
    T, E, k = 96, 32, 4
    x, _, dw = _case(8, T, E, k)
    dl = torch.tensor([3.0], device="cuda")
    ids, _, counts, _, _ = mm.mm_route_logits(x, k, True)
    whole = mm.mm_route_logits_backward(x, ids, counts, True, dw, dl)
    halves, c = [x[:40].contiguous(), x[40:].contiguous()], 0
    routed = [mm.mm_route_logits(h, k, True) for h in halves]
    c = routed[0][2] + routed[1][2]
    assert torch.equal(c, counts)
    parts = [mm.mm_route_logits_backward(h, r[0], c, True, d.contiguous(), dl)
             for h, r, d in zip(halves, routed, (dw[:40], dw[40:]))]
    assert torch.equal(torch.cat(parts), whole)


def test_backward_ignores_ids_that_are_none():
    T, E, k = 9, 16, 3
    x, _, dw = _case(9, T, E, k)
    ids, _, counts, _, _ = mm.mm_route_logits(x, k, False)
    bad = ids.clone()
    bad[2, 1], bad[4, 0], bad[6, 2] = -5, 1 << 30, ids[6, 0]
    g = mm.mm_route_logits_backward(x, bad, counts, False, dw)
    kept = dw.clone()
    kept[2, 1] = kept[4, 0] = kept[6, 2] = 0
    assert torch.equal(g, mm.mm_route_logits_backward(x, ids, counts, False, kept))
    assert mm.mm_poll_device_status() == mm.MM_OK


def test_logits_at_any_element_offset():
    # Views that begin at addresses aligned to one element only.
    for dtype in (torch.float32, torch.bfloat16):
        flat = torch.randn(1 + 50 * 21, device="cuda").to(dtype)
        x = flat[1:].view(50, 21)
        got = mm.mm_route_logits(x, 3, True)
        same = mm.mm_route_logits(x.clone(), 3, True)
        assert all(torch.equal(a, b) for a, b in zip(got, same))
        g = mm.mm_route_logits_backward(x, got[0], got[2], True, d_loss=got[4])
        assert torch.equal(g, mm.mm_route_logits_backward(x.clone(), got[0], got[2], True,
                                                          d_loss=got[4]))


def test_streams_and_captured_graphs():
    T, E, k = 3000, 64, 6
    cases = [_case(40 + i, T, E, k)[::2] for i in range(2)]

    def step(x, dw):
        ids, w, counts, sums, loss = mm.mm_route_logits(x, k, True)
        return ids, w, counts, sums, loss, mm.mm_route_logits_backward(x, ids, counts, True, dw,
                                                                       loss)

    want = [step(*c) for c in cases]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*c))
        graphs.append(g)
    side = torch.cuda.Stream()
    for _ in range(4):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
            eager = step(*cases[0])
    torch.cuda.synchronize()
    for o, w in zip(outs + [eager], want + [want[0]]):
        assert all(torch.equal(a, b) for a, b in zip(o, w))


def test_writes_only_its_outputs():
    from test_gpu_guards import Guarded
    L, st = mm.lib(), torch.cuda.current_stream().cuda_stream
    for T, E, k in ((5, 60, 4), (777, 130, 7)):
        x, mask, dw = _case(T, T, E, k, masked=0.3)
        b = {"x": Guarded((T, E), torch.float32, x), "mask": Guarded((T,), torch.uint8, mask),
             "ids": Guarded((T, k), torch.int32), "w": Guarded((T, k), torch.float32),
             "counts": Guarded((E,), torch.int32), "sums": Guarded((E,), torch.float32),
             "loss": Guarded((1,), torch.float32), "grad": Guarded((T, E), torch.float32),
             "dw": Guarded((T, k), torch.float32, dw)}
        n = int(L.mm_route_logits_workspace_size(T, E))
        b["ws"] = Guarded((max(n, 16),), torch.uint8)
        p = {name: g.t.data_ptr() for name, g in b.items()}
        assert L.mm_route_logits(p["x"], 0, p["mask"], T, E, k, 1, p["ids"], p["w"], p["counts"],
                                 p["sums"], p["loss"], p["ws"], n, st) == mm.MM_OK
        assert L.mm_route_logits_backward(p["x"], 0, p["mask"], p["ids"], p["counts"], p["dw"],
                                          p["loss"], T, E, k, 1, p["grad"], st) == mm.MM_OK
        torch.cuda.synchronize()
        for name, g in b.items():
            assert g.intact(), name


def test_as_many_tokens_as_an_index_counts():
    # One expert, 2^31 - 1 tokens: every token selects it with weight 1.
    T = (1 << 31) - 1
    x = torch.zeros(T, 1, dtype=torch.bfloat16, device="cuda")
    ids, w, counts, sums, loss = mm.mm_route_logits(x, 1, False)
    assert not ids.any() and int(counts) == T
    assert float(w.min()) == 1.0 and float(w.max()) == 1.0
    # Sums of ones: exact up to 2^24 in a lane (T / (304 * 16) ones) and a block,
    # then 320 additions at most.
    assert abs(float(sums) / T - 1) <= 320 * U and abs(float(loss) - 1) <= 324 * U
    dw = w  # ones
    g = mm.mm_route_logits_backward(x, ids, counts, False, dw, loss)
    del ids, w, dw
    # p = 1: dl = (dw + c) p - p (sum_i p_i (dw_i + c_i)), both terms the same value
    assert not g.any()


def _behind(step, x, src):
    """`step` on an x that is written late: by a copy on the same stream, by
    another stream that this one waits for, and by two streams at once."""
    cur = torch.cuda.current_stream()
    outs = []
    for way in range(3):
        x.zero_()
        if way == 0:
            torch.cuda._sleep(200_000)
            x.copy_(src)
        else:
            sides = [torch.cuda.Stream() for _ in range(way)]
            parts = list(zip(sides, x.chunk(way), src.chunk(way)))
            for s, a, b in parts:
                s.wait_stream(cur)
                with torch.cuda.stream(s):
                    torch.cuda._sleep(200_000)
                    a.copy_(b)
            for s in sides:
                cur.wait_stream(s)
        outs.append([t.clone() for t in step(x)])
    return outs


@pytest.mark.parametrize("T", [48, 3000])
def test_order_behind_copies_and_other_streams(T):
    # The kernels are launched programmatically: what the stream waits for comes
    # first all the same, in eager calls and in a captured graph.
    E, k, H, I = 8, 2, 128, 64
    rng = np.random.default_rng(T)
    src = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    gu = mm.mm_mxfp4_quantize(torch.from_numpy(
        rng.standard_normal((2 * E, I, H)).astype(np.float32)).cuda())
    dn = mm.mm_mxfp4_quantize(torch.from_numpy(
        rng.standard_normal((E, H, I)).astype(np.float32)).cuda())

    def step(x):
        logits = x[:, :E].contiguous()
        ids, w, counts, sums, loss = mm.mm_route_logits(logits, k, True)
        out = mm.mm_moe_experts_mxfp4(x, ids, w, *gu, *dn)
        g = mm.mm_route_logits_backward(logits, ids, counts, True, w, loss)
        codes, scales = mm.mm_mxfp4_quantize(x)
        c = mm.mm_mxfp4_gemm(codes, scales, gu[0][0], gu[1][0])
        return ids, w, counts, sums, loss, out, g, codes, c

    def first(x):  # each operator directly behind what wrote its input
        return (*mm.mm_mxfp4_quantize(x),)

    want = [[t.clone() for t in f(src)] for f in (step, first)]
    torch.cuda.synchronize()
    x = torch.empty_like(src)
    for f, w in zip((step, first), want):
        for got in _behind(f, x, src):
            assert all(torch.equal(a, b) for a, b in zip(got, w))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = _behind(f, x, src)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        for got in outs:
            assert all(torch.equal(a, b) for a, b in zip(got, w))
    assert mm.mm_poll_device_status() == mm.MM_OK


@pytest.mark.parametrize("E", [256, 200, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [4, 8])
def test_logits_aligned_to_less_than_a_lane_takes(E, dtype, offset):
    # A lane takes up to 32 bytes at once where the rows allow it; results do not
    # depend on it.
    flat = torch.randn(offset + 70 * E, device="cuda").to(dtype)
    x = flat[offset:].view(70, E)
    y = x.clone()
    dw = torch.randn(70, 5, device="cuda")
    got, same = mm.mm_route_logits(x, 5, True), mm.mm_route_logits(y, 5, True)
    assert all(torch.equal(a, b) for a, b in zip(got, same))
    g = mm.mm_route_logits_backward(x, got[0], got[2], True, dw, got[4])
    assert torch.equal(g, mm.mm_route_logits_backward(y, got[0], got[2], True, dw, got[4]))


@pytest.mark.parametrize("E,k", [(256, 8), (100, 5), (40, 3), (7, 7)])
@pytest.mark.parametrize("T", [31, 32, 33, 128, 129, 255, 256, 257])
def test_batches_around_one_block_and_one_cluster(T, E, k):
    x, mask, _ = _case(T + E, T, E, k, masked=0.2)
    got = mm.mm_route_logits(x, k, True, token_mask=mask)
    _check(x, mask, k, True, got)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in
                   zip(got, mm.mm_route_logits(x, k, True, token_mask=mask)))
    assert mm.mm_poll_device_status() == mm.MM_OK


def _nan_rows(rng, T, E, k):
    """Rows with 0 to E logits that are NaN, others -inf, and seldom k above it."""
    x = np.where(rng.random((T, E)) < rng.random((T, 1)), -np.inf, rng.standard_normal((T, E)))
    few = rng.random((T, 1)) < 0.7  # at most k - 1 above -inf
    rank = np.argsort(np.argsort(rng.random((T, E)), axis=1), axis=1)
    x = np.where(few & (rank >= rng.integers(0, k, (T, 1))), -np.inf, x)
    places = 32 if E <= 32 else 64 if E <= 64 else 128 if E <= 128 else 256
    count = rng.integers(0, E + 1, T)
    count[::3] = E                                   # all of them
    count[1::3] = np.clip(places - k, 0, E)          # as many as leave k places without
    count[::5] = 0
    order = np.argsort(rng.random((T, E)) - (x > -np.inf), axis=1)[:, ::-1]  # -inf first
    put = np.argsort(order, axis=1) < count[:, None]
    return np.where(put, np.nan, x)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T", [24, 200, 1500])  # one block, one cluster, many blocks
@pytest.mark.parametrize("E,k", [(60, 4), (24, 8), (30, 2), (31, 1), (63, 1), (120, 8), (127, 1),
                                 (248, 8), (255, 1), (250, 6), (32, 32), (30, 30), (40, 4),
                                 (128, 8), (256, 1), (1, 1)])
def test_rows_with_nan_select_experts_that_exist(E, k, T, masked):
    # NaN ranks as -inf, equal values by id, and a place past the experts never.
    rng = np.random.default_rng(E * 1000 + T + k)
    x64 = _nan_rows(rng, T, E, k)
    x = torch.from_numpy(x64.astype(np.float32)).cuda()
    x64 = _np64(x)
    rank = np.where(np.isnan(x64), -np.inf, x64)
    want = np.sort(np.argsort(-rank, axis=1, kind="stable")[:, :k], axis=1)
    mask = torch.from_numpy(rng.random(T) < 0.5).cuda() if masked else None
    ids, w, counts, sums, loss = mm.mm_route_logits(x, k, True, token_mask=mask)
    assert np.array_equal(ids.cpu().numpy(), want)
    counted = ~np.isneginf(x64).all(1)
    if masked:
        counted &= mask.cpu().numpy()
    assert np.array_equal(counts.cpu().numpy(), np.bincount(want[counted].ravel(), minlength=E))
    assert int(counts.sum()) == counted.sum() * k
    bad = counted & np.isnan(x64).any(1)
    assert torch.isnan(w[torch.from_numpy(bad).cuda()]).all()
    assert not w[torch.from_numpy(~counted).cuda()].any()
    assert torch.isnan(sums).all() == bad.any() and torch.isnan(loss).all() == bad.any()
    # The gradient of the rows that hold no NaN takes n from the counts.
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    g = _np64(mm.mm_route_logits_backward(x, ids, counts, True, dw, torch.ones(1, device="cuda"),
                                          mask))
    fine = counted & ~bad
    if fine.any():
        exact = ref.route_grad(x64[fine], k, True, _np64(dw)[fine], 1.0, ids=want[fine],
                               counts=counts.cpu().numpy())
        n = max(int(counted.sum()), 1)
        # terms of at most max |dw| and E k / (n k) n / n ..., each within 300 half steps
        size = np.abs(_np64(dw)).max() + E * counts.cpu().numpy().max() / (n * n * k)
        assert np.abs(g[fine] - exact).max() <= 300 * U * size
    assert not g[~counted].any()
    assert mm.mm_poll_device_status() == mm.MM_OK


@pytest.mark.parametrize("T", [30, 250, 20000])
def test_probabilities_far_below_the_largest(T):
    # Two experts d apart: p_1 = e^-d / (1 + e^-d), to the same relative error
    # for every d down to the smallest normal number.
    rng = np.random.default_rng(T)
    d = np.sort(rng.uniform(0, 87, T)).astype(np.float32)
    x = torch.from_numpy(np.stack([np.zeros_like(d), -d], 1)).cuda()
    ids, w, _, _, _ = mm.mm_route_logits(x, 2, False)
    want = np.exp(-d.astype(np.float64))
    want = want / (1 + want)
    # e^-d: the hardware's 2^t within 2^-22 = 4 U, the product with the rest's
    # factor 1 U; the sum 1 + e^-d 1 U of its own and at most half of that
    # error; its reciprocal and the product 1 U each.
    assert (np.abs(_np64(w)[:, 1] / want - 1) <= (5 + 1 + 2.5 + 2 + 0.5) * U).all()
    # dL/dl_1 = p_0 p_1 for dL/dw_1 = 1: p_1 (1 - p_1), one more rounding each in
    # the sum, the difference and the product.
    dw = torch.zeros(T, 2, device="cuda")
    dw[:, 1] = 1
    counts = torch.full((2,), T, dtype=torch.int32, device="cuda")
    g = _np64(mm.mm_route_logits_backward(x, ids, counts, False, dw))[:, 1]
    far = d > 2  # 1 - p_1 does not cancel
    assert (np.abs(g / (want * (1 - want)) - 1)[far] <= (11 + 4) * U).all()


@pytest.mark.parametrize("T", [4097, 100_000, 1 << 27])
@pytest.mark.parametrize("E", [3, 40, 200])
def test_sums_over_many_equal_tokens(T, E):
    # Every p is 1 / E, not a number of the type, so that a plain fp32 sum rounds
    # the same way at every token.
    if E > 3 and T > 100_000:
        T = (1 << 31) // E  # more than 2^31 logits
    x = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    _, _, counts, sums, loss = mm.mm_route_logits(x, 1, False)
    assert counts.tolist() == [T] + [0] * (E - 1)
    # p: the exponentials are 1 and their sum is exact, its reciprocal is within 1
    # U. A lane's partial sums of 8 tokens and what the last ones left: 9 U. Then
    # additions in pairs: 16 warps and the two kinds of sums 5, 8 blocks 3, 32
    # groups 5, and up to 480 blocks / (4 groups 8) = 15 U of those in turn.
    tol = (1 + 9 + 5 + 3 + 5 + 15) * U
    assert (np.abs(_np64(sums) / (T / E) - 1) <= tol).all()
    # loss = E (T / T) (T / E) / T = 1: the counts, the tree, two quotients, two
    # products
    assert abs(float(loss) - 1) <= tol + 14 * U
