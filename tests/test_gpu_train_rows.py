"""Slots by expert, token rows to their slots and back, against the definitions."""
import pytest
import torch

import mixture_experts_layer_mm_gb300 as mm
import train_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(mmlib):
    return mmlib


@pytest.fixture(autouse=True)
def _status():
    yield
    assert mm.mm_poll_device_status() == mm.MM_OK


def _ids(T, E, k, seed=0, skew=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, E, generator=g, device="cuda")
    if skew:
        x = x + torch.randn(1, E, generator=g, device="cuda")
    if k <= E:
        return x.topk(k, dim=-1)[1].to(torch.int32)
    return torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)


# One launch up to 16384 slots; spans of one chunk and of several beyond.
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (5, 3, 3), (33, 7, 2), (64, 128, 8),
                                   (1024, 60, 8), (1025, 60, 8), (4099, 256, 8), (9000, 1, 1),
                                   (700, 4, 32), (60001, 40, 10)])
@pytest.mark.parametrize("masked", [0.0, 0.3, 1.0])
def test_group(T, E, k, masked):
    ids = _ids(T, E, k)
    mask = None if masked == 0 else torch.rand(T, device="cuda") >= masked
    places, offsets = mm.mm_group_slots(ids, E, token_mask=mask)
    # by sorting: the definition's loop is slow for the long ones
    flat = ids.long() if mask is None else torch.where(mask[:, None], ids.long(), E)
    flat = flat.flatten()
    order = torch.sort(flat, stable=True)[1]
    want = torch.empty_like(flat)
    want[order] = torch.arange(T * k, device="cuda")
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    assert torch.equal(offsets[1:].long(), counts.cumsum(0)) and offsets[0] == 0
    assert torch.equal(places.flatten().long(), torch.where(flat < E, want, -1))
    if T * k < 3000:
        p, o = ref.group(ids.cpu(), E, None if mask is None else mask.cpu())
        assert torch.equal(places.cpu(), p) and torch.equal(offsets.cpu(), o)
    again = mm.mm_group_slots(ids, E, token_mask=mask)
    assert torch.equal(again[0], places) and torch.equal(again[1], offsets)


@pytest.mark.parametrize("T,E,k", [(128, 128, 8), (341, 5, 3), (1024, 256, 1), (32, 1, 32),
                                   (1000, 2, 1)])
def test_group_of_a_slot_a_thread(T, E, k):
    for masked in (0.0, 0.4):
        test_group(T, E, k, masked)


@pytest.mark.parametrize("T,E,k", [(205, 5, 5), (1025, 1, 1), (1031, 200, 7), (2048, 256, 8),
                                   (4096, 128, 4), (16383, 33, 1), (2731, 64, 6), (300, 256, 32)])
def test_group_of_a_cluster(T, E, k):
    """1025 to 16384 slots, and just beyond."""
    for masked in (0.0, 0.4):
        test_group(T, E, k, masked)


def test_group_of_a_cluster_flags_bad_ids():
    test_group_drops_and_flags_bad_ids(600)


def test_group_without_tokens():
    places, offsets = mm.mm_group_slots(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 9)
    assert places.shape == (0, 4) and offsets.tolist() == [0] * 10


@pytest.mark.parametrize("T", [50, 5000])
def test_group_drops_and_flags_bad_ids(T):
    ids = _ids(T, 16, 4)
    ids[3, 1], ids[7, 0], ids[9, 3] = 16, -1, 2 ** 31 - 1
    mask = torch.ones(T, dtype=torch.uint8, device="cuda")
    mask[9] = 0                                       # a masked token's ids do not matter
    places, offsets = mm.mm_group_slots(ids, 16, token_mask=mask)
    assert mm.mm_poll_device_status() == mm.MM_ERR_DEVICE
    p, o = ref.group(ids.cpu(), 16, mask.cpu())
    assert torch.equal(places.cpu(), p) and torch.equal(offsets.cpu(), o)
    ids[3, 1] = ids[7, 0] = 0
    mm.mm_group_slots(ids, 16, token_mask=mask)
    assert mm.mm_poll_device_status() == mm.MM_OK


@pytest.mark.parametrize("T,H,E,k", [(1, 8, 1, 1), (7, 264, 5, 3), (64, 2048, 128, 8),
                                     (300, 4104, 40, 10), (2000, 64, 256, 32), (33, 8200, 8, 2)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("masked", [0.0, 0.4])
def test_dispatch_and_combine(T, H, E, k, dtype, masked):
    g = torch.Generator(device="cuda").manual_seed(T)
    ids = _ids(T, E, k, seed=T)
    mask = None if masked == 0 else torch.rand(T, generator=g, device="cuda") >= masked
    x = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    w = torch.rand(T, k, generator=g, device="cuda")
    places, offsets = mm.mm_group_slots(ids, E, token_mask=mask)
    rows = torch.full((T * k + 3, H), 7.0, dtype=dtype, device="cuda")
    row_w = torch.full((T * k + 3,), 7.0, device="cuda")
    r, rw = mm.mm_dispatch_rows(x, places, w=w, rows=rows, row_w=row_w)
    assert r is rows and rw is row_w
    used = int(offsets[-1])
    p = places.flatten().long()
    slots = torch.nonzero(p >= 0).flatten()
    want, want_w = torch.full_like(rows, 7.0), torch.full_like(row_w, 7.0)
    want[p[slots]], want_w[p[slots]] = x[slots // k], w.flatten()[slots]
    assert torch.equal(rows, want) and torch.equal(row_w, want_w)   # rows behind are left alone
    plain, none = mm.mm_dispatch_rows(x, places)
    assert none is None and torch.equal(plain[:used], rows[:used])

    y = torch.randn(T * k, H, generator=g, device="cuda").to(dtype)
    y[used:] = float("nan")                                         # not read
    out = mm.mm_combine_rows(y, places, w=w)
    want, mag = ref.combine(y.nan_to_num(0), places, w)
    ref.close(out, want, mag, k + 1, "weighted")
    vals = torch.rand(T * k, generator=g, device="cuda")
    given = torch.empty(T, H, dtype=dtype, device="cuda")
    out, v = mm.mm_combine_rows(y, places, row_values=vals, out=given)
    assert out is given
    want, mag = ref.combine(y.nan_to_num(0), places)
    ref.close(out, want, mag, k + 1, "plain")
    assert torch.equal(v, torch.where(places >= 0, vals[places.clamp_min(0).long()], 0.0))


def test_combine_is_the_gradient_of_dispatch():
    """<dispatch(x), y> = <x, combine(y)>, also where a token has a row twice."""
    x = torch.randn(40, 64, device="cuda").bfloat16()
    ids = _ids(40, 6, 3)
    ids[5] = ids[5, 0]
    places, _ = mm.mm_group_slots(ids, 6)
    y = torch.randn(120, 64, device="cuda").bfloat16()
    rows, _ = mm.mm_dispatch_rows(x, places)
    left = (rows.double() * y.double()).sum()
    right = (x.double() * mm.mm_combine_rows(y, places).double()).sum()
    mag = (rows.double() * y.double()).abs().sum()
    assert abs(left - right) <= 2.0 ** -8 * mag


def test_bad_places_are_skipped_and_flagged():
    x = torch.randn(6, 64, device="cuda").bfloat16()
    places = torch.arange(12, dtype=torch.int32, device="cuda").view(6, 2)
    places[2, 1], places[4, 0] = 12, -2
    rows = torch.zeros(12, 64, dtype=torch.bfloat16, device="cuda")
    mm.mm_dispatch_rows(x, places, rows=rows)
    assert mm.mm_poll_device_status() == mm.MM_ERR_DEVICE
    good = places.clone()
    good[2, 1] = good[4, 0] = -1
    assert torch.equal(rows[5], torch.zeros(64, device="cuda").bfloat16())
    out = mm.mm_combine_rows(rows, places)
    assert mm.mm_poll_device_status() == mm.MM_ERR_DEVICE
    assert torch.equal(out, mm.mm_combine_rows(rows, good))


def test_rows_past_32_bit_offsets():
    """Rows whose elements lie beyond 2^31."""
    H, R = 65536, 40000                                    # 2.6e9 elements
    rows = torch.empty(R, H, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(2, H, device="cuda").bfloat16()
    places = torch.tensor([[R - 1, 5], [R - 2, 0]], dtype=torch.int32, device="cuda")
    mm.mm_dispatch_rows(x, places, rows=rows)
    for t in range(2):
        for j in range(2):
            assert torch.equal(rows[places[t, j]], x[t])
    out = mm.mm_combine_rows(rows, places)
    assert torch.equal(out, (2 * x.float()).bfloat16())


def test_no_rows_at_all():
    x = torch.randn(5, 64, device="cuda").bfloat16()
    places = torch.full((5, 2), -1, dtype=torch.int32, device="cuda")
    empty = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    mm.mm_dispatch_rows(x, places, rows=empty)
    out, v = mm.mm_combine_rows(empty, places, row_values=torch.empty(0, device="cuda"))
    assert not out.any() and not v.any()
    assert mm.mm_combine_rows(x, places[:0]).shape == (0, 64)


def test_streams_and_graphs_share_nothing():
    """The same calls on two streams at once, and captured and replayed on new inputs."""
    T, H, E, k = 3000, 256, 32, 8
    ids = [_ids(T, E, k, seed=s) for s in range(2)]
    xs = [torch.randn(T, H, device="cuda").bfloat16() for _ in range(2)]

    def run(i, stream=None):
        p, o = mm.mm_group_slots(ids[i], E, stream=stream)
        r, _ = mm.mm_dispatch_rows(xs[i], p, stream=stream)
        return p, o, r, mm.mm_combine_rows(r, p, stream=stream)

    want = [run(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [run(i, streams[i]) for i in range(2)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(0)
    ids[0].copy_(ids[1])
    xs[0].copy_(xs[1])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want[1]))


def test_groups_of_a_cluster_at_the_same_time():
    ids = [_ids(1000 + 400 * s, 64, 8, seed=s) for s in range(2)]
    want = [mm.mm_group_slots(i, 64) for i in ids]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[mm.mm_group_slots(ids[i], 64, stream=streams[i]) for i in range(2)] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        assert all(torch.equal(x, y) for a, b in zip(pair, want) for x, y in zip(a, b))


def test_good_places_are_written_beside_bad_ones():
    """Every row: copies of their tokens, and those that only a bad place would have had
    as they were."""
    x = torch.randn(6, 64, device="cuda").bfloat16()
    w = torch.rand(6, 2, device="cuda")
    places = torch.arange(11, -1, -1, dtype=torch.int32, device="cuda").view(6, 2)
    places[2, 1], places[4, 0], places[5, 1] = 12, -2, -1     # not 6, 3 and 0
    rows, row_w = torch.full((12, 64), 3.0, device="cuda").bfloat16(), torch.full((12,), 3.0, device="cuda")
    want, want_w = rows.clone(), row_w.clone()
    for f, p in enumerate(places.flatten().tolist()):
        if 0 <= p < 12:
            want[p], want_w[p] = x[f // 2], w[f // 2, f % 2]
    mm.mm_dispatch_rows(x, places, w=w, rows=rows, row_w=row_w)
    assert mm.mm_poll_device_status() == mm.MM_ERR_DEVICE
    assert torch.equal(rows, want) and torch.equal(row_w, want_w)
    assert (want == 3).all(1).sum() == 3
    vals = torch.rand(12, device="cuda")
    out, v = mm.mm_combine_rows(rows, places, row_values=vals)
    assert mm.mm_poll_device_status() == mm.MM_ERR_DEVICE
    good = torch.where((places >= 0) & (places < 12), places, -1)
    total, mag = ref.combine(rows, good)
    ref.close(out, total, mag, 3)
    assert torch.equal(v, torch.where(good >= 0, vals[good.clamp_min(0).long()], 0.0))


@pytest.mark.parametrize("E", [(1 << 32) + 8, 1 << 31, 257])
def test_too_many_experts_are_refused(E):
    with pytest.raises(mm.MMError) as e:
        mm.mm_group_slots(_ids(4, 8, 2), E)
    assert e.value.code == mm.MM_ERR_UNSUPPORTED
