"""Products grouped by expert over ragged segments and their gradients, against
float64."""
import pytest
import torch

import mixture_experts_layer_mm_gb300 as mm
import train_reference as ref

pytestmark = pytest.mark.gpu
B, H, F = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib(mmlib):
    return mmlib


@pytest.fixture(autouse=True)
def _status():
    yield
    assert mm.mm_poll_device_status() == mm.MM_OK


def _offsets(lens, lead=0):
    return torch.tensor([lead] + [lead + sum(lens[:i + 1]) for i in range(len(lens))],
                        dtype=torch.int32, device="cuda")


def _rand(g, *shape, dtype=B, std=1.0):
    return (std * torch.randn(*shape, generator=g, device="cuda")).to(dtype)


# Rows of the experts; lead and trail: rows outside of every segment, which hold NaN and
# infinities.
LENS = {
    "one row": ([1], 0, 0),
    "nothing": ([0, 0, 0], 2, 3),
    "few": ([1, 3, 0, 17, 65, 130, 0], 5, 9),
    "steps of 16": ([16, 48, 0, 32, 256], 0, 0),
    "chunk ends": ([255, 256, 257, 512, 0, 513], 1, 0),
    "one long": ([3001], 0, 7),
    "uneven": ([0, 2000, 3, 0, 0, 300], 0, 0),
}


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("N,K", [(64, 64), (8, 8), (264, 200), (1000, 1016), (520, 72)])
@pytest.mark.parametrize("dtype", [B, H])
def test_rows(lens, N, K, dtype):
    """Forward and dx. Rows outside of the segments stay as they are."""
    lens, lead, trail = LENS[lens]
    g = torch.Generator(device="cuda").manual_seed(N)
    R, E, off = sum(lens) + lead + trail, len(lens), _offsets(lens, lead)
    w = _rand(g, E, N, K, dtype=dtype, std=0.1)
    for way, cols, width in (("forward", K, N), ("dx", N, K)):
        x = _rand(g, R, cols, dtype=dtype)
        x[:lead] = float("inf")
        x[R - trail:] = float("nan")
        out = torch.full((R, width), 3.0, dtype=dtype, device="cuda")
        f = mm.mm_grouped_product if way == "forward" else mm.mm_grouped_product_dx
        assert f(x, w, off, out=out) is out
        a, b = lead, R - trail
        want, mag = ref.product(x, w, off, way)
        ref.close(out[a:b], want[a:b], mag[a:b], cols + 16, way)
        assert (out[:a] == 3).all() and (out[b:] == 3).all()
        if a == 0 and b == R:
            assert torch.equal(f(x, w, off), out)            # the same on every call


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("N,K", [(64, 64), (8, 8), (264, 200), (1000, 328), (520, 1024)])
@pytest.mark.parametrize("dtype,out_dtype", [(B, B), (H, H), (B, F), (H, F)])
def test_weights(lens, N, K, dtype, out_dtype):
    lens, lead, trail = LENS[lens]
    g = torch.Generator(device="cuda").manual_seed(K)
    R, E, off = sum(lens) + lead + trail, len(lens), _offsets(lens, lead)
    dy, x = _rand(g, R, N, dtype=dtype), _rand(g, R, K, dtype=dtype)
    dy[:lead], x[:lead] = float("inf"), float("nan")
    dy[R - trail:], x[R - trail:] = float("nan"), float("inf")
    a, b = lead, R - trail
    want, mag = ref.product(dy.nan_to_num(0, 0, 0), x.nan_to_num(0, 0, 0), off, "dw")
    got = mm.mm_grouped_product_dw(dy, x, off, out_dtype=out_dtype)
    assert got.dtype == out_dtype
    terms = max(lens) + 16
    ref.close(got, want, mag, terms, "dw")
    assert torch.equal(mm.mm_grouped_product_dw(dy, x, off, out_dtype=out_dtype), got)
    # Added to what is there: one more fp32 addition, and one rounding of the sum.
    old = _rand(g, E, N, K, dtype=out_dtype, std=3.0)
    acc = old.clone()
    assert mm.mm_grouped_product_dw(dy, x, off, out=acc, accumulate=True) is acc
    ref.close(acc, want + old.double(), mag + old.double().abs(), terms + 1, "accumulated")
    for e, n in enumerate(lens):
        if n == 0:
            assert not got[e].any() and torch.equal(acc[e], old[e])


def test_long_sums_keep_their_roundings():
    """An fp32 result of many rows of one sign: each 512 rows are one accumulation of the
    tensor cores (at most 32 steps of 16 that cut up to 2^-23 each), the rest fp32
    additions of up to 2^-24."""
    R = 16384
    dy = (1 + torch.rand(R, 72, device="cuda")).bfloat16()
    x = (1 + torch.rand(R, 136, device="cuda")).bfloat16()
    for E in (1, 2):
        off = _offsets([R // E] * E)
        got = mm.mm_grouped_product_dw(dy, x, off, out_dtype=F)
        want, _ = ref.product(dy, x, off, "dw")
        steps = 32 * 2.0 ** -23 + R // 512 * 2.0 ** -24
        assert ((got.double() - want).abs() <= steps * want).all()


@pytest.mark.parametrize("E,R,N,K,parts", [(1, 8192, 64, 64, True), (2, 30001, 128, 72, True),
                                           (1, 20000, 512, 512, True), (8, 9000, 640, 328, False),
                                           (128, 9000, 256, 256, False)])
def test_parts(E, R, N, K, parts):
    """Few tiles with long segments are cut into parts."""
    for out in (B, F):
        size = mm.mm_grouped_product_dw_workspace_size(R, E, N, K, out)
        assert (size > 0) == parts
    g = torch.Generator(device="cuda").manual_seed(R)
    lens = torch.bincount(torch.randint(0, E, (R,), generator=g, device="cuda"),
                          minlength=E).tolist()
    if E == 2:
        lens = [R - 5, 5]                                   # one of many parts, one of one
    dy, x, off = _rand(g, R, N), _rand(g, R, K), _offsets(lens)
    want, mag = ref.product(dy, x, off, "dw")
    for out in (B, F):
        ref.close(mm.mm_grouped_product_dw(dy, x, off, out_dtype=out), want, mag, max(lens) + 16)
        old = torch.randn(E, N, K, generator=g, device="cuda").to(out)
        acc = mm.mm_grouped_product_dw(dy, x, off, out=old.clone(), accumulate=True)
        ref.close(acc, want + old.double(), mag + old.double().abs(), max(lens) + 17)


def test_many_experts_of_uneven_load():
    g = torch.Generator(device="cuda").manual_seed(5)
    E, R, N, K = 256, 6000, 136, 264
    p = torch.exp(1.5 * torch.randn(E, generator=g, device="cuda"))
    lens = torch.bincount(torch.multinomial(p, R, replacement=True, generator=g),
                          minlength=E).tolist()
    off = _offsets(lens)
    x, dy, w = _rand(g, R, K), _rand(g, R, N), _rand(g, E, N, K)
    for f, a, b, way, terms in ((mm.mm_grouped_product, x, w, "forward", K),
                                (mm.mm_grouped_product_dx, dy, w, "dx", N),
                                (mm.mm_grouped_product_dw, dy, x, "dw", max(lens))):
        want, mag = ref.product(a, b, off, way)
        ref.close(f(a, b, off), want, mag, terms + 16, way)


@pytest.mark.parametrize("E,R,N,K", [(4, 5007, 1240, 2056), (1, 12300, 2040, 1992),
                                     (12, 11000, 1240, 1544), (1, 8200, 2048, 1000)])
@pytest.mark.parametrize("dtype", [B, H])
def test_weights_of_long_segments(E, R, N, K, dtype):
    """Mean lengths from which dw's MMAs run over both CTAs of a cluster."""
    g = torch.Generator(device="cuda").manual_seed(R)
    lens = torch.bincount(torch.randint(0, E, (R,), generator=g, device="cuda"),
                          minlength=E).tolist()
    if E == 12:
        lens = [6000, 0, 1, 17, 4982] + [0] * 7
    lead, trail = 3, 5
    dy, x = (_rand(g, R + 8, c, dtype=dtype) for c in (N, K))
    dy[:lead], x[:lead], dy[R + lead:], x[R + lead:] = [float("nan")] * 4
    off = _offsets(lens, lead)
    want, mag = ref.product(dy.nan_to_num(0), x.nan_to_num(0), off, "dw")
    got = mm.mm_grouped_product_dw(dy, x, off)
    ref.close(got, want, mag, max(lens) + 16, "dw")
    assert torch.equal(mm.mm_grouped_product_dw(dy, x, off), got)
    old = _rand(g, E, N, K, dtype=dtype, std=30.0)
    acc = mm.mm_grouped_product_dw(dy, x, off, out=old.clone(), accumulate=True)
    ref.close(acc, want + old.double(), mag + old.double().abs(), max(lens) + 17, "accumulated")


@pytest.mark.parametrize("E,R,N,K", [(200, 26000, 1000, 1016), (128, 24001, 136, 2056),
                                     (90, 25003, 1544, 520)])
def test_weights_of_many_segments_beyond_the_cache(E, R, N, K):
    """Rows of more bytes than L2 keeps, which dw brings there a tile ahead; one segment
    of many tiles' rows, some of none."""
    g = torch.Generator(device="cuda").manual_seed(R)
    p = torch.exp(0.7 * torch.randn(E, generator=g, device="cuda"))
    p[::17] = 0
    lens = torch.bincount(torch.multinomial(p, R - 2500, replacement=True, generator=g),
                          minlength=E).tolist()
    lens[7] += 2500
    lead, trail = 1, 3
    dy, x = (_rand(g, R + 4, c) for c in (N, K))
    dy[:lead], x[:lead], dy[R + lead:], x[R + lead:] = [float("nan")] * 4
    off = _offsets(lens, lead)
    want, mag = ref.product(dy.nan_to_num(0), x.nan_to_num(0), off, "dw")
    got = mm.mm_grouped_product_dw(dy, x, off)
    ref.close(got, want, mag, max(lens) + 16, "dw")
    assert torch.equal(mm.mm_grouped_product_dw(dy, x, off), got)


@pytest.mark.parametrize("lens,lead,trail", [([1], 0, 0), ([0, 3, 0, 1, 2], 2, 1), ([64], 0, 5),
                                             ([17, 0, 40], 3, 0), ([130], 0, 0), ([65, 33], 1, 1)])
@pytest.mark.parametrize("F,D", [(8, 2048), (72, 1416), (128, 1992), (520, 1096), (1000, 4104)])
@pytest.mark.parametrize("dtype", [B, H])
def test_few_rows_of_long_reductions(lens, lead, trail, F, D, dtype):
    """The reduction shared out among a cluster's blocks, forward and dx."""
    g = torch.Generator(device="cuda").manual_seed(D)
    R, off = sum(lens) + lead + trail, _offsets(lens, lead)
    a, b = lead, R - trail
    for way, shape in (("forward", (F, D)), ("dx", (D, F))):
        w = _rand(g, len(lens), *shape, dtype=dtype, std=0.1)
        x = _rand(g, R, D, dtype=dtype)
        x[:a], x[b:] = float("inf"), float("nan")
        out = torch.full((R, F), 3.0, dtype=dtype, device="cuda")
        f = mm.mm_grouped_product if way == "forward" else mm.mm_grouped_product_dx
        f(x, w, off, out=out)
        want, mag = ref.product(x, w, off, way)
        ref.close(out[a:b], want[a:b], mag[a:b], D + 16, way)
        assert (out[:a] == 3).all() and (out[b:] == 3).all()
        again = torch.full_like(out, 3.0)
        f(x, w, off, out=again)
        assert torch.equal(again, out)


def test_another_experts_infinities_stay_with_it():
    """Segments share tiles and stages of rows; their values do not meet."""
    lens = [37, 90, 5, 64]
    off = _offsets(lens)
    g = torch.Generator(device="cuda").manual_seed(2)
    x, dy, w = _rand(g, 196, 128), _rand(g, 196, 72), _rand(g, 4, 72, 128)
    want = [mm.mm_grouped_product(x, w, off), mm.mm_grouped_product_dx(dy, w, off),
            mm.mm_grouped_product_dw(dy, x, off)]
    x[37:127], dy[37:127], w[1] = float("nan"), float("inf"), float("nan")
    got = [mm.mm_grouped_product(x, w, off), mm.mm_grouped_product_dx(dy, w, off),
           mm.mm_grouped_product_dw(dy, x, off)]
    for a, b in zip(got[:2], want[:2]):
        assert torch.equal(a[:37], b[:37]) and torch.equal(a[127:], b[127:])
        assert not torch.isfinite(a[37:127]).any()
    assert torch.equal(got[2][[0, 2, 3]], want[2][[0, 2, 3]])
    assert not torch.isfinite(got[2][1]).any()


@pytest.mark.parametrize("bad", ["falls", "beyond", "negative"])
def test_bad_offsets_write_nothing(bad):
    off = {"falls": [0, 70, 60, 100], "beyond": [0, 10, 20, 101], "negative": [-1, 10, 20, 100]}[bad]
    off = torch.tensor(off, dtype=torch.int32, device="cuda")
    x = torch.randn(100, 64, device="cuda").bfloat16()
    w = torch.randn(3, 64, 64, device="cuda").bfloat16()
    for f in (lambda o: mm.mm_grouped_product(x, w, off, out=o),
              lambda o: mm.mm_grouped_product_dx(x, w, off, out=o)):
        o = torch.full((100, 64), 2.0, device="cuda").bfloat16()
        f(o)
        assert mm.mm_poll_device_status() == mm.MM_ERR_DEVICE
        assert (o == 2).all()
    o = torch.full((3, 64, 64), 2.0, device="cuda")
    mm.mm_grouped_product_dw(x, x, off, out=o)
    assert mm.mm_poll_device_status() == mm.MM_ERR_DEVICE
    assert (o == 2).all()
    long = torch.randn(8192, 64, device="cuda").bfloat16()          # in parts
    off = torch.tensor([0, 9000], dtype=torch.int32, device="cuda")
    o = torch.full((1, 64, 64), 2.0, device="cuda")
    mm.mm_grouped_product_dw(long, long, off, out=o)
    assert mm.mm_poll_device_status() == mm.MM_ERR_DEVICE
    assert (o == 2).all()


@pytest.mark.parametrize("bad", [[0, 30, 20, 50], [0, 10, 20, 51], [-1, 10, 20, 50]])
def test_bad_offsets_of_few_rows_write_nothing(bad):
    """Where a cluster's blocks share the reduction; the next call is sound again."""
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = _rand(g, 50, 2048), _rand(g, 3, 136, 2048, std=0.1)
    wt = w.transpose(1, 2).contiguous()
    good = _offsets([20, 0, 30])
    want, mag = ref.product(x, w, good, "forward")
    for f, m in ((mm.mm_grouped_product, w), (mm.mm_grouped_product_dx, wt)):
        o = torch.full((50, 136), 2.0, device="cuda").bfloat16()
        f(x, m, off, out=o)
        assert mm.mm_poll_device_status() == mm.MM_ERR_DEVICE
        assert (o == 2).all()
        ref.close(f(x, m, good, out=o), want, mag, 2048 + 16)


def test_few_rows_on_streams_and_in_graphs():
    """Calls that run at the same time, captured and not, with their own offsets."""
    g = torch.Generator(device="cuda").manual_seed(2)
    x = [_rand(g, 48, 2048) for _ in range(2)]
    w = [_rand(g, 4, 520, 2048, std=0.1) for _ in range(2)]
    off = [_offsets([10, 0, 33, 5]), _offsets([1, 40, 0, 7])]
    want = [mm.mm_grouped_product(x[i], w[i], off[i]) for i in range(2)]
    outs = [torch.empty_like(o) for o in want]
    graphs = []
    for i in range(2):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(3):
                mm.mm_grouped_product(x[i], w[i], off[i], out=outs[i])
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            outs[i].fill_(7)
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        with torch.cuda.stream(streams[2]):
            eager = [mm.mm_grouped_product(x[i], w[i], off[i]) for i in range(2)]
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], want[i]) and torch.equal(eager[i], want[i])


def test_buffers_aligned_to_16_bytes_only():
    g = torch.Generator(device="cuda").manual_seed(3)
    R, N, K = 70, 72, 136
    off = _offsets([30, 40])

    def odd(t):  # the same values 16 bytes behind a 256-byte boundary
        b = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")
        v = b[8:8 + t.numel()].view(t.shape)
        v.copy_(t)
        assert v.data_ptr() % 32 == 16
        return v

    x, dy, w = _rand(g, R, K), _rand(g, R, N), _rand(g, 2, N, K)
    for f, a, b in ((mm.mm_grouped_product, x, w), (mm.mm_grouped_product_dx, dy, w),
                    (mm.mm_grouped_product_dw, dy, x)):
        want = f(a, b, off)
        got = f(odd(a), odd(b), off, out=odd(torch.zeros_like(want)))
        assert torch.equal(got, want)


def test_no_rows():
    w = torch.randn(3, 64, 72, device="cuda").bfloat16()
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    x, dy = w.new_empty(0, 72), w.new_empty(0, 64)
    assert mm.mm_grouped_product(x, w, off).shape == (0, 64)
    assert mm.mm_grouped_product_dx(dy, w, off).shape == (0, 72)
    assert not mm.mm_grouped_product_dw(dy, x, off).any()
    acc = torch.ones(3, 64, 72, device="cuda")
    mm.mm_grouped_product_dw(dy, x, off, out=acc, accumulate=True)
    assert (acc == 1).all()


def test_results_past_32_bit_offsets():
    """Results and inputs of more than 2^31 elements: the first and the last rows."""
    R, N, K = 1_100_000, 2048, 8
    x = torch.randn(R, K, device="cuda").bfloat16()
    w = torch.randn(2, N, K, device="cuda").bfloat16()
    off = _offsets([3, R - 10], 0)
    y = mm.mm_grouped_product(x, w, off)
    for rows, e in ((slice(0, 3), 0), (slice(R - 700, R - 7), 1)):
        want = x[rows].double() @ w[e].double().T
        ref.close(y[rows], want, x[rows].double().abs() @ w[e].double().abs().T, K + 16)
    dx = mm.mm_grouped_product_dx(y, w, off)
    rows = slice(R - 700, R - 7)
    ref.close(dx[rows], y[rows].double() @ w[1].double(),
              y[rows].double().abs() @ w[1].double().abs(), N + 16)
    off = _offsets([300, 500], R - 900)
    dw = mm.mm_grouped_product_dw(y, x, off)
    want, mag = ref.product(y[R - 900:], x[R - 900:], off - (R - 900), "dw")
    ref.close(dw, want, mag, 516)


def test_weights_past_32_bit_offsets():
    E, N, K = 256, 4096, 2056                                # 2.2e9 values
    off = torch.full((E + 1,), 0, dtype=torch.int32, device="cuda")
    off[E] = 40
    dy, x = torch.randn(40, N, device="cuda").bfloat16(), torch.randn(40, K, device="cuda").bfloat16()
    dw = mm.mm_grouped_product_dw(dy, x, off)
    ref.close(dw[-1], dy.double().T @ x.double(), dy.double().abs().T @ x.double().abs(), 56)
    assert not dw[0].any() and not dw[E - 2].any()
    y = mm.mm_grouped_product(x, dw, off)
    ref.close(y, x.double() @ dw[-1].double().T, x.double().abs() @ dw[-1].double().abs().T, K + 16)
    back = mm.mm_grouped_product_dx(dy, dw, off)
    ref.close(back, dy.double() @ dw[-1].double(), dy.double().abs() @ dw[-1].double().abs(), N + 16)


def test_fp16_results_overflow_to_infinity():
    x = torch.full((16, 64), 200.0, dtype=H, device="cuda")
    w = torch.full((1, 64, 64), 200.0, dtype=H, device="cuda")
    off = _offsets([16])
    assert (mm.mm_grouped_product(x, w, off) == float("inf")).all()
    assert (mm.mm_grouped_product_dw(x, x, off, out_dtype=F) == 16 * 40000).all()


def test_streams_and_graphs_share_nothing():
    g = torch.Generator(device="cuda").manual_seed(9)
    R, N, K = 9000, 128, 72                                  # dw in parts
    off = [_offsets([R - 100, 100]), _offsets([4000, R - 4000])]
    x, dy, w = ([_rand(g, *s) for _ in range(2)] for s in ((R, K), (R, N), (2, N, K)))
    assert mm.mm_grouped_product_dw_workspace_size(R, 2, N, K, B) > 0

    def run(i, stream=None):
        return (mm.mm_grouped_product(x[i], w[i], off[i], stream=stream),
                mm.mm_grouped_product_dx(dy[i], w[i], off[i], stream=stream),
                mm.mm_grouped_product_dw(dy[i], x[i], off[i], stream=stream))

    want = [run(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [run(i, streams[i]) for i in range(2)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for i, gr in enumerate(graphs):
        with torch.cuda.graph(gr):
            outs.append(run(i))
    for i, s in enumerate(streams):                          # both at once
        with torch.cuda.stream(s):
            graphs[i].replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    for a in (x, dy, w, off):                                # other inputs, the same graph
        a[0].copy_(a[1])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(outs[0], want[1]))


def test_back_to_back_calls_wait_for_one_another():
    """Each product reads what the one before it wrote."""
    g = torch.Generator(device="cuda").manual_seed(4)
    off = _offsets([300, 0, 724])
    w = [_rand(g, 3, 256, 256, std=1 / 16) for _ in range(2)]
    x = _rand(g, 1024, 256)
    step = [x]
    for i in range(6):
        step.append(mm.mm_grouped_product(step[-1], w[i % 2], off))
        torch.cuda.synchronize()
    for _ in range(20):
        y = x
        for i in range(6):
            y = mm.mm_grouped_product(y, w[i % 2], off)
        assert torch.equal(y, step[-1])


@pytest.mark.parametrize("E,R,N,K", [(60, 15020, 1000, 1016), (128, 33000, 264, 520),
                                     (40, 15800, 1000, 1024), (2, 2100, 520, 2040),
                                     (1, 2049, 1000, 2048), (100, 51300, 264, 512)])
@pytest.mark.parametrize("dtype", [B, H])
def test_weights_where_copies_take_two_lines_a_row(E, R, N, K, dtype):
    """Mean lengths from which dw's MMAs run over both CTAs: of rows that are no whole number
    of 128-byte lines (of x, then of dy), and of others; a long segment, some of none."""
    g = torch.Generator(device="cuda").manual_seed(R)
    p = torch.exp(0.5 * torch.randn(E, generator=g, device="cuda"))
    p[1::9] = 0
    lens = torch.bincount(torch.multinomial(p, R, replacement=True, generator=g),
                          minlength=E).tolist()
    lead, trail = 2, 3
    dy, x = (_rand(g, R + 5, c, dtype=dtype) for c in (N, K))
    dy[:lead], x[:lead], dy[R + lead:], x[R + lead:] = [float("nan")] * 4
    off = _offsets(lens, lead)
    want, mag = ref.product(dy.nan_to_num(0), x.nan_to_num(0), off, "dw")
    for out in (dtype, F):
        got = mm.mm_grouped_product_dw(dy, x, off, out_dtype=out)
        ref.close(got, want, mag, max(lens) + 16, "dw")
        assert torch.equal(mm.mm_grouped_product_dw(dy, x, off, out_dtype=out), got)
        old = _rand(g, E, N, K, dtype=out, std=30.0)
        acc = mm.mm_grouped_product_dw(dy, x, off, out=old.clone(), accumulate=True)
        ref.close(acc, want + old.double(), mag + old.double().abs(), max(lens) + 17, "accumulated")


# fp32 results of segments of several slices: in the epilogue's registers, added up in
# memory, and in parts, which are sums of slices themselves. (E, N, K, rows of the
# segments, parts)
SLICED = {"registers": (8, 640, 328, [14000, 3000, 3000, 0, 1, 5, 4, 1], False),
          "memory": (128, 264, 512, [20000] + [300] * 127, False),
          "parts": (1, 512, 512, [20000], True)}


@pytest.mark.parametrize("name", SLICED)
def test_slices_of_long_segments_keep_their_roundings(name):
    """Values of one sign. A slice of 512 rows is 32 steps of 16 rows; each cuts up to 2^-23
    of the sum so far, which grows evenly: 16.5 of 2^-23 of the slice's at most (18 where
    the rows' sizes differ by chance), half of it on average. Then one fp32 addition a slice
    and a part, 2^-24 of the sum so far each. In one accumulation 2240 rows (the parts')
    would lose 2.4e-6 on average and 14000 rows 15e-6."""
    E, N, K, lens, parts = SLICED[name]
    R, off = sum(lens), _offsets(lens)
    assert (mm.mm_grouped_product_dw_workspace_size(R, E, N, K, F) > 0) == parts
    g = torch.Generator(device="cuda").manual_seed(8)
    dy, x = ((1 + torch.rand(R, c, generator=g, device="cuda")).bfloat16() for c in (N, K))
    got = mm.mm_grouped_product_dw(dy, x, off, out_dtype=F)
    for e in [e for e in range(E) if lens[e] > 512] + [E - 1]:
        a, b = off[e].item(), off[e + 1].item()
        want = dy[a:b].double().T @ x[a:b].double()
        err = (got[e].double() - want) / want
        adds = lens[e] // 512 + 2 + (lens[e] // 2240 + 1 if parts else 0)
        most = 18 * 2.0 ** -23 + (adds + 1) / 2 * 2.0 ** -24
        assert err.abs().max() <= most
        assert err.mean().abs() <= 9 * 2.0 ** -23 + 0.1 * (adds + 1) / 2 * 2.0 ** -24
