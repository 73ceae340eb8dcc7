"""The microscaled 4-bit operators against their float64 definitions."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_mm_gb300 as mm
import mx_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(mmlib):
    return mmlib


def _np64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def _status_ok():
    torch.cuda.synchronize()
    assert mm.mm_poll_device_status() == mm.MM_OK


def _spread(seed, *shape, std=1.0):
    """Values whose blocks cover many powers of two, some elements exactly on e2m1 borders."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-6, 7, (*shape[:-1], 1)))
    border = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5, -0.25, -3.5], shape)
    return (np.where(rng.random(shape) < 0.1, border, x) * std).astype(np.float32)


def _quantise_ref(x):
    s = ref.scale_bytes(x)
    return ref.codes_under(x, s), s


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("batch,rows,K", [(None, 1, 32), (None, 64, 2048), (3, 129, 96),
                                          (2, 128, 160), (1, 5, 640), (5, 33, 1056), (2, 1, 4096)])
def test_quantise_is_exact(batch, rows, K, dtype):
    shape = (rows, K) if batch is None else (batch, rows, K)
    x = torch.from_numpy(_spread(rows + K, *shape)).cuda().to(dtype)
    codes, scales = mm.mm_mxfp4_quantize(x)
    _status_ok()
    x64 = _np64(x).reshape(-1, rows, K)
    got_c = codes.cpu().numpy().reshape(-1, rows, K // 2)
    got_s = scales.cpu().numpy().reshape(len(x64), *mm.mm_mxfp4_scales_shape(rows, K))
    for b, m in enumerate(x64):
        c, s = _quantise_ref(m)
        assert np.array_equal(got_s[b], ref.tile(s))  # padding bytes are zero
        assert np.array_equal(got_c[b], ref.pack(c))
    want = np.stack([ref.quantised(m) for m in x64]).reshape(shape)
    for out in (torch.float32, torch.bfloat16):
        assert np.array_equal(_np64(mm.mm_mxfp4_dequantize(codes, scales, out)), want)
    half = mm.mm_mxfp4_dequantize(codes, scales, torch.float16).cpu()
    assert torch.equal(half, torch.from_numpy(want).to(torch.float32).to(torch.float16))


def test_quantise_extremes():
    rows = []
    rows.append(np.zeros(32))                                     # nothing
    rows.append(np.full(32, -0.0))
    rows.append(np.r_[np.full(31, 2.0 ** -149), 0.0])             # smallest subnormals
    rows.append(np.r_[2.0 ** -126, np.full(31, 2.0 ** -128)])     # under the smallest scale
    rows.append(np.r_[float(np.finfo(np.float32).max), -np.ones(31)])
    rows.append(np.r_[np.nextafter(np.float32(8), np.float32(0)), np.full(31, 6.9)])  # saturates
    rows.append(np.r_[8.0, np.full(31, 2.5)])
    rows.append(np.r_[4.0, np.linspace(-6, 6, 31)])
    rows.append(np.r_[np.inf, np.ones(31)])
    rows.append(np.r_[np.ones(31), np.nan])
    rows.append(np.r_[-np.inf, np.full(31, np.nan)])
    x = np.stack(rows).astype(np.float32)
    codes, scales = mm.mm_mxfp4_quantize(torch.from_numpy(x).cuda())
    c, s = _quantise_ref(x.astype(np.float64))
    assert np.array_equal(scales.cpu().numpy(), ref.tile(s))
    fine = (s != 255)[:, 0]
    assert np.array_equal(codes.cpu().numpy()[fine], ref.pack(c)[fine])
    out = _np64(mm.mm_mxfp4_dequantize(codes, scales, torch.float32))
    assert np.isnan(out[~fine]).all()
    assert np.array_equal(out[fine], ref.values(c, s)[fine])
    assert np.array_equal(np.signbit(out[fine]), np.signbit(x[fine]))
    _status_ok()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_buffers_aligned_to_16_bytes_only(dtype):
    size = torch.empty((), dtype=dtype).element_size()
    flat = torch.from_numpy(_spread(4, 1, 70 * 96 + 16)[0]).cuda().to(dtype)
    x = flat[16 // size:16 // size + 70 * 96].view(70, 96)
    assert x.data_ptr() % 32 == 16
    codes, scales = mm.mm_mxfp4_quantize(x)
    same = mm.mm_mxfp4_quantize(x.clone())
    assert torch.equal(codes, same[0]) and torch.equal(scales, same[1])
    out = torch.zeros(70 * 96 + 32, dtype=dtype, device="cuda")
    at = out[16 // size:16 // size + 70 * 96]
    rc = mm.lib().mm_mxfp4_dequantize(codes.data_ptr(), scales.data_ptr(), 1, 70, 96,
                                      at.data_ptr(), mm._lib._DTYPES[dtype],
                                      torch.cuda.current_stream().cuda_stream)
    assert rc == mm.MM_OK
    assert torch.equal(at.view(70, 96), mm.mm_mxfp4_dequantize(codes, scales, dtype))
    assert not out[:16 // size].any() and not out[16 // size + 70 * 96:].any()
    _status_ok()


def test_dequantise_every_code_and_scale():
    # Every byte of codes under every scale byte: row r has scale r.
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)          # K = 512
    s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    tiles = mm.mxfp4_tile_scales(torch.from_numpy(s))
    assert np.array_equal(tiles.numpy(), ref.tile(s))
    out = _np64(mm.mm_mxfp4_dequantize(codes.cuda(), tiles.cuda(), torch.float32))
    want = ref.values(ref.unpack(codes.numpy()), s)
    # 6 * 2^126 and 6 * 2^127, 3 * 2^127, 4 * 2^127 are beyond fp32
    with np.errstate(over="ignore"):
        want = want.astype(np.float32).astype(np.float64)
    assert np.array_equal(out, want, equal_nan=True)


def _matrix(seed, rows, K, std=1.0):
    x = _spread(seed, rows, K, std=std).astype(np.float64)
    c, s = _quantise_ref(x)
    return (torch.from_numpy(ref.pack(c)).cuda(), torch.from_numpy(ref.tile(s)).cuda(),
            ref.values(c, s))


GEMM = [(1, 1, 32), (16, 128, 64), (17, 129, 96), (128, 256, 256), (129, 257, 288), (300, 77, 2080),
        (5, 520, 4096), (1111, 1000, 544), (2, 3000, 128), (700, 16, 1024)]


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", GEMM)
def test_product(M, N, K, out):
    a, sa, av = _matrix(M + K, M, K)
    b, sb, bv = _matrix(N + 7 * K, N, K, std=0.02)
    c = _np64(mm.mm_mxfp4_gemm(a, sa, b, sb, out_dtype=out))
    _status_ok()
    want = av @ bv.T
    # The products are exact; K fp32 additions, each off by at most one step
    # (2^-23, whether rounded or cut) of a partial sum of at most sum |a b|.
    # Then one rounding to bf16 (half a step: 2^-8).
    tol = K * 2.0 ** -23 * (np.abs(av) @ np.abs(bv).T)
    if out == torch.bfloat16:
        tol = tol + (np.abs(want) + tol) * 2.0 ** -8
    assert c.shape == (M, N)
    assert (np.abs(c - want) <= tol).all(), np.abs(c - want).max()


def test_product_keeps_a_nan_block_to_its_own_row_and_column():
    a, sa, av = _matrix(1, 40, 288)
    b, sb, bv = _matrix(2, 140, 288)
    clean = mm.mm_mxfp4_gemm(a, sa, b, sb, out_dtype=torch.float32)
    row, col = 33, 130
    sa2, sb2 = sa.clone(), sb.clone()
    sa2[0, 2, (row % 32) * 16 + row // 32 * 4] = 255          # row 33, block 8
    sb2[1, 0, (col % 32) * 16 + (col % 128) // 32 * 4 + 3] = 255  # row 130, block 3
    got = mm.mm_mxfp4_gemm(a, sa2, b, sb2, out_dtype=torch.float32)
    _status_ok()
    nan = torch.zeros_like(got, dtype=torch.bool)
    nan[row], nan[:, col] = True, True
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], clean[~nan])


def test_product_reaches_past_32_bit_offsets():
    # C has more than 2^32 bytes and more than 2^31 elements; A's rows repeat,
    # so the far rows equal the near ones.
    M, N, K = 70000, 32768, 32
    a, sa, _ = _matrix(3, 128, K)
    b, sb, _ = _matrix(4, N, K)
    reps = -(-M // 128)
    big = a.repeat(reps, 1)[:M].contiguous()
    c = mm.mm_mxfp4_gemm(big, sa.repeat(reps, 1, 1), b, sb)
    near = mm.mm_mxfp4_gemm(a, sa, b, sb)
    _status_ok()
    for r0 in (0, 128 * 300, 128 * (reps - 2)):
        assert torch.equal(c[r0:r0 + 128], near)
    assert torch.equal(c[128 * (reps - 1):], near[:M - 128 * (reps - 1)])


# ---------------------------------------------------------------- experts ---

def _experts_case(seed, T, H, E, I, k, ids=None):
    rng = np.random.default_rng(seed)
    hidden = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
    if ids is None:
        ids = np.sort(np.argsort(rng.random((T, E)), axis=1)[:, :k], axis=1)
    w = rng.random((T, k)).astype(np.float32) + 0.05
    w = (w / w.sum(1, keepdims=True)).astype(np.float32)
    gu = (rng.standard_normal((2 * E, I, H)) * 1.5 / np.sqrt(H)).astype(np.float32)
    dn = (rng.standard_normal((E, H, I)) * 1.5 / np.sqrt(I)).astype(np.float32)
    d = {"hidden": hidden.cuda(), "ids": torch.from_numpy(ids.astype(np.int32)).cuda(),
         "w": torch.from_numpy(w).cuda()}
    d["gu"], d["sgu"] = mm.mm_mxfp4_quantize(torch.from_numpy(gu).cuda())
    d["dn"], d["sdn"] = mm.mm_mxfp4_quantize(torch.from_numpy(dn).cuda())
    return d


def _call(d, **kw):
    return mm.mm_moe_experts_mxfp4(d["hidden"], d["ids"], d["w"], d["gu"], d["sgu"], d["dn"],
                                   d["sdn"], **kw)


def _least_unit(v):
    """Power of two of which every value of each row is a multiple (rows of
    e2m1 values under powers of two)."""
    m, e = np.frexp(np.where(v == 0, np.inf, np.abs(v)))
    # m in {1/2, 3/4}: the value is a multiple of 2^(e - 2)
    return np.where(np.isinf(m), np.inf, np.ldexp(1.0, np.where(np.isinf(m), 0, e) - 2)).min(1)


def _sum_error(a, b, mag):
    """Bound of the fp32 accumulation of a b^T (mag = |a| |b|^T): none where
    every partial sum is an integer multiple, below 2^24, of the least
    product; else K steps as in test_product."""
    unit = _least_unit(a)[:, None] * _least_unit(b)[None, :]
    return np.where(mag < 2.0 ** 24 * unit, 0.0, a.shape[1] * 2.0 ** -23 * mag)


def _experts_ref(d):
    """The layer's definition in float64, and how far a kernel may be from it."""
    x = ref.quantised(_np64(d["hidden"]))
    ids, w = d["ids"].cpu().numpy(), _np64(d["w"])
    T, H = x.shape
    E, I = d["dn"].shape[0], d["dn"].shape[2] * 2
    gu = _np64(mm.mm_mxfp4_dequantize(d["gu"], d["sgu"], torch.float32))
    dn = _np64(mm.mm_mxfp4_dequantize(d["dn"], d["sdn"], torch.float32))
    y, tol, out_mag, block_mag = (np.zeros((T, H)) for _ in range(4))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if t.size == 0:
            continue
        g, u = x[t] @ gu[2 * e].T, x[t] @ gu[2 * e + 1].T
        ax = np.abs(x[t])
        eg = _sum_error(x[t], gu[2 * e], ax @ np.abs(gu[2 * e]).T)
        eu = _sum_error(x[t], gu[2 * e + 1], ax @ np.abs(gu[2 * e + 1]).T)
        act = g / (1 + np.exp(-g)) * u
        # |silu'| <= 1.1; the exponential's argument g log2(e) is rounded
        # (|g| 2^-24 relative), the exponential and the divide are within 2
        # ulp each, the additions and products within one: (8 + 2 |g|) 2^-23.
        silu = np.abs(g / (1 + np.exp(-g)))
        err = (1.1 * eg + silu * (8 + 2 * np.abs(g)) * 2.0 ** -23) * (np.abs(u) + eu) + silu * eu
        q = ref.quantised(act)
        da = ref.slack(act, err)
        wt = w[t, j][:, None]
        ad = np.abs(dn[e]).T
        np.add.at(y, t, wt * (q @ dn[e].T))
        np.add.at(tol, t, wt * (da @ ad + I * 2.0 ** -23 * ((np.abs(q) + da) @ ad)))
        row = np.abs(q @ dn[e].T) + da @ ad
        np.add.at(out_mag, t, wt * row)
        np.add.at(block_mag, t, wt * np.repeat(row.reshape(len(t), -1, 32).max(-1), 32, axis=1))
    k = ids.shape[1]
    # Each slot's output is held as fp16 (half a step: 2^-11) under a power of
    # two that keeps its block's largest value in [2^14, 2^15); below 2^-14
    # there the step is 2^-24, half of it 2^-39 of that value. Then the weighted
    # sum over the slots in fp32.
    tol = tol + (2.0 ** -11 + (k + 2) * 2.0 ** -24) * out_mag + 2.0 ** -39 * block_mag
    return y, tol + (np.abs(y) + tol) * 2.0 ** -8   # one rounding to bf16


EXPERTS = [(1, 128, 8, 64, 2), (16, 128, 8, 64, 2), (5, 64, 4, 192, 3), (33, 320, 7, 320, 4),
           (64, 256, 32, 128, 8), (300, 192, 3, 64, 2), (1100, 128, 40, 128, 5),
           (70, 2048, 16, 768, 8), (2, 4096, 3, 256, 1)]


@pytest.mark.parametrize("T,H,E,I,k", EXPERTS)
def test_experts(T, H, E, I, k):
    d = _experts_case(T + H, T, H, E, I, k)
    out = _call(d)
    _status_ok()
    want, tol = _experts_ref(d)
    off = np.abs(_np64(out) - want)
    assert (off <= tol).all(), (off.max(), (off / tol).max())
    # The bound has to be of use: the share that rounding borders take is small.
    assert np.linalg.norm(tol) <= 0.1 * np.linalg.norm(want)
    assert torch.equal(out, _call(d))  # the same on every call


@pytest.mark.parametrize("T", [1, 127, 128, 129, 400])
def test_experts_all_tokens_to_one_pair(T):
    # Two experts get every token, the others none: chunks that end at, before
    # and after a 128-row border.
    ids = np.tile([[2, 5]], (T, 1))
    d = _experts_case(T, T, 128, 9, 64, 2, ids=ids)
    out = _call(d)
    _status_ok()
    want, tol = _experts_ref(d)
    assert (np.abs(_np64(out) - want) <= tol).all()


def test_experts_bad_ids_are_dropped_and_flagged():
    T, H, E, I, k = 40, 128, 8, 64, 3
    d = _experts_case(9, T, H, E, I, k)
    good = d["ids"].clone()
    d["ids"][3, 0], d["ids"][7, 2], d["ids"][11, 1] = -1, E, d["ids"][11, 0]
    out = _call(d)
    torch.cuda.synchronize()
    assert mm.mm_poll_device_status() == mm.MM_ERR_DEVICE
    d2 = dict(d, ids=good, w=d["w"].clone())
    for t, j in ((3, 0), (7, 2), (11, 1)):
        d2["w"][t, j] = 0
    same = _call(d2)
    _status_ok()
    assert torch.equal(out, same)


def test_experts_on_streams_with_own_workspaces():
    # Two calls at once on two streams, each with its own workspace, and one on
    # a stream given by its handle.
    T, H, E, I, k = 200, 256, 16, 128, 4
    cases = [_experts_case(20 + i, T, H, E, I, k) for i in range(3)]
    want = [_call(d) for d in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    ws = [torch.empty(mm.mm_moe_experts_mxfp4_workspace_size(T, H, E, I, k), dtype=torch.uint8,
                      device="cuda") for _ in cases[:2]]
    got = []
    for rep in range(3):
        got = [_call(cases[0], stream=streams[0], workspace=ws[0]),
               _call(cases[1], stream=streams[1], workspace=ws[1]),
               _call(cases[2], stream=streams[2].cuda_stream)]
    for s in streams:
        s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    _status_ok()


def test_experts_in_two_captured_graphs():
    T, H, E, I, k = 30, 256, 16, 128, 4
    cases = [_experts_case(30 + i, T, H, E, I, k) for i in range(2)]
    want = [_call(d) for d in cases]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for d in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_call(d))
        graphs.append(g)
    side = torch.cuda.Stream()
    for _ in range(4):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    # New inputs under the same graph
    cases[0]["hidden"].copy_(cases[1]["hidden"])
    want0 = _call(cases[0])
    graphs[0].replay()
    _status_ok()
    assert torch.equal(outs[0], want0)


def test_writes_only_its_outputs():
    from test_gpu_guards import Guarded
    T, H, E, I, k = 37, 192, 6, 64, 3
    d = _experts_case(5, T, H, E, I, k)
    bufs = {n: Guarded(tuple(d[n].shape), d[n].dtype, d[n]) for n in d}
    out = Guarded((T, H), torch.bfloat16)
    ws = Guarded((mm.mm_moe_experts_mxfp4_workspace_size(T, H, E, I, k),), torch.uint8)
    _call({n: b.t for n, b in bufs.items()}, out=out.t, workspace=ws.t)
    L = mm.lib()
    st = torch.cuda.current_stream().cuda_stream
    x = Guarded((3, 45, 96), torch.bfloat16,
                torch.from_numpy(_spread(1, 3, 45, 96)).to(torch.bfloat16))
    codes, tiles = Guarded((3, 45, 48), torch.uint8), Guarded((3, 1, 1, 512), torch.uint8)
    back = Guarded((3, 45, 96), torch.float32)
    c = Guarded((45, 45), torch.float32)
    cb = Guarded((45, 45), torch.bfloat16)
    assert L.mm_mxfp4_quantize(x.t.data_ptr(), mm.MM_DTYPE_BF16, 3, 45, 96, codes.t.data_ptr(),
                               tiles.t.data_ptr(), st) == mm.MM_OK
    assert L.mm_mxfp4_dequantize(codes.t.data_ptr(), tiles.t.data_ptr(), 3, 45, 96,
                                 back.t.data_ptr(), mm.MM_DTYPE_FP32, st) == mm.MM_OK
    for o, dt in ((c, mm.MM_DTYPE_FP32), (cb, mm.MM_DTYPE_BF16)):
        assert L.mm_mxfp4_gemm(codes.t[0].data_ptr(), tiles.t[0].data_ptr(),
                               codes.t[1].data_ptr(), tiles.t[1].data_ptr(), 45, 45, 96,
                               o.t.data_ptr(), dt, st) == mm.MM_OK
    _status_ok()
    every = dict(bufs, out=out, ws=ws, x=x, codes=codes, tiles=tiles, back=back, c=c, cb=cb)
    for name, b in every.items():
        assert b.intact(), name


def test_routing_and_experts_together():
    """Router logits -> mm_route_logits -> 4-bit experts, as a layer uses them,
    beside mm_moe_forward on the same (dequantised) weights."""
    T, H, E, I, k = 130, 256, 16, 128, 4
    rng = np.random.default_rng(3)
    d = _experts_case(3, T, H, E, I, k)
    rw = torch.from_numpy((rng.standard_normal((E, H)) / np.sqrt(H)).astype(np.float32))
    rw = rw.to(torch.bfloat16).cuda()
    logits = d["hidden"].float() @ rw.float().T
    ids, w, counts, _, loss = mm.mm_route_logits(logits, k, True)
    ids2, w2 = mm.mm_route(d["hidden"], rw, k, True)
    top = torch.sort(logits, dim=-1, descending=True)[0]
    clear = (top[:, k - 1] - top[:, k]) > 1e-4  # elsewhere the two summation orders may differ
    assert torch.equal(ids[clear], ids2[clear])
    torch.testing.assert_close(w[clear], w2[clear], rtol=1e-4, atol=1e-7)
    assert int(counts.sum()) == T * k and 0.9 < float(loss) < 4
    out = mm.mm_moe_experts_mxfp4(d["hidden"], ids, w, d["gu"], d["sgu"], d["dn"], d["sdn"])
    gu = mm.mm_mxfp4_dequantize(d["gu"], d["sgu"]).view(E, 2 * I, H)
    dn = mm.mm_mxfp4_dequantize(d["dn"], d["sdn"])
    full = mm.mm_moe_forward(d["hidden"], rw, gu, dn, k, True)
    _status_ok()
    # The same layer but for the 4-bit activations. A value of a block is off
    # by at most a quarter of its size down to 1/4 of its unit; over normal
    # inputs the rounding's rms is about 0.12 of theirs, twice on the way
    # (hidden, activation), thrice counting that gate and up both carry the
    # first: sqrt(3) * 0.12 = 0.2.
    rel = (out.float() - full.float()).norm() / full.float().norm()
    assert rel < 0.3, rel


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 3e38])
def test_experts_keep_bad_tokens_to_themselves(bad):
    # Tokens that hold NaN, infinity or huge values share experts, chunks and
    # 32-row pieces with the others, whose outputs must not change at all.
    T, H, E, I, k = 100, 256, 6, 128, 3
    d = _experts_case(77, T, H, E, I, k)
    clean = _call(d)
    d["hidden"][7, 5] = bad
    d["hidden"][40] = bad
    d["hidden"][41, 200:] = -bad
    out = _call(d)
    _status_ok()
    rows = torch.ones(T, dtype=torch.bool, device="cuda")
    rows[[7, 40, 41]] = False
    assert torch.equal(out[rows], clean[rows])
    assert torch.isfinite(clean).all()
    if bad != 3e38:
        assert torch.isnan(out[~rows]).all()


def test_experts_with_tiny_and_huge_weights():
    # Expert outputs far below and above fp16's range pass through its block
    # powers of two, subnormal and large floats on the way out.
    T, H, E, I, k = 20, 128, 4, 64, 2
    for exponent in (-100, -60, 60, 100):
        d = _experts_case(78, T, H, E, I, k)
        want, tol = _experts_ref(d)
        scaled = dict(d, sdn=(d["sdn"].to(torch.int32) + exponent).clamp(1, 250).to(torch.uint8))
        # the padding bytes are not read as scales of anything but zeros
        out = _call(scaled)
        _status_ok()
        f = 2.0 ** exponent
        off = np.abs(_np64(out) - want * f)
        assert (off <= tol * f + 2.0 ** -133).all(), exponent


@pytest.mark.parametrize("T", [40, 900])  # grouped by every kernel itself, and by one of its own
def test_experts_bad_ids_in_small_and_large_batches(T):
    H, E, I, k = 128, 8, 64, 4
    d = _experts_case(80, T, H, E, I, k)
    rng = np.random.default_rng(1)
    hit = rng.choice(T * k, T // 4, replace=False)
    flat = d["ids"].view(-1)
    flat[torch.from_numpy(hit).cuda()] = torch.from_numpy(
        rng.choice([-1, E, 1 << 30, -(1 << 31)], hit.size).astype(np.int32)).cuda()
    d["ids"][T // 2] = 5        # one expert in every slot: the first stays
    d["w"][T // 2, 1:] = float("nan")  # weights of dropped slots are not read
    out = _call(d)
    torch.cuda.synchronize()
    assert mm.mm_poll_device_status() == mm.MM_ERR_DEVICE
    ok = dict(d, ids=d["ids"].clone(), w=d["w"].clone())
    drop = (ok["ids"] < 0) | (ok["ids"] >= E)
    drop[T // 2, 1:] = True
    # the same with the dropped slots' ids out of every float64 expert's way
    ok["ids"][drop] = -1
    ok["w"][drop] = 0
    want, tol = _experts_ref(ok)
    assert (np.abs(_np64(out) - want) <= tol).all()


@pytest.mark.parametrize("T", [3, 700])
def test_experts_without_a_valid_id(T):
    # Nothing to multiply: the call still writes zeros, after the kernels
    # before it, however often it runs.
    d = _experts_case(81, T, 128, 8, 64, 4)
    want = _call(d)
    none = dict(d, ids=torch.full_like(d["ids"], -7))
    for _ in range(20):
        out = torch.full((T, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        _call(none, out=out)
        assert not out.any()
        assert torch.equal(_call(d), want)
    torch.cuda.synchronize()
    assert mm.mm_poll_device_status() == mm.MM_ERR_DEVICE


def test_experts_back_to_back_in_one_workspace():
    # Calls of different sizes one after another in the same workspace, ids
    # written on the same stream just before: nothing starts too early.
    H, E, I, k = 256, 16, 128, 4
    cases = [_experts_case(90 + i, T, H, E, I, k) for i, T in enumerate((1, 600, 64, 512, 513, 5))]
    want = [_call(d) for d in cases]
    ws = torch.empty(mm.mm_moe_experts_mxfp4_workspace_size(600, H, E, I, k), dtype=torch.uint8,
                     device="cuda")
    got = []
    for rep in range(5):
        for d in cases:
            ids = torch.empty_like(d["ids"]).copy_(d["ids"])
            hid = torch.empty_like(d["hidden"]).copy_(d["hidden"])
            got.append(_call(dict(d, ids=ids, hidden=hid), workspace=ws))
            ids.zero_(), hid.zero_()
    _status_ok()
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % len(cases)]), i


def test_run_layer_with_4_bit_experts(capsys):
    from mixture_experts_layer_mm_gb300 import run_layer
    assert run_layer.main(["--workload", "tiny", "--passes", "2", "--mxfp4"]) == 0
    assert "status MM_OK" in capsys.readouterr().out


@pytest.mark.parametrize("M,N,K", [(1, 256, 1536), (64, 4096, 4096), (40, 1000, 2080),
                                   (130, 300, 4096), (128, 256, 8192), (257, 96, 3104),
                                   (33, 4864, 2048), (200, 640, 1568)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_product_with_a_long_reduction(M, N, K, out):
    # Few tiles and many stages: every ring slot is filled several times.
    a, sa, av = _matrix(M + K, M, K)
    b, sb, bv = _matrix(N + 7 * K, N, K, std=0.02)
    c = mm.mm_mxfp4_gemm(a, sa, b, sb, out_dtype=out)
    again = [mm.mm_mxfp4_gemm(a, sa, b, sb, out_dtype=out) for _ in range(3)]
    _status_ok()
    assert all(torch.equal(c, x) for x in again)
    want = av @ bv.T
    # as in test_product
    tol = K * 2.0 ** -23 * (np.abs(av) @ np.abs(bv).T)
    if out == torch.bfloat16:
        tol = tol + (np.abs(want) + tol) * 2.0 ** -8
    assert (np.abs(_np64(c) - want) <= tol).all()


def test_products_on_two_streams_and_in_a_graph():
    a, sa, _ = _matrix(1, 60, 4096)
    b, sb, _ = _matrix(2, 2000, 4096)
    want = mm.mm_mxfp4_gemm(a, sa, b, sb)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [mm.mm_mxfp4_gemm(a, sa, b, sb, stream=streams[i % 2]) for i in range(12)]
    g = torch.cuda.CUDAGraph()
    for s in streams:
        s.synchronize()
    with torch.cuda.graph(g):
        one = mm.mm_mxfp4_gemm(a, sa, b, sb)
    for _ in range(3):
        g.replay()
    _status_ok()
    assert all(torch.equal(x, want) for x in got + [one])


@pytest.mark.parametrize("M,N,K", [(2560, 2048, 2304), (8200, 700, 2080), (20000, 256, 256)])
def test_large_products(M, N, K):
    # Enough tiles for all SMs, in both orders of the weight rows; the float64
    # product on the GPU.
    g = torch.Generator(device="cuda").manual_seed(M)
    a = mm.mm_mxfp4_quantize(torch.randn(M, K, generator=g, device="cuda"))
    b = mm.mm_mxfp4_quantize(torch.randn(N, K, generator=g, device="cuda") * 0.05)
    av = mm.mm_mxfp4_dequantize(*a, dtype=torch.float32).double()
    bv = mm.mm_mxfp4_dequantize(*b, dtype=torch.float32).double()
    want, mag = av @ bv.T, av.abs() @ bv.abs().T
    for dt in (torch.float32, torch.bfloat16):
        c = mm.mm_mxfp4_gemm(*a, *b, out_dtype=dt).double()
        tol = K * 2.0 ** -23 * mag  # as in test_product
        if dt == torch.bfloat16:
            tol = tol + (want.abs() + tol) * 2.0 ** -8
        assert bool(((c - want).abs() <= tol).all())
    _status_ok()


# Few tiles (128 columns each, the reduction in two accumulators) next to many
# (256 columns, the last of them 128 or less), with whole groups of 32 columns
# and without, one stage of columns and several.
@pytest.mark.parametrize("M,N,K", [(1, 32, 32), (33, 100, 256), (96, 416, 288), (64, 1000, 544),
                                   (128, 19456, 512), (128, 19457, 512), (9984, 320, 96),
                                   (9900, 300, 512), (9900, 288, 2304), (13000, 290, 2080)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_products_of_few_and_many_tiles(M, N, K, out):
    a, sa, va = _matrix(M, M, K)
    b, sb, vb = _matrix(N + 1, N, K)
    got = _np64(mm.mm_mxfp4_gemm(a, sa, b, sb, out_dtype=out))
    ta, tb = torch.from_numpy(va).cuda(), torch.from_numpy(vb).cuda()
    want = _np64(ta @ tb.T)
    # fp32 sums of K exact products: every addition rounds once (or truncates: a
    # whole step), of partial sums below the sum of magnitudes.
    bound = (K + 2) * 2.0 ** -23 * _np64(ta.abs() @ tb.abs().T)
    if out == torch.bfloat16:
        bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want) + 2.0 ** -133
    assert (np.abs(got - want) <= bound).all()
    _status_ok()


@pytest.mark.parametrize("k", [1, 7, 8, 9, 20, 32])
def test_experts_of_many_slots_a_token(k):
    # Slots are read eight at a time: repeated and bad ids within and across the
    # eights are dropped, in a batch that is grouped by a kernel of its own.
    T, H, E, I = 2100 if k == 1 else 300, 64, 40, 64
    rng = np.random.default_rng(k)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    bad = rng.random((T, k)) < 0.1
    if k > 1:
        ids[bad] = np.where(rng.random(bad.sum()) < 0.5, -3, ids[np.nonzero(bad)[0], 0])
        first = np.nonzero(bad[:, 0])[0]
        ids[first, 0] = np.argsort(rng.random((len(first), E)), axis=1)[:, 0]
    # What counts by definition: an id in range that no earlier slot of its row has.
    clean = np.array([[e if 0 <= e < E and e not in row[:j] else E + 5
                       for j, e in enumerate(row)] for row in ids.tolist()], dtype=np.int32)
    assert (k == 1) == bool((clean == ids).all())
    d = _experts_case(5, T, H, E, I, k, ids=ids)
    got = _call(d)
    d["ids"] = torch.from_numpy(clean).cuda()
    want = _call(d)
    assert mm.mm_poll_device_status() == (mm.MM_OK if k == 1 else mm.MM_ERR_DEVICE)
    assert torch.equal(got, want)


def _scale_at(tiles, row, block):
    """The scale byte of (row, block) in every matrix of stored tiles [E, ...], as a view."""
    return tiles[:, row // 128, block // 4, row % 32 * 16 + row % 128 // 32 * 4 + block % 4]


@pytest.mark.parametrize("T", [9, 700])
def test_experts_keep_an_output_column_to_itself(T):
    # A column of the result takes its row of w_down alone, whatever the rows
    # beside it hold: NaN, products beyond fp32, values 2^60 times larger.
    H, E, I, k, h = 320, 8, 64, 4, 170
    d = _experts_case(82, T, H, E, I, k)
    clean = _call(d)
    others = torch.arange(H, device="cuda") != h
    for byte in (255, 254):
        s = d["sdn"].clone()
        _scale_at(s, h, 1)[2] = byte  # the columns 32 to 63 of w_down[2, h]
        out = _call(dict(d, sdn=s))
        assert torch.equal(out[:, others], clean[:, others])
        hit = (d["ids"] == 2).any(1)
        assert torch.equal(out[~hit, h], clean[~hit, h])
        bad = torch.isnan(out[hit, h]) if byte == 255 else ~torch.isfinite(out[hit, h])
        assert bad.all() if byte == 255 else bad.any()
    s = d["sdn"].clone()
    for block in range(I // 32):
        _scale_at(s, h, block)[:] += 60
    out = _call(dict(d, sdn=s))
    _status_ok()
    assert torch.equal(out[:, others], clean[:, others])
    assert torch.equal(out[:, h].float(), clean[:, h].float() * 2.0 ** 60)


@pytest.mark.parametrize("T", [3, 1100])
def test_experts_sum_their_slots_in_32_bits(T):
    # Two experts that differ in one intermediate of w_down, under weights 1 and
    # -1: the slots cancel but for that one, so that what each lost shows.
    H, I, i0 = 192, 128, 37
    d = _experts_case(83, T, H, 2, I, 2, ids=np.tile([[0, 1]], (T, 1)))
    d["gu"][2:], d["sgu"][2:] = d["gu"][:2].clone(), d["sgu"][:2].clone()
    d["dn"][1], d["sdn"][1] = d["dn"][0].clone(), d["sdn"][0].clone()
    d["dn"][1, :, i0 // 2] &= 0x0F  # the odd column's code
    d["w"][:, 0], d["w"][:, 1] = 1.0, -1.0
    out = _np64(_call(d))
    _status_ok()
    x = ref.quantised(_np64(d["hidden"]))
    gu = _np64(mm.mm_mxfp4_dequantize(d["gu"], d["sgu"], torch.float32))
    dn = _np64(mm.mm_mxfp4_dequantize(d["dn"], d["sdn"], torch.float32))
    assert not dn[1][:, i0].any() and np.array_equal(np.delete(dn[0], i0, 1), np.delete(dn[1], i0, 1))
    g, u = x @ gu[0].T, x @ gu[1].T
    silu = g / (1 + np.exp(-g))
    # As in _experts_ref; the sums of gate and up are within H steps.
    eg = H * 2.0 ** -23 * (np.abs(x) @ np.abs(gu[0]).T)
    eu = H * 2.0 ** -23 * (np.abs(x) @ np.abs(gu[1]).T)
    err = (1.1 * eg + np.abs(silu) * (8 + 2 * np.abs(g)) * 2.0 ** -23) * (np.abs(u) + eu) \
        + np.abs(silu) * eu
    q, da = ref.quantised(silu * u), ref.slack(silu * u, err)
    want = np.outer(q[:, i0], dn[0][:, i0]).reshape(T, H)
    # Both slots hold the same activation. Each sum is within I steps of its
    # magnitudes, the two additions of the slots within one each (of a value
    # below these magnitudes, 2^-24), then one rounding to bf16.
    mag = (np.abs(q) + da) @ np.abs(dn[0]).T
    tol = np.outer(da[:, i0], np.abs(dn[0][:, i0])) + (2 * I * 2.0 ** -23 + 2 * 2.0 ** -24) * mag
    tol = tol + (np.abs(want) + tol) * 2.0 ** -8
    assert (np.abs(out - want) <= tol).all(), (np.abs(out - want) / tol).max()


def _digits(value, unit, blocks, rng):
    """Codes [blocks, 32] and exponents [blocks]: under 2^exponent (7 apart, the
    last one `unit`) their sum is the integer `value` times 2^unit."""
    codes, left = np.zeros((blocks, 32), np.uint8), int(value)
    for b in range(blocks):
        step = 1 << 7 * (blocks - 1 - b)
        n = int(round(left / step))
        left -= n * step
        sign, n, i = (8 if n < 0 else 0), abs(n), 0
        while n:
            c = max(c for c in (2, 4, 5, 6, 7) if ref.LEVELS[c] <= n)  # 1, 2, 3, 4, 6
            codes[b, i] = c | sign
            n -= int(ref.LEVELS[c])
            i += 1
        codes[b] = codes[b, rng.permutation(32)]
    assert left == 0
    return codes, unit + 7 * np.arange(blocks - 1, -1, -1)


@pytest.mark.parametrize("low,high", [(-86, -60), (-60, -30), (-30, -8), (2, 40)])
def test_activations_next_to_a_border(low, high):
    # One token of ones, gate and up products g and u that are exact sums, and a
    # w_down that hands the activations out as they are. Every silu(g) u lies
    # 2^-20 to 2^-19 of itself beside a border between two 4-bit values; the
    # kernel's is within 10 half steps (2^-20.67) of it: 2^t 4, its factor, the sum
    # and two products 1 each, the reciprocal 2.
    rng = np.random.default_rng(low + 1000)
    H = I = 256
    gate, up = np.zeros((I, H), np.uint8), np.zeros((I, H), np.uint8)
    sg, su = np.full((I, H // 32), 127), np.full((I, H // 32), 127)
    want = np.zeros(I)
    silu = lambda g: g / (1 + np.exp(-g))  # noqa: E731
    for i in range(I):
        first = i % 32 == 0  # 4.5 in every block: the scale is 1
        gi = round(4 * 2 ** 7) if first else int(round(rng.uniform(low, high) * 2 ** 7))
        gate[i, :64], e = (a.reshape(-1) for a in _digits(gi, -7, 2, rng))
        sg[i, :2] = e + 127
        s = silu(gi / 2 ** 7)
        if first:
            ui, unit, want[i] = round(4.5 / s * 2 ** 20), -20, 4.0
        else:
            code = rng.integers(0, 7)
            lo, hi = ref.LEVELS[code], ref.LEVELS[code + 1]
            over = rng.random() < 0.5
            target = (lo + hi) / 2 * (1 + (1.5 if over else -1.5) * 2.0 ** -20)
            unit = int(np.floor(np.log2(target / abs(s)))) - 21
            ui = round(target / s * 2.0 ** -unit)
            want[i] = np.copysign(hi if over else lo, 1.0)
        exact = s * ui * 2.0 ** unit
        if not first:  # the products, not their targets, are what the test is about
            off = exact / ((lo + hi) / 2) - 1
            assert 2.0 ** -20 <= abs(off) <= 2.0 ** -19 and (off > 0) == over
        else:
            assert 4.4 < exact < 4.6
        codes, e = _digits(ui, unit, 4, rng)
        up[i, 64:192], su[i, 2:6] = codes.reshape(-1), e + 127
        # sums in 32 bits are exact: the magnitudes stay below 2^24 units
        assert sum(ref.LEVELS[codes & 7].sum(1) * 2.0 ** (e - unit)) < 2 ** 24
    assert su.max() <= 254 and su.min() >= 1
    dn = np.zeros((H, I), np.uint8)
    dn[np.arange(H), np.arange(H)] = 2  # 1.0

    def stored(c, s):
        return (torch.from_numpy(ref.pack(c)).cuda(),
                torch.from_numpy(ref.tile(s.astype(np.uint8))).cuda())

    (g, sg), (u, su) = stored(gate, sg), stored(up, su)
    dn, sdn = stored(dn, np.full((H, I // 32), 127))
    out = mm.mm_moe_experts_mxfp4(
        torch.ones(1, H, dtype=torch.bfloat16, device="cuda"),
        torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, 1, device="cuda"),
        torch.stack([g, u]), torch.stack([sg, su]), dn[None], sdn[None])
    _status_ok()
    assert np.array_equal(_np64(out)[0], want)
