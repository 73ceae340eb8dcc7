"""The SwiGLU with its pre-activations in 8 bits, forward and backward, against
the float64 definitions."""
import pytest
import torch

import mixture_experts_layer_mm_gb300 as mm
import train_reference as ref

pytestmark = pytest.mark.gpu
B, H = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib(mmlib):
    return mmlib


def _z(R, I, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(R, 2 * I, generator=g, device="cuda")
    z *= torch.exp(torch.randn(R, 1, generator=g, device="cuda"))
    z *= torch.exp(torch.randn(1, 2 * I, generator=g, device="cuda"))
    return z.to(dtype)


def _unequal(a, b):
    return int((a != b).sum())


# The formulas in fp32: sigma within 2^-20.5, 1 - sigma within 2^-22, a few products.
# In units of 2^-23 of the terms' magnitudes:
ACT_TERMS, GRAD_TERMS = 10, 24


def _check_backward(q, s, da, w, rows=None):
    dz, act, dw = mm.mm_swiglu_pack_backward(q, s, da, row_w=w, offsets=rows)
    n = da.shape[0] if rows is None else int(rows[-1])
    z, I = ref.decode(q, s)[:n], da.shape[1]
    ww = None if w is None else w[:n]
    wz, wa, wd = ref.swiglu_grad(z, da[:n], ww)
    g, u, d = z[:, :I].abs(), z[:, I:].abs(), da[:n].double().abs()
    k = 1.0 if w is None else ww.double().abs()[:, None]
    sig = torch.sigmoid(z[:, :I])
    # slope = sigma (1 + g (1 - sigma)): its terms may cancel
    mag = torch.cat((k * d * u * sig * (1 + g), k * d * g * sig), 1)
    ref.close(dz[:n], wz, mag, GRAD_TERMS, "dz", floor=ref.FLUSH * torch.cat((k * d * u, k * d), 1))
    ref.close(act[:n], wa, wa.abs(), ACT_TERMS, "act", floor=ref.FLUSH * k * u)
    if w is None:
        assert dw is None
    else:
        ref.close(dw[:n], wd, (da[:n].double() * ref.swiglu(z)).abs().sum(1), ACT_TERMS + I / 4 + 6,
                  "dw", rounding=False, floor=ref.FLUSH * (d * u).sum(1))
    return dz, act, dw


@pytest.mark.parametrize("R,I", [(1, 32), (3, 64), (33, 96), (70, 128), (9, 256), (129, 352),
                                 (17, 768), (5, 2048), (4, 4128), (1000, 32)])
@pytest.mark.parametrize("dtype", [B, H])
def test_pack_and_backward(R, I, dtype):
    z = _z(R, I, dtype)
    act, q, s = mm.mm_swiglu_pack(z)
    wq, ws = ref.encode(z)
    assert _unequal(q, wq) == 0 and _unequal(s, ws) == 0
    want = ref.swiglu(z.double())
    ref.close(act, want, want.abs(), ACT_TERMS, "act", floor=ref.FLUSH * z[:, I:].double().abs())
    for t in (torch.float32, B):                              # exact in both
        assert torch.equal(mm.mm_mxint8_dequantize(q, s, dtype=t).double(), ref.decode(q, s))
    g = torch.Generator(device="cuda").manual_seed(1)
    da = torch.randn(R, I, generator=g, device="cuda").to(dtype)
    _check_backward(q, s, da, None)
    w = torch.rand(R, generator=g, device="cuda")
    first = _check_backward(q, s, da, w)
    again = mm.mm_swiglu_pack_backward(q, s, da, row_w=w)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    assert mm.mm_poll_device_status() == mm.MM_OK


@pytest.mark.parametrize("R,I", [(65, 8192), (300, 1056), (1300, 768), (2001, 768), (3003, 800),
                                 (4001, 768), (5003, 352), (6001, 768), (9001, 352)])
def test_every_share_of_rows_and_lanes(R, I):
    """Rows over one lane group or several warps, one to three steps at a time."""
    test_pack_and_backward(R, I, B)


@pytest.mark.parametrize("dtype", [B, H])
def test_values_at_the_edges(dtype):
    """Zeros, the smallest and largest values, steps that tie, infinities and NaN."""
    big = torch.finfo(dtype).max
    tiny = torch.finfo(dtype).smallest_normal
    sub = 2.0 ** -133 if dtype == B else 2.0 ** -24
    z = torch.zeros(16, 64, dtype=dtype, device="cuda")
    z[1, 0], z[1, 33] = big, -big
    z[2, 5], z[2, 40] = tiny, -tiny
    z[3, 5], z[3, 40] = sub, -sub
    z[4, :8] = torch.tensor([127.5, 126.5, 0.5, 1.5, 2.5, -0.5, -1.5, 64.0], device="cuda")
    z[5, 3], z[6, 3], z[7, 40] = float("inf"), float("nan"), float("-inf")
    z[8, :32] = torch.linspace(-64, 64, 32, device="cuda")
    z[9, 0], z[9, 1] = 1.0, 2.0 ** -20
    z[10, :32] = -100.0
    z[10, 32:] = 3.0
    z[11, :32] = 100.0
    z[11, 32:] = 3.0
    z[12, 0], z[12, 32] = -big, 1.0                           # sigma is 0, whatever g
    act, q, s = mm.mm_swiglu_pack(z)
    wq, ws = ref.encode(z)
    assert torch.equal(q, wq) and torch.equal(s, ws)
    v = mm.mm_mxint8_dequantize(q, s, dtype=torch.float32).double()
    w = ref.decode(q, s)
    assert torch.equal(v.isnan(), w.isnan()) and torch.equal(v.nan_to_num(0), w.nan_to_num(0))
    fine = [i for i in range(16) if i not in (1, 5, 6, 7)]
    want = ref.swiglu(z.double())[fine]
    ref.close(act[fine], want, want.abs() + 2.0 ** -100, ACT_TERMS)
    assert act[6, 3].isnan() and act[5, 0] == 0 and act[1, 0].abs() == 0
    da = torch.ones(16, 32, dtype=dtype, device="cuda")
    dz, a, _ = mm.mm_swiglu_pack_backward(q, s, da)
    assert dz[5, :32].isnan().all() and dz[6, :32].isnan().all() and a[7].isnan().all()
    rest = [i for i in range(16) if i not in (1, 5, 6, 7, 12)]
    _check_backward(q[rest].contiguous(), s[rest].contiguous(), da[rest].contiguous(), None)
    assert not torch.isnan(dz[12]).any()                      # the gate's slope and value are 0
    assert dz[12, 0] == 0 and dz[12, 32] == 0 and a[12, 0] == 0


def test_dequantise_every_code_and_scale():
    q = torch.arange(-128, 128, dtype=torch.int16).to(torch.int8).repeat(256, 1).cuda()
    s = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 8).cuda()
    want = ref.decode(q, s)
    for t in (torch.float32, B, H):
        got = mm.mm_mxint8_dequantize(q, s, dtype=t)
        exact = want.to(torch.float32).to(t)                  # inf beyond the range
        assert torch.equal(got.isnan(), exact.isnan())
        assert torch.equal(got.nan_to_num(7), exact.nan_to_num(7))


def test_rows_behind_the_last_segment_are_left_alone():
    R, I, used = 200, 96, 77
    off = torch.tensor([0, 30, used], dtype=torch.int32, device="cuda")
    z = _z(R, I, B)
    z[used:] = float("nan")
    L = mm.lib()
    act = torch.full((R, I), 5.0, device="cuda").bfloat16()
    q = torch.full((R, 2 * I), 5, dtype=torch.int8, device="cuda")
    s = torch.full((R, I // 16), 5, dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    assert L.mm_swiglu_pack(z.data_ptr(), mm.MM_DTYPE_BF16, off.data_ptr() + 8, R, I,
                            act.data_ptr(), q.data_ptr(), s.data_ptr(), st) == mm.MM_OK
    wa, wq, ws = mm.mm_swiglu_pack(z[:used].contiguous())
    assert torch.equal(act[:used], wa) and torch.equal(q[:used], wq) and torch.equal(s[:used], ws)
    assert (act[used:] == 5).all() and (q[used:] == 5).all() and (s[used:] == 5).all()
    a2, q2, s2 = mm.mm_swiglu_pack(z, offsets=off)
    assert torch.equal(a2[:used], wa) and torch.equal(q2[:used], wq) and torch.equal(s2[:used], ws)
    da, w = torch.randn(R, I, device="cuda").bfloat16(), torch.rand(R, device="cuda")
    dz = torch.full((R, 2 * I), 5.0, device="cuda").bfloat16()
    ra, rw = torch.full_like(act, 5.0), torch.full((R,), 5.0, device="cuda")
    assert L.mm_swiglu_pack_backward(q.data_ptr(), s.data_ptr(), da.data_ptr(), mm.MM_DTYPE_BF16,
                                     w.data_ptr(), off.data_ptr() + 8, R, I, dz.data_ptr(),
                                     ra.data_ptr(), rw.data_ptr(), st) == mm.MM_OK
    torch.cuda.synchronize()
    assert (dz[used:] == 5).all() and (ra[used:] == 5).all() and (rw[used:] == 5).all()
    got = _check_backward(q2, s2, da, w, rows=off)
    assert torch.equal(got[0][:used], dz[:used]) and torch.equal(got[2][:used], rw[:used])
    off[2] = R + 50                                           # more than there are: all of them
    z = _z(R, I, B)
    assert torch.equal(mm.mm_swiglu_pack(z, offsets=off)[0], mm.mm_swiglu_pack(z)[0])


def test_rows_past_32_bit_offsets():
    R, I = 140_000, 8192                                      # 2.3e9 pre-activations
    z = torch.empty(R, 2 * I, dtype=B, device="cuda")
    z.zero_()
    z[-3:] = _z(3, I, B)
    act, q, s = mm.mm_swiglu_pack(z)
    wq, ws = ref.encode(z[-3:])
    assert torch.equal(q[-3:], wq) and torch.equal(s[-3:], ws)
    want = ref.swiglu(z[-3:].double())
    ref.close(act[-3:], want, want.abs(), ACT_TERMS)
    v = mm.mm_mxint8_dequantize(q, s)
    assert torch.equal(v[-3:].double(), ref.decode(wq, ws))
    del v
    da = torch.ones(R, I, dtype=B, device="cuda")
    dz, a, _ = mm.mm_swiglu_pack_backward(q, s, da)
    wz, wa, _ = ref.swiglu_grad(ref.decode(wq, ws), da[-3:])
    ref.close(a[-3:], wa, wa.abs(), ACT_TERMS)
    assert (dz[-3:].double() - wz).abs().max() <= 2.0 ** -7 * wz.abs().max()
    assert not dz[0].any() and not a[0].any()


def test_streams_and_graphs_share_nothing():
    z = [_z(3000, 256, B, seed=i) for i in range(2)]
    da, w = torch.randn(3000, 256, device="cuda").bfloat16(), torch.rand(3000, device="cuda")

    def run(i, stream=None):
        act, q, s = mm.mm_swiglu_pack(z[i], stream=stream)
        return (act, q, s, mm.mm_mxint8_dequantize(q, s, stream=stream),
                *mm.mm_swiglu_pack_backward(q, s, da, row_w=w, stream=stream))

    want = [run(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [run(i, streams[i]) for i in range(2)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, r) for p, r in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(0)
    z[0].copy_(z[1])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, r) for p, r in zip(got, want[1]))


def test_rows_of_the_interchange_format():
    """MXINT8 of the OCP formats, q / 64 under 2^(s' - 127): its bytes less six."""
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randint(-127, 128, (40, 96), generator=g, device="cuda").to(torch.int8)
    theirs = torch.randint(6, 254, (40, 3), generator=g, device="cuda").to(torch.uint8)
    theirs[3, 1] = 255
    ours = torch.where(theirs == 255, theirs, theirs - 6)
    unit = torch.ldexp(torch.ones((), dtype=torch.float64), theirs.cpu().int() - 127)
    want = q.cpu().double().view(40, 3, 32) / 64 * unit[..., None]
    want[3, 1] = float("nan")
    got = mm.mm_mxint8_dequantize(q, ours, dtype=torch.float32).cpu().double().view(40, 3, 32)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(0), want.nan_to_num(0))
