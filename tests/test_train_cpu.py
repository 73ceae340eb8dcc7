"""The operators that train the experts on a machine without a GPU: what they
refuse before any CUDA call, the sizes they report, and the float64 definitions
that the GPU tests use, by hand and by differences."""
import pytest
import torch

import mixture_experts_layer_mm_gb300 as mm
import train_reference as ref

INV, UNS, MEM, OK = (mm.MM_ERR_INVALID_ARG, mm.MM_ERR_UNSUPPORTED, mm.MM_ERR_NO_MEMORY, mm.MM_OK)
F32, BF16, F16 = mm.MM_DTYPE_FP32, mm.MM_DTYPE_BF16, mm.MM_DTYPE_FP16


@pytest.fixture(scope="module")
def L(mmlib):
    return mm.lib()


def test_group_slots_refusals(L):
    def call(ids=16, T=4, k=2, E=8, places=16, off=16, ws=None, n=0):
        return L.mm_group_slots(ids, None, T, k, E, places, off, ws, n, None)

    assert call(T=-1) == INV and call(k=0) == INV and call(E=0) == INV and call(E=257) == UNS
    assert call(k=33) == UNS and call(T=1 << 30) == UNS
    assert call(ids=None) == INV and call(places=None) == INV and call(off=None) == INV
    assert call(ids=18) == INV and call(places=18) == INV and call(off=18) == INV
    size = L.mm_group_slots_workspace_size
    assert size(0, 1, 1) == 0 and size(64, 8, 128) == 0
    assert size(-1, 1, 1) == -1 and size(4, 33, 8) == -1 and size(4, 2, 257) == -1
    need = size(4096, 8, 128)
    assert need == 32 * 128 * 4
    assert size(1 << 26, 8, 256) <= 152 * 256 * 4  # a count an expert for each of the blocks
    assert call(T=4096, k=8, E=128) == INV                     # a workspace is needed
    assert call(T=4096, k=8, E=128, ws=16, n=need - 1) == MEM
    assert call(T=4096, k=8, E=128, ws=24, n=need) == INV


def test_rows_refusals(L):
    def dis(x=16, dt=BF16, places=16, w=None, T=4, k=2, H=64, R=8, rows=16, rw=None):
        return L.mm_dispatch_rows(x, dt, places, w, T, k, H, R, rows, rw, None)

    def com(rows=16, dt=BF16, places=16, w=None, rv=None, T=4, k=2, H=64, R=8, out=16, v=None):
        return L.mm_combine_rows(rows, dt, places, w, rv, T, k, H, R, out, v, None)

    for f in (dis, com):
        assert f(T=-1) == INV and f(k=0) == INV and f(H=0) == INV and f(R=-1) == INV
        assert f(H=60) == UNS and f(k=33) == UNS and f(H=(1 << 20) + 8) == UNS
        assert f(dt=F32) == UNS and f(dt=9) == INV and f(rows=None) == INV and f(rows=24) == INV
        assert f(places=None) == INV and f(places=18) == INV
    assert dis(x=None) == INV and dis(x=8) == INV and dis(w=16) == INV and dis(rw=16) == INV
    assert dis(w=18, rw=16) == INV and dis(T=0, x=None, places=None, rows=None) == OK
    assert com(out=None) == INV and com(out=8) == INV and com(rv=16) == INV and com(v=16) == INV
    assert com(T=0, rows=None, places=None, out=None) == OK


def test_product_refusals(L):
    def y(x=16, w=16, dt=BF16, off=16, R=4, E=2, N=64, K=64, out=16):
        return L.mm_grouped_product(x, w, dt, off, R, E, N, K, out, None)

    def dx(x=16, w=16, dt=BF16, off=16, R=4, E=2, N=64, K=64, out=16):
        return L.mm_grouped_product_dx(x, w, dt, off, R, E, N, K, out, None)

    def dw(x=16, w=16, dt=BF16, off=16, R=4, E=2, N=64, K=64, out=16, odt=BF16, add=0, ws=None,
           n=0):
        return L.mm_grouped_product_dw(x, w, dt, off, R, E, N, K, out, odt, add, ws, n, None)

    for f in (y, dx, dw):
        assert f(R=-1) == INV and f(E=0) == INV and f(N=0) == INV and f(K=0) == INV
        assert f(N=60) == UNS and f(K=60) == UNS and f(E=257) == UNS and f(R=(1 << 31) - 1) == UNS
        assert f(N=(1 << 20) + 8) == UNS and f(K=(1 << 20) + 8) == UNS
        assert f(N=1 << 19, K=1 << 18) == UNS and f(R=1 << 30, N=1 << 20, K=8) == UNS
        assert f(dt=F32) == UNS and f(dt=5) == INV
        assert f(x=None) == INV and f(w=None) == INV and f(off=None) == INV and f(out=None) == INV
        assert f(x=8) == INV and f(w=8) == INV and f(off=18) == INV and f(out=8) == INV
    assert y(R=0, x=None, w=None, off=None, out=None) == OK
    assert dx(R=0, x=None, w=None, off=None, out=None) == OK
    assert dw(R=0, x=None, w=None, off=None, add=1) == OK      # nothing to add
    assert dw(odt=F16) == UNS and dw(dt=F16, odt=BF16) == UNS and dw(odt=7) == INV
    size = L.mm_grouped_product_dw_workspace_size
    assert size(-1, 1, 8, 8, F32) == -1 and size(4, 1, 12, 8, F32) == -1
    assert size(4, 1, 8, 8, 7) == -1 and size(0, 4, 64, 64, BF16) == 0
    assert size(32768, 128, 1536, 2048, BF16) == 0             # many tiles: whole segments
    need = size(32768, 1, 64, 64, F32)                         # one tile: parts
    assert 0 < need < 1 << 24
    assert dw(R=32768, E=1, odt=F32) == INV
    assert dw(R=32768, E=1, odt=F32, ws=16, n=need - 1) == MEM
    assert dw(R=32768, E=1, odt=F32, ws=24, n=need) == INV


def test_swiglu_refusals(L):
    def pack(z=16, dt=BF16, end=None, R=4, I=64, act=16, q=16, s=16):
        return L.mm_swiglu_pack(z, dt, end, R, I, act, q, s, None)

    def back(q=16, s=16, da=16, dt=BF16, w=None, end=None, R=4, I=64, dz=16, act=16, dw=None):
        return L.mm_swiglu_pack_backward(q, s, da, dt, w, end, R, I, dz, act, dw, None)

    def deq(q=16, s=16, R=4, I=64, out=16, dt=BF16):
        return L.mm_mxint8_dequantize(q, s, R, I, out, dt, None)

    for f in (pack, back, deq):
        assert f(R=-1) == INV and f(I=0) == INV and f(I=48) == UNS and f(dt=9) == INV
        assert f(I=1 << 21) == UNS and f(R=(1 << 31) - 1) == UNS
        assert f(q=None) == INV and f(s=None) == INV and f(q=8) == INV
    assert pack(dt=F32) == UNS and back(dt=F32) == UNS
    assert pack(z=None) == INV and pack(act=None) == INV and pack(z=8) == INV and pack(end=18) == INV
    assert back(da=None) == INV and back(dz=8) == INV and back(act=None) == INV
    assert back(w=18) == INV and back(dw=18) == INV and back(end=18) == INV
    assert deq(out=None) == INV and deq(out=8) == INV
    assert pack(R=0, z=None, act=None, q=None, s=None) == OK
    assert back(R=0, q=None, s=None, da=None, dz=None, act=None) == OK
    assert deq(R=0, q=None, s=None, out=None) == OK


def test_binding_refuses_what_is_not_on_a_gpu(mmlib):
    b, i = torch.bfloat16, torch.int32
    x, w, off = torch.zeros(4, 64, dtype=b), torch.zeros(2, 32, 64, dtype=b), torch.zeros(3, dtype=i)
    ids = torch.zeros(4, 2, dtype=i)
    for f in (lambda: mm.mm_group_slots(ids, 8), lambda: mm.mm_dispatch_rows(x, ids),
              lambda: mm.mm_combine_rows(x, ids), lambda: mm.mm_grouped_product(x, w, off),
              lambda: mm.mm_grouped_product_dw(x, x, off), lambda: mm.mm_swiglu_pack(x),
              lambda: mm.mm_mxint8_dequantize(torch.zeros(4, 64, dtype=torch.int8),
                                              torch.zeros(4, 2, dtype=torch.uint8))):
        with pytest.raises(ValueError, match="CUDA"):
            f()
    for f in (lambda: mm.mm_dispatch_rows(x.float(), ids), lambda: mm.mm_swiglu_pack(x.double()),
              lambda: mm.mm_grouped_product(3, w, off)):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(ValueError, match="dimensions"):
        mm.mm_dispatch_rows(x, ids[0])
    with pytest.raises(ValueError, match="shape"):
        mm.mm_grouped_product(x, w, off[:2])


def test_stored_values_by_hand():
    z = torch.zeros(2, 64)
    z[0, :4] = torch.tensor([1.0, -0.5, 1 / 128, 1 / 256])       # unit 2^-6
    z[0, 32:36] = torch.tensor([127.5, 127.4, -127.6, 0.5])      # unit 1: to 128, cut to 127
    z[1, 0] = 2.0 ** -140
    z[1, 32] = float("inf")
    q, s = ref.encode(z)
    assert s.tolist() == [[121, 127], [0, 255]]
    assert q[0, :4].tolist() == [64, -32, 0, 0]                  # 0.5 steps: ties to even
    assert q[0, 32:36].tolist() == [127, 127, -127, 0]
    assert q[1].abs().sum() == 0                                 # 2^-13 steps of 2^-127; a NaN block
    v = ref.decode(q, s)
    assert v[0, 0] == 1.0 and v[0, 32] == 127 and v[1, :32].abs().sum() == 0
    assert v[1, 32:].isnan().all()


def test_stored_values_are_within_half_a_step():
    g = torch.Generator().manual_seed(0)
    z = torch.randn(64, 256, generator=g) * torch.exp(2 * torch.randn(64, 1, generator=g))
    z = z.to(torch.bfloat16)
    q, s = ref.encode(z)
    unit = torch.exp2(s.double() - 127).repeat_interleave(32, 1)
    assert ((ref.decode(q, s) - z.double()).abs() <= unit / 2).all()


def test_gradients_by_differences():
    """swiglu_grad and experts against central differences and autograd in float64."""
    g = torch.Generator().manual_seed(1)

    def rand(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)

    z, da, w = rand(3, 128), rand(3, 64), rand(3).abs()
    dz, act, dw = ref.swiglu_grad(z, da, w)
    h, dirz, dirw = 1e-6, rand(3, 128), rand(3)

    def f(z, w):
        return (da * w[:, None] * ref.swiglu(z)).sum()

    num = (f(z + h * dirz, w + h * dirw) - f(z - h * dirz, w - h * dirw)) / (2 * h)
    assert abs(num - (dz * dirz).sum() - (dw * dirw).sum()) < 1e-7
    assert torch.allclose(act, w[:, None] * ref.swiglu(z))
    E, H, I = 3, 8, 32
    args = [rand(4, H), rand(4, 2), rand(E, 2 * I, H), rand(E, H, I)]
    ids, mask = torch.tensor([[0, 2], [1, 2], [2, 0], [1, 1]]), torch.tensor([1, 1, 0, 1])
    leaves = [a.clone().requires_grad_(True) for a in args]
    d = rand(4, H)
    grads = torch.autograd.grad(
        (d * ref.experts(leaves[0], ids, *leaves[1:], mask=mask)).sum(), leaves)
    dirs = [rand(*a.shape) for a in args]
    ends = [(d * ref.experts(*(lambda a: (a[0], ids, *a[1:]))(
        [x + s * 1e-6 * v for x, v in zip(args, dirs)]), mask=mask)).sum() for s in (1, -1)]
    assert abs((ends[0] - ends[1]) / 2e-6 - sum((a * b).sum() for a, b in zip(grads, dirs))) < 1e-5


def test_group_by_hand():
    ids = torch.tensor([[2, 0], [0, 2], [5, 1], [0, 0]])
    places, offsets = ref.group(ids, 3, torch.tensor([True, True, True, False]))
    assert offsets.tolist() == [0, 2, 3, 5]
    assert places.tolist() == [[3, 0], [1, 4], [-1, 2], [-1, -1]]


def test_a_refused_backward_makes_no_call(mmlib, monkeypatch):
    """Both gradients are looked at before the first call, which would add to one."""
    from mixture_experts_layer_mm_gb300 import _lib, experts_train
    made = []
    for name in ("mm_dispatch_rows", "mm_grouped_product_dx", "mm_grouped_product_dw",
                 "mm_swiglu_pack_backward", "mm_combine_rows"):
        monkeypatch.setattr(_lib, name, lambda *a, name=name, **k: made.append(name) or (a[0],) * 3)
    b, E, H, I, T, k = torch.bfloat16, 3, 16, 32, 4, 2
    s = experts_train.ExpertsSaved(
        torch.zeros(T, H, dtype=b), torch.zeros(T, k, dtype=torch.int32),
        torch.zeros(E + 1, dtype=torch.int32), torch.zeros(T * k),
        torch.zeros(T * k, 2 * I, dtype=torch.int8), torch.zeros(T * k, I // 16, dtype=torch.uint8))
    gu, dn = torch.zeros(E, 2 * I, H, dtype=b), torch.zeros(E, H, I, dtype=b)
    d_gu, d_dn = torch.zeros(gu.shape), torch.zeros(dn.shape)

    def call(match, error=ValueError, d_out=s.hidden, gu=gu, dn=dn, accumulate=True, **given):
        with pytest.raises(error, match=match):
            mm.moe_experts_train_backward(d_out, s, gu, dn, accumulate=accumulate, **given)

    call("accumulate needs", d_w_down=d_dn)
    call("accumulate needs", d_w_gate_up=d_gu)
    call("accumulate needs")
    call("d_w_gate_up must have shape", d_w_down=d_dn, d_w_gate_up=d_gu[:2], accumulate=False)
    call("d_out must have shape", d_out=s.hidden[:2], d_w_down=d_dn, d_w_gate_up=d_gu)
    call("w_gate_up must have shape", gu=gu[:, :32], d_w_down=d_dn, d_w_gate_up=d_gu)
    call("CUDA", d_w_down=d_dn, d_w_gate_up=d_gu)
    call("d_out must be torch", TypeError, d_out=s.hidden.float(), d_w_down=d_dn, d_w_gate_up=d_gu)
    assert not made


def test_the_byte_is_six_less_than_the_interchange_formats():
    """In OCP's MXINT8 a block whose largest value is 1 has the byte 127 and codes q / 64."""
    z = torch.zeros(1, 32)
    z[0, :3] = torch.tensor([1.0, -0.75, 1 / 64])
    q, s = ref.encode(z)
    assert s.item() == 127 - 6 and q[0, :3].tolist() == [64, -48, 1]
    assert torch.equal(ref.decode(q, s), (q.double() / 64) * 2.0 ** (s.double().item() + 6 - 127))


def test_sizes_beyond_an_int_are_refused(mmlib):
    """Not taken as what their lower 32 bits say."""
    big = (1 << 32) + 4
    assert mm.mm_group_slots_workspace_size(4096, 8, 128) > 0
    for sizes in ((big, 2, 8), (4, big, 8), (4, 2, big), (1 << 31, 1, 8)):
        assert mm.mm_group_slots_workspace_size(*sizes) == -1
    for i in range(4):
        sizes = [32768, 1, 64, 64]
        assert mm.mm_grouped_product_dw_workspace_size(*sizes, torch.float32) > 0
        sizes[i] += 1 << 32
        assert mm.mm_grouped_product_dw_workspace_size(*sizes, torch.float32) == -1
    b, i32 = torch.bfloat16, torch.int32
    rows, slots = torch.zeros(1, 8, dtype=b).expand(big, 8), torch.zeros(1, 1, dtype=i32).expand(big, 1)
    w, off = torch.zeros(1, 8, 8, dtype=b), torch.zeros(2, dtype=i32)
    for f in (lambda: mm.mm_group_slots(slots, 8), lambda: mm.mm_dispatch_rows(rows, slots),
              lambda: mm.mm_combine_rows(rows[:4], slots), lambda: mm.mm_combine_rows(rows, slots[:4]),
              lambda: mm.mm_grouped_product(rows, w, off), lambda: mm.mm_grouped_product_dx(rows, w, off),
              lambda: mm.mm_grouped_product_dw(rows, rows, off),
              lambda: mm.mm_swiglu_pack(rows[:, :1].expand(big, 64)),
              lambda: mm.mm_mxint8_dequantize(torch.zeros(1, 32, dtype=torch.int8).expand(big, 32),
                                              torch.zeros(1, 1, dtype=torch.uint8).expand(big, 1))):
        with pytest.raises(ValueError, match="below 2"):
            f()
