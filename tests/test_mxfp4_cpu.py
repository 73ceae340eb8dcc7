"""Routing from logits and the 4-bit operators on a machine without a GPU:
what the entry points refuse before any CUDA call, the sizes they report, the
stored order of the scales, and the float64 definitions the GPU tests use."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_mm_gb300 as mm
import mx_reference as ref

INV, UNS, MEM, OK = (mm.MM_ERR_INVALID_ARG, mm.MM_ERR_UNSUPPORTED, mm.MM_ERR_NO_MEMORY, mm.MM_OK)
F32, BF16, F16 = mm.MM_DTYPE_FP32, mm.MM_DTYPE_BF16, mm.MM_DTYPE_FP16


@pytest.fixture(scope="module")
def L(mmlib):
    return mm.lib()


def test_route_logits_refusals(L):
    def call(logits=16, dt=F32, T=4, E=8, k=2, ids=16, w=16, counts=16, sums=16, loss=16, ws=None,
             n=0):
        return L.mm_route_logits(logits, dt, None, T, E, k, 1, ids, w, counts, sums, loss, ws, n,
                                 None)

    assert call(T=-1) == INV and call(E=0) == INV and call(k=0) == INV and call(dt=7) == INV
    assert call(dt=F16) == UNS and call(E=257) == UNS and call(k=9) == UNS
    assert call(E=64, k=33) == UNS and call(T=1 << 30, E=8, k=2) == UNS
    assert call(logits=None) == INV and call(ids=None) == INV and call(w=None) == INV
    assert call(counts=None) == INV and call(sums=None) == INV and call(loss=None) == INV
    assert call(logits=18) == INV and call(w=18) == INV and call(loss=18) == INV
    assert call(dt=BF16, logits=17) == INV
    need = L.mm_route_logits_workspace_size(1000, 8)
    assert need > 0
    assert call(T=1000) == INV                       # a workspace is needed
    assert call(T=1000, ws=16, n=need - 1) == MEM
    assert call(T=1000, ws=24, n=need) == INV        # misaligned
    assert L.mm_route_logits_workspace_size(8, 64) == 0
    assert L.mm_route_logits_workspace_size(-1, 64) == -1
    assert L.mm_route_logits_workspace_size(8, 300) == -1
    # grows to a fixed number of rows of 2 values an expert
    assert L.mm_route_logits_workspace_size(1 << 20, 256) == \
        L.mm_route_logits_workspace_size(1 << 16, 256) <= 1 << 20


def test_route_logits_backward_refusals(L):
    def call(logits=16, dt=F32, ids=16, counts=16, dw=16, dl=16, T=4, E=8, k=2, grad=16):
        return L.mm_route_logits_backward(logits, dt, None, ids, counts, dw, dl, T, E, k, 1, grad,
                                          None)

    assert call(T=-1) == INV and call(dt=F16) == UNS and call(E=300) == UNS and call(k=9) == UNS
    assert call(logits=None) == INV and call(ids=None) == INV and call(counts=None) == INV
    assert call(grad=None) == INV and call(dw=18) == INV and call(dl=18) == INV
    assert call(grad=18) == INV and call(dt=BF16, logits=17) == INV
    assert call(T=0, logits=None, ids=None, counts=None, grad=None) == OK


def test_mxfp4_refusals(L):
    assert L.mm_mxfp4_scales_size(3, 129, 160) == 3 * 2 * 2 * 512
    assert L.mm_mxfp4_scales_size(0, 5, 32) == 0 and L.mm_mxfp4_scales_size(1, 0, 32) == 0
    assert L.mm_mxfp4_scales_size(1, 5, 33) == -1 and L.mm_mxfp4_scales_size(-1, 5, 32) == -1
    assert L.mm_mxfp4_scales_size(1, 5, 0) == -1
    assert L.mm_mxfp4_scales_size(1 << 20, 1 << 12, 32) == -1
    q = L.mm_mxfp4_quantize
    assert q(16, BF16, 1, 4, 33, 16, 16, None) == UNS and q(16, 3, 1, 4, 32, 16, 16, None) == INV
    assert q(16, BF16, -1, 4, 32, 16, 16, None) == INV
    assert q(None, BF16, 1, 4, 32, 16, 16, None) == INV
    assert q(16, BF16, 1, 4, 32, 24, 16, None) == INV
    assert q(None, BF16, 0, 4, 32, None, None, None) == OK
    assert q(None, F16, 1, 0, 32, None, None, None) == OK
    d = L.mm_mxfp4_dequantize
    assert d(16, 16, 1, 4, 48, 16, BF16, None) == UNS and d(16, 16, 1, 4, 32, 16, 9, None) == INV
    assert d(16, 16, 1, 4, 32, 8, BF16, None) == INV and d(16, None, 1, 4, 32, 16, F32, None) == INV
    assert d(None, None, 2, 0, 32, None, F32, None) == OK
    g = L.mm_mxfp4_gemm
    assert g(16, 16, 16, 16, 4, 4, 40, 16, BF16, None) == UNS
    assert g(16, 16, 16, 16, 4, 4, 32, 16, F16, None) == UNS
    assert g(16, 16, 16, 16, -4, 4, 32, 16, BF16, None) == INV
    assert g(16, 16, 16, 16, 4, -4, 32, 16, BF16, None) == INV
    assert g(16, 16, 16, 16, 4, 4, 32, 16, 5, None) == INV
    assert g(16, 16, None, 16, 4, 4, 32, 16, BF16, None) == INV
    assert g(16, 16, 16, 24, 4, 4, 32, 16, BF16, None) == INV
    assert g(None, None, None, None, 0, 4, 32, None, BF16, None) == OK
    assert g(None, None, None, None, 4, 0, 32, None, F32, None) == OK


def test_experts_refusals(L):
    size = L.mm_moe_experts_mxfp4_workspace_size

    def call(T=4, H=64, E=8, I=64, k=2, hidden=16, ids=16, w=16, gu=16, out=16, ws=256, n=None):
        n = max(size(4, 64, 8, 64, 2), 0) if n is None else n
        return L.mm_moe_experts_mxfp4(hidden, ids, w, gu, 16, 16, 16, T, H, E, I, k, out, ws, n,
                                      None)

    assert call(T=-1) == INV and call(H=0) == INV and call(k=0) == INV
    assert call(H=96) == UNS and call(I=32) == UNS and call(E=300) == UNS and call(k=9) == UNS
    assert call(hidden=None) == INV and call(ids=None) == INV and call(gu=24) == INV
    assert call(out=8) == INV and call(ws=None) == INV and call(ws=128) == INV
    assert call(n=size(4, 64, 8, 64, 2) - 1) == MEM
    assert call(T=0, hidden=None, ids=None, w=None, gu=None, out=None, ws=None, n=0) == OK
    assert size(4, 96, 8, 64, 2) == -1 and size(-1, 64, 8, 64, 2) == -1
    assert size(1 << 30, 64, 8, 64, 2) == -1
    # token rows, activations, fp16 rows of the down product
    assert size(64, 2048, 128, 768, 8) >= 512 * (2048 // 2 + 768 // 2 + 2048 * 2)


def test_sizes_at_the_end_of_the_index_range(L):
    top = (1 << 31) - 1
    # The most tokens: the workspace of any long batch, not one of a wrapped count.
    assert L.mm_route_logits_workspace_size(top, 8) == L.mm_route_logits_workspace_size(1 << 20, 8)
    # Rows and columns end 4096 short of 2^31, so that steps beyond them stay in range.
    last = (1 << 31) - 4096
    assert L.mm_mxfp4_scales_size(1, 1, last) == last // 128 * 512
    assert L.mm_mxfp4_scales_size(1, last, 32) == last // 128 * 512
    assert L.mm_mxfp4_scales_size(1, 1, last + 32) == -1
    assert L.mm_mxfp4_scales_size(1, last + 1, 32) == -1
    assert L.mm_mxfp4_scales_size(2, 1 << 30, 32) == -1
    for K in (last + 32, (1 << 31) - 32):
        assert L.mm_mxfp4_quantize(16, F32, 1, 1, K, 16, 16, None) == UNS
        assert L.mm_mxfp4_dequantize(16, 16, 1, 1, K, 16, F32, None) == UNS
        assert L.mm_mxfp4_gemm(16, 16, 16, 16, 1, 1, K, 16, F32, None) == UNS
    for rows in (last + 1, (1 << 31) - 128, top):
        assert L.mm_mxfp4_gemm(16, 16, 16, 16, 1, rows, 32, 16, F32, None) == UNS
        assert L.mm_mxfp4_gemm(16, 16, 16, 16, rows, 1, 32, 16, F32, None) == UNS


def test_experts_workspace_counts_the_segments_that_can_hold_rows(L):
    size = L.mm_moe_experts_mxfp4_workspace_size
    # One token of 8 slots: 8 segments of 128 rows, whatever the number of experts.
    row = 2048 // 2 + 768 // 2 + 2048 * 2 + 2048 // 32 + (2048 + 768) // 32  # bytes a row
    assert 8 * 128 * row <= size(1, 2048, 256, 768, 8) <= 8 * 128 * row + 16384
    assert size(1, 2048, 128, 768, 8) <= size(1, 2048, 256, 768, 8)


def test_binding_refusals(mmlib):
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        mm.mm_mxfp4_quantize(x)
    with pytest.raises(ValueError, match="CUDA"):
        mm.mm_route_logits(x, 2, True)
    with pytest.raises(TypeError):
        mm.mm_route_logits(x.double(), 2, True)
    with pytest.raises(TypeError):
        mm.mm_mxfp4_quantize(x.to(torch.int32))
    with pytest.raises(ValueError, match="dimensions"):
        mm.mm_mxfp4_quantize(torch.zeros(64))
    c, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 1, 512, dtype=torch.uint8)
    with pytest.raises(ValueError, match="shape"):
        mm.mm_mxfp4_gemm(c, s[:, :, :256], c, s)
    with pytest.raises(ValueError, match="one matrix"):
        mm.mm_mxfp4_gemm(c.repeat(2, 1, 1), s, c, s)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="shape"):
        mm.mm_route_logits_backward(x, ids[:3], torch.zeros(64, dtype=torch.int32), True)
    with pytest.raises(ValueError, match="one value"):
        mm.mm_route_logits_backward(x, ids, torch.zeros(64, dtype=torch.int32), True,
                                    d_loss=torch.zeros(2))
    with pytest.raises(ValueError, match="shape"):
        mm.mm_moe_experts_mxfp4(torch.zeros(4, 128), ids, torch.zeros(3, 2), c, s, c[None], s[None])


@pytest.mark.parametrize("rows,K", [(1, 32), (128, 128), (129, 160), (300, 1056)])
def test_scale_order(rows, K, mmlib):
    s = np.random.default_rng(rows).integers(0, 256, (rows, K // 32)).astype(np.uint8)
    got = mm.mxfp4_tile_scales(torch.from_numpy(s))
    assert tuple(got.shape) == mm.mm_mxfp4_scales_shape(rows, K)
    assert np.array_equal(got.numpy(), ref.tile(s))
    two = mm.mxfp4_tile_scales(torch.from_numpy(np.stack([s, s[::-1]])))
    assert np.array_equal(two[0].numpy(), ref.tile(s))
    assert np.array_equal(two[1].numpy(), ref.tile(s[::-1]))


def test_reference_rounding_by_hand():
    x = np.zeros(32)
    x[:16] = [4, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 5.01, 7.9, -0.1, -2.5, -0.75, 0.74, 3.6]
    s = ref.scale_bytes(x)
    assert s.tolist() == [127]
    want = [4, 0, .5, 1, 1, 2, 2, 4, 4, 6, 6, -0.0, -2, -1, .5, 4]
    assert ref.values(ref.codes_under(x, s), s)[:16].tolist() == want
    assert ref.scale_bytes(x * 2 - 0.0).tolist() == [127 + 1]
    assert ref.scale_bytes(np.zeros(32)).tolist() == [0]
    assert ref.scale_bytes(np.r_[np.inf, np.zeros(31)]).tolist() == [255]
    assert np.array_equal(ref.unpack(ref.pack(ref.codes_under(x, s))), ref.codes_under(x, s))


def test_reference_balance_loss_by_hand():
    # Two tokens, two experts, one each: p = (3/4, 1/4) and (1/4, 3/4).
    l = np.log(np.array([[3.0, 1.0], [1.0, 3.0]]))
    r = ref.route(l, 1, False)
    assert r["ids"].tolist() == [[0], [1]] and r["counts"].tolist() == [1, 1]
    assert np.allclose(r["w"], 0.75) and np.isclose(r["loss"], 1.0)
    # Both to expert 0: f = (1, 0), P = (3/4, 1/4): loss = 2 * 3/4
    r = ref.route(np.log(np.array([[3.0, 1.0], [3.0, 1.0]])), 1, False)
    assert np.isclose(r["loss"], 1.5)
    # its gradient: p (c - sum p c), c = (1, 0) * 2 / 2
    g = ref.route_grad(np.log(np.array([[3.0, 1.0], [3.0, 1.0]])), 1, False, None, 1.0)
    assert np.allclose(g, [[3 / 16, -3 / 16]] * 2)
