"""Measured calls of the router-training and 4-bit expert operators.

Four groups of calls, each in a plain form (elementary torch operations in 32
bits) and through the package:

  route     routing from given router logits with the balance loss, the
            per-expert counts and (training) the gradient of the logits
  quantize  rows to microscaled 4-bit floats (blocks of 32 e2m1 values under
            one e8m0 power of two) and back to bf16
  product   C = A B^T of two microscaled 4-bit matrices
  experts   the routed SwiGLU experts of an MoE layer with 4-bit weights

4-bit values are stored two to a byte (even column in the low nibble). The
scale bytes of a [rows, K] matrix are stored in tiles of 128 rows x 128
columns: tile (r / 128, k / 128) is 512 contiguous bytes, and the scale of
row r, columns [32 c, 32 c + 32) is its byte
(r % 32) * 16 + ((r % 128) / 32) * 4 + c % 4; rows and columns are padded up
to whole tiles with zero bytes.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# e2m1 magnitudes by code, and the borders between neighbours: a value on a
# border goes to the even code, so borders 1, 3, 5 (0.75, 1.75, 3.5) round up.
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # One decode step's routing (the 64-token decode shape): latency.
        dict(name="route_decode", op="route", T=64, E=128, k=8, renorm=True, dtype="fp32",
             masked=0.0, train=False),
        # A training micro-batch of 4096 tokens with padded sequences, bf16 logits.
        dict(name="route_train", op="route", T=4096, E=128, k=8, renorm=True, dtype="bf16",
             masked=0.1, train=True),
        # An odd token count and an expert count that fills no power of two.
        dict(name="route_train_odd", op="route", T=5003, E=60, k=4, renorm=False, dtype="fp32",
             masked=0.05, train=True),
        # A large global batch over the most experts the router takes.
        dict(name="route_train_large", op="route", T=131072, E=256, k=8, renorm=True,
             dtype="fp32", masked=0.02, train=True),
        # The activations of one decode step.
        dict(name="quantize_tokens", op="quantize", batch=1, rows=64, K=2048, dtype="bf16"),
        # The gate_up weights of one whole layer (128 experts, gate and up).
        dict(name="quantize_weights", op="quantize", batch=256, rows=768, K=2048, dtype="bf16"),
        # A projection of a decode batch: the weights' bytes are the work.
        dict(name="product_decode", op="product", M=64, N=4096, K=4096, out="bf16"),
        # Ragged in every dimension, fp32 result.
        dict(name="product_odd", op="product", M=1111, N=1000, K=2080, out="fp32"),
        # A projection of a prefill batch: arithmetic is the work.
        dict(name="product_prefill", op="product", M=8192, N=4096, K=4096, out="bf16"),
        # One new token through the experts.
        dict(name="experts_token", op="experts", T=1, H=2048, I=768, E=128, k=8),
        # A decode batch: nearly every expert is read for a few tokens.
        dict(name="experts_decode", op="experts", T=64, H=2048, I=768, E=128, k=8),
        # A prefill batch.
        dict(name="experts_prefill", op="experts", T=4096, H=2048, I=768, E=128, k=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "quantize", "product", "experts"])
    if op == "route":
        E = rng.choice([8, 16, 40, 60, 64, 100, 128, 160, 256])
        return dict(op=op, T=_log(rng, 1, 131072), E=E, k=rng.randint(1, min(E, 10)),
                    renorm=rng.random() < 0.5, dtype=rng.choice(["fp32", "bf16"]),
                    masked=rng.choice([0.0, 0.0, 0.1, 0.4]), train=rng.random() < 0.7)
    if op == "quantize":
        K = 32 * _log(rng, 1, 256)
        rows = _log(rng, 1, 4096)
        batch = _log(rng, 1, max(1, min(64, 400_000_000 // (K * rows * 2))))
        return dict(op=op, batch=batch, rows=rows, K=K,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    if op == "product":
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 16, 4096), K=32 * _log(rng, 1, 128),
                    out=rng.choice(["bf16", "bf16", "fp32"]))
    H, I, E = rng.choice([(2048, 768, 128), (1024, 512, 64), (640, 320, 40), (2048, 1024, 32),
                          (256, 64, 8)])
    return dict(op=op, T=_log(rng, 1, 4096), H=H, I=I, E=E, k=rng.randint(1, min(E, 8)))


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["dtype"] == "fp32" else 2
        n = T * E * size + T * k * 8 + E * 8 + 4
        flops = T * E * 6
        if case["train"]:
            n += T * E * size + T * k * 4
            flops += T * E * 6
        return {"bytes": n + T * (case["masked"] > 0), "flops": flops}
    if op == "quantize":
        n = case["batch"] * case["rows"] * case["K"]
        return {"bytes": n * ((4 if case["dtype"] == "fp32" else 2) + 2), "flops": 4 * n}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * K * 17 / 32 + M * N * (4 if case["out"] == "fp32" else 2),
                "flops": 2 * M * N * K}
    T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
    distinct = E * (1 - (1 - k / E) ** T)  # experts that some token chose (expected)
    return {"bytes": distinct * 3 * H * I * 17 / 32 + T * H * 4 + T * k * 8,
            "flops": 2 * T * k * 3 * H * I}


# ----------------------------------------------------------------- inputs ---

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _encode(x):
    """Codes (uint8, two to a byte) and block exponents (uint8) of x [..., K] float32."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = (torch.frexp(amax)[1] - 3).clamp(-127, 127)  # floor(log2 amax) - 2
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    v = torch.ldexp(b, -e.unsqueeze(-1))
    a = v.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(v).to(torch.uint8)).flatten(-2).unflatten(-1, (-1, 2))
    return code[..., 0] + 16 * code[..., 1], (e + 127).to(torch.uint8)


def _tile(s):
    """Scale bytes [batch, rows, K / 32] in the stored tile order."""
    rows, cols = s.shape[1:]
    s = torch.nn.functional.pad(s, (0, -cols % 4, 0, -rows % 128))
    s = s.view(s.shape[0], s.shape[1] // 128, 4, 32, s.shape[2] // 4, 4)
    return s.permute(0, 1, 4, 3, 2, 5).flatten(3).contiguous()  # [batch, rows/128, K/128, 512]


def _untile(t, rows, cols):
    b, r, c = t.shape[:3]
    s = t.view(b, r, c, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(b, r * 128, c * 4)
    return s[:, :rows, :cols]


def _rows_with_range(g, batch, rows, K):
    """Rows whose magnitudes spread as activations' and weights' do, with some
    larger columns."""
    x = _normal(g, batch, rows, K)
    x *= torch.exp(0.5 * _normal(g, batch, rows, 1))
    x *= torch.exp(0.7 * _normal(g, batch, 1, K))
    return x


def _weights(g, batch, rows, K, std=0.02):
    codes = torch.empty(batch, rows, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(batch, rows, K // 32, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (rows * K))
    for b in range(0, batch, step):
        n = min(step, batch - b)
        codes[b:b + n], scales[b:b + n] = _encode(std * _normal(g, n, rows, K))
    return codes, _tile(scales)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        # Logits with a per-expert offset: the uneven load a balance loss is for.
        s["logits"] = (_normal(g, T, E) + 0.5 * _normal(g, 1, E)).to(_DTYPES[case["dtype"]])
        s["mask"] = None
        if case["masked"] > 0:
            s["mask"] = torch.rand(T, generator=g, device="cuda") >= case["masked"]
        if case["train"]:
            s["d_topk_w"] = _normal(g, T, k) / T
            s["d_loss"] = torch.full((1,), 0.01, device="cuda")
    elif op == "quantize":
        x = _rows_with_range(g, case["batch"], case["rows"], case["K"])
        s["x"] = x.to(_DTYPES[case["dtype"]])
    elif op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        a, sa = _encode(_rows_with_range(g, 1, M, K))
        s["a"], s["sa"] = a, _tile(sa)
        s["b"], s["sb"] = _weights(g, 1, N, K)
    else:
        T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
        s["hidden"] = _normal(g, T, H).to(torch.bfloat16)
        logits = _normal(g, T, E) + 0.3 * _normal(g, 1, E)
        w, ids = torch.sort(torch.softmax(logits, -1), dim=-1, descending=True, stable=True)
        ids, order = torch.sort(ids[:, :k], -1)
        w = w[:, :k].gather(1, order)
        s["ids"] = ids.to(torch.int32).contiguous()
        s["w"] = (w / w.sum(-1, keepdim=True)).contiguous()
        s["gu"], s["sgu"] = _weights(g, 2 * E, I, H)
        s["dn"], s["sdn"] = _weights(g, E, H, I)
        # The plan of the plain form: the experts that some token chose, and
        # the longest list of tokens of one expert.
        count = torch.bincount(ids.flatten(), minlength=E)
        s["used"] = torch.nonzero(count).flatten()
        s["most"] = int(count.max())
    return s


# ------------------------------------------------------------- plain form ---

def _decode(codes, scales, rows, K):
    """float32 values [batch, rows, K] of stored codes and tiled scales."""
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int32)
    e = _untile(scales, rows, K // 32).to(torch.int32) - 127
    v = torch.ldexp(table[c].unflatten(-1, (-1, 32)), e.unsqueeze(-1))
    return v.flatten(-2)


def _rounded(x):
    """x [..., K] float32 rounded to the nearest microscaled 4-bit values."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax)[1] - 3).clamp(-127, 127)
    a = torch.ldexp(b.abs(), -e)
    q = (0.5 * (a > 0.25) + 0.5 * (a >= 0.75) + 0.5 * (a > 1.25) + 0.5 * (a >= 1.75)
         + 1.0 * (a > 2.5) + 1.0 * (a >= 3.5) + 2.0 * (a > 5.0))
    return torch.ldexp(torch.copysign(q.float(), b), e).flatten(-2)


def _plain_route(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    x = s["logits"].float()
    valid = torch.ones(T, 1, device=x.device) if s["mask"] is None else s["mask"][:, None].float()
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    ids = torch.sort(torch.sort(x, dim=-1, descending=True, stable=True)[1][:, :k], -1)[0]
    chosen = p.gather(1, ids)
    total = chosen.sum(-1, keepdim=True)
    w = (chosen / total if c["renorm"] else chosen) * valid
    picked = torch.zeros(T, E, device=x.device).scatter_(1, ids, 1.0) * valid
    counts = picked.sum(0, dtype=torch.float64)
    prob_sums = (p * valid).sum(0, dtype=torch.float64)
    n = counts.sum() / k
    n = torch.where(n > 0, n, torch.ones_like(n))
    loss = E * (counts / (n * k) * prob_sums / n).sum()
    out = {"ids": ids.to(torch.int32), "w": w, "counts": counts.to(torch.int32),
           "prob_sums": prob_sums.float(), "loss": loss.float().reshape(1)}
    if c["train"]:
        dw = s["d_topk_w"]
        if c["renorm"]:
            r = chosen / total
            d = torch.zeros_like(p).scatter_(1, ids, r * (dw - (dw * r).sum(-1, keepdim=True)))
        else:
            d = torch.zeros_like(p).scatter_(1, ids, chosen * dw)
            d = d - p * (chosen * dw).sum(-1, keepdim=True)
        f = (s["d_loss"].double() * E * counts / (n * k) / n).float()
        d = (d + p * (f - (p * f).sum(-1, keepdim=True))) * valid
        out["d_logits"] = d.to(s["logits"].dtype)
    return out


def _plain_experts(s):
    c = s["case"]
    T, H, I, k, most = c["T"], c["H"], c["I"], c["k"], s["most"]
    x = _rounded(s["hidden"].float())
    used = s["used"]
    n = used.numel()
    flat = torch.bucketize(s["ids"].flatten().long(), used)  # place among the used experts
    order = torch.sort(flat, dim=0, stable=True)[1]
    counts = torch.zeros(n, dtype=torch.long, device=flat.device).scatter_add_(
        0, flat, torch.ones_like(flat))
    first = torch.cumsum(counts, 0) - counts
    place = torch.empty_like(flat)
    place[order] = torch.arange(T * k, device=flat.device)
    place = place - first[flat]
    rows = torch.zeros(n, most, H, device=x.device)
    rows[flat, place] = x.repeat_interleave(k, 0)
    pair = torch.stack((2 * used, 2 * used + 1), 1).flatten()
    gu = _decode(s["gu"][pair], s["sgu"][pair], I, H).view(n, 2 * I, H)
    z = torch.bmm(rows, gu.transpose(1, 2))
    gate, up = z[..., :I], z[..., I:]
    act = _rounded(gate / (1 + torch.exp(-gate)) * up)
    y = torch.bmm(act, _decode(s["dn"][used], s["sdn"][used], H, I).transpose(1, 2))
    y = (y[flat, place].view(T, k, H) * s["w"][..., None]).sum(1)
    return y.to(torch.bfloat16)


# ------------------------------------------------------------------- run ---

def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        if op == "route":
            return _plain_route(s)
        if op == "quantize":
            return _rounded(s["x"].float()).to(torch.bfloat16)
        if op == "product":
            a = _decode(s["a"], s["sa"], c["M"], c["K"])[0]
            b = _decode(s["b"], s["sb"], c["N"], c["K"])[0]
            return (a @ b.T).to(_DTYPES[c["out"]])
        return _plain_experts(s)
    import mixture_experts_layer_mm_gb300 as mm
    if op == "route":
        ids, w, counts, prob_sums, loss = mm.mm_route_logits(
            s["logits"], c["k"], c["renorm"], token_mask=s["mask"])
        out = {"ids": ids, "w": w, "counts": counts, "prob_sums": prob_sums, "loss": loss}
        if c["train"]:
            out["d_logits"] = mm.mm_route_logits_backward(
                s["logits"], ids, counts, c["renorm"], d_topk_w=s["d_topk_w"],
                d_loss=s["d_loss"], token_mask=s["mask"])
        return out
    if op == "quantize":
        codes, scales = mm.mm_mxfp4_quantize(s["x"])
        return mm.mm_mxfp4_dequantize(codes, scales, dtype=torch.bfloat16)
    if op == "product":
        return mm.mm_mxfp4_gemm(s["a"], s["sa"], s["b"], s["sb"], out_dtype=_DTYPES[c["out"]])
    return mm.mm_moe_experts_mxfp4(s["hidden"], s["ids"], s["w"], s["gu"], s["sgu"], s["dn"],
                                   s["sdn"])


# ----------------------------------------------------------------- exact ---

_LEVELS = np.array(_E2M1)


def _exact_values(codes, scales, rows, K):
    """float64 values of one stored matrix [rows, K]: codes [rows, K / 2], scales [tiles, ...]."""
    r = torch.arange(rows, device=codes.device)[:, None]
    c = torch.arange(K // 32, device=codes.device)[None, :]
    byte = scales[r // 128, c // 4, r % 32 * 16 + r % 128 // 32 * 4 + c % 4].double()
    v = torch.empty(rows, K, dtype=torch.float64, device=codes.device)
    level = torch.tensor(_LEVELS, device=codes.device)
    for half, nibble in enumerate((codes & 15, codes >> 4)):
        n = nibble.long()
        v[:, half::2] = level[n & 7] * (1 - 2 * (n >> 3)).double()
    return v * torch.exp2(byte - 127).repeat_interleave(32, 1)


def _exact_round(x):
    """float64 x [rows, K] to the nearest 4-bit values (ties to the even code) under the power of
    two that brings each block's largest magnitude into [4, 8)."""
    b = x.reshape(-1, 32)
    amax = b.abs().amax(1)
    unit = torch.exp2(torch.floor(torch.log2(amax.clamp_min(2.0 ** -125))) - 2)
    unit = torch.where(4 * unit > amax, unit / 2, unit)  # log2 rounded up
    unit = torch.where(8 * unit <= amax, unit * 2, unit)[:, None].clamp_min(2.0 ** -127)
    m = (b / unit).abs().clamp_max(6.0)
    # spacing of the e2m1 numbers around m: 1/2 below 2, 1 up to 4, 2 up to 6
    gap = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).double()
    q = torch.round(m / gap) * gap  # torch.round takes ties to even multiples
    return (torch.sign(b) * q * unit).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "product":
        a = _exact_values(s["a"][0], s["sa"][0], case["M"], case["K"])
        b = _exact_values(s["b"][0], s["sb"][0], case["N"], case["K"])
        return a @ b.T
    if op == "quantize":
        x = s["x"]
        return torch.stack([_exact_round(m.double()).to(torch.bfloat16) for m in x])
    if op == "route":
        x = s["logits"].double()
        T, E, k = case["T"], case["E"], case["k"]
        keep = torch.ones(T, dtype=torch.bool, device=x.device) if s["mask"] is None else s["mask"]
        p = torch.softmax(x, -1)
        # rank of each expert: how many are larger, or equal with a lower id
        ids = torch.argsort(x, dim=-1, descending=True, stable=True)[:, :k].sort(-1)[0]
        sel = torch.zeros(T, E, dtype=torch.bool, device=x.device).scatter_(1, ids, True)
        w = p.gather(1, ids)
        if case["renorm"]:
            w = w / w.sum(-1, keepdim=True)
        w[~keep] = 0
        n = max(1, int(keep.sum()))
        counts = (sel & keep[:, None]).sum(0)
        mean = p[keep].sum(0) / n
        frac = counts.double() / (n * k)
        out = {"ids": ids.to(torch.int32), "w": w, "counts": counts.to(torch.int32),
               "prob_sums": p[keep].sum(0), "loss": (E * (frac * mean).sum()).reshape(1)}
        if case["train"]:
            leaf = x.clone().requires_grad_(True)
            q = torch.softmax(leaf, -1)
            v = q.gather(1, ids)
            if case["renorm"]:
                v = v / v.sum(-1, keepdim=True)
            total = (v[keep] * s["d_topk_w"][keep].double()).sum()
            total = total + s["d_loss"].double() * E * (frac * (q[keep].sum(0) / n)).sum()
            out["d_logits"] = torch.autograd.grad(total, leaf)[0]
        return out
    T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
    x = _exact_round(s["hidden"].double())
    y = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    for e in range(E):
        t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        if t.numel() == 0:
            continue
        gate = x[t] @ _exact_values(s["gu"][2 * e], s["sgu"][2 * e], I, H).T
        up = x[t] @ _exact_values(s["gu"][2 * e + 1], s["sgu"][2 * e + 1], I, H).T
        act = _exact_round(gate * torch.sigmoid(gate) * up)
        y.index_add_(0, t, s["w"][t, j].double()[:, None]
                     * (act @ _exact_values(s["dn"][e], s["sdn"][e], H, I).T))
    return y
