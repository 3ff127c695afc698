"""Operators of a block-128 FP8 linear layer with the norm in front of it, and the cases they are timed on.

Four operators:
  quantize   bf16 -> FP8 codes with one fp32 scale for each block of 128 (block_quantize, block_quantize_dual)
  gemm       the product of two such operands, scales applied block by block (block_gemm)
  norm       layer norm / RMS norm, to bf16 or straight to the quantized operand of the next
             product (layer_norm, layer_norm_quantize)
  norm_bwd   its backward pass, with the reductions of the weight's and the bias's gradients
             (layer_norm_backward)

Definitions, with BLK = 128, FMAX = 448 (E4M3) or 57344 (E5M2):
  a block is 128 neighbouring elements of one row along the product's reduction dimension ("row"
  of the matrix, or of its transpose), or a 128 x 128 tile; the last block of a row may be shorter.
    amax  = max(largest |v| of the block, 2^-100)
    scale = amax / FMAX, code = FP8(clamp(v * (FMAX / amax), -FMAX, FMAX)), nearest, ties to even
  scales are stored with the reduction dimension's blocks outermost: scales[block][row]
  (tiles: scales[block][row of tiles]).
    C[m, n] = sum_b sa[b][m] * sb[b][n or tile of n] * sum_{k in b} A[m, k] B[n, k]
    y = (x - mean) * rstd * weight + bias, rstd = 1 / sqrt(mean((x - mean)^2) + eps); the RMS form
    has mean = 0.
    xh = (x - mean) * rstd, g = dy * weight: dx = rstd * (g - mean(g) - xh * mean(g * xh)) (RMS: without
    mean(g)), dweight = sum_rows dy * xh, dbias = sum_rows dy.

Where `own` is true, run() calls the library; otherwise it computes the plain form in torch.
"""
import torch

own = False

BLK = 128
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FLOOR = 2.0 ** -100


def _cdiv(a, b):
    return -(-a // b)


def listed():
    return [
        # one new token through the QKV projection of an 8B model: latency, bound by the weight's bytes
        {"name": "gemm_token_qkv", "op": "gemm", "M": 1, "N": 6144, "K": 4096, "fa": "e4m3", "fb": "e4m3",
         "tile_b": True, "out": "bf16"},
        # a serving batch of 48 tokens through the MLP's down projection: few rows, a long reduction
        {"name": "gemm_batch_down", "op": "gemm", "M": 48, "N": 4096, "K": 14336, "fa": "e4m3", "fb": "e4m3",
         "tile_b": True, "out": "bf16"},
        # training, forward: 8192 tokens through the QKV projection
        {"name": "gemm_fprop_qkv", "op": "gemm", "M": 8192, "N": 6144, "K": 4096, "fa": "e4m3", "fb": "e4m3",
         "tile_b": True, "out": "bf16"},
        # training, activation gradient of the gate and up projections for a ragged 1000 tokens, E5M2 gradients
        {"name": "gemm_dgrad_ragged", "op": "gemm", "M": 1000, "N": 4096, "K": 28672, "fa": "e5m2", "fb": "e4m3",
         "tile_b": True, "out": "bf16"},
        # training, weight gradient of the QKV projection: both operands scaled along tokens, fp32 out
        {"name": "gemm_wgrad_qkv", "op": "gemm", "M": 6144, "N": 4096, "K": 8192, "fa": "e5m2", "fb": "e4m3",
         "tile_b": False, "out": "f32"},
        # activations of 8192 tokens, one form only (forward without a backward pass)
        {"name": "quantize_row_x", "op": "quantize", "rows": 8192, "cols": 4096, "fmt": "e4m3", "form": "row"},
        # the output gradient of a ragged 1000 tokens in both forms of the backward pass
        {"name": "quantize_dual_dy", "op": "quantize", "rows": 1000, "cols": 6144, "fmt": "e5m2", "form": "dual"},
        # the gate and up weight after an optimizer step, in both forms, 128 x 128 tiles
        {"name": "quantize_tile_w", "op": "quantize", "rows": 28672, "cols": 4096, "fmt": "e4m3", "form": "tile_dual"},
        # one new token's norm in front of the QKV projection (RMS, as the 8B configuration has it)
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 4096, "rms": True, "to": "block"},
        # training: 8192 tokens' layer norm written as the next product's operand
        {"name": "norm_train", "op": "norm", "rows": 8192, "cols": 4096, "rms": False, "to": "block"},
        # its backward pass
        {"name": "norm_bwd_train", "op": "norm_bwd", "rows": 8192, "cols": 4096, "rms": False},
        # RMS, a ragged number of tokens of the 70B configuration's width
        {"name": "norm_bwd_ragged", "op": "norm_bwd", "rows": 1001, "cols": 8192, "rms": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def _some(rng, lo, hi, steps):
    """A size of [lo, hi], even over its logarithm, rounded to one of `steps`."""
    s = rng.choice(steps)
    return max(lo, min(hi, _cdiv(_log(rng, lo, hi), s) * s))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "quantize", "norm", "norm_bwd"])
    if op == "gemm":
        while True:
            c = {"op": op, "M": _log(rng, 1, 8192), "N": _some(rng, 128, 8192, (1, 16, 128)),
                 "K": _some(rng, 64, 28672, (1, 16, 128, 128)), "fa": rng.choice(["e4m3", "e5m2"]), "fb": "e4m3",
                 "tile_b": rng.random() < 0.7, "out": rng.choice(["bf16", "bf16", "f32"])}
            if c["M"] * c["N"] * c["K"] <= 6144 * 4096 * 8192:
                return c
    if op == "quantize":
        return {"op": op, "rows": _some(rng, 1, 16384, (1, 1, 128)), "cols": _some(rng, 128, 7168, (1, 16, 128)),
                "fmt": rng.choice(["e4m3", "e5m2"]), "form": rng.choice(["row", "transpose", "dual", "tile", "tile_dual"])}
    if op == "norm":
        return {"op": op, "rows": _log(rng, 1, 8192), "cols": _some(rng, 128, 4096, (1, 16, 128)),
                "rms": rng.random() < 0.5, "to": rng.choice(["bf16", "block"])}
    return {"op": op, "rows": _log(rng, 1, 8192), "cols": _some(rng, 128, 4096, (1, 16, 128)), "rms": rng.random() < 0.5}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _act(g, rows, cols):
    """activations: normal, a few channels 50 times as large"""
    x = torch.randn(rows, cols, device="cuda", generator=g)
    x[:, torch.randint(cols, (max(1, cols // 1000),), device="cuda", generator=g)] *= 50.0
    return x.bfloat16()


def _grad(g, rows, cols):
    """gradients: small, heavy-tailed"""
    x = torch.randn(rows, cols, device="cuda", generator=g)
    return (1e-3 * x * torch.rand(rows, cols, device="cuda", generator=g).add_(0.05).reciprocal_().sqrt_()).bfloat16()


def _weight(g, rows, cols):
    return (0.02 * torch.randn(rows, cols, device="cuda", generator=g)).bfloat16()


def _operand(x, fmt, tile):
    """codes in a buffer of rows padded to 16 bytes, as the quantizer lays them out, and scales"""
    codes, scales = _quantize(x, fmt, tile)
    rows, k = x.shape
    buf = torch.zeros(rows, _cdiv(k, 16) * 16, dtype=torch.uint8, device=x.device)
    buf[:, :k] = codes
    return buf[:, :k], scales


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        a = (_grad if case["fa"] == "e5m2" else _act)(g, M, K)
        b = (_weight if case["tile_b"] else _act)(g, N, K)
        return {"case": case, "a": _operand(a, case["fa"], False), "b": _operand(b, case["fb"], case["tile_b"])}
    rows, cols = case["rows"], case["cols"]
    if op == "quantize":
        make = _weight if case["form"].startswith("tile") else _grad if case["fmt"] == "e5m2" else _act
        return {"case": case, "x": make(g, rows, cols)}
    s = {"case": case, "x": _act(g, rows, cols), "weight": (1 + 0.1 * torch.randn(cols, device="cuda", generator=g)).bfloat16(),
         "bias": None if case["rms"] else (0.1 * torch.randn(cols, device="cuda", generator=g)).bfloat16(), "eps": 1e-5}
    if op == "norm_bwd":
        s["dy"] = _grad(g, rows, cols)
        s["mean"], s["rstd"] = _statistics(s["x"].float(), case["rms"], s["eps"])
    return s


# ---- plain forms, in 32 bits ----

def _blocks(x):
    """[rows, K] -> [rows, blocks, 128], padded with zeros"""
    rows, k = x.shape
    return torch.nn.functional.pad(x, (0, _cdiv(k, BLK) * BLK - k)).view(rows, _cdiv(k, BLK), BLK)


def _quantize(x, fmt, tile):
    """(codes [rows, K] as bytes, scales [blocks, rows] or [blocks, tiles of rows])"""
    x = x.float()
    rows, k = x.shape
    xb = _blocks(x)
    amax = xb.abs().amax(2)
    if tile:
        nt = _cdiv(rows, BLK)
        amax = torch.nn.functional.pad(amax, (0, 0, 0, nt * BLK - rows)).view(nt, BLK, -1).amax(1)
    amax = amax.clamp(min=FLOOR)
    scales, inv = amax / FMAX[fmt], FMAX[fmt] / amax
    if tile:
        inv = inv.repeat_interleave(BLK, 0)[:rows]
    q = (xb * inv[:, :, None]).view(rows, -1)[:, :k].clamp(-FMAX[fmt], FMAX[fmt]).to(F8[fmt])
    return q.view(torch.uint8), scales.t().contiguous()


def _values(codes, scales, fmt):
    """[rows, K] in 32 bits"""
    rows, k = codes.shape
    s = scales.t()
    if s.shape[0] != rows:
        s = s.repeat_interleave(BLK, 0)[:rows]
    return codes.contiguous().view(F8[fmt]).float() * s.repeat_interleave(BLK, 1)[:, :k]


def _statistics(x, rms, eps):
    mean = None if rms else x.mean(1)
    d = x if rms else x - mean[:, None]
    return mean, (d.square().mean(1) + eps).rsqrt()


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "gemm":
        a = _values(*s["a"], case["fa"])
        b = _values(*s["b"], case["fb"])
        c = a @ b.t()
        return c if case["out"] == "f32" else c.bfloat16()
    if op == "quantize":
        form, fmt, tile, out = case["form"], case["fmt"], case["form"].startswith("tile"), []
        if form != "transpose":
            out += list(_quantize(s["x"], fmt, tile))
        if form in ("transpose", "dual", "tile_dual"):
            out += list(_quantize(s["x"].t().contiguous(), fmt, tile))
        return [t.contiguous().view(F8[fmt]) if t.dtype == torch.uint8 else t for t in out]
    x, w = s["x"].float(), s["weight"].float()
    if op == "norm":
        mean, rstd = _statistics(x, case["rms"], s["eps"])
        y = (x if mean is None else x - mean[:, None]) * rstd[:, None] * w
        y = y if s["bias"] is None else y + s["bias"].float()
        if case["to"] == "bf16":
            out = [y.bfloat16()]
        else:
            codes, scales = _quantize(y, "e4m3", False)
            out = [codes.contiguous().view(F8["e4m3"]), scales]
        return out + ([rstd] if mean is None else [mean, rstd])
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (x if case["rms"] else x - s["mean"][:, None]) * rstd
    g = dy * w
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    if not case["rms"]:
        dx = dx - g.mean(1, keepdim=True)
    out = [(dx * rstd).bfloat16(), (dy * xh).sum(0)]
    return out if case["rms"] else out + [dy.sum(0)]


# ---- the library's calls ----

def _run_own(s):
    import precision_block_amax_amd as mx
    case, op = s["case"], s["case"]["op"]
    if op == "gemm":
        return mx.block_gemm(*s["a"], case["fa"], *s["b"], case["fb"],
                             out_dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16)
    if op == "quantize":
        form, fmt = case["form"], case["fmt"]
        if form in ("dual", "tile_dual"):
            out = mx.block_quantize_dual(s["x"], fmt, fmt, tile=form == "tile_dual")
        else:
            out = mx.block_quantize(s["x"], fmt, mode=form)
        return [t.view(F8[fmt]) if t.dtype == torch.uint8 else t for t in out]
    if op == "norm":
        if case["to"] == "bf16":
            y, mean, rstd = mx.layer_norm(s["x"], s["weight"], s["bias"], eps=s["eps"], rms=case["rms"])
            out = [y]
        else:
            codes, scales, mean, rstd = mx.layer_norm_quantize(s["x"], s["weight"], s["bias"], "e4m3", eps=s["eps"],
                                                               rms=case["rms"])
            out = [codes.view(F8["e4m3"]), scales]
        return out + ([rstd] if mean is None else [mean, rstd])
    dx, dw, db = mx.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], rms=case["rms"],
                                        bias_grad=not case["rms"])
    return [dx, dw] if case["rms"] else [dx, dw, db]


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op = case["op"]
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        kb = _cdiv(K, BLK)
        scales = 4 * kb * (M + (_cdiv(N, BLK) if case["tile_b"] else N))
        return {"bytes": M * K + N * K + scales + M * N * (4 if case["out"] == "f32" else 2), "flops": 2 * M * N * K}
    rows, cols = case["rows"], case["cols"]
    n, rb, cb = rows * cols, _cdiv(rows, BLK), _cdiv(cols, BLK)
    if op == "quantize":
        form, b, f = case["form"], 2 * n, 0
        if form != "transpose":
            b, f = b + n + 4 * cb * (rb if form.startswith("tile") else rows), f + 3 * n
        if form in ("transpose", "dual", "tile_dual"):
            b, f = b + n + 4 * rb * (cb if form.startswith("tile") else cols), f + 3 * n
        return {"bytes": b, "flops": f}
    params = 2 * cols * (1 if case["rms"] else 2)
    stats = 4 * rows * (1 if case["rms"] else 2)
    if op == "norm":
        return {"bytes": 2 * n + params + stats + (2 * n if case["to"] == "bf16" else n + 4 * cb * rows), "flops": 8 * n}
    return {"bytes": 6 * n + 2 * cols + stats + 4 * cols * (1 if case["rms"] else 2), "flops": 12 * n}


# ---- the definitions in 64 bits ----

def _exact_scale(v, fmt, tile):
    """v (float64 [rows, K]) -> (v / scale, scales), without the rounding to 8 bits"""
    rows, k = v.shape
    inv, scales = torch.empty_like(v), []
    for k0 in range(0, k, BLK):
        m = v[:, k0:k0 + BLK].abs().max(dim=1).values
        if tile:
            m = torch.stack([t.max() for t in m.split(BLK)])
        m = torch.maximum(m, torch.full_like(m, FLOOR))
        scales.append(m / FMAX[fmt])
        per_row = torch.cat([t.expand(min(BLK, rows - BLK * i)) for i, t in enumerate(scales[-1].unbind())]) if tile else scales[-1]
        inv[:, k0:k0 + BLK] = v[:, k0:k0 + BLK] / per_row[:, None]
    return inv, torch.stack(scales)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        (ca, sa), (cb, sb) = s["a"], s["b"]
        N, K = case["N"], case["K"]
        per = torch.arange(N, device="cuda") // BLK if case["tile_b"] else torch.arange(N, device="cuda")
        c = torch.zeros(case["M"], N, dtype=torch.float64, device="cuda")
        step = 8 * BLK  # scales multiplied into each side, a few blocks at a time
        for k0 in range(0, K, step):
            kb = torch.arange(k0, min(K, k0 + step), device="cuda") // BLK
            a = ca[:, k0:k0 + step].contiguous().view(F8[case["fa"]]).double() * sa.double()[kb].t()
            b = cb[:, k0:k0 + step].contiguous().view(F8[case["fb"]]).double() * sb.double()[kb][:, per].t()
            c += torch.mm(a, b.t())
        return c
    x = s["x"].double()
    if op == "quantize":
        form, tile, out = case["form"], case["form"].startswith("tile"), []
        if form != "transpose":
            out += _exact_scale(x, case["fmt"], tile)
        if form in ("transpose", "dual", "tile_dual"):
            out += _exact_scale(x.t().contiguous(), case["fmt"], tile)
        return out
    w, n = s["weight"].double(), case["cols"]
    if op == "norm":
        mean = torch.zeros(case["rows"], dtype=torch.float64, device="cuda") if case["rms"] else x.sum(1) / n
        x = x - mean[:, None]
        rstd = 1.0 / torch.sqrt((x * x).sum(1) / n + s["eps"])
        y = x * rstd[:, None] * w[None, :]
        if s["bias"] is not None:
            y = y + s["bias"].double()[None, :]
        out = [y] if case["to"] == "bf16" else list(_exact_scale(y, "e4m3", False))
        return out + ([rstd] if case["rms"] else [mean, rstd])
    dy, rstd = s["dy"].double(), s["rstd"].double()
    xh = (x if case["rms"] else x - s["mean"].double()[:, None]) * rstd[:, None]
    g = dy * w[None, :]
    inner = g - xh * ((g * xh).sum(1) / n)[:, None]
    if not case["rms"]:
        inner = inner - (g.sum(1) / n)[:, None]
    out = [inner * rstd[:, None], (dy * xh).sum(0)]
    return out if case["rms"] else out + [dy.sum(0)]
