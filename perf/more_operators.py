"""Operators of a layer with experts and normalised queries and keys, and the cases they are timed on.

Five operators:
  grouped    the product of block-128 FP8 rows, sorted by expert, with their experts' weights (block_gemm_grouped)
  grouped_k  the experts' weight gradients: a product for each group of tokens, tokens as the reduction
             dimension (block_gemm_grouped_k)
  quantize   bf16 -> FP8 codes with blocks of 128 tokens that start anew at every group, written transposed, alone or
             beside the row form (block_quantize_grouped, block_quantize_grouped_dual)
  rope       rotary positions of queries and keys; its inverse is its backward pass (rope)
  qk_norm    RMS norm of each head of queries and keys and the rotation in one pass, forward and backward
             (qk_norm_rope, qk_norm_rope_backward)

Definitions, with BLK = 128, FMAX = 448 (E4M3) or 57344 (E5M2):
  group g is the rows ends[g - 1] .. ends[g] - 1 (0 before the first); rows from the last end on belong to none.
    block of 128 elements:  amax = max(largest |v|, 2^-100), scale = amax / FMAX, code = FP8(v * (FMAX / amax))
  grouped:    C[t, n] = sum_b sa[b][t] * sb[g][b][n's tile] * sum_{k in b} A[t, k] B[g, n, k] for t in g
  transposed form: the tokens of a group become columns from 128 * (blocks of the groups before it) on, the last block
    of a group filled with zeros; scales[block][row].  What lies behind the last group's blocks stays as it was.
  grouped_k:  C[g, m, n] = sum over the blocks b of g of sa[b][m] * sb[b][n] * sum_{k in b} A[m, k] B[n, k]
  rope: pair i of the first 2 F elements of a head, F frequencies: (a, b) = (x_i, x_{i + F}) (half) or
    (x_2i, x_2i+1) (interleaved); with angle p * freq_i at position p and c, s its cosine and sine times `scale`:
    (a c - b s, b c + a s), inverse (a c + b s, b c - a s); the head's other elements stay
  qk_norm: xh = x * rstd, rstd = 1 / sqrt(mean(x^2) + eps) over a head; y = rope(xh * weight).
    With u = rope_inverse(dy): dweight = sum over tokens and heads of u * xh, g = u * weight,
    dx = rstd * (g - xh * mean(g * xh))

Where `own` is true, run() calls the library; otherwise it computes the plain form in torch.
"""
import math

import torch

own = False

BLK = 128
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FLOOR = 2.0 ** -100
EPS = 1e-6


def _cdiv(a, b):
    return -(-a // b)


def listed():
    return [
        # one new token, 8 of 128 experts, gate and up projections: latency, bound by the chosen weights' bytes
        {"name": "grouped_token", "op": "grouped", "rows": 8, "pad": 0, "groups": 128, "N": 1536, "K": 2048, "fa": "e4m3",
         "out": "bf16"},
        # training, forward: 8192 tokens, 2 of 8 experts each, gate and up projections of an 8B model's MLP
        {"name": "grouped_fprop", "op": "grouped", "rows": 16384, "pad": 0, "groups": 8, "N": 28672, "K": 4096, "fa": "e4m3",
         "out": "bf16"},
        # training, activation gradient: 1000 tokens, 8 of 128 experts, E5M2 gradients, in a buffer with rows to spare
        {"name": "grouped_dgrad_ragged", "op": "grouped", "rows": 8000, "pad": 192, "groups": 128, "N": 2048, "K": 1536,
         "fa": "e5m2", "out": "bf16"},
        # training, weight gradient of the down projections of 8 experts
        {"name": "grouped_wgrad", "op": "grouped_k", "rows": 16384, "groups": 8, "M": 4096, "N": 14336, "fa": "e5m2",
         "out": "f32"},
        # the same of 128 small experts with few tokens each: bound by writing the gradients
        {"name": "grouped_wgrad_ragged", "op": "grouped_k", "rows": 8000, "groups": 128, "M": 1536, "N": 2048, "fa": "e5m2",
         "out": "f32"},
        # activations sorted by expert, as the weight gradient's right operand
        {"name": "quantize_x", "op": "quantize", "rows": 16384, "cols": 4096, "groups": 8, "fmt": "e4m3", "dual": False},
        # the output gradient of 1000 tokens' 8 choices of 128 experts, in both forms of the backward pass
        {"name": "quantize_dual_dy", "op": "quantize", "rows": 8000, "cols": 1536, "groups": 128, "fmt": "e5m2", "dual": True},
        # one new token at a far position, heads of an 8B model: latency
        {"name": "rope_token", "op": "rope", "tokens": 1, "q_heads": 32, "k_heads": 8, "dim": 128, "rot": 128,
         "layout": "half", "scaling": "bands", "inverse": False, "from": 131000},
        # training at 8192 tokens, heads of a 70B model, the gradient's way back, interleaved pairs
        {"name": "rope_backward", "op": "rope", "tokens": 8192, "q_heads": 64, "k_heads": 8, "dim": 128, "rot": 128,
         "layout": "interleaved", "scaling": "bands", "inverse": True, "from": 0},
        # a serving batch of 48 new tokens
        {"name": "qk_norm_batch", "op": "qk_norm", "tokens": 48, "q_heads": 32, "k_heads": 4, "dim": 128, "rot": 128,
         "layout": "half", "scaling": "none", "backward": False, "from": 30000},
        # training, forward and backward, heads of an 8B model
        {"name": "qk_norm_train", "op": "qk_norm", "tokens": 8192, "q_heads": 32, "k_heads": 8, "dim": 128, "rot": 128,
         "layout": "half", "scaling": "none", "backward": False, "from": 0},
        {"name": "qk_norm_backward", "op": "qk_norm", "tokens": 8192, "q_heads": 32, "k_heads": 8, "dim": 128, "rot": 128,
         "layout": "half", "scaling": "none", "backward": True, "from": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def _some(rng, lo, hi, steps):
    """A size of [lo, hi], even over its logarithm, rounded to one of `steps`."""
    s = rng.choice(steps)
    return max(lo, min(hi, _cdiv(_log(rng, lo, hi), s) * s))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "grouped_k", "quantize", "rope", "qk_norm", "qk_norm"])
    if op == "grouped":
        while True:
            c = {"op": op, "rows": _log(rng, 1, 16384), "pad": rng.choice([0, 0, 1, 77]), "groups": _log(rng, 1, 128),
                 "N": _some(rng, 128, 28672, (1, 16, 128, 128)), "K": _some(rng, 64, 14336, (1, 16, 128, 128)),
                 "fa": rng.choice(["e4m3", "e5m2"]), "out": rng.choice(["bf16", "bf16", "f32"])}
            if c["groups"] * c["N"] * c["K"] <= 2 ** 29 and c["rows"] * c["N"] * c["K"] <= 2 ** 39:
                return c
    if op == "grouped_k":
        while True:
            c = {"op": op, "rows": _log(rng, 1, 16384), "groups": _log(rng, 1, 128), "M": _some(rng, 64, 8192, (1, 16, 128)),
                 "N": _some(rng, 64, 8192, (1, 16, 128)), "fa": rng.choice(["e4m3", "e5m2"]),
                 "out": rng.choice(["f32", "f32", "bf16"])}
            if c["groups"] * c["M"] * c["N"] <= 2 ** 28 and c["rows"] * c["M"] * c["N"] <= 2 ** 39:
                return c
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 16384), "cols": _some(rng, 128, 4096, (1, 16, 128)), "groups": _log(rng, 1, 128),
                "fmt": rng.choice(["e4m3", "e5m2"]), "dual": rng.random() < 0.5}
    dim = rng.choice([64, 128, 128, 128, 256, 80, 96, 40])
    c = {"op": op, "tokens": _log(rng, 1, 8192), "q_heads": rng.choice([1, 6, 16, 32, 32]), "k_heads": rng.choice([1, 2, 8, 8]),
         "dim": dim, "rot": rng.choice([dim, dim, dim // 2, dim // 4]), "layout": rng.choice(["half", "interleaved"]),
         "scaling": rng.choice(["none", "linear", "bands"]), "from": rng.choice([0, 0, 5000, 500000])}
    c["rot"] -= c["rot"] % 2
    c["inverse" if op == "rope" else "backward"] = rng.random() < 0.5
    while c["tokens"] * (c["q_heads"] + c["k_heads"]) * dim > 8192 * 40 * 128:
        c["tokens"] //= 2
    return c


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


def _popularity(groups):
    """what share of the rows an expert gets: the last of many gets a tenth of what the first gets"""
    p = torch.tensor([1.0 / (1.0 + 9.0 * i / max(1, groups - 1)) for i in range(groups)], dtype=torch.float64)
    return p / p.sum()


def _route(rows, groups, seed):
    """rows dealt out to groups: their ends, as numbers"""
    g = torch.Generator().manual_seed(int(seed) + 1)
    p = _popularity(groups)[torch.randperm(groups, generator=g)]
    picks = torch.multinomial(p, rows, replacement=True, generator=g)
    return torch.bincount(picks, minlength=groups).cumsum(0).tolist()


def _padded(ends):
    """first and last block of every group, in the transposed form"""
    out, b, at = [], 0, 0
    for e in ends:
        out.append((b, b + _cdiv(e - at, BLK)))
        b, at = out[-1][1], e
    return out


def _pitched(codes):
    """rows padded to 16 bytes, as the quantizers lay them out"""
    k = codes.shape[-1]
    buf = torch.zeros(*codes.shape[:-1], _cdiv(k, 16) * 16, dtype=torch.uint8, device=codes.device)
    buf[..., :k] = codes
    return buf[..., :k]


def _weights(g, groups, n, k):
    """stacked weights in 128 x 128 tiles: codes [groups, n, k], scales [groups, blocks of k, tiles of n]"""
    codes = torch.empty(groups, n, _cdiv(k, 16) * 16, dtype=torch.uint8, device="cuda")[:, :, :k]
    scales = torch.empty(groups, _cdiv(k, BLK), _cdiv(n, BLK), device="cuda")
    for i in range(groups):
        codes[i], scales[i] = _quantize(0.02 * torch.randn(n, k, device="cuda", generator=g), "e4m3", True)
    return codes, scales


def _frequencies(rot, scaling):
    """radians per position for each pair, in 64 bits, and the factor of the cosines and sines"""
    theta = 500000.0 if scaling == "bands" else 10000.0
    f = [theta ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        f = [v / 4.0 for v in f]
    if scaling == "bands":  # long wavelengths slowed down 8 times, short ones kept, those between in proportion
        for i, v in enumerate(f):
            turns = 8192.0 * v / (2.0 * math.pi)
            keep = min(1.0, max(0.0, (turns - 1.0) / (4.0 - 1.0)))
            f[i] = v * keep + v / 8.0 * (1.0 - keep)
    return torch.tensor(f, dtype=torch.float64, device="cuda")


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op in ("grouped", "grouped_k", "quantize"):
        s["ends"] = _route(case["rows"], case["groups"], seed)
        s["ends_gpu"] = torch.tensor(s["ends"], dtype=torch.int32, device="cuda")
    if op == "grouped":
        make = _grad if case["fa"] == "e5m2" else _act
        codes, scales = _quantize(make(g, case["rows"] + case["pad"], case["K"]), case["fa"], False)
        s["a"] = (_pitched(codes), scales)
        s["b"] = _weights(g, case["groups"], case["N"], case["K"])
    elif op == "grouped_k":
        dy = (_grad if case["fa"] == "e5m2" else _act)(g, case["rows"], case["M"])
        s["a"] = _quantize_grouped(dy, case["fa"], s["ends"])
        s["b"] = _quantize_grouped(_act(g, case["rows"], case["N"]), "e4m3", s["ends"])
    elif op == "quantize":
        s["x"] = (_grad if case["fmt"] == "e5m2" else _act)(g, case["rows"], case["cols"])
        # buffers that a training program keeps: the transposed form has room for any groups
        cols, blocks = case["cols"], _bound(case["rows"], case["groups"])
        s["out"] = [torch.zeros(cols, blocks * BLK, dtype=torch.uint8, device="cuda"), torch.zeros(blocks, cols, device="cuda")]
        if case["dual"]:
            codes = torch.zeros(case["rows"], _cdiv(cols, 16) * 16, dtype=torch.uint8, device="cuda")[:, :cols]
            s["out"] = [codes, torch.zeros(_cdiv(cols, BLK), case["rows"], device="cuda")] + s["out"]
    else:
        t, hq, hk, d = case["tokens"], case["q_heads"], case["k_heads"], case["dim"]
        make = _grad if op == "rope" and case["inverse"] else _act
        # queries, keys and values as the QKV product leaves them
        qkv = make(g, t, (hq + 2 * hk) * d).view(t, hq + 2 * hk, d)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        s["positions"] = case["from"] + torch.arange(t, device="cuda")
        s["freqs"] = _frequencies(case["rot"], case["scaling"])
        if op == "qk_norm":
            s["qw"], s["kw"] = ((1 + 0.1 * torch.randn(d, device="cuda", generator=g)).bfloat16() for _ in range(2))
            if case["backward"]:
                s["dq"], s["dk"] = _grad(g, t, hq * d).view(t, hq, d), _grad(g, t, hk * d).view(t, hk, d)
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


def _bound(rows, groups):
    """the most blocks that the rows can take, whatever their groups"""
    return (rows + (BLK - 1) * min(rows, groups)) // BLK


def _spread(x, ends):
    """[rows, cols] -> [cols, 128 * blocks], every group from a block of its own on"""
    at = _padded(ends)
    out = torch.zeros(x.shape[1], at[-1][1] * BLK, dtype=x.dtype, device=x.device)
    for (b, _), lo, hi in zip(at, [0] + ends[:-1], ends):
        out[:, b * BLK:b * BLK + hi - lo] = x[lo:hi].t()
    return out


def _quantize_grouped(x, fmt, ends):
    return _quantize(_spread(x, ends), fmt, False)


def _values(codes, scales, fmt):
    """[rows, K] in 32 bits"""
    rows, k = codes.shape
    s = scales.t()
    if s.shape[0] != rows:
        s = s.repeat_interleave(BLK, 0)[:rows]
    return codes.contiguous().view(F8[fmt]).float() * s.repeat_interleave(BLK, 1)[:, :k]


def _angles(s, dtype):
    a = s["positions"].double()[:, None] * s["freqs"]
    return a.cos().to(dtype)[:, None], a.sin().to(dtype)[:, None]


def _rotate(x, cos, sin, layout, inverse):
    f = cos.shape[-1]
    sin = -sin if inverse else sin
    a, b = (x[..., :f], x[..., f:2 * f]) if layout == "half" else (x[..., 0:2 * f:2], x[..., 1:2 * f:2])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.cat([u, v], -1) if layout == "half" else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([r, x[..., 2 * f:]], -1)


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "grouped":
        (ca, sa), (cb, sb) = s["a"], s["b"]
        a = _values(ca, sa, case["fa"])
        c = torch.empty(case["rows"], case["N"], device="cuda")
        for i, (lo, hi) in enumerate(zip([0] + s["ends"][:-1], s["ends"])):
            if hi > lo:
                torch.mm(a[lo:hi], _values(cb[i], sb[i], "e4m3").t(), out=c[lo:hi])
        return c if case["out"] == "f32" else c.bfloat16()
    if op == "grouped_k":
        a, b = _values(*s["a"], case["fa"]), _values(*s["b"], "e4m3")
        c = torch.empty(case["groups"], case["M"], case["N"], device="cuda")
        for i, (lo, hi) in enumerate(_padded(s["ends"])):
            torch.mm(a[:, lo * BLK:hi * BLK], b[:, lo * BLK:hi * BLK].t(), out=c[i])
        return c if case["out"] == "f32" else c.bfloat16()
    if op == "quantize":
        fmt = case["fmt"]
        out = list(_quantize(s["x"], fmt, False)) if case["dual"] else []
        codes, scales = _quantize_grouped(s["x"], fmt, s["ends"])
        left = _bound(case["rows"], case["groups"]) - scales.shape[0]
        pad = torch.nn.functional.pad
        out += [pad(codes, (0, left * BLK)), pad(scales, (0, 0, 0, left))]
        return [t.contiguous().view(F8[fmt]) if t.dtype == torch.uint8 else t for t in out]
    cos, sin = _angles(s, torch.float32)
    if op == "rope":
        return [_rotate(x.float(), cos, sin, case["layout"], case["inverse"]).bfloat16() for x in (s["q"], s["k"])]
    out, grads = [], []
    for x, w, dy in ((s["q"], s["qw"], s.get("dq")), (s["k"], s["kw"], s.get("dk"))):
        x, w = x.float(), w.float()
        rstd = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
        xh = x * rstd
        if dy is None:
            out.append(_rotate(xh * w, cos, sin, case["layout"], False).bfloat16())
            continue
        u = _rotate(dy.float(), cos, sin, case["layout"], True)
        g = u * w
        out.append((rstd * (g - xh * (g * xh).mean(-1, keepdim=True))).bfloat16())
        grads.append((u * xh).sum((0, 1)))
    return out + grads


# ---- the library's calls ----

def _run_own(s):
    import precision_block_amax_amd as mx
    case, op = s["case"], s["case"]["op"]
    if op in ("grouped", "grouped_k"):
        out = torch.float32 if case["out"] == "f32" else torch.bfloat16
        call = mx.block_gemm_grouped if op == "grouped" else mx.block_gemm_grouped_k
        c = call(*s["a"], case["fa"], *s["b"], "e4m3", s["ends_gpu"], out_dtype=out)
        return c[:case["rows"]] if op == "grouped" else c
    if op == "quantize":
        fmt = case["fmt"]
        if case["dual"]:
            out = mx.block_quantize_grouped_dual(s["x"], s["ends_gpu"], fmt, fmt, out=s["out"])
        else:
            out = mx.block_quantize_grouped(s["x"], s["ends_gpu"], fmt, out=s["out"])
        return [t.view(F8[fmt]) if t.dtype == torch.uint8 else t for t in out]
    if op == "rope":
        return mx.rope(s["q"], s["k"], s["positions"], s["freqs"], layout=case["layout"], inverse=case["inverse"])
    args = (s["q"], s["k"], s["qw"], s["kw"], s["positions"], s["freqs"])
    if not case["backward"]:
        return mx.qk_norm_rope(*args, eps=EPS, layout=case["layout"])
    return mx.qk_norm_rope_backward(s["dq"], s["dk"], *args, eps=EPS, layout=case["layout"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op = case["op"]
    if op == "grouped":
        T, N, K, G = case["rows"], case["N"], case["K"], case["groups"]
        # groups that get at least one row, on average
        met = float((1 - (1 - _popularity(G)).pow(T)).sum())
        b = T * K + 4 * T * _cdiv(K, BLK) + met * (N * K + 4 * _cdiv(N, BLK) * _cdiv(K, BLK))
        return {"bytes": int(b) + T * N * (4 if case["out"] == "f32" else 2), "flops": 2 * T * N * K}
    if op == "grouped_k":
        T, M, N, G = case["rows"], case["M"], case["N"], case["groups"]
        b = (M + N) * (T + 4 * _cdiv(T, BLK)) + G * M * N * (4 if case["out"] == "f32" else 2)
        return {"bytes": b, "flops": 2 * M * N * T}
    if op == "quantize":
        rows, cols = case["rows"], case["cols"]
        n = rows * cols
        b, f = 3 * n + 4 * _cdiv(rows, BLK) * cols, 3 * n
        if case["dual"]:
            b, f = b + n + 4 * rows * _cdiv(cols, BLK), f + 3 * n
        return {"bytes": b, "flops": f}
    t, d = case["tokens"], case["dim"]
    n = t * (case["q_heads"] + case["k_heads"]) * d
    b = 8 * t + 4 * case["rot"]
    if op == "rope":
        return {"bytes": 4 * n + b, "flops": 3 * n}
    if case["backward"]:
        return {"bytes": 6 * n + b + 12 * d, "flops": 14 * n}
    return {"bytes": 4 * n + b + 4 * d, "flops": 7 * n}


# ---- the definitions in 64 bits ----

def _scaled(codes, scales, fmt):
    """a block-128 operand's values; scales [blocks, rows]"""
    v = codes.contiguous().view(F8[fmt]).double()
    for i in range(scales.shape[0]):
        v[:, i * BLK:(i + 1) * BLK] *= scales[i].double()[:, None]
    return v


def _exact_blocks(v, fmt):
    """v (float64 [rows, K]) -> (v / scale, scales), without the rounding to 8 bits"""
    q, scales = v.clone(), []
    for k0 in range(0, v.shape[1], BLK):
        scales.append(v[:, k0:k0 + BLK].abs().max(dim=1).values.clamp(min=FLOOR) / FMAX[fmt])
        q[:, k0:k0 + BLK] /= scales[-1][:, None]
    return q, torch.stack(scales)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "grouped":
        a = _scaled(*s["a"], case["fa"])
        c = torch.zeros(case["rows"], case["N"], dtype=torch.float64, device="cuda")
        tile = torch.arange(case["N"], device="cuda") // BLK
        at = 0
        for i, end in enumerate(s["ends"]):
            if end > at:
                c[at:end] = torch.mm(a[at:end], _scaled(s["b"][0][i], s["b"][1][i][:, tile], "e4m3").t())
            at = end
        return c
    if op == "grouped_k":
        a, b = _scaled(*s["a"], case["fa"]), _scaled(*s["b"], "e4m3")
        c = torch.zeros(case["groups"], case["M"], case["N"], dtype=torch.float64, device="cuda")
        at = col = 0
        for i, end in enumerate(s["ends"]):
            if end > at:
                c[i] = torch.mm(a[:, col:col + end - at], b[:, col:col + end - at].t())
            col += _cdiv(end - at, BLK) * BLK
            at = end
        return c
    if op == "quantize":
        x, out = s["x"].double(), []
        if case["dual"]:
            out += _exact_blocks(x, case["fmt"])
        codes, scales, at = [], [], 0
        for end in s["ends"]:
            if end > at:
                part = torch.zeros(_cdiv(end - at, BLK) * BLK, case["cols"], dtype=torch.float64, device="cuda")
                part[:end - at] = x[at:end]
                q, sc = _exact_blocks(part.t().contiguous(), case["fmt"])
                codes.append(q)
                scales.append(sc)
            at = end
        left = _bound(case["rows"], case["groups"]) - sum(len(t) for t in scales)
        codes.append(torch.zeros(case["cols"], left * BLK, dtype=torch.float64, device="cuda"))
        scales.append(torch.zeros(left, case["cols"], dtype=torch.float64, device="cuda"))
        return out + [torch.cat(codes, 1), torch.cat(scales)]
    n, inter = case["rot"] // 2, case["layout"] == "interleaved"
    first = torch.arange(n, device="cuda") * (2 if inter else 1)
    second = first + (1 if inter else n)
    angle = s["positions"].double()[:, None, None] * s["freqs"][None, None]
    turn = torch.polar(torch.ones_like(angle), angle)

    def rotated(x, by):  # pairs as complex numbers
        y, z = x.clone(), torch.complex(x[..., first], x[..., second]) * by
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out, grads = [], []
    for x, name in ((s["q"].double(), "q"), (s["k"].double(), "k")):
        if op == "rope":
            out.append(rotated(x, turn.conj() if case["inverse"] else turn))
            continue
        w = s[name + "w"].double()
        r = 1.0 / torch.sqrt((x * x).sum(-1, keepdim=True) / case["dim"] + EPS)
        if not case["backward"]:
            out.append(rotated(x * r * w, turn))
            continue
        u = rotated(s["d" + name].double(), turn.conj())
        grads.append((u * x * r).flatten(0, 1).sum(0))
        inner = (u * w * x).sum(-1, keepdim=True) / case["dim"]
        out.append(u * w * r - x * inner * r ** 3)
    return out + grads
