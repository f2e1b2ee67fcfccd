"""The norm before an expert layer, FP8 with one scale for each block of 128, and the expert MLP on such weights, as
measured cases: what a serving or training step calls from the residual stream to the experts' outputs, in plain torch
and through the library.

Operators:
  norm      rmsnorm_fwd: the residual's addition, the root-mean-square norm, and its output in bf16 and in 8 bits with scales
  norm_bwd  rmsnorm_bwd: the gradients of its input (the residual's own added) and of its weight
  quant     fp8_block_quantize and fp8_block_dequantize: bf16 -> E4M3 with one fp32 scale for 1 x 128 or 128 x 128 values,
            row and transposed forms, the rows gathered by the routing's map, and back
  gemm      fp8_block_grouped_gemm: every expert's rows (1 x 128 scales) times its own weight (128 x 128 scales)
  wgrad     fp8_block_grouped_wgrad: the gradient of every expert's weight, both operands with scales along the tokens
  mlp       grouped_mlp_fwd_fp8_block and unpermute_combine: the expert MLP on such weights
"""
import math
import types

import numpy as np
import torch

own = False

# Mixtral-shaped layer of this repository's benchmark: 8 experts, hidden 4096, ffn 14336, top-2.
H_MIX, F_MIX = 4096, 14336
BLOCK = 128
EPS = 1e-6


def _lib():
    import moe_grouped_expert_amd as m
    return m


def listed():
    return [
        # eight requests with one new token each: the residual added, the norm for the router in bf16 and for the experts in 8 bits
        {"name": "norm serve", "op": "norm", "T": 8, "H": H_MIX, "x": "bf16", "weight": "bf16", "residual": True, "form": "fp8_block"},
        # the tokens of a training step or of prompts
        {"name": "norm prompt", "op": "norm", "T": 16384, "H": H_MIX, "x": "bf16", "weight": "bf16", "residual": True, "form": "fp8_block"},
        # the backward of a training step's tokens, the gradient that reaches the residual stream added
        {"name": "norm_bwd train", "op": "norm_bwd", "T": 8192, "H": H_MIX, "x": "bf16", "weight": "bf16", "residual": True},
        # a small ragged batch of a residual stream in fp32
        {"name": "norm_bwd odd", "op": "norm_bwd", "T": 777, "H": 2080, "x": "f32", "weight": "f32", "residual": False},
        # a training step's tokens, top-2: permuted, and quantized for the product and, transposed, for the weight gradient
        {"name": "quant tokens", "op": "quant", "batch": 1, "R": 8192, "C": H_MIX, "k": 2, "E": 8, "block": "1x128", "orient": "both"},
        # one expert's gate-up weight, for the product and, transposed, for the input gradient
        {"name": "quant weight", "op": "quant", "batch": 1, "R": 2 * F_MIX, "C": H_MIX, "k": 0, "E": 0, "block": "128x128", "orient": "both"},
        # one token through a dense projection: latency and one read of the weight
        {"name": "gemm one token", "op": "gemm", "E": 1, "rows": 1, "N": 2048, "K": H_MIX, "k": 0, "spread": 0.0},
        # the down projection of a prompt's rows, uneven odd groups
        {"name": "gemm prompt", "op": "gemm", "E": 8, "rows": 8191, "N": H_MIX, "K": F_MIX, "k": 0, "spread": 0.3},
        # the down projection's weight gradient of a training step
        {"name": "wgrad train", "op": "wgrad", "E": 8, "rows": 8192, "N": H_MIX, "K": F_MIX, "spread": 0.3},
        # a short ragged batch, experts without a token among them, odd sizes
        {"name": "wgrad odd", "op": "wgrad", "E": 16, "rows": 301, "N": 1056, "K": 2080, "spread": 2.5},
        # the whole expert MLP, eight requests with one new token each
        {"name": "mlp serve", "op": "mlp", "T": 8, "E": 8, "k": 2, "H": H_MIX, "F": F_MIX},
        # the whole expert MLP on a long prompt
        {"name": "mlp prompt", "op": "mlp", "T": 8192, "E": 8, "k": 2, "H": H_MIX, "F": F_MIX},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "quant", "gemm", "gemm", "wgrad", "mlp"])
    if op in ("norm", "norm_bwd"):
        c = {"op": op, "T": _log(rng, 1, 16384), "H": 32 * _log(rng, 1, 256), "x": rng.choice(["bf16", "bf16", "f32"]),
             "weight": rng.choice(["bf16", "f32"]), "residual": rng.random() < 0.7}
        if op == "norm":
            c["form"] = rng.choice(["none", "fp8_block", "fp8_block"])
        return c
    if op == "quant":
        block = rng.choice(["1x128", "1x128", "128x128"])
        c = {"op": op, "batch": 1, "R": _log(rng, 1, 8192), "C": 32 * _log(rng, 1, 448), "k": 0, "E": 0, "block": block,
             "orient": rng.choice(["row", "col", "both"])}
        if block == "1x128" and rng.random() < 0.5:
            c.update(E=rng.choice([4, 8, 16]), k=rng.randint(1, 4), C=32 * _log(rng, 1, 128))
        elif rng.random() < 0.3:
            c.update(batch=3, R=_log(rng, 1, 2048))
        return c
    if op == "gemm":
        return {"op": op, "E": rng.choice([1, 3, 8, 16]), "rows": _log(rng, 1, 8192), "N": 32 * _log(rng, 4, 256),
                "K": 32 * _log(rng, 2, 256), "k": rng.choice([0, 0, 2]), "spread": rng.choice([0.0, 0.3, 1.0])}
    if op == "wgrad":
        return {"op": op, "E": rng.choice([1, 3, 8, 16]), "rows": _log(rng, 1, 8192), "N": 32 * _log(rng, 1, 128),
                "K": 32 * _log(rng, 1, 128), "spread": rng.choice([0.0, 0.3, 2.0])}
    E = rng.choice([4, 8, 16])
    return {"op": op, "T": _log(rng, 1, 4096), "E": E, "k": rng.randint(1, 4), "H": 32 * _log(rng, 4, 128),
            "F": 32 * _log(rng, 4, 224)}


# ------------------------------------------------------------------------------ number formats, in plain torch

def _blocks(n):
    return -(-n // BLOCK)


def _factors(amax):
    """fp32 scale of a block from its largest magnitude (448 is E4M3's largest value; tiny blocks count as 2^-100), and
    what its values are multiplied by."""
    m = amax.clamp(min=2.0 ** -100)
    return m / 448, 448 / m


def _e4m3(v):
    return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _quant_rows(x):
    """fp32 [..., C] -> E4M3 codes uint8 [..., C] and fp32 scales [..., ceil(C / 128)]."""
    C = x.shape[-1]
    b = torch.nn.functional.pad(x, (0, -C % BLOCK)).reshape(*x.shape[:-1], -1, BLOCK)
    s, inv = _factors(b.abs().amax(-1))
    return _e4m3(b * inv[..., None]).reshape(*x.shape[:-1], -1)[..., :C].contiguous(), s


def _quant_tiles(x):
    """fp32 [..., R, C] -> codes [..., R, C] and scales [..., ceil(R / 128), ceil(C / 128)]."""
    R, C = x.shape[-2:]
    b = torch.nn.functional.pad(x, (0, -C % BLOCK, 0, -R % BLOCK))
    b = b.reshape(*x.shape[:-2], _blocks(R), BLOCK, _blocks(C), BLOCK)
    s, inv = _factors(b.abs().amax((-3, -1)))
    q = _e4m3(b * inv[..., :, None, :, None])
    return q.reshape(*x.shape[:-2], _blocks(R) * BLOCK, _blocks(C) * BLOCK)[..., :R, :C].contiguous(), s


def _decode(codes, scales):
    """fp32 values; scales for 1 x 128 or for 128 x 128 values, by their shape."""
    R, C = codes.shape[-2:]
    s = scales.repeat_interleave(BLOCK, -1)[..., :C]
    if s.shape[-2] != R:
        s = s.repeat_interleave(BLOCK, -2)[..., :R, :]
    return codes.view(torch.float8_e4m3fn).to(torch.float32) * s


# ------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _stream(T, H, g):
    """A residual stream: every channel has a spread of its own, a few channels much larger than the others."""
    spread = torch.exp(0.5 * torch.randn(H, generator=g, device="cuda"))
    spread = torch.where(torch.rand(H, generator=g, device="cuda") < 0.005, 20 * spread, spread)
    return torch.randn(T, H, generator=g, device="cuda") * spread


def _sizes(rows, E, spread, seed):
    """Rows of each expert: `rows` in all, weights exp(spread * normal); spread 0 is an even split."""
    r = np.random.RandomState(seed % (1 << 31))
    w = np.exp(spread * r.standard_normal(E))
    cut = np.floor(np.concatenate([[0.0], np.cumsum(w) / w.sum()]) * rows + 0.5).astype(np.int64)
    return np.diff(cut)


def _weights(E, N, K, g):
    """E normal weights [N][K] in E4M3 with 128 x 128 scales, one expert at a time (bounded memory)."""
    codes = torch.empty(E, N, K, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, _blocks(N), _blocks(K), device="cuda")
    for e in range(E):
        w = torch.randn(N, K, generator=g, device="cuda").mul_(0.02)
        codes[e], scales[e] = _quant_tiles(w.to(torch.bfloat16).float())
    return codes, scales


def _routes(T, E, k, align, g):
    """The maps of a routing call: experts in order, each group at a multiple of `align` rows, tokens in order inside."""
    logits = torch.randn(T, E, generator=g, device="cuda") + 0.3 * torch.randn(E, generator=g, device="cuda")
    top = torch.sort(logits, dim=1, descending=True, stable=True)
    idx, prob = top.indices[:, :k], torch.softmax(top.values[:, :k], 1)
    flat = idx.reshape(-1)
    sizes = torch.bincount(flat, minlength=E)
    offsets = torch.cat([sizes.new_zeros(1), ((sizes + align - 1) // align * align).cumsum(0)])
    R = (T * k + E * (align - 1) + 31) // 32 * 32
    order = torch.sort(flat, stable=True).indices
    first = sizes.cumsum(0) - sizes
    pos = torch.empty_like(flat)
    pos[order] = offsets[flat[order]] + torch.arange(T * k, device="cuda") - first[flat[order]]
    src = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    src[pos] = torch.arange(T, device="cuda", dtype=torch.int32).repeat_interleave(k)
    prob_perm = torch.zeros(R, device="cuda")
    prob_perm[pos] = prob.reshape(-1)
    return types.SimpleNamespace(T=T, E=E, k=k, align=align, R=R, split_sizes=sizes.to(torch.int32),
                                 group_offsets=offsets.to(torch.int32), perm_src=src, prob_perm=prob_perm,
                                 perm_pos=pos.reshape(T, k).to(torch.int32))


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    op = c["op"]
    s = {"c": c}
    if op in ("norm", "norm_bwd"):
        T, H, dt = c["T"], c["H"], _dtype(c["x"])
        s["weight"] = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(_dtype(c["weight"]))
        s["x"] = _stream(T, H, g).to(dt)
        if op == "norm":
            s["residual"] = _stream(T, H, g).to(dt) if c["residual"] else None
        else:
            s["dy"] = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
            s["d_residual"] = torch.randn(T, H, generator=g, device="cuda").to(dt) if c["residual"] else None
            s["rstd"] = (1 / torch.sqrt((s["x"].double() ** 2).mean(1) + EPS)).float()
    elif op == "quant":
        if c["E"]:
            s["x"] = _stream(c["R"], c["C"], g).to(torch.bfloat16)
            s["rows"] = _routes(c["R"], c["E"], c["k"], BLOCK, g).perm_src
        else:
            s["rows"] = None
            s["x"] = torch.randn(c["batch"], c["R"], c["C"], generator=g, device="cuda").mul_(0.02).to(torch.bfloat16)
    elif op == "gemm":
        E, rows, N, K = c["E"], c["rows"], c["N"], c["K"]
        sizes = _sizes(rows, E, c["spread"], seed)
        # with k: the rows of a product are the tokens, each named by k rows
        T = rows // c["k"] + 1 if c["k"] else rows
        s["a"], s["a_scale"] = _quant_rows(_stream(T, K, g).to(torch.bfloat16).float())
        s["a_rows"] = torch.randint(0, T, (rows,), generator=g, device="cuda", dtype=torch.int32) if c["k"] else None
        s["w"], s["w_scale"] = _weights(E, N, K, g)
        s["sizes"] = torch.from_numpy(sizes).to(torch.int32).cuda()
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)])).to(torch.int32).cuda()
        s["cap"] = int(sizes.max())
    elif op == "wgrad":
        E, rows, N, K = c["E"], c["rows"], c["N"], c["K"]
        sizes = _sizes(rows, E, c["spread"], seed)
        offsets = np.concatenate([[0], np.cumsum(-(-sizes // BLOCK) * BLOCK)])
        R = (rows + E * (BLOCK - 1) + 31) // 32 * 32
        live = torch.zeros(R, 1, device="cuda")
        for n, o in zip(sizes.tolist(), offsets.tolist()):
            live[o:o + n] = 1
        s["dy"], s["dy_scale"] = _quant_rows((torch.randn(R, N, generator=g, device="cuda").to(torch.bfloat16) * live).float().T.contiguous())
        s["x"], s["x_scale"] = _quant_rows((_stream(R, K, g).to(torch.bfloat16) * live).float().T.contiguous())
        s["sizes"] = torch.from_numpy(sizes).to(torch.int32).cuda()
        s["offsets"] = torch.from_numpy(offsets).to(torch.int32).cuda()
        s["cap"] = int(sizes.max())
    else:
        T, E, k, H, F = c["T"], c["E"], c["k"], c["H"], c["F"]
        s["rt"] = _routes(T, E, k, 32, g)
        s["x"], s["x_scale"] = _quant_rows(torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16).float())
        s["wgu"], s["wgu_scale"] = _weights(E, 2 * F, H, g)
        s["wd"], s["wd_scale"] = _weights(E, H, F, g)
        s["cap"] = int(s["rt"].split_sizes.max())
    return s


# ------------------------------------------------------------------------------ the plain forms

def _norm(s):
    c = s["c"]
    r = s["x"].float()
    out = {}
    if s["residual"] is not None:
        out["residual"] = (r + s["residual"].float()).to(s["x"].dtype)
        r = out["residual"].float()
    rstd = 1 / torch.sqrt((r * r).mean(1, keepdim=True) + EPS)
    y = r * rstd * s["weight"].float()
    out["y"], out["rstd"] = y.to(torch.bfloat16), rstd[:, 0]
    if c["form"] == "fp8_block":
        out["q"] = _decode(*_quant_rows(y)).to(torch.bfloat16)
    return out


def _norm_bwd(s):
    r, rstd = s["x"].float(), s["rstd"][:, None]
    dy, xhat = s["dy"].float(), r * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if s["d_residual"] is not None:
        dx = dx + s["d_residual"].float()
    return dx.to(s["x"].dtype), (dy * xhat).sum(0)


def _forms(s, quant, decode):
    c, x = s["c"], s["x"].float()
    if s["rows"] is not None:
        x = torch.cat([x, x.new_zeros(1, x.shape[1])])[s["rows"].long()]
    out = {}
    if c["orient"] != "col":
        out["row"] = decode(*quant(x)).to(torch.bfloat16)
    if c["orient"] != "row":
        # the transpose, its rows' length a multiple of 32
        xt = torch.nn.functional.pad(x.transpose(-1, -2), (0, -x.shape[-2] % 32))
        out["col"] = decode(*quant(xt.contiguous())).to(torch.bfloat16)
    return out


def _padded(a, sizes, offsets, cap):
    """Where each group's rows stand, each padded to the largest one's rows (past the end of `a` where there is none)."""
    row = offsets[:-1, None].long() + torch.arange(cap, device=a.device)
    return torch.where(torch.arange(cap, device=a.device) < sizes[:, None], row, torch.full_like(row, a.shape[0]))


def _grouped(a, w, sizes, offsets, cap):
    """Rows of `a` times their own expert's w^T."""
    R, E = a.shape[0], w.shape[0]
    row = _padded(a, sizes, offsets, cap)
    out = torch.bmm(torch.cat([a, a.new_zeros(1, a.shape[1])])[row], w.transpose(1, 2))
    return a.new_zeros(R + 1, w.shape[1]).index_copy_(0, row.reshape(-1), out.reshape(E * cap, -1))[:R]


def _wgrad(s):
    dy, x = _decode(s["dy"], s["dy_scale"]).T, _decode(s["x"], s["x_scale"]).T
    row = _padded(dy, s["sizes"], s["offsets"], s["cap"])
    dy, x = (torch.cat([v, v.new_zeros(1, v.shape[1])])[row] for v in (dy, x))
    return torch.bmm(dy.transpose(1, 2), x).to(torch.bfloat16)


def _mlp(s):
    rt, F = s["rt"], s["c"]["F"]
    x = _decode(s["x"], s["x_scale"])
    x = torch.cat([x, x.new_zeros(1, x.shape[1])])[rt.perm_src.long()]
    gu = _grouped(x, _decode(s["wgu"], s["wgu_scale"]), rt.split_sizes, rt.group_offsets, s["cap"])
    G, U = gu[:, :F], gu[:, F:]
    h = _decode(*_quant_rows(rt.prob_perm[:, None] * (G / (1 + torch.exp(-G))) * U))
    y = _grouped(h, _decode(s["wd"], s["wd_scale"]), rt.split_sizes, rt.group_offsets, s["cap"]).to(torch.bfloat16)
    return y[rt.perm_pos.long()].float().sum(1).to(torch.bfloat16)


def _run_plain(s):
    op = s["c"]["op"]
    if op == "norm":
        return _norm(s)
    if op == "norm_bwd":
        return _norm_bwd(s)
    if op == "quant":
        return _forms(s, _quant_rows if s["c"]["block"] == "1x128" else _quant_tiles, _decode)
    if op == "gemm":
        a = _decode(s["a"], s["a_scale"])
        a = a if s["a_rows"] is None else a[s["a_rows"].long()]
        return _grouped(a, _decode(s["w"], s["w_scale"]), s["sizes"], s["offsets"], s["cap"]).to(torch.bfloat16)
    if op == "wgrad":
        return _wgrad(s)
    return _mlp(s)


def _run_own(s):
    m, c = _lib(), s["c"]
    op = c["op"]
    if op == "norm":
        o = m.rmsnorm_fwd(s["x"], s["weight"], EPS, residual=s["residual"], form=None if c["form"] == "none" else c["form"])
        out = {"y": o.y, "rstd": o.rstd}
        if s["residual"] is not None:
            out["residual"] = o.residual
        if c["form"] == "fp8_block":
            out["q"] = m.fp8_block_dequantize(o.codes, o.scales)
        return out
    if op == "norm_bwd":
        return m.rmsnorm_bwd(s["dy"], s["x"], s["weight"], s["rstd"], d_residual=s["d_residual"])
    if op == "quant":
        rc, rs, cc, cs = m.fp8_block_quantize(s["x"], c["orient"], c["block"], rows=s["rows"])
        out = {}
        if rc is not None:
            out["row"] = m.fp8_block_dequantize(rc, rs)
        if cc is not None:
            out["col"] = m.fp8_block_dequantize(cc, cs)
        return out
    if op == "gemm":
        return m.fp8_block_grouped_gemm(s["a"], s["a_scale"], s["w"], s["w_scale"], s["sizes"], s["offsets"], a_rows=s["a_rows"])
    if op == "wgrad":
        return m.fp8_block_grouped_wgrad(s["dy"], s["dy_scale"], s["x"], s["x_scale"], s["sizes"], s["offsets"], out_dtype="bf16")
    f = m.grouped_mlp_fwd_fp8_block(s["rt"], s["x"], s["x_scale"], s["wgu"], s["wd"], s["wgu_scale"], s["wd_scale"])
    return m.unpermute_combine(f.y_perm, s["rt"].perm_pos)


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    """Inputs read once and outputs written once; two operations for each product and sum of the matrix products."""
    c = case
    op = c["op"]
    if op in ("norm", "norm_bwd"):
        n, b = c["T"] * c["H"], 2 if c["x"] == "bf16" else 4
        if op == "norm":
            q = {"none": 0, "fp8_block": 132 / 128}[c["form"]]
            return {"bytes": int(n * (b * (3 if c["residual"] else 1) + 2 + q + (q > 0) * 2)), "flops": 8 * n}
        return {"bytes": n * (b * (3 if c["residual"] else 2) + 2) + 4 * c["H"], "flops": 12 * n}
    if op == "quant":
        forms = 2 if c["orient"] == "both" else 1
        n = c["batch"] * c["R"] * c["C"]
        m = c["R"] * c["k"] * c["C"] if c["E"] else n
        return {"bytes": 2 * n + forms * 3 * m, "flops": 4 * m * forms}
    # experts without a row need no weight: at most as many experts as rows are read
    if op == "gemm":
        E = min(c["E"], c["rows"])
        a = (c["rows"] // c["k"] + 1 if c["k"] else c["rows"]) * c["K"]
        return {"bytes": E * c["N"] * c["K"] + a * 33 // 32 + 2 * c["rows"] * c["N"], "flops": 2 * c["rows"] * c["N"] * c["K"]}
    if op == "wgrad":
        return {"bytes": c["rows"] * (c["N"] + c["K"]) * 33 // 32 + 2 * c["E"] * c["N"] * c["K"],
                "flops": 2 * c["rows"] * c["N"] * c["K"]}
    rows = c["T"] * c["k"]
    return {"bytes": 3 * min(c["E"], rows) * c["F"] * c["H"] + c["T"] * c["H"] * 33 // 32 + 2 * rows * c["F"] * 33 // 32
            + 4 * rows * c["H"] + 2 * c["T"] * c["H"], "flops": 6 * rows * c["H"] * c["F"]}


# ------------------------------------------------------------------------------ the definitions in 64 bits

def _table():
    """The magnitudes of E4M3 in order of their codes."""
    return [m / 512 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]


def _values(codes, scales, both=False):
    """By table, in 64 bits; both: a scale for 128 x 128 values."""
    t = torch.tensor(_table() + [math.nan], dtype=torch.float64, device=codes.device)
    v = t[(codes & 127).int()]
    v = torch.where(codes >= 128, -v, v)
    at = torch.arange(codes.shape[-1], device=codes.device) // BLOCK
    s = scales.double()[..., at]
    if both:
        s = s[..., torch.arange(codes.shape[-2], device=codes.device) // BLOCK, :]
    return v * s


def _nearest(a):
    """The nearest E4M3 value, ties to the even code, at most 448; by search in the table."""
    t = torch.tensor(_table(), dtype=torch.float64, device=a.device)
    m = a.abs().clamp(max=448)
    hi = torch.searchsorted(t, m).clamp(max=len(t) - 1)
    lo = (hi - 1).clamp(min=0)
    mid = (t[lo] + t[hi]) / 2
    pick = torch.where(m > mid, hi, torch.where(m < mid, lo, torch.where(hi % 2 == 0, hi, lo)))
    return torch.copysign(t[pick], a)


def _through(x, rows_too=False):
    """What is left of x (64 bits) after one scale for each block: each block's largest magnitude becomes 448."""
    out = torch.empty_like(x)
    R, C = x.shape[-2:]
    step = BLOCK if rows_too else R
    for r in range(0, R, step):
        for k in range(0, C, BLOCK):
            b = x[..., r:r + step, k:k + BLOCK]
            top = b.abs().amax((-2, -1) if rows_too else -1, keepdim=True).clamp(min=2.0 ** -100) / 448
            out[..., r:r + step, k:k + BLOCK] = _nearest(b / top) * top
    return out


def _by_group(a, w, sizes, offsets):
    """Each group's rows times its own weight, group after group."""
    out = torch.zeros(a.shape[0], w(0).shape[0], dtype=torch.float64, device=a.device)
    for e, (n, o) in enumerate(zip(sizes.tolist(), offsets.tolist())):
        if n:
            out[o:o + n] = a[o:o + n] @ w(e).T
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    op = c["op"]
    if op == "norm":
        x, out = s["x"].double(), {}
        if s["residual"] is not None:
            out["residual"] = x + s["residual"].double()
            x = out["residual"].to(s["x"].dtype).double()   # the norm is taken of the sum as it is stored
        ms = torch.einsum("th,th->t", x, x) / c["H"]
        y = x / torch.sqrt(ms + EPS)[:, None] * s["weight"].double()
        out["y"], out["rstd"] = y, torch.rsqrt(ms + EPS)
        if c["form"] != "none":
            out["q"] = _through(y)
        return out
    if op == "norm_bwd":
        # the Jacobian of y = x w / sqrt(mean x^2 + eps), with the forward's statistic
        x, q, dy, w = s["x"].double(), s["rstd"].double()[:, None], s["dy"].double(), s["weight"].double()
        along = ((dy * w) * x).sum(1, keepdim=True)
        dx = dy * w * q - x * q ** 3 * along / c["H"]
        if s["d_residual"] is not None:
            dx = dx + s["d_residual"].double()
        return dx, torch.einsum("th,th->h", dy, x * q)
    if op == "quant":
        x = s["x"].double()
        if s["rows"] is not None:
            got = torch.zeros(s["rows"].numel(), c["C"], dtype=torch.float64, device="cuda")
            there = s["rows"] >= 0
            got[there] = x[s["rows"][there].long()]
            x = got
        out = {}
        if c["orient"] != "col":
            out["row"] = _through(x, c["block"] == "128x128")
        if c["orient"] != "row":
            xt = torch.nn.functional.pad(x.transpose(-1, -2), (0, -x.shape[-2] % 32)).contiguous()
            out["col"] = _through(xt, c["block"] == "128x128")
        return out
    if op == "gemm":
        a = _values(s["a"], s["a_scale"])
        a = a if s["a_rows"] is None else a[s["a_rows"].long()]
        return _by_group(a, lambda e: _values(s["w"][e], s["w_scale"][e], True), s["sizes"], s["offsets"])
    if op == "wgrad":
        dy, x = _values(s["dy"], s["dy_scale"]), _values(s["x"], s["x_scale"])
        out = torch.zeros(c["E"], c["N"], c["K"], dtype=torch.float64, device="cuda")
        for e, (n, o) in enumerate(zip(s["sizes"].tolist(), s["offsets"].tolist())):
            out[e] = dy[:, o:o + n] @ x[:, o:o + n].T
        return out
    rt, F = s["rt"], c["F"]
    x = torch.zeros(rt.R, c["H"], dtype=torch.float64, device="cuda")
    there = rt.perm_src >= 0
    x[there] = _values(s["x"], s["x_scale"])[rt.perm_src[there].long()]
    gu = _by_group(x, lambda e: _values(s["wgu"][e], s["wgu_scale"][e], True), rt.split_sizes, rt.group_offsets)
    h = rt.prob_perm.double()[:, None] * gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
    y = _by_group(_through(h), lambda e: _values(s["wd"][e], s["wd_scale"][e], True), rt.split_sizes, rt.group_offsets)
    return y[rt.perm_pos.long()].sum(1)
