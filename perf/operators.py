"""The router and the 4-bit expert products as measured cases: what a serving or training step calls
around the grouped expert MLP, in plain torch and through the library.

Operators:
  topk      moe_route_topk: expert scores (softmax or sigmoid of the router logits), a balance bias that takes
            part in the choice only, groups of experts, top-k, renormalised and scaled weights
  topk_bwd  moe_route_topk_bwd: the gradient of those weights with respect to the logits
  quant     mxfp4_quantize and mxfp4_dequantize: bf16 -> E2M1 codes with one E8M0 scale per 32 values, and back
  gemm      mxfp4_grouped_gemm: every expert's rows times its own MXFP4 weight, rows in MXFP8 or MXFP4
  mlp       grouped_mlp_fwd_mxfp4 and unpermute_combine: the expert MLP on MXFP4 weights, MXFP8 activations
"""
import math
import types

import numpy as np
import torch

own = False

# Mixtral-shaped layer of this repository's benchmark: 8 experts, hidden 4096, ffn 14336, top-2.
H_MIX, F_MIX = 4096, 14336


def _lib():
    import moe_grouped_expert_amd as m
    return m


def listed():
    return [
        # one step of token-by-token serving: four requests, many small experts in groups; latency only
        {"name": "topk serve sigmoid groups", "op": "topk", "T": 4, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "topk_groups": 4, "topn": 2, "renorm": True, "scale": 2.5, "dtype": "f32", "masked": 0.0},
        # a training step of the same router: all tokens of a batch, some experts masked out
        {"name": "topk train sigmoid groups", "op": "topk", "T": 16384, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "topk_groups": 4, "topn": 2, "renorm": True, "scale": 2.5, "dtype": "f32", "masked": 0.02},
        # the Mixtral-shaped router on one long sequence, bf16 logits
        {"name": "topk train softmax", "op": "topk", "T": 32768, "E": 8, "k": 2, "score": "softmax", "bias": False,
         "groups": 1, "topk_groups": 1, "topn": 1, "renorm": True, "scale": 1.0, "dtype": "bf16", "masked": 0.0},
        # backward of the grouped sigmoid router
        {"name": "topk_bwd sigmoid", "op": "topk_bwd", "T": 16384, "E": 256, "k": 8, "score": "sigmoid", "renorm": True,
         "scale": 2.5, "dtype": "f32", "masked": 0.02},
        # weights that are not renormalised: every expert's logit gets a gradient; odd sizes, bf16
        {"name": "topk_bwd softmax odd", "op": "topk_bwd", "T": 5001, "E": 60, "k": 4, "score": "softmax", "renorm": False,
         "scale": 1.0, "dtype": "bf16", "masked": 0.01},
        # one expert's gate-up weight, both orientations (forward and input gradient)
        {"name": "quant weight both", "op": "quant", "batch": 1, "R": 2 * F_MIX, "C": H_MIX, "orient": "both", "std": 0.02},
        # the activations of a small odd batch
        {"name": "quant activations", "op": "quant", "batch": 1, "R": 333, "C": H_MIX, "orient": "row", "std": 1.0},
        # one token through a dense projection: latency and one read of the weight
        {"name": "gemm one token", "op": "gemm", "E": 1, "rows": 1, "N": 2048, "K": H_MIX, "a": "mxfp8", "spread": 0.0},
        # serving 16 requests: two rows for each expert on average, the whole gate-up weight is read
        {"name": "gemm serve", "op": "gemm", "E": 8, "rows": 32, "N": 2 * F_MIX, "K": H_MIX, "a": "mxfp8", "spread": 0.5},
        # a prompt's rows with both operands in 4 bits, uneven odd groups
        {"name": "gemm prompt 4-bit", "op": "gemm", "E": 8, "rows": 8191, "N": H_MIX, "K": F_MIX, "a": "mxfp4", "spread": 0.3},
        # the whole expert MLP, eight requests with one new token each
        {"name": "mlp serve", "op": "mlp", "T": 8, "E": 8, "k": 2, "H": H_MIX, "F": F_MIX},
        # the whole expert MLP on a long prompt
        {"name": "mlp prompt", "op": "mlp", "T": 8192, "E": 8, "k": 2, "H": H_MIX, "F": F_MIX},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["topk", "topk_bwd", "quant", "gemm", "gemm", "mlp"])
    if op in ("topk", "topk_bwd"):
        E = rng.choice([4, 8, 12, 16, 30, 32, 60, 64, 96, 128, 160, 200, 256])
        c = {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(8, E // 2)),
             "score": rng.choice(["softmax", "sigmoid"]), "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5, 0.5]),
             "dtype": rng.choice(["f32", "bf16"]), "masked": rng.choice([0.0, 0.01, 0.1])}
        if op == "topk_bwd" and c["k"] == 1:
            c["renorm"] = False   # one renormalised weight is a constant: its gradient is 0
        if op == "topk":
            groups = rng.choice([g for g in (1, 2, 4, 8) if E % g == 0 and E // g >= 2])
            need = -(-c["k"] * groups // E)
            c.update(bias=rng.random() < 0.6, groups=groups, topk_groups=rng.randint(need, groups), topn=rng.choice([1, 2]))
        return c
    if op == "quant":
        return {"op": op, "batch": rng.choice([1, 1, 3]), "R": _log(rng, 1, 9000), "C": 32 * _log(rng, 1, 448),
                "orient": rng.choice(["row", "col", "both"]), "std": rng.choice([0.02, 1.0])}
    if op == "gemm":
        return {"op": op, "E": rng.choice([1, 3, 8, 16]), "rows": _log(rng, 1, 8192), "N": 32 * _log(rng, 4, 256),
                "K": 32 * _log(rng, 2, 256), "a": rng.choice(["mxfp8", "mxfp4"]), "spread": rng.choice([0.0, 0.3, 1.0])}
    E = rng.choice([4, 8, 16])
    return {"op": op, "T": _log(rng, 1, 4096), "E": E, "k": rng.randint(1, 4), "H": 32 * _log(rng, 4, 128),
            "F": 32 * _log(rng, 4, 224)}


# ------------------------------------------------------------------------------ number formats, in plain torch

def _floor_log2(a):
    """floor(log2 a) of positive fp32 values (frexp: a = mantissa in [0.5, 1) times 2^e)."""
    return torch.frexp(a).exponent - 1


def _mx_scale(x, emax):
    """E8M0 bytes of the blocks of 32 along the last axis: floor(log2 amax) - emax, kept in [-127, 127], plus 127."""
    amax = x.reshape(*x.shape[:-1], -1, 32).abs().amax(-1)
    e = torch.where(amax > 0, _floor_log2(amax) - emax, torch.full_like(amax, -127, dtype=torch.int32)).clamp(-127, 127)
    return e + 127


def _pow2(s):
    """2^(s - 127) of E8M0 bytes, exact in fp32 (2^-127 is subnormal, so in two factors)."""
    half = torch.div(s.to(torch.int32) - 127, 2, rounding_mode="floor")
    one = torch.ones((), device=s.device, dtype=torch.float32)
    return torch.ldexp(one, half) * torch.ldexp(one, s.to(torch.int32) - 127 - half)


def _div_pow2(x, s):
    """x / 2^(s - 127), x blocked by 32 along the last axis."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    half = torch.div(s.to(torch.int32) - 127, 2, rounding_mode="floor")
    rest = s.to(torch.int32) - 127 - half
    return torch.ldexp(torch.ldexp(b, -half[..., None]), -rest[..., None])


def _quant4(x):
    """fp32 [..., C] -> packed E2M1 codes uint8 [..., C/2] (even element in the low half) and E8M0 bytes [..., C/32].
    The magnitudes are 0, .5, 1, 1.5, 2, 3, 4, 6; nearest, ties to the even code, at most 6."""
    s = _mx_scale(x, 2)
    v = _div_pow2(x, s)
    a = v.abs()
    q = torch.where(a < 2, (2 * a).round(), torch.where(a < 4, a.round() + 2, (a / 2).round() + 4)).clamp(max=7)
    code = q.to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    code = code.reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.to(torch.uint8)


def _decode4(codes, scales):
    """Packed E2M1 codes and their scales -> fp32 values."""
    c = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    m = (c & 7).to(torch.float32)
    mag = torch.where(m < 4, m * 0.5, torch.where(m < 6, m - 2, 2 * m - 8))
    v = torch.where(c >= 8, -mag, mag)
    return (v.reshape(*v.shape[:-1], -1, 32) * _pow2(scales)[..., None]).reshape(v.shape)


def _quant8(x):
    """fp32 [..., C] -> E4M3 codes and E8M0 bytes (the same block rule, largest exponent 8, at most 448)."""
    s = _mx_scale(x, 8)
    v = _div_pow2(x, s).clamp(-448, 448).reshape(x.shape)
    return v.to(torch.float8_e4m3fn).view(torch.uint8), s.to(torch.uint8)


def _decode8(codes, scales):
    v = codes.view(torch.float8_e4m3fn).to(torch.float32)
    return (v.reshape(*v.shape[:-1], -1, 32) * _pow2(scales)[..., None]).reshape(v.shape)


# ------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _logits(c, g):
    """Router logits of a trained layer: a spread of about one, some experts preferred by all tokens; masked experts
    are -inf, and one row in 500 has every expert masked."""
    T, E = c["T"], c["E"]
    l = torch.randn(T, E, generator=g, device="cuda") * 1.2 + torch.randn(E, generator=g, device="cuda") * 0.5
    if c["masked"] > 0:
        u = torch.rand(T, E, generator=g, device="cuda")
        row = torch.rand(T, 1, generator=g, device="cuda") < 0.002
        l = torch.where((u < c["masked"]) | row, torch.full_like(l, -math.inf), l)
    return l.to(torch.bfloat16) if c["dtype"] == "bf16" else l


def _sizes(rows, E, spread, seed):
    """Rows of each expert: `rows` in all, weights exp(spread * normal); spread 0 is an even split."""
    r = np.random.RandomState(seed % (1 << 31))
    w = np.exp(spread * r.standard_normal(E))
    cut = np.floor(np.concatenate([[0.0], np.cumsum(w) / w.sum()]) * rows + 0.5).astype(np.int64)
    return np.diff(cut)


def _weights(E, N, K, g):
    """MXFP4 codes and scales of E normal weights [N][K], one expert at a time (bounded memory)."""
    codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, N, K // 32, dtype=torch.uint8, device="cuda")
    for e in range(E):
        w = torch.randn(N, K, generator=g, device="cuda").mul_(0.02)
        codes[e], scales[e] = _quant4(w.to(torch.bfloat16).float())
    return codes, scales


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    op = c["op"]
    s = {"c": c}
    if op == "topk":
        s["logits"] = _logits(c, g)
        s["bias"] = torch.randn(c["E"], generator=g, device="cuda") * 0.05 if c["bias"] else None
    elif op == "topk_bwd":
        s["logits"] = _logits(c, g)
        # the forward's choice: the k largest logits, masked experts last
        s["idx"] = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True).indices[:, :c["k"]].to(torch.int32).contiguous()
        s["d_prob"] = torch.randn(c["T"], c["k"], generator=g, device="cuda")
    elif op == "quant":
        shape = (c["batch"], c["R"], c["C"])
        s["w"] = torch.randn(shape, generator=g, device="cuda").mul_(c["std"]).to(torch.bfloat16)
    elif op == "gemm":
        E, rows, N, K = c["E"], c["rows"], c["N"], c["K"]
        sizes = _sizes(rows, E, c["spread"], seed)
        a = torch.randn(rows, K, generator=g, device="cuda").to(torch.bfloat16).float()
        s["a"], s["a_scale"] = _quant8(a) if c["a"] == "mxfp8" else _quant4(a)
        s["w"], s["w_scale"] = _weights(E, N, K, g)
        s["sizes"] = torch.from_numpy(sizes).to(torch.int32).cuda()
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)])).to(torch.int32).cuda()
        s["cap"] = int(sizes.max())
    else:
        T, E, k, H, F = c["T"], c["E"], c["k"], c["H"], c["F"]
        logits = torch.randn(T, E, generator=g, device="cuda") + 0.3 * torch.randn(E, generator=g, device="cuda")
        top = torch.sort(logits, dim=1, descending=True, stable=True)
        idx, prob = top.indices[:, :k], torch.softmax(top.values[:, :k], 1)
        # the maps of a routing call: experts in order, each group at a multiple of 32 rows, tokens in order inside
        flat = idx.reshape(-1)
        sizes = torch.bincount(flat, minlength=E)
        padded = (sizes + 31) // 32 * 32
        offsets = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
        R = (T * k + E * 31 + 31) // 32 * 32
        order = torch.sort(flat, stable=True).indices
        first = sizes.cumsum(0) - sizes
        pos = torch.empty_like(flat)
        pos[order] = offsets[flat[order]] + torch.arange(T * k, device="cuda") - first[flat[order]]
        x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16).float()
        xp = torch.zeros(R, H, device="cuda")
        xp[pos] = x.repeat_interleave(k, 0)
        prob_perm = torch.zeros(R, device="cuda")
        prob_perm[pos] = prob.reshape(-1)
        xc, xs = _quant8(xp)
        s["rt"] = types.SimpleNamespace(T=T, E=E, k=k, H=H, align=32, prec="mxfp8", R=R, split_sizes=sizes.to(torch.int32),
                                        group_offsets=offsets.to(torch.int32), prob_perm=prob_perm,
                                        perm_pos=pos.reshape(T, k).to(torch.int32), x_perm=xc, x_perm_scale=xs)
        s["wgu"], s["wgu_scale"] = _weights(E, 2 * F, H, g)
        s["wd"], s["wd_scale"] = _weights(E, H, F, g)
        s["cap"] = int(sizes.max())
    return s


# ------------------------------------------------------------------------------ the plain forms

def _keys(logits, bias, score):
    """What the choice goes by, in 64 bits (two experts may be nearly equal): the logit, or with a bias score + bias."""
    l = logits.double()
    off = torch.isneginf(l)
    if bias is None:
        return l, off, _scores(l, off, score)
    sc = _scores(l, off, score)
    return torch.where(off, torch.full_like(l, -math.inf), sc + bias.double()), off, sc


def _scores(l, off, score):
    """Scores of the experts, 0 for a masked one."""
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    m = l.amax(1, keepdim=True)
    e = torch.where(off, torch.zeros_like(l), torch.exp(l - torch.where(torch.isneginf(m), torch.zeros_like(m), m)))
    t = e.sum(1, keepdim=True)
    return e / torch.where(t > 0, t, torch.ones_like(t))


def _topk(c, logits, bias):
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    key, off, sc = _keys(logits, bias, c["score"])
    if G > 1 and c["topk_groups"] < G:
        # a group's score: its best experts' scores, summed (with the bias where there is one); none left: last
        by = key if bias is not None or c["topn"] == 1 else torch.where(off, key, sc)
        best = torch.sort(by.reshape(T, G, E // G), dim=2, descending=True).values[..., :c["topn"]]
        gs = torch.where(torch.isneginf(best), torch.zeros_like(best), best).sum(2)
        gs = torch.where(torch.isneginf(best[..., 0]), best[..., 0], gs)
        rank = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=key.device).scatter_(1, rank, True)
        keep = keep[:, :, None].expand(T, G, E // G).reshape(T, E)
        # kept, then kept but masked, then the other groups' experts
        key = torch.where(keep, torch.where(off, torch.full_like(key, -1e300), key), torch.full_like(key, -math.inf))
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(sc, 1, idx)
    if c["renorm"]:
        t = w.sum(1, keepdim=True)
        w = w / torch.where(t > 0, t, torch.ones_like(t))
    return idx.to(torch.int32), (w * c["scale"]).float()


def _topk_bwd(c, logits, idx, d_prob):
    l = logits.float()
    sc = _scores(l, torch.isneginf(l), c["score"])
    i = idx.long()
    w = torch.gather(sc, 1, i)
    d = d_prob * c["scale"]
    if c["renorm"]:
        t = w.sum(1, keepdim=True)
        t = torch.where(t > 0, t, torch.ones_like(t))
        d = (d - (w / t * d).sum(1, keepdim=True)) / t
    ds = torch.zeros_like(sc).scatter_add_(1, i, d)
    if c["score"] == "sigmoid":
        dl = ds * sc * (1 - sc)
    else:
        dl = sc * (ds - (sc * ds).sum(1, keepdim=True))
    return dl.to(logits.dtype)


def _grouped(a, w, sizes, offsets, cap):
    """Rows of `a` times their own expert's w^T: the groups side by side, each padded to the largest one's rows."""
    R, E = a.shape[0], w.shape[0]
    row = offsets[:-1, None].long() + torch.arange(cap, device=a.device)
    ok = torch.arange(cap, device=a.device) < sizes[:, None]
    row = torch.where(ok, row, torch.full_like(row, R))
    padded = torch.cat([a, a.new_zeros(1, a.shape[1])])[row]
    out = torch.bmm(padded, w.transpose(1, 2))
    return a.new_zeros(R + 1, w.shape[1]).index_copy_(0, row.reshape(-1), out.reshape(E * cap, -1))[:R]


def _mlp(s):
    rt, c = s["rt"], s["c"]
    F = c["F"]
    gu = _grouped(_decode8(rt.x_perm, rt.x_perm_scale), _decode4(s["wgu"], s["wgu_scale"]), rt.split_sizes, rt.group_offsets, s["cap"])
    G, U = gu[:, :F], gu[:, F:]
    h = rt.prob_perm[:, None] * (G / (1 + torch.exp(-G))) * U
    h = _decode8(*_quant8(h))
    y = _grouped(h, _decode4(s["wd"], s["wd_scale"]), rt.split_sizes, rt.group_offsets, s["cap"]).to(torch.bfloat16)
    return y[rt.perm_pos.long()].float().sum(1).to(torch.bfloat16)


def _run_plain(s):
    c = s["c"]
    op = c["op"]
    if op == "topk":
        return _topk(c, s["logits"], s["bias"])
    if op == "topk_bwd":
        return _topk_bwd(c, s["logits"], s["idx"], s["d_prob"])
    if op == "quant":
        x, out = s["w"].float(), {}
        if c["orient"] != "col":
            out["row"] = _decode4(*_quant4(x)).to(torch.bfloat16)
        if c["orient"] != "row":
            xt = torch.nn.functional.pad(x.transpose(1, 2), (0, -c["R"] % 32)).contiguous()
            out["col"] = _decode4(*_quant4(xt)).to(torch.bfloat16)
        return out
    if op == "gemm":
        a = _decode8(s["a"], s["a_scale"]) if c["a"] == "mxfp8" else _decode4(s["a"], s["a_scale"])
        return _grouped(a, _decode4(s["w"], s["w_scale"]), s["sizes"], s["offsets"], s["cap"]).to(torch.bfloat16)
    return _mlp(s)


def _run_own(s):
    m, c = _lib(), s["c"]
    op = c["op"]
    if op == "topk":
        return m.moe_route_topk(s["logits"], c["k"], score=c["score"], bias=s["bias"], num_groups=c["groups"],
                                topk_groups=c["topk_groups"], group_topn=c["topn"], renormalize=c["renorm"], scale=c["scale"])
    if op == "topk_bwd":
        return m.moe_route_topk_bwd(s["logits"], s["idx"], s["d_prob"], score=c["score"], renormalize=c["renorm"],
                                    scale=c["scale"])
    if op == "quant":
        rc, rs, cc, cs = m.mxfp4_quantize(s["w"], c["orient"])
        out = {}
        if rc is not None:
            out["row"] = m.mxfp4_dequantize(rc, rs)
        if cc is not None:
            out["col"] = m.mxfp4_dequantize(cc, cs)
        return out
    if op == "gemm":
        return m.mxfp4_grouped_gemm(s["a"], s["a_scale"], s["w"], s["w_scale"], s["sizes"], s["offsets"])
    f = m.grouped_mlp_fwd_mxfp4(s["rt"], s["wgu"], s["wd"], s["wgu_scale"], s["wd_scale"])
    return m.unpermute_combine(f.y_perm, s["rt"].perm_pos)


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    """Inputs read once and outputs written once; two operations for each product and sum of the matrix products."""
    c = case
    op = c["op"]
    if op in ("topk", "topk_bwd"):
        b = 2 if c["dtype"] == "bf16" else 4
        n = c["T"] * c["E"]
        return {"bytes": n * b * (2 if op == "topk_bwd" else 1) + c["T"] * c["k"] * 8, "flops": 10 * n}
    if op == "quant":
        n = c["batch"] * c["R"] * c["C"]
        forms = 2 if c["orient"] == "both" else 1
        return {"bytes": 2 * n + forms * (n // 2 + n // 32) + forms * 2 * n, "flops": 4 * n * forms}
    # experts without a row need no weight: at most as many experts as rows are read
    if op == "gemm":
        E = min(c["E"], c["rows"])
        a = c["rows"] * c["K"] * (33 if c["a"] == "mxfp8" else 17) // (32 if c["a"] == "mxfp8" else 32)
        return {"bytes": E * c["N"] * c["K"] * 17 // 32 + a + 2 * c["rows"] * c["N"], "flops": 2 * c["rows"] * c["N"] * c["K"]}
    rows = c["T"] * c["k"]
    E = min(c["E"], rows)
    w = 3 * E * c["F"] * c["H"] * 17 // 32
    return {"bytes": w + rows * c["H"] * 33 // 32 + 2 * rows * c["F"] * 33 // 32 + 4 * rows * c["H"] + 2 * c["T"] * c["H"],
            "flops": 6 * rows * c["H"] * c["F"]}


# ------------------------------------------------------------------------------ the definitions in 64 bits

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _values4(codes, scales):
    """By table, in 64 bits."""
    table = torch.tensor(_E2M1 + [-v for v in _E2M1], dtype=torch.float64, device=codes.device)
    v = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device=codes.device)
    v[..., 0::2] = table[(codes & 15).int()]
    v[..., 1::2] = table[(codes >> 4).int()]
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _values8(codes, scales):
    n = torch.arange(256, device=codes.device)
    e, m = (n >> 3) & 15, (n & 7).double()
    mag = torch.where(e == 0, m / 512, (1 + m / 8) * torch.exp2(e.double() - 7))
    return torch.where(n >= 128, -mag, mag)[codes.int()] * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _nearest(x, values, emax):
    """Each block's scale from its largest magnitude, each value to the nearest representable one (ties to the one of
    even place in the table), in 64 bits; returns the values they stand for."""
    table = torch.tensor(values, dtype=torch.float64, device=x.device)
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax))))
    e = torch.where(torch.exp2(e) > amax, e - 1, torch.where(torch.exp2(e + 1) <= amax, e + 1, e)) - emax
    scale = torch.exp2(torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127))
    a = (b / scale).abs().clamp(max=values[-1])
    hi = torch.searchsorted(table, a).clamp(max=len(values) - 1)
    lo = (hi - 1).clamp(min=0)
    mid = (table[lo] + table[hi]) / 2
    pick = torch.where(a > mid, hi, torch.where(a < mid, lo, torch.where(hi % 2 == 0, hi, lo)))
    return (torch.copysign(table[pick], b) * scale).reshape(x.shape)


def _e4m3_table():
    return [m / 512 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]


def _rows(a, wc, ws, sizes, offsets):
    """Each group's rows times its own weight, group after group, in 64 bits."""
    out = torch.zeros(a.shape[0], wc.shape[1], dtype=torch.float64, device=a.device)
    for e, (n, o) in enumerate(zip(sizes.tolist(), offsets.tolist())):
        if n:
            out[o:o + n] = a[o:o + n] @ _values4(wc[e], ws[e]).T
    return out


def _first(v):
    """The lowest place of each row's largest value."""
    n = torch.arange(v.shape[1], device=v.device)
    return torch.where(v == v.amax(1, keepdim=True), n, torch.full_like(n, v.shape[1])).amin(1)


def _best(c, key, p, live):
    """One expert after the other: the largest key among the groups that are left, masked experts after all others."""
    T, E, G = c["T"], c["E"], c["groups"]
    none = torch.full_like(key, -math.inf)
    low = torch.full_like(key, -1e300)
    pool = torch.where(live, key, low)
    if c["topk_groups"] < G:
        by = p if c["topn"] == 2 and not c["bias"] else key
        by = torch.where(live, by, none).reshape(T, G, E // G)
        a = by.amax(2)
        if c["topn"] == 2:
            place = _first(by.reshape(T * G, -1)).reshape(T, G, 1)
            b = by.scatter(2, place, -math.inf).amax(2)
            a = torch.where(torch.isneginf(b), a, a + b)
        a = torch.where(torch.isneginf(a), low[:, :G], a)
        keep = torch.zeros(T, G, dtype=torch.bool, device=key.device)
        for _ in range(c["topk_groups"]):
            g = _first(a)[:, None]
            keep.scatter_(1, g, True)
            a = a.scatter(1, g, -math.inf)
        pool = torch.where(keep.repeat_interleave(E // G, 1), pool, none)
    idx = []
    for _ in range(c["k"]):
        i = _first(pool)[:, None]
        idx.append(i)
        pool = pool.scatter(1, i, -math.inf)
    return torch.cat(idx, 1).to(torch.int32)


def exact(case, seed):
    s = prepare(case, seed)
    c, op = s["c"], s["c"]["op"]
    if op in ("topk", "topk_bwd"):
        l = s["logits"].double()
        live = ~torch.isneginf(l)
        if c["score"] == "sigmoid":
            p = torch.sigmoid(l)
        else:
            p = torch.nan_to_num(torch.softmax(l, 1), nan=0.0)
    if op == "topk":
        idx = _best(c, l if s["bias"] is None else p + s["bias"].double(), p, live)
        w = p.gather(1, idx.long())
        if c["renorm"]:
            w = torch.nan_to_num(w / w.sum(1, keepdim=True), nan=0.0)
        return idx, w * c["scale"]
    if op == "topk_bwd":
        # the Jacobian of the weights, written out: dw_i/dl_e for every slot i and expert e
        T, E, k = c["T"], c["E"], c["k"]
        i = s["idx"].long()
        d = s["d_prob"].double() * c["scale"]
        hot = torch.nn.functional.one_hot(i, E).double()
        ps = p.gather(1, i)
        if c["score"] == "sigmoid":
            J = hot * (ps * (1 - ps))[..., None]
        else:
            J = ps[..., None] * (hot - p[:, None, :])
        if c["renorm"]:
            t = ps.sum(1, keepdim=True)
            J = torch.nan_to_num(J / t[..., None] - ps[..., None] * J.sum(1, keepdim=True) / (t * t)[..., None], nan=0.0)
        return (J * d[..., None]).sum(1) * live
    if op == "quant":
        x, out = s["w"].double(), {}
        if c["orient"] != "col":
            out["row"] = _nearest(x, _E2M1, 2)
        if c["orient"] != "row":
            out["col"] = _nearest(torch.nn.functional.pad(x.transpose(1, 2), (0, -c["R"] % 32)).contiguous(), _E2M1, 2)
        return out
    if op == "gemm":
        a = _values8(s["a"], s["a_scale"]) if c["a"] == "mxfp8" else _values4(s["a"], s["a_scale"])
        return _rows(a, s["w"], s["w_scale"], s["sizes"], s["offsets"])
    rt, F = s["rt"], c["F"]
    gu = _rows(_values8(rt.x_perm, rt.x_perm_scale), s["wgu"], s["wgu_scale"], rt.split_sizes, rt.group_offsets)
    h = rt.prob_perm.double()[:, None] * gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
    y = _rows(_nearest(h, _e4m3_table(), 8), s["wd"], s["wd_scale"], rt.split_sizes, rt.group_offsets)
    return y[rt.perm_pos.long()].sum(1)
