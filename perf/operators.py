"""Operators next to the W4A16 expert layer, measured against their plain forms.

  route    router_topk: the top-k experts and weights of each token from router logits, and router_topk_grad
  gemm     grouped_gemm: y[rows of e] = a[rows of e] . w[e]^T for ragged groups of rows, and its two gradients
           (grouped_gemm_dgrad: dy . w[e]; grouped_gemm_wgrad: dy_e^T . a_e)
  mxq      mx_quant / mx_dequant: rows of FP4 (e2m1) codes with one power-of-two scale per 32 values
  mxgemm   mx_grouped_gemm: the grouped product of MXFP4 rows with MXFP4 expert weights, activations quantised in the pass

A case is a dict of plain values. `own` False computes the plain form in
elementary torch operations, True calls the package's kernels.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # one decoded token of the 384-expert layer: launch latency
        dict(name="route one token", op="route", T=1, E=384, topk=8, score="sigmoid", bias=True, renorm=True, scale=2.5,
             dtype="fp32", grad=False),
        # a training micro-batch: routing and the gradient of its logits
        dict(name="route train step", op="route", T=8192, E=384, topk=8, score="softmax", bias=False, renorm=True, scale=1.0,
             dtype="bf16", grad=True),
        # the tiny layer of the smoke test, 32 tokens x top-2: launch latency
        dict(name="gemm tiny", op="gemm", way="fwd", E=8, N=1024, K=256, rows=64, dtype="fp16", skew=False),
        # gate|up of one GPU's 48 of 384 experts, 448 decoded tokens x top-8: the weights' bytes
        dict(name="gemm decode share", op="gemm", way="fwd", E=48, N=4096, K=7168, rows=448, dtype="bf16", skew=False),
        # the same share at prefill, about 512 rows an expert, uneven
        dict(name="gemm prefill share", op="gemm", way="fwd", E=48, N=4096, K=7168, rows=24576, dtype="bf16", skew=True),
        # down projection of a TP8 shard (I = 256), 4096 tokens x top-8: short contraction, the output's bytes
        dict(name="gemm tp8 down", op="gemm", way="fwd", E=384, N=7168, K=256, rows=32768, dtype="bf16", skew=False),
        # gradients of the gate|up product in training: of its input, and of 8 experts' weights
        dict(name="gemm input gradient", op="gemm", way="dgrad", E=48, N=4096, K=7168, rows=8192, dtype="bf16", skew=True),
        dict(name="gemm weight gradient", op="gemm", way="wgrad", E=8, N=4096, K=7168, rows=16384, dtype="bf16", skew=True),
        # activations of a decode batch, and a stack of weights as they are converted at load
        dict(name="mxq decode batch", op="mxq", rows=448, K=7168, dtype="bf16"),
        dict(name="mxq weights", op="mxq", rows=98304, K=7168, dtype="bf16"),
        # the gate|up share in MXFP4: decode and prefill
        dict(name="mxgemm decode share", op="mxgemm", E=48, N=4096, K=7168, rows=448, dtype="bf16", skew=False),
        dict(name="mxgemm prefill share", op="mxgemm", E=48, N=4096, K=7168, rows=24576, dtype="bf16", skew=True),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["route", "gemm", "gemm", "gemm", "mxq", "mxgemm", "mxgemm"])
    if op == "route":
        E = _log_int(rng, 4, 512)
        return dict(op=op, T=_log_int(rng, 1, 8192), E=E, topk=rng.randint(1, min(E, 16)),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, renorm=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["bf16", "fp16", "fp32"]), grad=rng.random() < 0.5)
    if op == "mxq":
        return dict(op=op, rows=_log_int(rng, 1, 98304), K=_log_int(rng, 32, 7168, 32),
                    dtype=rng.choice(["bf16", "fp16"]))
    step = 32 if op == "mxgemm" else 8
    while True:
        c = dict(op=op, E=_log_int(rng, 1, 384), N=_log_int(rng, 64, 7168, 8), K=_log_int(rng, 64, 7168, step),
                 rows=_log_int(rng, 1, 24576), dtype=rng.choice(["bf16", "fp16"]), skew=rng.random() < 0.5)
        if c["E"] * c["N"] * c["K"] <= 48 * 4096 * 7168 and c["rows"] * c["N"] * c["K"] <= 24576 * 4096 * 7168:
            return dict(c, way=rng.choice(["fwd", "dgrad", "wgrad"])) if op == "gemm" else c


# ---- inputs ---------------------------------------------------------------------


def _randn(shape, dtype, g, scale=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=g)


def _counts(case, seed):
    """Rows of each expert: independent draws of one expert a row, evenly, or
    (skew) by a popularity that falls with the square root of the rank, with
    one expert in eight that no row goes to."""
    g = torch.Generator().manual_seed(seed)
    E = case["E"]
    p = torch.ones(E)
    if case["skew"]:
        p = torch.arange(1, E + 1).float().rsqrt()
        p[7::8] = 0.0
        p = p[torch.randperm(E, generator=g)]
    return torch.bincount(torch.multinomial(p, case["rows"], replacement=True, generator=g), minlength=E)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]
    op = case["op"]
    s = dict(case)
    if op == "route":
        T, E = case["T"], case["E"]
        s["logits"] = _randn((T, E), dt, g, 1.5)
        s["bias"] = _randn((E,), torch.float32, g, 0.05) if case["bias"] else None
        s["dw"] = _randn((T, case["topk"]), torch.float32, g) if case["grad"] else None
        return s
    if op == "mxq":
        s["x"] = _activations(case["rows"], case["K"], dt, g)
        return s
    E, N, K, rows = case["E"], case["N"], case["K"], case["rows"]
    counts = _counts(case, seed)
    s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32).cuda()
    s["cap"] = int(counts.max())     # the most rows of one expert, as the program that made the groups knows it
    if op == "mxgemm":
        s["a"] = _activations(rows, K, dt, g)
        s["wq"] = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
        s["ws"] = torch.zeros((E, N, (K // 32 + 15) // 16 * 16), dtype=torch.uint8, device="cuda")
        s["ws"][:, :, : K // 32] = torch.randint(116, 121, (E, N, K // 32), dtype=torch.uint8, device="cuda", generator=g)
        return s
    if case["way"] != "dgrad":
        s["a"] = _randn((rows, K), dt, g)
    if case["way"] != "fwd":
        s["dy"] = _randn((rows, N), dt, g)
    if case["way"] != "wgrad":
        s["w"] = _randn((E, N, K), dt, g, K ** -0.5)
    return s


def _activations(rows, K, dt, g):
    """Normal values, one feature in 64 sixteen times as large (outlier channels)."""
    x = _randn((rows, K), dt, g)
    x[:, 5::64] *= 16.0
    return x


# ---- one pass -------------------------------------------------------------------


def run(s):
    if own:
        return _own(s)
    return {"route": _plain_route, "gemm": _plain_gemm, "mxq": _plain_mxq, "mxgemm": _plain_mxgemm}[s["op"]](s)


def _own(s):
    import w4a16_int4_grouped_amd as M
    op = s["op"]
    if op == "route":
        ids, w = M.router_topk(s["logits"], s["topk"], score=s["score"], bias=s["bias"], renorm=s["renorm"], scale=s["scale"])
        if s["dw"] is None:
            return ids, w
        return ids, w, M.router_topk_grad(s["logits"], ids, s["dw"], score=s["score"], renorm=s["renorm"], scale=s["scale"])
    if op == "mxq":
        q, scales = M.mx_quant(s["x"])
        return M.mx_dequant(q, scales, dtype=s["x"].dtype)
    if op == "mxgemm":
        aq, a_scales = M.mx_quant(s["a"])
        return M.mx_grouped_gemm(aq, a_scales, s["wq"], s["ws"], s["offsets"], out_dtype=s["a"].dtype)
    if s["way"] == "fwd":
        return M.grouped_gemm(s["a"], s["w"], s["offsets"])
    if s["way"] == "dgrad":
        return M.grouped_gemm_dgrad(s["dy"], s["w"], s["offsets"])
    return M.grouped_gemm_wgrad(s["dy"], s["a"], s["offsets"])


def _plain_route(s):
    """Keys in 64 bits, where near ones decide; a stable sort gives ties to the lowest index."""
    logits = s["logits"]
    key = logits.double()
    if s["bias"] is not None:
        key = (torch.sigmoid(key) if s["score"] == "sigmoid" else torch.softmax(key, -1)) + s["bias"].double()
    ids = torch.sort(key, dim=1, descending=True, stable=True)[1][:, : s["topk"]]
    x = logits.float()
    chosen = x.gather(1, ids)
    if s["score"] == "softmax":
        score = torch.softmax(chosen if s["renorm"] else x, -1)
        w = score if s["renorm"] else score.gather(1, ids)
    else:
        w = torch.sigmoid(chosen)
        if s["renorm"]:
            w = w / w.sum(1, keepdim=True)
    out = (ids.to(torch.int32), w * s["scale"])
    if s["dw"] is None:
        return out
    dw = s["dw"] * s["scale"]
    if s["score"] == "softmax" and not s["renorm"]:
        dl = torch.zeros_like(x).scatter_(1, ids, dw) - (dw * w).sum(1, keepdim=True)
        return out + ((dl * score).to(logits.dtype),)
    if s["renorm"]:
        d = w * (dw - (dw * w).sum(1, keepdim=True))
    else:
        d = dw * w
    if s["score"] == "sigmoid":
        d = d * torch.sigmoid(-chosen)
    return out + (torch.zeros_like(x).scatter_(1, ids, d).to(logits.dtype),)


def _padded(x, offsets, cap):
    """FP32 [E, cap, width]: each expert's rows, zeros behind its last."""
    at = offsets[:-1, None].long() + torch.arange(cap, device=x.device)
    live = at < offsets[1:, None]
    return torch.where(live[:, :, None], x.float()[at.clamp(max=x.shape[0] - 1)], 0.0)


def _unpadded(y, offsets, rows):
    """The rows of FP32 [E, cap, width], one after another."""
    r = torch.arange(rows, device=y.device)
    e = torch.searchsorted(offsets[1:].long(), r, right=True)
    return y[e, r - offsets[e]]


def _plain_gemm(s):
    off, cap = s["offsets"], s["cap"]
    dt = _DT[s["dtype"]]
    if s["way"] == "fwd":
        y = torch.bmm(_padded(s["a"], off, cap), s["w"].float().transpose(1, 2).contiguous())
        return _unpadded(y, off, s["rows"]).to(dt)
    dy = _padded(s["dy"], off, cap)
    if s["way"] == "dgrad":
        return _unpadded(torch.bmm(dy, s["w"].float()), off, s["rows"]).to(dt)
    return torch.bmm(dy.transpose(1, 2).contiguous(), _padded(s["a"], off, cap)).to(dt)


def _plain_round_mx(x):
    """FP32 rows rounded to e2m1 values times a power of two per 32: the scale's exponent is that of the block's
    largest magnitude less 2 (the exponent of e2m1's largest, 6), and larger values than 6 become 6."""
    b = x.reshape(x.shape[0], -1, 32)
    e = torch.frexp(b.abs().amax(2, keepdim=True))[1] - 3
    v = b * _power(-e)
    m = v.abs()
    code = ((m > 0.25).int() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    return (_e2m1(x.device)[code] * _power(e) * torch.where(v < 0, -1.0, 1.0)).reshape(x.shape)


def _e2m1(device):
    return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=device)


def _power(e):
    """FP32 2^e, exactly, for -126 <= e <= 127."""
    return ((e + 127) << 23).view(torch.float32)


def _plain_mxq(s):
    return _plain_round_mx(s["x"].float()).to(s["x"].dtype)


def _plain_mx_values(q, scales):
    """FP32 values of packed codes, low nibble first, and their biased exponents."""
    code = torch.stack([q & 15, q >> 4], -1).flatten(-2).int()
    v = _e2m1(q.device)[code & 7] * torch.where(code > 7, -1.0, 1.0)
    v = v.reshape(*q.shape[:-1], -1, 32) * _power(scales[..., : q.shape[-1] // 16].int() - 127)[..., None]
    return v.flatten(-2)


def _plain_mxgemm(s):
    a = _plain_round_mx(s["a"].float())
    w = _plain_mx_values(s["wq"], s["ws"])
    y = torch.bmm(_padded(a, s["offsets"], s["cap"]), w.transpose(1, 2).contiguous())
    return _unpadded(y, s["offsets"], s["rows"]).to(s["a"].dtype)


# ---- what a pass cannot do without ----------------------------------------------


def work(case):
    op, b = case["op"], _SIZE[case["dtype"]]
    if op == "route":
        T, E, k = case["T"], case["E"], case["topk"]
        n = T * E * b + T * k * 8 + (E * 4 if case["bias"] else 0)
        if case["grad"]:
            n += T * E * b + T * k * 4
        return {"bytes": n, "flops": T * E * (8 if case["grad"] else 4)}
    if op == "mxq":
        n = case["rows"] * case["K"]
        return {"bytes": 2 * n * b, "flops": 4 * n}
    E, N, K, rows = case["E"], case["N"], case["K"], case["rows"]
    live = E - E // 8 if case["skew"] else E
    live = live * (1.0 - (1.0 - 1.0 / live) ** rows)     # experts that some row goes to, about
    if op == "mxgemm":
        n = rows * K * b + live * N * K * 17 / 32 + rows * N * b
    elif case["way"] == "wgrad":
        n = rows * (K + N) * b + E * N * K * b
    else:
        n = rows * (K + N) * b + live * N * K * b
    return {"bytes": int(n), "flops": 2 * rows * N * K}


# ---- the definitions in 64 bits ---------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s)
    if case["op"] == "mxq":
        return _exact_mx(s["x"])
    ends = s["offsets"].tolist()
    groups = [(e, ends[e], ends[e + 1]) for e in range(case["E"]) if ends[e + 1] > ends[e]]
    N, K, rows = case["N"], case["K"], case["rows"]
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    if case["op"] == "mxgemm":
        a, y = _exact_mx(s["a"]), new(rows, N)
        table = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12, 0, -1, -2, -3, -4, -6, -8, -12], dtype=torch.float64, device="cuda") / 2
        for e, lo, hi in groups:
            q = s["wq"][e].int()
            w = new(N, K)
            w[:, 0::2], w[:, 1::2] = table[q % 16], table[q // 16]
            w *= (2.0 ** (s["ws"][e, :, : K // 32].double() - 127.0)).repeat_interleave(32, 1)
            y[lo:hi] = a[lo:hi] @ w.T
        return y
    if case["way"] == "wgrad":
        d = new(case["E"], N, K)
        for e, lo, hi in groups:
            d[e] = s["dy"][lo:hi].double().T @ s["a"][lo:hi].double()
        return d
    y = new(rows, N if case["way"] == "fwd" else K)
    for e, lo, hi in groups:
        w = s["w"][e].double()
        y[lo:hi] = s["a"][lo:hi].double() @ w.T if case["way"] == "fwd" else s["dy"][lo:hi].double() @ w
    return y


def _exact_mx(x):
    """The nearest of the sixteen e2m1 values (the even code of two as near) under each block's scale."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    for lo in range(0, x.shape[0], 4096):
        b = x[lo:lo + 4096].double().reshape(-1, 32)
        top = b.abs().amax(1, keepdim=True)
        step = 2.0 ** (torch.floor(torch.log2(torch.where(top > 0, top, 1.0))) - 2.0)
        v = (b / step).abs()
        up = torch.bucketize(v, grid).clamp(max=7)       # grid[up - 1] < v <= grid[up]
        dn = (up - 1).clamp(min=0)
        far_up, far_dn = (grid[up] - v).abs(), (v - grid[dn]).abs()
        code = torch.where((far_up < far_dn) | ((far_up == far_dn) & (up % 2 == 0)), up, dn)
        out[lo:lo + 4096] = (grid[code] * torch.sign(b) * step).reshape(-1, x.shape[1])
    return out


def _exact_route(s):
    x = s["logits"].double()
    T, k = x.shape[0], s["topk"]
    p = torch.exp(x - x.max(1, keepdim=True)[0])
    p = p / p.sum(1, keepdim=True) if s["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-x))
    key = x.clone() if s["bias"] is None else p + s["bias"].double()
    ids = torch.empty((T, k), dtype=torch.int64, device=x.device)
    place = torch.arange(x.shape[1], device=x.device)
    for j in range(k):
        best = key.max(1, keepdim=True)[0]
        ids[:, j] = torch.where(key == best, place, x.shape[1]).min(1)[0]
        key.scatter_(1, ids[:, j:j + 1], -math.inf)
    part = p.gather(1, ids)
    total = part.sum(1, keepdim=True) if s["renorm"] else torch.ones_like(part[:, :1])
    w = s["scale"] * part / total
    if s["dw"] is None:
        return ids, w
    dw = s["scale"] * s["dw"].double()
    ds = dw / total                                     # gradient of the chosen scores
    if s["renorm"]:
        ds = ds - (dw * part).sum(1, keepdim=True) / total ** 2
    ds = torch.zeros_like(x).scatter_(1, ids, ds)
    if s["score"] == "sigmoid":
        return ids, w, ds * p * (1.0 - p)
    return ids, w, p * (ds - (ds * p).sum(1, keepdim=True))
