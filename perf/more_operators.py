"""Operators of a training step around the experts' products, measured against their plain forms.

  balance  router_balance / router_balance_grad: rows per expert and the load-balance loss of each sequence, and the
           gradient of the router logits
  combine  combine / combine_grad: a token's weighted sum of its experts' rows, the gradients of the rows (0 in a
           group's padding) and of the weights; without weights the gradient of a permutation
  mx8      mx8_quant / mx8_dequant: checkpoints of activations in 8 bits (integers with one power-of-two scale per 32
           values), read back as they are or as the rows of a routing
  swiglu   swiglu_save / swiglu_grad: SwiGLU that keeps its input as such a checkpoint, and its gradient, which computes
           the output again; or the gradient from the input itself
  linear   grouped_linear: the experts' product with bias, SwiGLU and residual in its epilogue; grouped_bias_grad: the
           gradient of the biases

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
        # the smoke test's tiny layer: launch latency
        dict(name="balance tiny", op="balance", T=32, E=8, topk=2, S=1, score="softmax", masked=False, grad=False,
             add=False, dtype="fp32"),
        # a micro-batch of the 384-expert router: a loss for each of 13 uneven sequences, experts masked for some
        # tokens, the gradient added to that of the experts' weights
        dict(name="balance train step", op="balance", T=16411, E=384, topk=8, S=13, score="sigmoid", masked=True,
             grad=True, add=True, dtype="bf16"),
        # one decoded token of the 384-expert layer
        dict(name="combine one token", op="combine", T=1, E=384, topk=8, H=7168, block=16, weighted=True, drop=0.0,
             grad=False, dtype="bf16"),
        # a training micro-batch, forward and backward: 65536 rows and each expert's padding
        dict(name="combine train step", op="combine", T=8192, E=384, topk=8, H=7168, block=128, weighted=True, drop=0.0,
             grad=True, dtype="bf16"),
        # activations of a decode batch
        dict(name="mx8 decode batch", op="mx8", T=448, E=0, topk=0, K=7168, dtype="bf16"),
        # the layer's input kept for the backward pass, read back as the rows of its routing
        dict(name="mx8 routed rows", op="mx8", T=8192, E=384, topk=8, K=7168, dtype="bf16"),
        # gate | up rows of a decode batch
        dict(name="swiglu decode rows", op="swiglu", rows=3584, I=2048, way="save", dtype="bf16"),
        # gate | up rows of a training micro-batch: forward with a checkpoint, backward from it
        dict(name="swiglu train step", op="swiglu", rows=65536, I=2048, way="both", dtype="bf16"),
        # gate | up with SwiGLU of one GPU's 48 of 384 experts, 448 decoded tokens x top-8: the weights' bytes
        dict(name="linear decode share", op="linear", way="fwd", E=48, N=4096, K=7168, rows=448, bias=False, act="swiglu",
             residual=False, dtype="bf16", skew=False),
        # the same share at prefill with biases, about 512 rows an expert, uneven
        dict(name="linear prefill share", op="linear", way="fwd", E=48, N=4096, K=7168, rows=24576, bias=True, act="swiglu",
             residual=False, dtype="bf16", skew=True),
        # down projection of a TP8 shard (I = 256) onto a residual, 4096 tokens x top-8: the output's bytes
        dict(name="linear tp8 down", op="linear", way="fwd", E=384, N=7168, K=256, rows=32768, bias=True, act="none",
             residual=True, dtype="fp16", skew=False),
        # gradient of the gate | up biases of the prefill share
        dict(name="linear bias gradient", op="linear", way="bgrad", E=48, N=4096, K=0, rows=24576, bias=True, act="none",
             residual=False, dtype="bf16", skew=True),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["balance", "combine", "mx8", "swiglu", "linear"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    if op == "balance":
        E = _log_int(rng, 4, 512)
        return dict(op=op, T=_log_int(rng, 1, 12000), E=E, topk=rng.randint(1, min(E, 16)), S=_log_int(rng, 1, 64),
                    score=rng.choice(["softmax", "sigmoid"]), masked=rng.random() < 0.5, grad=rng.random() < 0.6,
                    add=rng.random() < 0.5, dtype=dtype)
    if op == "combine":
        E = _log_int(rng, 4, 512)
        return dict(op=op, T=_log_int(rng, 1, 4000), E=E, topk=rng.randint(1, min(E, 10)), H=_log_int(rng, 64, 7168, 8),
                    block=rng.choice([1, 16, 128]), weighted=rng.random() < 0.7, drop=rng.choice([0.0, 0.5, 0.875]),
                    grad=rng.random() < 0.6, dtype=dtype)
    if op == "mx8":
        E = rng.choice([0, 8, 48, 384])
        return dict(op=op, T=_log_int(rng, 1, 4000 if E else 24576), E=E, topk=rng.randint(1, 8) if E else 0,
                    K=_log_int(rng, 32, 7168, 8), dtype=dtype)
    if op == "swiglu":
        return dict(op=op, rows=_log_int(rng, 1, 32768), I=_log_int(rng, 32, 2048, 8),
                    way=rng.choice(["save", "both", "grad"]), dtype=dtype)
    while True:
        act = rng.choice(["none", "swiglu"])
        c = dict(op=op, way="fwd" if rng.random() < 0.75 else "bgrad", E=_log_int(rng, 1, 384),
                 N=_log_int(rng, 64, 7168, 16 if act == "swiglu" else 8), K=_log_int(rng, 64, 7168, 8),
                 rows=_log_int(rng, 1, 24576), bias=rng.random() < 0.7, act=act, residual=rng.random() < 0.4,
                 dtype=rng.choice(["bf16", "fp16"]), skew=rng.random() < 0.5)
        if c["E"] * c["N"] * c["K"] <= 48 * 4096 * 7168 and c["rows"] * c["N"] * c["K"] <= 24576 * 4096 * 7168:
            return c


# ---- inputs ---------------------------------------------------------------------


def _randn(shape, dtype, g, scale=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=g)


def _uniform(shape, g):
    return torch.empty(shape, dtype=torch.float32, device="cuda").uniform_(1e-6, 1.0, generator=g)


def _routing(s, T, E, topk, block, drop, g):
    """Each token's distinct experts as rows grouped by expert, groups padded
    to multiples of `block`, in buffers for R rows, as many as any routing may
    need: slots [T, topk] (-1 for the share `drop` of the experts, which lie
    elsewhere), row_src [R] (t * topk + j, or T * topk in the padding and
    behind the last group) and offsets."""
    ids = torch.topk(_uniform((T, E), g), topk, dim=1)[1]
    here = E - int(E * drop)
    e = torch.where(ids < here, ids, here).flatten()
    order = torch.sort(e, stable=True)[1]
    counts = torch.bincount(e, minlength=here + 1)[:here]
    starts = torch.cat([counts.new_zeros(1), ((counts + block - 1) // block * block).cumsum(0)])
    s["R"], live = T * topk + here * (block - 1), int(counts.sum())
    before = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    kept = order[:live]
    slot = starts[e[kept]] + torch.arange(live, device="cuda") - before[e[kept]]
    s["slots"] = torch.full((T * topk,), -1, dtype=torch.int32, device="cuda")
    s["slots"][kept] = slot.int()
    s["slots"] = s["slots"].view(T, topk)
    s["row_src"] = torch.full((s["R"],), T * topk, dtype=torch.int32, device="cuda")
    s["row_src"][slot] = kept.int()
    s["offsets"] = starts.int()


def _counts(case, seed):
    """Rows of each expert: independent draws of one expert a row, evenly, or
    (skew) by a popularity that falls with the square root of the rank, with
    one expert in eight that no row goes to."""
    g = torch.Generator().manual_seed(seed)
    p = torch.ones(case["E"])
    if case["skew"]:
        p = torch.arange(1, case["E"] + 1).float().rsqrt()
        p[7::8] = 0.0
        p = p[torch.randperm(case["E"], generator=g)]
    return torch.bincount(torch.multinomial(p, case["rows"], replacement=True, generator=g), minlength=case["E"])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]
    s = dict(case)
    if case["op"] == "balance":
        T, E, S = case["T"], case["E"], case["S"]
        s["logits"] = _randn((T, E), dt, g, 1.5) + _randn((E,), torch.float32, g, 0.5).to(dt)   # some experts are popular
        if case["masked"]:
            s["logits"].masked_fill_(_uniform((T, E), g) < 0.1, -math.inf)
            s["logits"][96::97] = -math.inf       # padding tokens
        top = torch.topk(s["logits"].float(), case["topk"], dim=1)
        s["ids"] = torch.where(top[0] > -math.inf, top[1], -1).int()
        cuts = torch.randint(0, T + 1, (S - 1,), generator=torch.Generator().manual_seed(seed)).sort()[0].tolist()
        s["ends"] = [0] + cuts + [T]
        s["offsets"] = torch.tensor(s["ends"], dtype=torch.int32, device="cuda") if S > 1 else None
        # a gradient per logit is d_loss * S / (T * E), about: scaled as mixed-precision training does, 16 bits hold it
        s["d_loss"] = _randn((S,), torch.float32, g, 0.01 * T * E / S) if case["grad"] else None
        s["add"] = _randn((T, E), dt, g, 0.01) if case["add"] else None
        return s
    if case["op"] == "combine":
        T, k, H = case["T"], case["topk"], case["H"]
        _routing(s, T, case["E"], k, case["block"], case["drop"], g)
        s["y"] = _randn((s["R"], H), dt, g)
        s["w"] = _uniform((T, k), g) if case["weighted"] else None
        s["d_out"] = _randn((T, H), dt, g) if case["grad"] else None
        s["d_y"] = torch.zeros_like(s["y"]) if case["grad"] else None     # rows behind the last group stay as they are
        return s
    if case["op"] == "mx8":
        s["x"] = _activations(case["T"], case["K"], dt, g)
        if case["E"]:
            _routing(s, case["T"], case["E"], case["topk"], 16, 0.0, g)
            s["out"] = torch.zeros((s["R"], case["K"]), dtype=dt, device="cuda")
        return s
    if case["op"] == "linear":
        E, N, K, rows = case["E"], case["N"], case["K"], case["rows"]
        counts = _counts(case, seed)
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32).cuda()
        s["cap"] = int(counts.max())     # the most rows of one expert, as the program that made the groups knows it
        if case["way"] == "bgrad":
            s["dy"] = _randn((rows, N), dt, g)
            return s
        s["a"] = _randn((rows, K), dt, g)
        s["w"] = _randn((E, N, K), dt, g, K ** -0.5)
        s["bias"] = _randn((E, N), dt, g, 0.5) if case["bias"] else None
        s["residual"] = _randn((rows, N // 2 if case["act"] == "swiglu" else N), dt, g) if case["residual"] else None
        return s
    rows, I = case["rows"], case["I"]
    s["h"] = _activations(rows, 2 * I, dt, g)
    s["d_a"] = _randn((rows, I), dt, g) if case["way"] != "save" else None
    return s


def _activations(rows, K, dt, g):
    """Normal values, one feature in 64 eight times as large (outlier channels)."""
    x = _randn((rows, K), dt, g)
    x[:, 5::64] *= 8.0
    return x


# ---- one pass -------------------------------------------------------------------


def run(s):
    if own:
        return _own(s)
    return {"balance": _plain_balance, "combine": _plain_combine, "mx8": _plain_mx8, "swiglu": _plain_swiglu,
            "linear": _plain_linear}[s["op"]](s)


def _own(s):
    import w4a16_int4_grouped_amd as M
    op = s["op"]
    if op == "balance":
        loss, counts = M.router_balance(s["logits"], s["ids"], score=s["score"], offsets=s["offsets"])
        if s["d_loss"] is None:
            return loss, counts
        return loss, counts, M.router_balance_grad(s["logits"], counts, s["d_loss"], s["topk"], score=s["score"],
                                                   offsets=s["offsets"], add=s["add"])
    if op == "combine":
        out = M.combine(s["y"], s["slots"], s["w"])
        if s["d_out"] is None:
            return out
        if s["w"] is None:
            return out, M.combine_grad(s["d_out"], s["slots"], row_src=s["row_src"], offsets=s["offsets"],
                                       out=(s["d_y"], None))[0]
        d_w = torch.empty_like(s["w"])
        return (out,) + tuple(M.combine_grad(s["d_out"], s["slots"], y=s["y"], w=s["w"], row_src=s["row_src"],
                                             offsets=s["offsets"], out=(s["d_y"], d_w)))
    if op == "mx8":
        q, scales = M.mx8_quant(s["x"])
        if not s["E"]:
            return M.mx8_dequant(q, scales, dtype=s["x"].dtype)
        return M.mx8_dequant(q, scales, row_src=s["row_src"], topk=s["topk"], offsets=s["offsets"], out=s["out"])
    if op == "linear":
        if s["way"] == "bgrad":
            return M.grouped_bias_grad(s["dy"], s["offsets"])
        return M.grouped_linear(s["a"], s["w"], s["offsets"], bias=s["bias"], act=s["act"], residual=s["residual"])
    h = s["h"]
    if s["way"] == "grad":
        return M.swiglu_grad(h, s["d_a"])
    a, q, scales = M.swiglu_save(h)
    if s["way"] == "both":
        return (a,) + tuple(M.swiglu_grad(q, s["d_a"], scales=scales))
    v = M.mx8_dequant(q.view(2 * s["rows"], s["I"]), scales.view(2 * s["rows"], -1), dtype=h.dtype)
    return a, v.view(s["rows"], 2 * s["I"])


def _plain_scores(logits, score):
    """FP32 scores that sum to 1 in a row (0 in a row without an expert), and 1 - sigmoid, or 1."""
    x = logits.float()
    if score == "sigmoid":
        v = 1.0 / (1.0 + torch.exp(-x))
        rest = 1.0 / (1.0 + torch.exp(x))
    else:
        top = x.max(1, keepdim=True)[0]
        v, rest = torch.exp(x - torch.where(top > -math.inf, top, 0.0)), 1.0
    total = v.sum(1, keepdim=True)
    return v / torch.where(total > 0, total, 1.0), rest


def _plain_balance(s):
    T, E, S, k = s["T"], s["E"], s["S"], s["topk"]
    p, rest = _plain_scores(s["logits"], s["score"])
    seq = torch.zeros(T, dtype=torch.int64, device=p.device)
    if s["offsets"] is not None:
        seq = torch.searchsorted(s["offsets"][1:].long(), torch.arange(T, device=p.device), right=True)
    ids = s["ids"].long()
    place = torch.where(ids >= 0, seq[:, None] * E + ids, S * E).flatten()
    counts = torch.zeros(S * E + 1, dtype=torch.int32, device=p.device)
    counts = counts.scatter_add_(0, place, torch.ones_like(place, dtype=torch.int32))[:-1].view(S, E)
    sums = torch.stack([p[lo:hi].sum(0) for lo, hi in zip(s["ends"], s["ends"][1:])])
    n = torch.bincount(seq, minlength=S)[:S].float()
    scale = E / (k * torch.where(n > 0, n * n, 1.0))
    loss = scale * (counts.float() * sums).sum(1)
    if s["d_loss"] is None:
        return loss, counts
    c = ((s["d_loss"] * scale)[:, None] * counts.float())[seq]
    d = p * (c - (c * p).sum(1, keepdim=True)) * rest
    if s["add"] is not None:
        d = d + s["add"].float()
    return loss, counts, d.to(s["logits"].dtype)


def _plain_combine(s):
    T, k, H, dt = s["T"], s["topk"], s["H"], s["y"].dtype
    live = s["slots"] >= 0
    slot = s["slots"].long().clamp(min=0)
    rows = torch.where(live[:, :, None], s["y"].float()[slot], 0.0)
    w = torch.ones(T, k, device=live.device) if s["w"] is None else s["w"]
    out = (rows * w[:, :, None]).sum(1).to(dt)
    if s["d_out"] is None:
        return out
    d = s["d_out"].float()
    src = s["row_src"].long()
    own_row = src < T * k
    src = src.clamp(max=T * k - 1)
    dy = torch.where(own_row[:, None], d[src // k] * w.flatten()[src][:, None], 0.0).to(dt)
    if s["w"] is None:
        return out, dy
    return out, dy, (rows * d[:, None, :]).sum(2)


def _power(e):
    """FP32 2^e, exactly, for -126 <= e <= 127."""
    return ((e + 127) << 23).view(torch.float32)


def _plain_round8(x):
    """FP32 rows as integers from -127 to 127 times 2^(e - 6) per 32 values, 2^e the power of two at or below the
    block's largest magnitude."""
    K = x.shape[1]
    b = torch.nn.functional.pad(x, (0, -K % 32)).view(x.shape[0], -1, 32)
    e = (torch.frexp(b.abs().amax(2, keepdim=True))[1] - 1).clamp(-120, 120)
    v = torch.round(b * _power(6 - e)).clamp(-127.0, 127.0) * _power(e - 6)
    return v.view(x.shape[0], -1)[:, :K]


def _plain_mx8(s):
    v = _plain_round8(s["x"].float())
    if s["E"]:
        src, n = s["row_src"].long(), s["T"] * s["topk"]
        v = torch.where((src < n)[:, None], v[src.clamp(max=n - 1) // s["topk"]], 0.0)
    return v.to(s["x"].dtype)


def _plain_swiglu(s):
    h, I, dt = s["h"].float(), s["I"], s["h"].dtype

    def act(h):
        g, u = h[:, :I], h[:, I:]
        sig = 1.0 / (1.0 + torch.exp(-g))
        return g, u, sig, (g * sig * u).to(dt)

    out = ()
    if s["way"] != "grad":
        out = (act(h)[3],)
        h = _plain_round8(h.reshape(-1, I)).reshape(-1, 2 * I)
        if s["way"] == "save":
            return out + (h.to(dt),)
    g, u, sig, a = act(h)
    d = s["d_a"].float()
    dh = torch.cat([d * u * sig * (1.0 + g * (1.0 - sig)), d * g * sig], 1)
    return out + (dh.to(dt), a)


def _padded(x, offsets, cap):
    """FP32 [E, cap, width]: each expert's rows, zeros behind its last."""
    at = offsets[:-1, None].long() + torch.arange(cap, device=x.device)
    live = at < offsets[1:, None]
    return torch.where(live[:, :, None], x.float()[at.clamp(max=x.shape[0] - 1)], 0.0)


def _plain_linear(s):
    off, cap, dt = s["offsets"], s["cap"], _DT[s["dtype"]]
    if s["way"] == "bgrad":
        return _padded(s["dy"], off, cap).sum(1).to(dt)
    z = torch.bmm(_padded(s["a"], off, cap), s["w"].float().transpose(1, 2).contiguous())
    if s["bias"] is not None:
        z = z + s["bias"].float()[:, None, :]
    r = torch.arange(s["rows"], device=z.device)
    e = torch.searchsorted(off[1:].long(), r, right=True)
    y = z[e, r - off[e]]
    if s["act"] == "swiglu":
        g, u = y[:, : s["N"] // 2], y[:, s["N"] // 2:]
        y = g / (1.0 + torch.exp(-g)) * u
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(dt)


# ---- what a pass cannot do without ----------------------------------------------


def work(case):
    op, b = case["op"], _SIZE[case["dtype"]]
    if op == "balance":
        T, E, k, S = case["T"], case["E"], case["topk"], case["S"]
        n = T * E * b + T * k * 4 + S * (E + 1) * 4
        if case["grad"]:
            n += T * E * b * (2 if case["add"] else 1) + S * 4
        return {"bytes": n, "flops": T * E * (12 if case["grad"] else 5)}
    if op == "combine":
        T, k, H = case["T"], case["topk"], case["H"]
        here = case["E"] - int(case["E"] * case["drop"])
        live = T * k * here / case["E"]                        # rows here, about
        n = live * H * b + T * H * b + T * k * (8 if case["weighted"] else 4)
        f = 2 * live * H
        if case["grad"]:
            pad = min(here, live) * (case["block"] - 1) / 2    # half a block an expert with rows, about
            n += T * H * b + (live + pad) * H * b + (live + pad) * 4 + (T * k * 4 if case["weighted"] else 0)
            f += (4 if case["weighted"] else 1) * live * H
        return {"bytes": int(n), "flops": int(f)}
    if op == "mx8":
        out = case["T"] * max(case["topk"], 1) + min(case["E"], case["T"] * case["topk"]) * 7.5
        return {"bytes": int((case["T"] + out) * case["K"] * b), "flops": int((4 * case["T"] + out) * case["K"])}
    if op == "linear":
        E, N, K, rows = case["E"], case["N"], case["K"], case["rows"]
        if case["way"] == "bgrad":
            return {"bytes": (rows + E) * N * b, "flops": rows * N}
        live = E - E // 8 if case["skew"] else E
        live = live * (1.0 - (1.0 - 1.0 / live) ** rows)     # experts that some row goes to, about
        n_out = N // 2 if case["act"] == "swiglu" else N
        n = rows * (K + n_out * (2 if case["residual"] else 1)) * b + live * N * (K + (1 if case["bias"] else 0)) * b
        return {"bytes": int(n), "flops": 2 * rows * N * K}
    n = case["rows"] * case["I"]
    # save: h in, its values and a out; grad: h and d_a in, d_h and a out; both: h and d_a in, d_h and a twice out
    return {"bytes": n * b * {"save": 5, "grad": 6, "both": 7}[case["way"]],
            "flops": n * {"save": 20, "grad": 20, "both": 40}[case["way"]]}


# ---- the definitions in 64 bits ---------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"balance": _exact_balance, "combine": _exact_combine, "mx8": _exact_mx8, "swiglu": _exact_swiglu,
            "linear": _exact_linear}[case["op"]](s)


def _exact_balance(s):
    """Row by row of each sequence: f_e = rows of e / (n k), P_e = the mean score, loss = E sum_e f_e P_e."""
    x, E = s["logits"].double(), s["E"]
    out = torch.zeros_like(x) if s["add"] is None else s["add"].double()
    losses, counts = [], []
    for i, (lo, hi) in enumerate(zip(s["ends"], s["ends"][1:])):
        n = hi - lo
        ids = s["ids"][lo:hi]
        counts.append(torch.bincount(ids[ids >= 0].long().flatten(), minlength=E))
        if n == 0:
            losses.append(x.new_zeros(()))
            continue
        f = counts[-1].double() / (n * s["topk"])
        v = torch.sigmoid(x[lo:hi]) if s["score"] == "sigmoid" else torch.exp(x[lo:hi] - x[lo:hi].amax(1, True))
        v = torch.nan_to_num(v, nan=0.0)
        total = v.sum(1, True)
        p = torch.where(total > 0, v / total, torch.zeros_like(v))
        losses.append(E * (f * p.mean(0)).sum())
        if s["d_loss"] is not None:
            dp = s["d_loss"][i].double() * E / n * f           # of the scores
            dv = dp - (p * dp).sum(1, True)                    # of the unnormalised ones, times their sum
            out[lo:hi] += p * dv * (1.0 - v if s["score"] == "sigmoid" else 1.0)
    res = (torch.stack(losses), torch.stack(counts))
    return res if s["d_loss"] is None else res + (out,)


def _exact_combine(s):
    T, k, H = s["T"], s["topk"], s["H"]
    y, slots = s["y"], s["slots"].long()
    out = torch.zeros(T, H, dtype=torch.float64, device=y.device)
    grad = s["d_out"] is not None
    dy = torch.zeros(s["R"], H, dtype=torch.float64, device=y.device) if grad else None
    dw = torch.zeros(T, k, dtype=torch.float64, device=y.device)
    for j in range(k):
        t = (slots[:, j] >= 0).nonzero()[:, 0]
        r = slots[t, j]
        w = torch.ones(len(t), 1, dtype=torch.float64, device=y.device) if s["w"] is None else s["w"][t, j, None].double()
        v = y[r].double()
        out[t] += w * v
        if grad:
            d = s["d_out"][t].double()
            dy[r] = w * d
            dw[t, j] = (d * v).sum(1)
    if not grad:
        return out
    return (out, dy) if s["w"] is None else (out, dy, dw)


def _exact_values8(x):
    """The nearest multiple (the even one of two as near) of a 64th of the block's scale, at most 127 of them."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for c in range(0, x.shape[1], 32):
        b = x[:, c:c + 32].double()
        top = b.abs().amax(1, keepdim=True)
        # the magnitude's exponent field, less 6, as a number of its own
        step = ((torch.where(top > 0, top, 1.0).view(torch.int64) >> 52) - 6 << 52).view(torch.float64)
        out[:, c:c + 32] = torch.clamp(torch.round(b / step), -127, 127) * step
    return out


def _exact_mx8(s):
    v = _exact_values8(s["x"])
    if not s["E"]:
        return v
    out = torch.zeros(s["R"], s["K"], dtype=torch.float64, device=v.device)
    for j in range(s["topk"]):
        out[s["slots"][:, j].long()] = v
    return out


def _exact_swiglu(s):
    I, h = s["I"], s["h"].double()
    g, u = h[:, :I], h[:, I:]
    res = [] if s["way"] == "grad" else [g * torch.sigmoid(g) * u]
    if s["way"] != "grad":
        g, u = _exact_values8(s["h"][:, :I]), _exact_values8(s["h"][:, I:])
        if s["way"] == "save":
            return res[0], torch.cat([g, u], 1)
    sig = torch.sigmoid(g)
    d = s["d_a"].double()
    dg = d * u * (sig + g * sig * torch.sigmoid(-g))
    res += [torch.cat([dg, d * g * sig], 1), g * sig * u]
    return tuple(res)


def _exact_linear(s):
    """Expert by expert."""
    ends, N = s["offsets"].tolist(), s["N"]
    E, rows = s["E"], s["rows"]
    if s["way"] == "bgrad":
        return torch.stack([s["dy"][lo:hi].double().sum(0) for lo, hi in zip(ends, ends[1:])])
    out = torch.zeros(rows, N // 2 if s["act"] == "swiglu" else N, dtype=torch.float64, device=s["a"].device)
    for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
        if hi == lo:
            continue
        z = s["a"][lo:hi].double() @ s["w"][e].double().T
        if s["bias"] is not None:
            z += s["bias"][e].double()
        out[lo:hi] = z if s["act"] == "none" else z[:, : N // 2] * torch.sigmoid(z[:, : N // 2]) * z[:, N // 2:]
        if s["residual"] is not None:
            out[lo:hi] += s["residual"][lo:hi].double()
    return out
