"""64-bit references of the operators of a training step (CPU)."""
import math

import torch

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def close(got, exact, slack, what):
    """|got - exact| <= slack and one rounding to got's type (half a step of the value, or of the subnormals)."""
    f = torch.finfo(got.dtype)
    tol = slack + (exact.abs() + slack) * (f.eps / 2) + f.smallest_normal * f.eps / 2
    err = (got.double().cpu() - exact).abs()
    worst = float((err / tol.clamp(min=1e-300)).max()) if err.numel() else 0.0
    print(f"  {what}: worst error {worst:.3g} of its bound", flush=True)
    assert torch.isfinite(got).all(), what
    assert (err <= tol).all(), what


# ---- balance ----------------------------------------------------------------------


def clean(logits):
    x = logits.double()
    x = torch.where(torch.isnan(x), -math.inf, x)
    return x.clamp(max=torch.finfo(torch.float32).max)


def scores(logits, score):
    """p of each row, and 1 - sigmoid (softmax: 1)."""
    x = clean(logits)
    out = x == -math.inf
    empty = out.all(1, keepdim=True)
    if score == "softmax":
        key, rest = x, torch.ones_like(x)
    else:
        key, rest = torch.nn.functional.logsigmoid(x), torch.sigmoid(-x)
    p = torch.softmax(torch.where(out & empty, 0.0, torch.where(out, -math.inf, key)), 1)
    return torch.where(out, 0.0, p), rest


def sequences(T, offsets):
    if offsets is None:
        return [(0, T)]
    off = [min(max(int(v), 0), T) for v in offsets]
    return list(zip(off, off[1:]))


def balance(logits, ids, score, offsets):
    T, E = logits.shape
    p, _ = scores(logits, score)
    loss, counts = [], []
    for lo, hi in sequences(T, offsets):
        n = hi - lo
        c = ids[lo:hi].flatten().long()
        c = torch.bincount(c[(c >= 0) & (c < E)], minlength=E)
        counts.append(c)
        loss.append(float(E * (c.double() / max(n * ids.shape[1], 1) * (p[lo:hi].sum(0) / max(n, 1))).sum()))
    return torch.tensor(loss, dtype=torch.float64), torch.stack(counts).int()


def score_error(logits):
    """Relative error of p in FP32: the rounding of l - top (half a step of it) moves e^(l - top) by as much as the step,
    exp, 1 + exp, reciprocals and products add 8 steps, the sum of E terms one for each that a lane adds and 6 lanes'
    steps."""
    x = clean(logits)
    x = torch.where(x == -math.inf, math.nan, x)
    far = torch.nan_to_num((x - torch.nan_to_num(x, nan=-math.inf).amax(1, keepdim=True)).abs(), nan=0.0, posinf=0.0)
    return (far.clamp(max=104) + logits.shape[1] / 64 + 14) * 2.0 ** -23      # (e^-104 is 0 in FP32)


def balance_grad(logits, counts, d_loss, topk, score, offsets, add=None):
    """(gradient, what FP32 may add to its error)."""
    T, E = logits.shape
    p, rest = scores(logits, score)
    c = torch.zeros_like(p)
    for s, (lo, hi) in enumerate(sequences(T, offsets)):
        if hi > lo:
            c[lo:hi] = d_loss[s].double() * E / ((hi - lo) ** 2 * topk) * counts[s].double()
    dot = (c * p).sum(1, keepdim=True)
    d = p * (c - dot) * rest
    rel = score_error(logits)
    slack = p * rest * (rel * 2 * (c.abs() + dot.abs()) + (c.abs() * p * rel).sum(1, keepdim=True)) * 2
    slack = slack + 2.0 ** -130     # products below the normal numbers
    if add is not None:
        slack = slack + (d.abs() + add.double().abs()) * 2.0 ** -24
        d = d + add.double()
    return d, slack


# ---- rows of a routing ---------------------------------------------------------------


def routing(T, E, topk, block, seed, lost=0.0, spare=0):
    """slots [T, topk], row_src [R], offsets [E + 1]: distinct experts a token,
    a share `lost` of them elsewhere, groups padded to `block`, `spare` rows
    behind the last."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand(T, E, generator=g).argsort(1)[:, :topk]
    ids = torch.where(torch.rand(T, topk, generator=g) < lost, -1, ids)
    slots = torch.full((T * topk,), -1, dtype=torch.int32)
    flat = ids.flatten()
    src, off = [], [0]
    for e in range(E):
        mine = (flat == e).nonzero()[:, 0]
        slots[mine] = (off[-1] + torch.arange(len(mine))).int()
        pad = -len(mine) % block
        src += mine.tolist() + [T * topk] * pad
        off.append(off[-1] + len(mine) + pad)
    src += [T * topk] * spare
    return slots.view(T, topk), torch.tensor(src, dtype=torch.int32), torch.tensor(off, dtype=torch.int32)


# ---- rows in 8 bits -------------------------------------------------------------------


def mx8(x):
    """(values, codes, scale bytes [rows, blocks]) of rows in 64 bits; values NaN where a block is not finite."""
    rows, K = x.shape
    b = torch.nn.functional.pad(x.double(), (0, -K % 32)).view(rows, -1, 32)
    bad = ~torch.isfinite(b).all(-1)
    b = torch.where(bad[..., None], 0.0, b)
    m = b.abs().amax(-1)
    e = (torch.frexp(m)[1] - 1).clamp(min=-127)
    e = torch.where(m == 0, -127, e)
    step = torch.ldexp(torch.ones_like(m), e - 6)[..., None]
    code = torch.round(b / step).clamp(-127, 127)
    byte = torch.where(bad, 255, (e + 127) * (m >= 2.0 ** -126))    # a subnormal's exponent field is 0
    val = torch.where(bad[..., None], math.nan, code * step)
    flat = lambda t: t.reshape(rows, -1)[:, :K]  # noqa: E731
    return flat(val), flat(code).to(torch.int8), byte.to(torch.uint8)


# ---- SwiGLU ---------------------------------------------------------------------------


def swiglu(h):
    I = h.shape[1] // 2
    g, u = h.double()[:, :I], h.double()[:, I:]
    return g * torch.sigmoid(g) * u


def swiglu_slack(h):
    """FP32 error of a: s(g) within (2 |g| + 8) steps of 2^-23 (the exponent g log2 e rounded, exp, 1 + x, reciprocal).
    Where 1 + e^-g is above 2^126 its reciprocal is subnormal, and 0 where e^-g is infinite: s is off by up to 2^-126
    then, and a by |g u| times that."""
    I = h.shape[1] // 2
    g, u = h.double()[:, :I], h.double()[:, I:]
    return swiglu(h).abs() * (2 * g.abs() + 10) * 2.0 ** -23 + 2.0 ** -126 * (1 + (g * u).abs() * (g < -87))


def swiglu_grad(h, d_a):
    """(d_h, slack)."""
    I = h.shape[1] // 2
    g, u, d = h.double()[:, :I], h.double()[:, I:], d_a.double()
    s = torch.sigmoid(g)
    dg, du = d * u * s * (1 + g * (1 - s)), d * g * s
    rel = (2 * g.abs() + 12) * 2.0 ** -23
    slack = torch.cat([(d * u).abs() * s * rel * (2 + 2 * g.abs()), du.abs() * rel], 1)
    lost = 2.0 ** -126 * (g < -87) * (1 + g.abs())       # of s, as in swiglu_slack
    return torch.cat([dg, du], 1), slack + torch.cat([(d * u).abs() * lost, d.abs() * lost], 1) + 2.0 ** -126


# ---- product with an epilogue --------------------------------------------------------


def linear(a, w, counts, bias, act, residual, start=0):
    """(out, FP32's error before the last rounding) for the rows of the groups; 0 elsewhere."""
    from tests.ops_util import groups
    K, N = a.shape[1], w.shape[1]
    half = N // 2
    out = torch.zeros(a.shape[0], half if act == "swiglu" else N, dtype=torch.float64)
    slack = torch.zeros_like(out)
    for e, lo, hi in groups(counts, start):
        x, v = a[lo:hi].double(), w[e].double()
        b = torch.zeros(N, dtype=torch.float64) if bias is None else bias[e].double()
        z = x @ v.T + b
        err = (x.abs() @ v.abs().T) * (K + 1) * 2.0 ** -23 + z.abs() * 2.0 ** -24     # of the sum, of adding the bias
        if act == "swiglu":
            g, u, eg, eu = z[:, :half], z[:, half:], err[:, :half], err[:, half:]
            s = torch.sigmoid(g)
            z = g * s * u
            # |d silu / dg| <= 1.1; s(g) within (2 |g| + 10) steps; lost where 1 / (1 + e^-g) is subnormal
            err = 1.1 * eg * (u.abs() + eu) + (g * s).abs() * eu + z.abs() * (2 * g.abs() + 10) * 2.0 ** -23
            err = err + 2.0 ** -126 * (1 + (g * u).abs() * (g < -87))
        if residual is not None:
            z = z + residual[lo:hi].double()
            err = err + (z.abs() + err) * 2.0 ** -24
        out[lo:hi], slack[lo:hi] = z, err
    return out, slack
