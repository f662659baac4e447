"""Helpers of the operator tests: 64-bit references on the CPU and the
tolerances of products.

A product's output differs from the exact one by its FP32 accumulation, at
most C * 2^-23 * sum |q p| over the contraction length C (one rounding or
truncation of at most 2^-23 of the running sum, itself at most sum |q p|, per
addition), and by one rounding to the output type, at most eps / 2 of the
value (or half the smallest subnormal).
"""
import torch


def bound(exact, magnitude, C, dtype):
    f = torch.finfo(dtype)
    acc = (C + 1) * 2.0 ** -23 * magnitude
    return acc + (exact.abs() + acc) * (f.eps / 2) + f.smallest_normal * f.eps


def check(got, exact, magnitude, C, what):
    err = (got.double().cpu() - exact).abs()
    tol = bound(exact, magnitude, C, got.dtype)
    worst = float((err / tol.clamp(min=1e-300)).max()) if err.numel() else 0.0
    print(f"  {what}: worst error {worst:.3g} of its bound", flush=True)
    assert torch.isfinite(got).all(), what
    assert (err <= tol).all(), what


def offsets_of(counts, start=0):
    return torch.cumsum(torch.tensor([start] + list(counts)), 0).to(torch.int32)


def groups(counts, start=0):
    lo = start
    for e, n in enumerate(counts):
        yield e, lo, lo + n
        lo += n


def random_counts(E, rows, seed, empty=0.2):
    g = torch.Generator().manual_seed(seed)
    p = torch.rand(E, generator=g) + 0.05
    p[torch.rand(E, generator=g) < empty] = 0
    if float(p.sum()) == 0:
        p[0] = 1.0
    return torch.bincount(torch.multinomial(p, rows, replacement=True, generator=g), minlength=E).tolist()


E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def mx_values(q, scales):
    """64-bit values of codes [..., K/2] and scale bytes [..., >= K/32] (CPU)."""
    code = torch.stack([q & 15, q >> 4], -1).flatten(-2).long()
    s = scales[..., : q.shape[-1] // 16].double()
    s = torch.where(s == 255, torch.nan, 2.0 ** (s - 127.0))
    return E2M1[code] * s.repeat_interleave(32, -1)


def mx_reference(x):
    """(values, scale bytes) of rows quantised in 64 bits (CPU)."""
    b = x.double().reshape(*x.shape[:-1], -1, 32)
    m = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    e = torch.floor(torch.log2(torch.where((m > 0) & ~bad, m, 1.0)))
    e = torch.where(m >= 2.0 ** (e + 1), e + 1, torch.where(m < 2.0 ** e, e - 1, e))   # log2 may round across a power
    byte = torch.where(m > 0, (e - 2 + 127).clamp(min=0), 0.0)
    v = torch.where(bad[..., None], 0.0, b) * 2.0 ** (127 - byte)[..., None]
    grid = E2M1[:8]
    far = (v.abs()[..., None] - grid).abs()
    near = far.amin(-1, keepdim=True)
    even = torch.arange(8) % 2 * 0.5
    code = torch.where(far == near, even, 9.0).argmin(-1)     # nearest, the even code of two as near
    val = grid[code] * torch.where(v < 0, -1.0, 1.0) * 2.0 ** (byte - 127)[..., None]
    val = torch.where(bad[..., None], torch.nan, val)
    return val.reshape(x.shape), torch.where(bad, 255.0, byte).to(torch.uint8)
