"""The token step in fp64 with a bound on the error of a kernel that keeps everything between the raw row and y in fp32,
value by value (u = 2^-24):
  * convolution: four fused sums, 4 u of the sum of magnitudes, times SiLU's slope (at most 1.1); SiLU from a 2^x within
    2^-22 of its value (its argument rounded twice: |v| 2^-23 more), a reciprocal within 2^-23 and a product: in all below
    2^-20 of the channel's sum of magnitudes, dc.
  * time step: raw = dt + bias rounded (u |raw|, which softplus passes on with a relative slope of at most
    max(1, |raw|)), exp, log1p and a sum: (|raw| + 6) u of the step, dl.
  * decay: its exponent takes dl, the rate (3 u) and a product: |a| (dl + 4 u) of the decay, and exp itself 2 u.
  * state: S' = decay S + step B x: the above, the products step x and times B, and the sum: 3 u of the magnitudes,
    and step (|B| dx + dB |x| + dB dx).
  * read-out: |C| dS + dC |S'| + dC dS, a sum of N terms (N + 4) u of its magnitudes, D dx, the gate (2^-21 + |z| 2^-23
    of it and a product), and the result's own rounding where it is bf16.
"""
import torch

import ssm_ref as ref

U, UBF = 2.0 ** -24, 2.0 ** -8


def inputs(n, H, P, G, N, dtype, seed):
    """A projection's rows [z | x B C | dt] of n sequences, a history, weights and a state (CPU)."""
    g = torch.Generator().manual_seed(seed)
    C = H * P + 2 * G * N
    r = lambda *s: torch.randn(*s, generator=g)
    rows = r(n, H * P + C + H).to(dtype)
    step = torch.exp(torch.rand(H, generator=g) * 4.6 - 6.9)
    return dict(z=rows[:, :H * P].unflatten(1, (H, P)), u=rows[:, H * P:H * P + C], dt=rows[:, H * P + C:], w=r(C, 4) * 0.5,
                bias=r(C) * 0.1, hist=r(n, 3, C).to(dtype), A_log=torch.log(torch.rand(H, generator=g) * 15 + 1),
                D=1 + r(H) * 0.1, dt_bias=torch.log(torch.expm1(step)), S=r(n, H, N, P) * 0.3)


def step(b, G, dtype, full, between=lambda v: v):
    """(y, S', tolerance of y, tolerance of S', history).  `between` is applied to the convolution's results."""
    n, H, N, P = b["S"].shape
    f = {k: v.double() for k, v in b.items()}
    c, hist, mag = ref.conv(b["u"], b["w"], b["bias"] if full else None, b["hist"], [(i, i + 1) for i in range(n)])
    c, dc = between(c), 2.0 ** -20 * mag

    def split(v):
        x, Bm, Cm = v.split([H * P, G * N, G * N], -1)
        heads = lambda t: t.unflatten(-1, (G, N)).repeat_interleave(H // G, 1)
        return x.unflatten(-1, (H, P))[:, :, None], heads(Bm)[..., None], heads(Cm)[..., None]

    (x, Bm, Cm), (dx, dB, dC) = split(c), split(dc)
    raw = f["dt"] + (f["dt_bias"] if full else 0)
    lam = torch.log1p(torch.exp(-raw.abs())) + raw.clamp(min=0)
    a = lam * torch.exp(f["A_log"])
    lam, a, raw = lam[..., None, None], a[..., None, None], raw[..., None, None]
    dl = (raw.abs() + 6) * U
    fade, upd = torch.exp(-a), lam * Bm * x
    S = fade * f["S"] + upd
    Smag = fade * f["S"].abs() + upd.abs()
    dS = fade * f["S"].abs() * (a * (dl + 4 * U) + 2 * U) + upd.abs() * dl + 3 * U * Smag \
        + lam * (Bm.abs() * dx + dB * x.abs() + dB * dx)
    skip = f["D"][:, None] if full else torch.zeros(H, 1, dtype=torch.float64)
    x, dx = x[:, :, 0], dx[:, :, 0]
    o = (Cm * S).sum(2) + skip * x
    do = (Cm.abs() * dS + dC * S.abs() + dC * dS + (N + 4) * U * Cm.abs() * (S.abs() + dS)).sum(2) \
        + skip.abs() * (dx + 2 * U * x.abs())
    if full:
        gate = f["z"] / (1 + torch.exp(-f["z"]))
        do = gate.abs() * (do + (o.abs() + do) * (2.0 ** -21 + f["z"].abs() * 2.0 ** -23 + 2 * U))
        o = o * gate
    if dtype is torch.bfloat16:
        do = do + UBF * (o.abs() + do)
    return o, S, do + 1e-30, dS + 1e-30, hist
