"""Plain fp64 forms of the state space block and of the norms around a block, token by token from
their definitions, and the same sums taken over absolute values (the scale that rounding errors are
measured against).  CPU, torch; used by the tests only."""
import torch


def f64(t):
    return None if t is None else t.detach().cpu().double()


def spans(total, cu=None, B=None, T=None, max_len=None):
    """(first, last) row of every sequence."""
    if cu is None:
        return [(b * T, (b + 1) * T) for b in range(B)]
    cu = [int(c) for c in cu]
    return [(cu[i], min(cu[i + 1], cu[i] + (total if max_len is None else max_len)))
            for i in range(len(cu) - 1)]


def conv(x, w, bias, hist, sp):
    """x [rows, C] -> (out [rows, C] (NaN outside the sequences), hist_out [nseq, 3, C], the sum of
    |w u| + |bias| per value)."""
    x, w, bias = f64(x), f64(w), f64(bias)
    C = x.shape[1]
    out, mag = torch.full_like(x, float("nan")), torch.zeros_like(x)
    hout = torch.zeros(len(sp), 3, C, dtype=torch.float64)
    for s, (a, b) in enumerate(sp):
        past = torch.zeros(3, C, dtype=torch.float64) if hist is None else f64(hist[s])
        rows = torch.cat([past, x[a:b]])
        hout[s] = rows[-3:]
        if b > a:
            win = torch.stack([rows[j:j + b - a] for j in range(4)])      # [4, n, C], oldest first
            acc = (win * w.T[:, None]).sum(0) + (0 if bias is None else bias)
            out[a:b] = acc / (1 + torch.exp(-acc))
            mag[a:b] = (win * w.T[:, None]).abs().sum(0) + (0 if bias is None else bias.abs())
    return out, hout, mag


def scan(x, dt, A_log, Bm, Cm, D, z, dt_bias, S0, sp):
    """[rows, ...] token tensors -> y [rows, H, P] (NaN outside the sequences), S_T, and the scales
    of y and S_T: the same recurrence over absolute values."""
    x, dt, A_log, Bm, Cm, D, z, dt_bias, S0 = map(f64, (x, dt, A_log, Bm, Cm, D, z, dt_bias, S0))
    rows, H, P = x.shape
    G, N = Bm.shape[1:]
    Bh, Ch = Bm.repeat_interleave(H // G, 1), Cm.repeat_interleave(H // G, 1)
    raw = dt if dt_bias is None else dt + dt_bias
    lam = torch.log1p(torch.exp(-raw.abs())) + raw.clamp(min=0)
    fade = torch.exp(-lam * torch.exp(A_log))
    y, ymag = torch.full_like(x, float("nan")), torch.zeros_like(x)
    S_T = torch.zeros(len(sp), H, N, P, dtype=torch.float64)
    Smag = torch.zeros_like(S_T)
    skip = torch.zeros(H, dtype=torch.float64) if D is None else D
    for s, (a, b) in enumerate(sp):
        S = torch.zeros(H, N, P, dtype=torch.float64) if S0 is None else S0[s].clone()
        M = S.abs()
        for t in range(a, b):
            upd = Bh[t][:, :, None] * (x[t] * lam[t][:, None])[:, None]
            S = S * fade[t][:, None, None] + upd
            M = M * fade[t][:, None, None] + upd.abs()
            y[t] = (S * Ch[t][:, :, None]).sum(1) + skip[:, None] * x[t]
            ymag[t] = (M * Ch[t][:, :, None].abs()).sum(1) + (skip[:, None] * x[t]).abs()
        S_T[s], Smag[s] = S, M
    if z is not None:
        gate = z / (1 + torch.exp(-z))
        y, ymag = y * gate, ymag * gate.abs()
    return y, S_T, ymag, Smag


def rms(v, eps):
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)


def block_norm(y, h, w_post, w_pre, z, scale, eps):
    """All arguments fp64 (autograd runs through it); returns (h_out, x or None)."""
    u = y if w_post is None else rms(y, eps) * w_post
    if z is not None:
        u = u * z / (1 + torch.exp(-z))
    if scale is not None:
        u = u * scale
    out = h + u
    return out, None if w_pre is None else rms(out, eps) * w_pre
