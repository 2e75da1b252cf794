"""Cases of the selective state space operators and of the norms around a block.

Five calls are covered: the short causal convolution of the state space block (``conv``), its scan
over prompts (``scan``), its step for single tokens (``step``), and the norms before and after a
block fused with its gate and residual scale, forward (``norm``) and backward (``norm_bwd``).

``run`` computes a case either in its plain form (elementary torch operations, fp32 with long sums
of logarithms in fp64, rounded once at the end) or, where ``own`` is true, through the package's
public calls.  ``exact`` computes the same from the definitions in fp64, token by token.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------
def listed():
    return [
        # a long prompt's projection rows [z | x B C | dt] through the convolution, in one sequence
        dict(name="conv_prompt", op="conv", B=1, T=16384, H=64, P=64, G=8, N=128, dtype="bf16", packed=0),
        # a serving batch of short ragged requests that go on from earlier pieces (history in, out)
        dict(name="conv_packed", op="conv", B=24, T=300, H=48, P=64, G=1, N=64, dtype="bf16", packed=7),
        # one long prompt, eight groups of eight heads, gated output: few chains, a long axis
        dict(name="scan_prompt", op="scan", B=1, T=8192, H=64, P=64, G=8, N=128, dtype="bf16", packed=0, z=True, s0=False),
        # prefill batch with the head counts of the delta layers (16 shared heads for 48, width 128)
        dict(name="scan_batch", op="scan", B=4, T=2048, H=48, P=128, G=16, N=128, dtype="bf16", packed=0, z=False, s0=False),
        # packed requests of 1 to 2000 tokens that continue from a state, one group for all heads
        dict(name="scan_packed", op="scan", B=32, T=2000, H=64, P=64, G=1, N=128, dtype="bf16", packed=3, z=True, s0=True),
        # a small fp32 model's odd-length prompt (the reference precision)
        dict(name="scan_f32_odd", op="scan", B=2, T=333, H=6, P=32, G=2, N=16, dtype="f32", packed=0, z=True, s0=True),
        # one request, one token: the latency of a chat turn
        dict(name="step_one", op="step", B=1, H=64, P=64, G=8, N=128, dtype="bf16", z=True),
        # a full decode batch with the delta layers' head counts
        dict(name="step_batch", op="step", B=256, H=48, P=128, G=16, N=128, dtype="bf16", z=True),
        # a training batch's residual stream in bf16, the block's output normed, gated and scaled
        dict(name="norm_rows", op="norm", rows=8192, D=6144, dtype="bf16", h="bf16", post=True, pre=True, z=True, scale=True),
        # a few decode tokens with the residual kept in fp32
        dict(name="norm_tokens", op="norm", rows=5, D=5120, dtype="bf16", h="f32", post=True, pre=True, z=False, scale=True),
        # the backward of the training batch
        dict(name="norm_bwd_rows", op="norm_bwd", rows=8192, D=6144, dtype="bf16", h="bf16", post=True, pre=True, z=True, scale=True),
        # an odd width in fp32, as a small model's tests have it
        dict(name="norm_bwd_odd", op="norm_bwd", rows=333, D=1001, dtype="f32", h="f32", post=True, pre=True, z=True, scale=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "step", "norm", "norm_bwd"])
    if op in ("norm", "norm_bwd"):
        c = dict(op=op, rows=_log(rng, 1, 8192), D=_log(rng, 64, 8192), dtype=rng.choice(["bf16", "bf16", "f32"]))
        c["D"] = c["D"] // 8 * 8 if rng.random() < 0.7 else c["D"]
        c["h"] = "f32" if c["dtype"] == "f32" else rng.choice(["bf16", "f32"])
        c["post"], c["pre"] = rng.choice([(True, True), (True, True), (False, True), (True, False)])
        c["z"], c["scale"] = rng.random() < 0.6, rng.random() < 0.6
        while c["rows"] * c["D"] * (1 if c["h"] == "bf16" else 2) > 8192 * 6144:
            c["rows"] = max(1, c["rows"] // 2)
        return c
    P, N = rng.choice([(64, 128), (64, 128), (64, 64), (128, 128), (128, 64), (32, 16)])
    G = rng.choice([1, 2, 4, 8])
    H = G * rng.choice([1, 2, 3, 4, 6, 8]) * (2 if G < 4 else 1)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "step":
        c = dict(op=op, B=_log(rng, 1, 256), H=H, P=P, G=G, N=N, dtype=dtype, z=rng.random() < 0.6)
        while c["B"] * H * P * N > 256 * 48 * 128 * 128:
            c["B"] //= 2
        return c
    packed = rng.choice([0, rng.randrange(1, 1000)])
    B = _log(rng, 2, 32) if packed else rng.choice([1, 1, 2, 3, 4])
    T = _log(rng, 1, 16384 if op == "conv" else 8192)
    c = dict(op=op, B=B, T=T, H=H, P=P, G=G, N=N, dtype=dtype, packed=packed)
    while c["B"] * c["T"] * H * P * (1 if dtype == "bf16" else 8) > 8192 * 4096:
        c["T"] = max(1, c["T"] // 2)
    if op == "scan":
        c["z"], c["s0"] = rng.random() < 0.5, rng.random() < 0.5
    return c


def _lengths(c):
    """The requests' lengths of a packed case: 1 .. T tokens, spread over the logarithm, the longest T."""
    if not c["packed"]:
        return [c["T"]] * c["B"]
    r = random.Random(c["packed"])
    return [c["T"]] + [_log(r, 1, c["T"]) for _ in range(c["B"] - 1)]


def _el(dtype):
    return 2 if dtype == "bf16" else 4


def work(case):
    c = case
    if c["op"] in ("norm", "norm_bwd"):
        n, el, eh = c["rows"] * c["D"], _el(c["dtype"]), _el(c["h"])
        vec = 4 * c["D"] * (c["post"] + c["pre"] + c["scale"])
        if c["op"] == "norm":      # y, h (z) in; h after the block (and x) out
            return {"bytes": n * (el * (1 + c["z"] + c["pre"]) + 2 * eh) + vec, "flops": 12 * n}
        # y, h after the block, its gradient (z, dx) in; dy, dh (dz) and the vectors' gradients out
        return {"bytes": n * (el * (2 + 2 * c["z"] + c["pre"]) + 3 * eh) + 2 * vec, "flops": 30 * n}
    H, P, G, N, el = c["H"], c["P"], c["G"], c["N"], _el(c["dtype"])
    C = H * P + 2 * G * N
    if c["op"] == "step":
        per = el * (2 * H * P * (1 + 0.5 * c["z"]) + 2 * G * N + H + 6 * C) + 8 * H * N * P
        return {"bytes": c["B"] * per + 20 * C + 12 * H, "flops": c["B"] * (5 * H * N * P + 8 * C)}
    rows, B = sum(_lengths(c)), c["B"]
    if c["op"] == "conv":
        hist = 6 * el * B * C if c["packed"] else 3 * el * B * C
        return {"bytes": 2 * el * rows * C + hist + 20 * C, "flops": 12 * rows * C}
    st = 4 * B * H * N * P
    return {"bytes": el * rows * (H * P * (2 + c["z"]) + 2 * G * N + H) + st * (1 + c["s0"]) + 12 * H,
            "flops": 5 * rows * H * N * P}


# --------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------
def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]

    def randn(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)

    def rand(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=g, device=DEV) * (hi - lo) + lo

    s = {"case": c}
    if c["op"] in ("norm", "norm_bwd"):
        rows, D, th = c["rows"], c["D"], DTYPES[c["h"]]
        s["y"] = randn(rows, D, std=0.7)
        s["h"] = randn(rows, D, std=2.0, dtype=th)      # the residual stream is wider than a block's output
        s["z"] = randn(rows, D) if c["z"] else None
        s["w_post"] = 1.0 + randn(D, std=0.1, dtype=torch.float32) if c["post"] else None
        s["w_pre"] = 1.0 + randn(D, std=0.1, dtype=torch.float32) if c["pre"] else None
        s["scale"] = 0.5 + randn(D, std=0.1, dtype=torch.float32) if c["scale"] else None
        if c["op"] == "norm_bwd":
            s["dh_out"] = randn(rows, D, std=1e-2, dtype=th)
            s["dx"] = randn(rows, D, std=1e-2) if c["pre"] else None
        return s
    H, P, G, N, B = c["H"], c["P"], c["G"], c["N"], c["B"]
    C = H * P + 2 * G * N
    s["A_log"] = torch.log(rand(H, lo=1.0, hi=16.0))
    step = torch.exp(rand(H, lo=math.log(1e-3), hi=math.log(1e-1)))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))     # softplus(dt_bias) = step
    s["D"] = 1.0 + randn(H, std=0.1, dtype=torch.float32)
    s["w"] = randn(C, 4, std=0.5, dtype=torch.float32)
    s["bias"] = randn(C, std=0.1, dtype=torch.float32)
    if c["op"] == "step":
        proj = randn(B, H * P + C + H)                       # [z | x B C | dt], as one projection makes it
        s["z"] = proj[:, :H * P].view(B, H, P) if c["z"] else None
        s["xbc"], s["dt"] = proj[:, H * P:H * P + C], proj[:, H * P + C:]
        s["hist"], s["hist_next"] = randn(B, 3, C), torch.empty(B, 3, C, device=DEV, dtype=dt)
        s["S"] = randn(B, H, N, P, std=0.3, dtype=torch.float32)
        return s
    lens = _lengths(c)
    rows = sum(lens)
    s["rows"], s["max_len"] = rows, max(lens)
    if c["packed"]:
        s["cu"] = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
    if c["op"] == "conv":
        proj = randn(rows, H * P + C + H)
        s["xbc"] = proj[:, H * P:H * P + C]
        s["hist"] = randn(B, 3, C) if c["packed"] else None
        return s
    conv = torch.randn(rows, C, generator=g, device=DEV)
    conv = (conv * torch.sigmoid(conv)).to(dt)               # the convolution's output rows [x | B | C]
    proj = randn(rows, H * P + H)                            # the projection's z and dt columns
    s["x"], s["z"] = conv[:, :H * P].view(rows, H, P), proj[:, :H * P].view(rows, H, P) if c["z"] else None
    s["Bm"], s["Cm"] = conv[:, H * P:H * P + G * N].view(rows, G, N), conv[:, H * P + G * N:].view(rows, G, N)
    s["dt"] = proj[:, H * P:]
    s["S0"] = randn(B, H, N, P, std=0.3, dtype=torch.float32) if c["s0"] else None
    if not c["packed"]:
        for k in ("x", "z", "Bm", "Cm", "dt"):
            s[k] = None if s[k] is None else s[k].unflatten(0, (B, c["T"]))
    return s


# --------------------------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------------------------
def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _softplus(x):
    return torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-torch.abs(x)))


def _where(s):
    """For each row its sequence, its place there and each sequence's first row."""
    c = s["case"]
    first = s["cu"].long() if c["packed"] else torch.arange(c["B"] + 1, device=DEV) * c["T"]
    row = torch.arange(s["rows"], device=DEV)
    seq = torch.searchsorted(first, row, right=True) - 1
    return seq, row - first[seq], first


def _plain_conv(s):
    x, w, c = s["xbc"], s["w"], s["case"]
    seq, pos, first = _where(s)
    hist = torch.zeros(c["B"], 3, x.shape[1], device=DEV, dtype=x.dtype) if s["hist"] is None else s["hist"]
    table = torch.cat([hist.flatten(0, 1), x])
    row = torch.arange(s["rows"], device=DEV)
    n = 3 * c["B"]

    def tap(j):    # the row j tokens back, from the history where the sequence is shorter
        return table[torch.where(pos >= j, n + row - j, 3 * seq + 3 + pos - j)].float() * w[:, 3 - j]

    a = tap(3) + tap(2) + tap(1) + tap(0) + s["bias"]
    last = torch.arange(3, device=DEV) - 3 + (first[1:] - first[:-1])[:, None]
    at = torch.where(last >= 0, n + first[:-1, None] + last, 3 * torch.arange(c["B"], device=DEV)[:, None] + 3 + last)
    return _silu(a).to(x.dtype), table[at]


def _plain_scan(s):
    c = s["case"]
    H, P, G, N, B, L = c["H"], c["P"], c["G"], c["N"], c["B"], s["max_len"]
    Q = 64
    nc = -(-L // Q)
    R = H // G

    def lay(v):    # [B, nc, Q, ...] with zeros behind each sequence's end
        v = v if c["packed"] else v.flatten(0, 1)
        out = torch.zeros(B, nc * Q, *v.shape[1:], device=DEV)
        out[seq, pos] = v.float()
        return out.view(B, nc, Q, *v.shape[1:])

    seq, pos, _ = _where(s)
    x, Bm, Cm = lay(s["x"]), lay(s["Bm"]), lay(s["Cm"])
    step = lay(_softplus(s["dt"].float() + s["dt_bias"]))                      # [B, nc, Q, H]
    cum = torch.cumsum(step.double() * -torch.exp(s["A_log"]).double(), dim=2)  # log decay from the chunk's start
    end = cum[:, :, -1]                                                        # [B, nc, H]
    xd = (x * step[..., None]).permute(0, 1, 3, 2, 4)                          # [B, nc, H, Q, P]
    tri = torch.ones(Q, Q, device=DEV, dtype=torch.bool).tril()
    ch = cum.permute(0, 1, 3, 2)
    gap = (ch[..., :, None] - ch[..., None, :]).masked_fill(~tri, -math.inf)
    dec = torch.exp(gap).float()                                               # [B, nc, H, Q, Q]
    Bg, Cg = Bm.permute(0, 1, 3, 2, 4), Cm.permute(0, 1, 3, 2, 4)              # [B, nc, G, Q, N]
    score = Cg @ Bg.transpose(-1, -2)
    within = (score[:, :, :, None] * dec.unflatten(2, (G, R))).flatten(2, 3) @ xd
    fade = torch.exp(end[:, :, None] - cum).float().permute(0, 1, 3, 2)        # [B, nc, H, Q]
    piece = (Bg[:, :, :, None].transpose(-1, -2) @ (xd * fade[..., None]).unflatten(2, (G, R))).flatten(2, 3)
    S0 = torch.zeros(B, H, N, P, device=DEV) if s["S0"] is None else s["S0"]
    every = torch.cat([S0[:, None], piece], 1)                                 # [B, nc + 1, H, N, P]
    total = torch.cumsum(torch.cat([torch.zeros_like(end[:, :1]), end], 1), 1).permute(0, 2, 1)
    keep = torch.ones(nc + 1, nc + 1, device=DEV, dtype=torch.bool).tril()
    carry = torch.exp((total[..., :, None] - total[..., None, :]).masked_fill(~keep, -math.inf)).float()
    states = (carry @ every.permute(0, 2, 1, 3, 4).flatten(3)).view(B, H, nc + 1, N, P)
    before = states[:, :, :-1].permute(0, 2, 1, 3, 4)                          # [B, nc, H, N, P]
    across = (Cg[:, :, :, None] @ before.unflatten(2, (G, R))).flatten(2, 3) * torch.exp(ch).float()[..., None]
    y = (within + across).permute(0, 1, 3, 2, 4) + x * s["D"][:, None]
    y = y.reshape(B, nc * Q, H, P)[seq, pos]
    if s["z"] is not None:
        y = y * _silu((s["z"] if c["packed"] else s["z"].flatten(0, 1)).float())
    y = y.to(s["x"].dtype)
    return y if c["packed"] else y.unflatten(0, (B, c["T"])), states[:, :, -1]


def _plain_step(s):
    c = s["case"]
    H, P, G, N, B = c["H"], c["P"], c["G"], c["N"], c["B"]
    win = torch.cat([s["hist"], s["xbc"][:, None]], 1)                         # [B, 4, C]
    a = _silu((win.float() * s["w"].T).sum(1) + s["bias"])
    x = a[:, :H * P].view(B, H, P)
    Bm = a[:, H * P:H * P + G * N].view(B, G, N).repeat_interleave(H // G, 1)
    Cm = a[:, H * P + G * N:].view(B, G, N).repeat_interleave(H // G, 1)
    step = _softplus(s["dt"].float() + s["dt_bias"])
    fade = torch.exp(-step * torch.exp(s["A_log"]))
    S = s["S"].mul_(fade[..., None, None]).add_(Bm[..., None] * (x * step[..., None])[:, :, None])
    y = (S * Cm[..., None]).sum(2) + x * s["D"][:, None]
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["hist_next"].copy_(win[:, 1:])
    s["hist"], s["hist_next"] = s["hist_next"], s["hist"]
    return y.to(s["xbc"].dtype), S, s["hist"]


def _plain_norm(s, eps=1e-5):
    y, h = s["y"].float(), s["h"].float()
    if s["w_post"] is not None:
        y = y * torch.rsqrt((y * y).mean(1, keepdim=True) + eps) * s["w_post"]
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    if s["scale"] is not None:
        y = y * s["scale"]
    h = h + y
    if s["w_pre"] is None:
        return h.to(s["h"].dtype), None
    x = h * torch.rsqrt((h * h).mean(1, keepdim=True) + eps) * s["w_pre"]
    return h.to(s["h"].dtype), x.to(s["y"].dtype)


def _plain_norm_bwd(s, eps=1e-5):
    y, h, dh = s["y"].float(), s["h"].float(), s["dh_out"].float()
    one = torch.ones(y.shape[1], device=DEV)
    dw_pre = dw_post = dscale = dz = None
    if s["w_pre"] is not None:
        r = torch.rsqrt((h * h).mean(1, keepdim=True) + eps)
        dx = s["dx"].float()
        dw_pre = (dx * h * r).sum(0)
        v = dx * s["w_pre"]
        dh = dh + r * (v - h * r * r * (v * h).mean(1, keepdim=True))
    rho = torch.rsqrt((y * y).mean(1, keepdim=True) + eps) if s["w_post"] is not None else None
    n = y if rho is None else y * rho * s["w_post"]
    z = None if s["z"] is None else s["z"].float()
    gate = one if z is None else _silu(z)
    scale = one if s["scale"] is None else s["scale"]
    if s["scale"] is not None:
        dscale = (dh * gate * n).sum(0)
    if z is not None:
        sg = 1.0 / (1.0 + torch.exp(-z))
        dz = (dh * scale * n * sg * (1.0 + z * (1.0 - sg))).to(s["z"].dtype)
    dn = dh * scale * gate
    if rho is not None:
        dw_post = (dn * y * rho).sum(0)
        v = dn * s["w_post"]
        dn = rho * (v - y * rho * rho * (v * y).mean(1, keepdim=True))
    return {"dy": dn.to(s["y"].dtype), "dh": dh.to(s["h"].dtype), "dz": dz, "dw_post": dw_post,
            "dw_pre": dw_pre, "dres_scale": dscale}


# --------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------
def _own(s):
    import gated_deltanet_linear_18_b200 as gdn

    c = s["case"]
    if c["op"] == "conv":
        if c["packed"]:
            return gdn.ssm_conv_varlen(s["xbc"], s["w"], s["bias"], s["cu"], s["max_len"], hist=s["hist"],
                                       want_hist=True)
        x = s["xbc"].unflatten(0, (c["B"], c["T"]))
        out, hist = gdn.ssm_conv(x, s["w"], s["bias"], want_hist=True)
        return out.flatten(0, 1), hist
    if c["op"] == "scan":
        if c["packed"]:
            return gdn.ssm_scan_varlen(s["x"], s["dt"], s["A_log"], s["Bm"], s["Cm"], s["cu"], s["max_len"],
                                       D=s["D"], z=s["z"], dt_bias=s["dt_bias"], S0=s["S0"])
        return gdn.ssm_scan(s["x"], s["dt"], s["A_log"], s["Bm"], s["Cm"], D=s["D"], z=s["z"],
                            dt_bias=s["dt_bias"], S0=s["S0"])
    if c["op"] == "step":
        y, _ = gdn.ssm_step(s["xbc"], s["dt"], s["hist"], s["w"], s["bias"], s["A_log"], s["S"], groups=c["G"],
                            D=s["D"], z=s["z"], dt_bias=s["dt_bias"], hist_out=s["hist_next"])
        s["hist"], s["hist_next"] = s["hist_next"], s["hist"]
        return y, s["S"], s["hist"]
    if c["op"] == "norm":
        return gdn.block_norm(s["y"], s["h"], w_post=s["w_post"], w_pre=s["w_pre"], z=s["z"], res_scale=s["scale"],
                              eps=1e-5)
    return gdn.block_norm_bwd(s["y"], s["h"], s["dh_out"], s["dx"], w_post=s["w_post"], w_pre=s["w_pre"],
                              z=s["z"], res_scale=s["scale"], eps=1e-5)


def run(state):
    if own:
        return _own(state)
    return {"conv": _plain_conv, "scan": _plain_scan, "step": _plain_step, "norm": _plain_norm,
            "norm_bwd": _plain_norm_bwd}[state["case"]["op"]](state)


# --------------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------------
def exact(case, seed):
    c, s = case, prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}

    def norm(v, w):
        return v / torch.sqrt(torch.square(v).sum(-1, keepdim=True) / v.shape[-1] + 1e-5) * w

    def block(y, h, w_post, w_pre, z, scale):
        u = y if w_post is None else norm(y, w_post)
        u = u if z is None else u * (z * torch.sigmoid(z))
        out = h + (u if scale is None else u * scale)
        return out, None if w_pre is None else norm(out, w_pre)

    if c["op"] == "norm":
        return block(d["y"], d["h"], d["w_post"], d["w_pre"], d["z"], d["scale"])
    if c["op"] == "norm_bwd":
        # h is the residual after the block: the gradients at it are those of h = after - update
        leaf = {k: d[k].requires_grad_() for k in ("y", "z", "w_post", "scale", "w_pre") if d[k] is not None}
        after = d["h"].requires_grad_()
        dh = d["dh_out"]
        dw_pre = None
        if c["pre"]:
            back = torch.autograd.grad(norm(after, leaf["w_pre"]), (after, leaf["w_pre"]), d["dx"])
            dh, dw_pre = dh + back[0], back[1]
        names = [k for k in ("y", "z", "w_post", "scale") if k in leaf]
        upd, _ = block(d["y"], torch.zeros_like(d["h"]), d["w_post"], None, d["z"], d["scale"])
        got = dict(zip(names, torch.autograd.grad(upd, [leaf[k] for k in names], dh.detach())))
        return {"dy": got["y"], "dh": dh.detach(), "dz": got.get("z"), "dw_post": got.get("w_post"), "dw_pre": dw_pre,
                "dres_scale": got.get("scale")}

    H, P, G, N, B = c["H"], c["P"], c["G"], c["N"], c["B"]

    def conv(window):      # [.., 4, C], oldest token first
        a = torch.einsum("...jc,cj->...c", window, d["w"]) + d["bias"]
        return a * torch.sigmoid(a)

    def advance(S, x, Bm, Cm, dt):
        lam = torch.nn.functional.softplus(dt + d["dt_bias"], threshold=200.0)
        S = S * torch.exp(-lam * torch.exp(d["A_log"]))[..., None, None]
        S = S + torch.einsum("bhn,bhp->bhnp", Bm, x * lam[..., None])
        return S, torch.einsum("bhnp,bhn->bhp", S, Cm) + x * d["D"][:, None]

    def heads(v):
        return v.repeat_interleave(H // G, dim=-2)

    if c["op"] == "step":
        win = torch.cat([d["hist"], d["xbc"][:, None]], 1)
        a = conv(win)
        S, y = advance(d["S"], a[:, :H * P].view(B, H, P), heads(a[:, H * P:-G * N].view(B, G, N)),
                       heads(a[:, -G * N:].view(B, G, N)), d["dt"])
        if d["z"] is not None:
            y = y * d["z"] * torch.sigmoid(d["z"])
        return y, S, win[:, 1:]
    lens = _lengths(c)
    cuts = [sum(lens[:i]) for i in range(len(lens) + 1)]
    if c["op"] == "conv":
        outs, hists = [], []
        for i, n in enumerate(lens):
            past = torch.zeros(3, d["xbc"].shape[1], device=DEV, dtype=torch.float64) if d["hist"] is None else d["hist"][i]
            rows = torch.cat([past, d["xbc"][cuts[i]:cuts[i + 1]]])
            outs.append(conv(rows.unfold(0, 4, 1).transpose(1, 2)))
            hists.append(rows[n:])
        return torch.cat(outs), torch.stack(hists)
    flat = {k: None if d[k] is None else d[k] if c["packed"] else d[k].flatten(0, 1) for k in ("x", "Bm", "Cm", "dt", "z")}
    S = torch.zeros(B, H, N, P, device=DEV, dtype=torch.float64) if d["S0"] is None else d["S0"].clone()
    y = torch.empty(cuts[-1], H, P, device=DEV, dtype=torch.float64)
    order = sorted(range(B), key=lambda i: -lens[i])       # the longest first: the live ones are a prefix
    S = S[order]
    start = torch.tensor([cuts[i] for i in order], device=DEV)
    for t in range(max(lens)):
        live = sum(n > t for n in lens)
        r = start[:live] + t
        S[:live], y[r] = advance(S[:live], flat["x"][r], heads(flat["Bm"][r]), heads(flat["Cm"][r]), flat["dt"][r])
    back = torch.empty_like(S)
    back[order] = S
    if flat["z"] is not None:
        y = y * flat["z"] * torch.sigmoid(flat["z"])
    return y if c["packed"] else y.unflatten(0, (B, c["T"])), back
