"""The state space block's calls (short convolution, prompt scan, token step) against the plain fp64
forms, through the public Python calls.

Tolerances, per value, from counting roundings (u = 2^-24 for fp32, 2^-8 for bf16):
  * convolution: five products and sums in fp32 and SiLU (slope below 1.1, exp within 2^-21 of its
    value): 2^-20 (sum |w u| + |bias|); a bf16 result adds 2^-8 |out|.
  * scan on CUDA cores: every token rounds the state a few times and the decay's exponent once, so
    after t tokens the state is off by at most 8 (t + 8) u times the recurrence over absolute values
    (exponents here stay below 16, whose rounding the same count covers); y adds its sum of N terms,
    64 u; a bf16 y adds 2^-8 |y|.
  * scan on the tensor cores: the weights of a chunk's products and the state that the read-out
    takes are rounded to bf16 once each: 2^-8 of the absolute read-out (plus the fp32 terms above);
    the state's updates are three bf16 terms (2^-24), summed in fp32 by the tensor core, whose sums
    are truncated (2^-23 for each of the 384 products of a chunk): 400 2^-23 per chunk that the
    state still holds; the recurrence over absolute values is its scale.
"""
import pytest
import torch

import gated_deltanet_linear_18_b200 as gdn
import ssm_ref as ref

pytestmark = pytest.mark.gpu

U32, UBF = 2.0 ** -24, 2.0 ** -8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def within(got, want, tol, name):
    """|got - want| <= tol per value; where the reference has none (NaN) nothing is said."""
    got = got.detach().cpu().double()
    live = ~torch.isnan(want)
    bad = ((got - want).abs() > tol) & live | (torch.isnan(got) & live)
    if bad.any():
        i = int(torch.argmax(((got - want).abs() / tol.clamp(min=1e-300)).masked_fill(~live, 0).flatten()))
        raise AssertionError(f"{name}: {int(bad.sum())} of {got.numel()} off; worst {got.flatten()[i]} "
                             f"for {want.flatten()[i]} (allowed {tol.flatten()[i]})")


def conv_inputs(rows, C, nseq, dtype, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn(rows, C + pad, generator=g).to(DT[dtype])
    return dict(x=wide.cuda()[:, pad:] if pad else wide.cuda(), w=(torch.randn(C, 4, generator=g) * 0.5).cuda(),
                bias=(torch.randn(C, generator=g) * 0.1).cuda(),
                hist=torch.randn(nseq, 3, C, generator=g).to(DT[dtype]).cuda())


def check_conv(out, want, mag, dtype, name="conv"):
    tol = 2.0 ** -20 * mag + (UBF * want.abs().nan_to_num() if dtype == "bf16" else 0) + 1e-30
    within(out, want, tol, name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,C,pad,hist", [(1, 8, 0, True), (2, 16, 0, False), (3, 40, 8, True), (4, 1, 0, True),
                                          (7, 33, 3, True), (8, 256, 0, True), (9, 1032, 16, False),
                                          (131, 264, 0, True), (500, 24, 5, False)])
def test_conv_dense(dtype, T, C, pad, hist):
    B = 3
    d = conv_inputs(B * T, C, B, dtype, seed=T * 7 + C, pad=pad)
    x = d["x"].unflatten(0, (B, T))
    out, hout = gdn.ssm_conv(x, d["w"], d["bias"], hist=d["hist"] if hist else None, want_hist=True)
    want, hwant, mag = ref.conv(d["x"], d["w"], d["bias"], d["hist"] if hist else None, ref.spans(B * T, B=B, T=T))
    check_conv(out.flatten(0, 1), want, mag, dtype)
    assert torch.equal(hout.cpu().double(), hwant)


LENS = [[5, 0, 1, 2, 0, 3, 40, 0], [0, 0], [1] * 9, [64, 200, 3]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_conv_packed_rows_behind_and_empty(dtype, lens):
    """Ragged and empty sequences, rows behind the last sequence left as they were."""
    C, behind = 48, 4
    total = sum(lens) + behind
    d = conv_inputs(total, C, len(lens), dtype, seed=len(lens))
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    out = torch.full((total, C), 7.0, dtype=DT[dtype], device="cuda")
    _, hout = gdn.ssm_conv_varlen(d["x"], d["w"], d["bias"], cu.cuda(), max(max(lens), 1), hist=d["hist"],
                                  want_hist=True, out=out)
    want, hwant, mag = ref.conv(d["x"], d["w"], d["bias"], d["hist"], ref.spans(total, cu=cu))
    check_conv(out, want, mag, dtype)
    assert torch.equal(hout.cpu().double(), hwant)
    assert (out[total - behind:] == 7.0).all()


@pytest.mark.parametrize("lead", [1, 2, 5, 70])
def test_packed_sequences_that_start_behind_the_first_row(lead):
    """Rows before the first sequence belong to none: they reach no window and keep their outputs."""
    lens, C = [9, 0, 70, 3], 40
    total = lead + sum(lens)
    d = conv_inputs(total, C, len(lens), "bf16", seed=lead)
    cu = torch.tensor([lead] + lens).cumsum(0).to(torch.int32)
    for hist in (d["hist"], None):
        out = torch.full((total, C), 7.0, dtype=torch.bfloat16, device="cuda")
        _, hout = gdn.ssm_conv_varlen(d["x"], d["w"], d["bias"], cu.cuda(), 70, hist=hist, want_hist=True, out=out)
        want, hwant, mag = ref.conv(d["x"], d["w"], d["bias"], hist, ref.spans(total, cu=cu))
        check_conv(out, want, mag, "bf16")
        assert torch.equal(hout.cpu().double(), hwant) and (out[:lead] == 7.0).all()
    for P, N, dtype in ((64, 64, "bf16"), (16, 16, "f32")):
        d = scan_inputs(total, len(lens), 2, P, 1, N, dtype, seed=lead)
        out = torch.full((total, 2, P), 7.0, device="cuda", dtype=DT[dtype])
        y, sT = gdn.ssm_scan_varlen(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], cu.cuda(), 70, D=d["D"], z=d["z"],
                                    dt_bias=d["dt_bias"], S0=d["S0"], out=out)
        check_scan(y, sT, d, ref.spans(total, cu=cu), dtype, uses_tensor_cores(P, N, dtype))
        assert (out[:lead] == 7.0).all()


def test_packed_calls_with_the_largest_max_seqlen():
    """A max_seqlen that no sequence comes near, up to 2^31 - 1: what the longest one's length gives."""
    lens = [5, 40, 3]
    total, most = sum(lens), 2 ** 31 - 1
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    d = conv_inputs(total, 24, 3, "bf16", seed=61)
    call = lambda m: gdn.ssm_conv_varlen(d["x"], d["w"], d["bias"], cu, m, hist=d["hist"], want_hist=True)
    for a, b in zip(call(40), call(most)):
        assert torch.equal(a, b)
    for dtype, m in (("f32", most), ("bf16", 5000)):
        s = scan_inputs(total, 3, 2, 64, 1, 64, dtype, seed=62)
        scan = lambda m: gdn.ssm_scan_varlen(s["x"], s["dt"], s["A_log"], s["Bm"], s["Cm"], cu, m, D=s["D"], S0=s["S0"])
        for a, b in zip(scan(40), scan(m)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_packed_sequences_longer_than_told(dtype):
    """A sequence takes max_seqlen rows at most; the rows behind them belong to none."""
    lens, most, H, P, G, N = [90, 40, 200], 64, 2, 64, 1, 64
    total = sum(lens)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    sp = ref.spans(total, cu=cu, max_len=most)
    inside = torch.zeros(total, dtype=torch.bool)
    for a, b in sp:
        inside[a:b] = True
    d = conv_inputs(total, 24, 3, dtype, seed=6)
    out = torch.full((total, 24), 7.0, dtype=DT[dtype], device="cuda")
    _, hout = gdn.ssm_conv_varlen(d["x"], d["w"], d["bias"], cu.cuda(), most, hist=d["hist"], want_hist=True, out=out)
    want, hwant, mag = ref.conv(d["x"], d["w"], d["bias"], d["hist"], sp)
    check_conv(out, want, mag, dtype)
    assert torch.equal(hout.cpu().double(), hwant) and (out.cpu()[~inside] == 7.0).all()
    d = scan_inputs(total, 3, H, P, G, N, dtype, seed=7)
    out = torch.full((total, H, P), 7.0, device="cuda", dtype=DT[dtype])
    y, sT = gdn.ssm_scan_varlen(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], cu.cuda(), most, D=d["D"], z=d["z"],
                                dt_bias=d["dt_bias"], S0=d["S0"], out=out)
    check_scan(y, sT, d, sp, dtype, uses_tensor_cores(P, N, dtype))
    assert (out.cpu()[~inside] == 7.0).all()


def test_conv_large_takes_long_tiles_and_equals_short_ones():
    """A call whose tiles are long gives what its pieces (tiles of a few rows) give, bit for bit, with the
    history handed on."""
    T, C = 9000, 1024 + 8
    d = conv_inputs(T, C, 1, "bf16", seed=5)
    big = gdn.ssm_conv(d["x"][None].expand(1, T, C), d["w"], d["bias"])
    x5 = torch.cat([d["x"]] * 5)                       # 45000 x 1032: tiles of over 100 rows
    cu = torch.arange(6, dtype=torch.int32) * T
    five = gdn.ssm_conv_varlen(x5, d["w"], d["bias"], cu.cuda(), T)
    for i in range(5):
        assert torch.equal(five[i * T:(i + 1) * T], big[0])
    hist, outs = None, []
    for a in range(0, T, 1777):
        o, hist = gdn.ssm_conv(d["x"][None, a:a + 1777].contiguous(), d["w"], d["bias"], hist=hist, want_hist=True)
        outs.append(o)
    assert torch.equal(torch.cat(outs, 1), big)


def test_conv_packed_neighbours_stay_isolated():
    lens = [3, 5, 4]
    d = conv_inputs(12, 16, 3, "bf16", seed=3)
    cu = torch.tensor([0, 3, 8, 12], dtype=torch.int32).cuda()
    clean = gdn.ssm_conv_varlen(d["x"], d["w"], d["bias"], cu, 5, hist=d["hist"])
    x = d["x"].clone()
    x[3:8] = float("nan")
    out = gdn.ssm_conv_varlen(x, d["w"], d["bias"], cu, 5, hist=d["hist"])
    assert torch.equal(out[:3], clean[:3]) and torch.equal(out[8:], clean[8:])
    assert torch.isnan(out[3:8]).all() and sum(lens) == 12


# ------------------------------------------------------------------------------------------------
# scan
# ------------------------------------------------------------------------------------------------
def scan_inputs(rows, nseq, H, P, G, N, dtype, seed=0, pad=0, fast=False):
    g = torch.Generator().manual_seed(seed)
    C = H * P + 2 * G * N
    c = torch.randn(rows, C + pad, generator=g)
    c = (c * torch.sigmoid(c)).to(DT[dtype]).cuda()[:, pad:]
    p = torch.randn(rows, H * P + H + pad, generator=g).to(DT[dtype]).cuda()[:, pad:]
    step = torch.exp(torch.rand(H, generator=g) * 4.6 - 6.9)
    d = dict(x=c[:, :H * P].unflatten(1, (H, P)), Bm=c[:, H * P:H * P + G * N].unflatten(1, (G, N)),
             Cm=c[:, H * P + G * N:].unflatten(1, (G, N)), z=p[:, :H * P].unflatten(1, (H, P)), dt=p[:, H * P:],
             A_log=torch.log(torch.rand(H, generator=g) * 15 + 1).cuda(),
             D=(torch.randn(H, generator=g) * 0.1 + 1).cuda(),
             dt_bias=((2.0 if fast else 1.0) * torch.log(torch.expm1(step))).cuda() + (6.0 if fast else 0.0),
             S0=(torch.randn(nseq, H, N, P, generator=g) * 0.3).cuda())
    return d


def uses_tensor_cores(P, N, dtype, aligned=True):
    return dtype == "bf16" and P in (64, 128) and N in (64, 128) and aligned


def check_scan(y, sT, d, sp, dtype, tc, z=True, s0=True, D=True, bias=True, extra=0.0):
    want, S, ymag, Smag = ref.scan(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], d["D"] if D else None,
                                   d["z"] if z else None, d["dt_bias"] if bias else None,
                                   d["S0"] if s0 else None, sp)
    longest = max([b - a for a, b in sp] + [1])
    per = 8 * (longest + 8) * U32
    if tc:
        per = max(per, 400 * 2 ** -23 * (longest // 128 + 2))
    tol_y = (per + 64 * U32 + (2.02 * UBF + extra if tc else 0)) * ymag + (UBF * want.abs().nan_to_num()
                                                                  if dtype == "bf16" else 0) + 1e-30
    within(y, want, tol_y, "y")
    if sT is not None:
        within(sT, S, per * Smag + 1e-30, "S_T")


SCAN = [  # T, H, P, G, N
    (1, 2, 64, 1, 128), (2, 4, 64, 2, 64), (3, 1, 16, 1, 16), (17, 3, 32, 1, 16), (40, 2, 128, 2, 128),
    (63, 6, 64, 2, 128), (64, 2, 128, 1, 64), (65, 4, 64, 4, 128), (127, 3, 64, 1, 128), (128, 2, 64, 1, 64),
    (129, 5, 64, 1, 128), (130, 2, 16, 1, 128), (257, 4, 64, 2, 128), (300, 2, 128, 1, 128), (33, 4, 128, 2, 32),
    (513, 2, 64, 1, 128),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,P,G,N", SCAN, ids=str)
def test_scan_dense(dtype, T, H, P, G, N):
    B = 2
    d = scan_inputs(B * T, B, H, P, G, N, dtype, seed=T + H)
    v = {k: t.unflatten(0, (B, T)) if k in ("x", "dt", "Bm", "Cm", "z") else t for k, t in d.items()}
    y, sT = gdn.ssm_scan(v["x"], v["dt"], v["A_log"], v["Bm"], v["Cm"], D=v["D"], z=v["z"], dt_bias=v["dt_bias"],
                         S0=v["S0"])
    gdn.check_error()
    ok = uses_tensor_cores(P, N, dtype, (H * P + 2 * G * N) % 8 == 0)
    check_scan(y.flatten(0, 1), sT, d, ref.spans(B * T, B=B, T=T), dtype, ok)


@pytest.mark.parametrize("z,s0,D,bias", [(False, False, False, False), (True, False, False, True),
                                         (False, True, True, False), (False, False, True, True)])
@pytest.mark.parametrize("P,N,dtype", [(64, 128, "bf16"), (32, 16, "f32")])
def test_scan_optional_arguments(z, s0, D, bias, P, N, dtype):
    T, H, G = 150, 4, 2
    d = scan_inputs(T, 1, H, P, G, N, dtype, seed=11)
    one = lambda t: t.unsqueeze(0)
    y, sT = gdn.ssm_scan(one(d["x"]), one(d["dt"]), d["A_log"], one(d["Bm"]), one(d["Cm"]), D=d["D"] if D else None,
                         z=one(d["z"]) if z else None, dt_bias=d["dt_bias"] if bias else None,
                         S0=d["S0"] if s0 else None)
    check_scan(y[0], sT, d, ref.spans(T, B=1, T=T), dtype, uses_tensor_cores(P, N, dtype), z, s0, D, bias)


@pytest.mark.parametrize("P,N", [(64, 128), (128, 64)])
@pytest.mark.parametrize("fast", [False, True], ids=["slow", "fast"])
def test_scan_long_and_fast_decays(P, N, fast):
    """A long sequence (segments of it run side by side), and decays so fast that a state lives for
    a token or two (steps up to 20, decays below 2^-100 in a chunk)."""
    T, H, G = 2100, 2, 1
    d = scan_inputs(T, 1, H, P, G, N, "bf16", seed=21, fast=fast)
    one = lambda t: t.unsqueeze(0)
    y, sT = gdn.ssm_scan(one(d["x"]), one(d["dt"]), d["A_log"], one(d["Bm"]), one(d["Cm"]), D=d["D"],
                         z=one(d["z"]), dt_bias=d["dt_bias"], S0=d["S0"])
    gdn.check_error()
    check_scan(y[0], sT, d, ref.spans(T, B=1, T=T), "bf16", True)


@pytest.mark.parametrize("P,N,dtype", [(64, 128, "bf16"), (128, 64, "bf16"), (32, 16, "f32")])
def test_scan_tokens_that_reset_the_state(P, N, dtype):
    """Time steps of 3e4 among ordinary ones, and heads whose rate overflows fp32: such a token leaves nothing of the
    state, and the ordinary tokens after it keep their accuracy.  Beyond the usual bound: a weight inside a block of
    32 tokens takes the difference of two prefix sums of exponents held above -128 each, at most 10 of them in a block
    here: 2 x 5 roundings of 2^-24 x 1280, times ln 2: below 2^-11."""
    T, H = 300, 2
    d = scan_inputs(T, 1, H, P, 1, N, dtype, seed=23)
    d["dt"] = d["dt"].clone()
    d["dt"][5::7] = 3e4                                         # 4 or 5 in a block
    d["dt"][6::14] = -200.0                                     # and steps that are 0 in fp32
    for a_log in (2.7, 100.0):
        d["A_log"] = torch.tensor([a_log, 0.0], device="cuda")
        one = lambda t: t.unsqueeze(0)
        y, sT = gdn.ssm_scan(one(d["x"]), one(d["dt"]), d["A_log"], one(d["Bm"]), one(d["Cm"]), D=d["D"],
                             z=one(d["z"]), S0=d["S0"])
        check_scan(y[0], sT, d, ref.spans(T, B=1, T=T), dtype, uses_tensor_cores(P, N, dtype), bias=False,
                   extra=2.0 ** -11)


RAGGED = [[0, 1, 127, 128, 129, 0, 300, 2], [64, 0], [1, 1, 1], [700, 5]]


@pytest.mark.parametrize("P,N,dtype", [(64, 128, "bf16"), (128, 128, "bf16"), (64, 64, "f32")])
@pytest.mark.parametrize("lens", RAGGED, ids=str)
def test_scan_packed(P, N, dtype, lens):
    """Ragged and empty sequences; an empty one hands its state on; rows behind the last sequence
    are left as they were."""
    H, G, behind = 4, 2, 3
    total = sum(lens) + behind
    d = scan_inputs(total, len(lens), H, P, G, N, dtype, seed=len(lens) + P)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    out = torch.full((total, H, P), 7.0, device="cuda", dtype=DT[dtype])
    y, sT = gdn.ssm_scan_varlen(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], cu.cuda(), max(lens), D=d["D"],
                                z=d["z"], dt_bias=d["dt_bias"], S0=d["S0"], out=out)
    gdn.check_error()
    assert y is out and (out[total - behind:] == 7.0).all()
    check_scan(y, sT, d, ref.spans(total, cu=cu), dtype, uses_tensor_cores(P, N, dtype))
    for s, n in enumerate(lens):
        if n == 0:
            assert torch.equal(sT[s], d["S0"][s])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_packed_neighbours_stay_isolated(dtype):
    """NaN and infinities in one sequence and behind the last one reach no other sequence."""
    lens, H, P, G, N = [100, 90, 70], 2, 64, 1, 128
    total = sum(lens) + 5
    d = scan_inputs(total, 3, H, P, G, N, dtype, seed=4)
    cu = torch.tensor([0, 100, 190, 260], dtype=torch.int32).cuda()
    call = lambda: gdn.ssm_scan_varlen(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], cu, 100, D=d["D"], z=d["z"],
                                       dt_bias=d["dt_bias"], S0=d["S0"])
    y0, s0 = call()
    for k in ("x", "Bm", "Cm", "dt"):
        d[k] = d[k].clone()
        d[k][100:190] = float("nan") if k != "Bm" else float("inf")
        d[k][260:] = float("nan")
    y, sT = call()
    for a, b, s in ((0, 100, 0), (190, 260, 2)):
        assert torch.equal(y[a:b], y0[a:b]) and torch.equal(sT[s], s0[s])
    assert torch.isnan(y[100:190].float()).all() and torch.isnan(sT[1]).all()


@pytest.mark.parametrize("P,N", [(64, 64), (128, 128)])
def test_scan_many_short_sequences(P, N):
    """More items than SMs: the same CTA goes from sequence to sequence, among them empty ones and longer ones."""
    g = torch.Generator().manual_seed(71)
    lens = torch.randint(0, 40, (330,), generator=g).tolist()
    lens[::37] = [0] * len(lens[::37])
    lens[5], lens[200], lens[329] = 300, 129, 256
    H = 128 // P
    total = sum(lens)
    d = scan_inputs(total, len(lens), H, P, 1, N, "bf16", seed=72)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    y, sT = gdn.ssm_scan_varlen(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], cu.cuda(), max(lens), D=d["D"], z=d["z"],
                                dt_bias=d["dt_bias"], S0=d["S0"])
    gdn.check_error()
    check_scan(y, sT, d, ref.spans(total, cu=cu), "bf16", True)
    y2, s2 = gdn.ssm_scan_varlen(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], cu.cuda(), max(lens), D=d["D"], z=d["z"],
                                 dt_bias=d["dt_bias"], S0=d["S0"])
    assert torch.equal(y, y2) and torch.equal(sT, s2)          # whichever CTA took what


def test_scan_whole_and_cut_pairs_together():
    """150 pairs of (sequence, two heads): 148 run whole, two in segments."""
    B, T, H, P, G, N = 3, 1030, 100, 64, 2, 64
    d = scan_inputs(B * T, B, H, P, G, N, "bf16", seed=81)
    v = {k: t.unflatten(0, (B, T)) if k in ("x", "dt", "Bm", "Cm", "z") else t for k, t in d.items()}
    y, sT = gdn.ssm_scan(v["x"], v["dt"], v["A_log"], v["Bm"], v["Cm"], D=v["D"], z=v["z"], dt_bias=v["dt_bias"],
                         S0=v["S0"])
    gdn.check_error()
    check_scan(y.flatten(0, 1), sT, d, ref.spans(B * T, B=B, T=T), "bf16", True)


def test_scan_given_outputs_and_no_state():
    T, H, P, G, N = 140, 2, 64, 1, 128
    d = scan_inputs(T, 1, H, P, G, N, "bf16", seed=91)
    one = {k: t.unsqueeze(0) if k in ("x", "dt", "Bm", "Cm", "z") else t for k, t in d.items()}
    a = (one["x"], one["dt"], one["A_log"], one["Bm"], one["Cm"])
    y0, s0 = gdn.ssm_scan(*a, D=d["D"], S0=d["S0"])
    out, st = torch.empty_like(y0), torch.empty_like(s0)
    ws = torch.empty(gdn.ssm_scan_workspace_bytes(1, T, H, G, P, N, torch.bfloat16), dtype=torch.uint8, device="cuda")
    y1, s1 = gdn.ssm_scan(*a, D=d["D"], S0=d["S0"], out=out, state_out=st, workspace=ws)
    assert y1 is out and s1 is st and torch.equal(y0, y1) and torch.equal(s0, s1)
    y2, s2 = gdn.ssm_scan(*a, D=d["D"], S0=d["S0"], want_state=False)
    assert s2 is None and torch.equal(y0, y2)


@pytest.mark.parametrize("P,N,dtype", [(64, 128, "bf16"), (32, 16, "f32")])
def test_no_tokens(P, N, dtype):
    """Without tokens the state and the history are handed on."""
    d = scan_inputs(1, 2, 2, P, 1, N, dtype, seed=95)
    e = {k: d[k][:0].unflatten(0, (2, 0)) for k in ("x", "dt", "Bm", "Cm")}
    y, sT = gdn.ssm_scan(e["x"], e["dt"], d["A_log"], e["Bm"], e["Cm"], S0=d["S0"])
    assert y.shape == (2, 0, 2, P) and torch.equal(sT, d["S0"])
    _, s0 = gdn.ssm_scan(e["x"], e["dt"], d["A_log"], e["Bm"], e["Cm"])
    assert (s0 == 0).all()
    hist = torch.randn(2, 3, 8, device="cuda").to(DT[dtype])
    out, h = gdn.ssm_conv(torch.empty(2, 0, 8, device="cuda", dtype=DT[dtype]), torch.ones(8, 4, device="cuda"),
                          hist=hist, want_hist=True)
    assert out.shape == (2, 0, 8) and torch.equal(h, hist)


def test_scan_unaligned_rows_take_the_other_kernel():
    """Rows whose distance is not a multiple of 8 values (an odd number of dt columns before them)."""
    T, H, P, G, N = 140, 3, 64, 1, 64
    d = scan_inputs(T, 1, H, P, G, N, "bf16", seed=8, pad=3)
    one = lambda t: t.unsqueeze(0)
    y, sT = gdn.ssm_scan(one(d["x"]), one(d["dt"]), d["A_log"], one(d["Bm"]), one(d["Cm"]), D=d["D"],
                         z=one(d["z"]), dt_bias=d["dt_bias"], S0=d["S0"])
    check_scan(y[0], sT, d, ref.spans(T, B=1, T=T), "bf16", False)


@pytest.mark.parametrize("P,N,dtype", [(64, 128, "bf16"), (16, 32, "f32")])
def test_scan_in_pieces_continues(P, N, dtype):
    """A sequence in two pieces, the state handed on, against the fp64 form of the whole."""
    T, cut, H, G = 390, 201, 2, 1
    d = scan_inputs(T, 1, H, P, G, N, dtype, seed=31)
    sT, ys = d["S0"], []
    for a, b in ((0, cut), (cut, T)):
        y, sT = gdn.ssm_scan(*(d[k][None, a:b] for k in ("x", "dt")), d["A_log"],
                             *(d[k][None, a:b] for k in ("Bm", "Cm")), D=d["D"], z=d["z"][None, a:b],
                             dt_bias=d["dt_bias"], S0=sT)
        ys.append(y[0])
    check_scan(torch.cat(ys), sT, d, ref.spans(T, B=1, T=T), dtype, uses_tensor_cores(P, N, dtype))


@pytest.mark.parametrize("T,H,P,N", [(2100, 2, 64, 128), (130, 2, 32, 16)])
def test_scan_is_reproducible_captured_and_on_another_stream(T, H, P, N):
    """The same bits from a second call, on another stream, and from a captured graph that is
    replayed on other values, two graphs with a workspace of their own."""
    d = scan_inputs(T, 1, H, P, 1, N, "bf16", seed=41)
    v = {k: t.unsqueeze(0).contiguous() if k in ("x", "dt", "Bm", "Cm", "z") else t for k, t in d.items()}
    call = lambda: gdn.ssm_scan(v["x"], v["dt"], v["A_log"], v["Bm"], v["Cm"], D=v["D"], z=v["z"],
                                dt_bias=v["dt_bias"], S0=v["S0"])
    y0, s0 = call()
    y1, s1 = call()
    assert torch.equal(y0, y1) and torch.equal(s0, s1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2, s2 = call()
    torch.cuda.synchronize()
    assert torch.equal(y0, y2) and torch.equal(s0, s2)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        graphs.append((g, out))
    v["x"].mul_(0.5)
    want = call()
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    gdn.check_error()


# ------------------------------------------------------------------------------------------------
# token step, and the calls together
# ------------------------------------------------------------------------------------------------
def block_inputs(n, T, H, P, G, N, dtype, seed=0):
    """A projection's rows [z | x B C | dt] of n sequences of T tokens, as one tensor."""
    g = torch.Generator().manual_seed(seed)
    C = H * P + 2 * G * N
    proj = torch.randn(n, T, H * P + C + H, generator=g).to(DT[dtype]).cuda()
    d = scan_inputs(1, n, H, P, G, N, dtype, seed=seed)
    return dict(proj=proj, z=proj[..., :H * P].unflatten(2, (H, P)), u=proj[..., H * P:H * P + C],
                dt=proj[..., H * P + C:], w=(torch.randn(C, 4, generator=g) * 0.5).cuda(),
                bias=(torch.randn(C, generator=g) * 0.1).cuda(),
                hist=torch.randn(n, 3, C, generator=g).to(DT[dtype]).cuda(), A_log=d["A_log"], D=d["D"],
                dt_bias=d["dt_bias"], S0=d["S0"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,H,P,G,N", [(1, 2, 64, 1, 128), (3, 6, 16, 2, 16), (2, 3, 128, 1, 32), (5, 8, 64, 8, 64),
                                       (70, 4, 128, 2, 128), (1, 1, 16, 1, 128), (2, 2, 32, 2, 64)], ids=str)
@pytest.mark.parametrize("full", [True, False])
def test_step(dtype, n, H, P, G, N, full):
    """One token against the fp64 form (x, B, C in fp64 between convolution and scan)."""
    b = block_inputs(n, 1, H, P, G, N, dtype, seed=n + H)
    S = b["S0"].clone()
    opt = dict(D=b["D"], z=b["z"][:, 0], dt_bias=b["dt_bias"]) if full else {}
    bias = b["bias"] if full else None
    y, hist = gdn.ssm_step(b["u"][:, 0], b["dt"][:, 0], b["hist"], b["w"], bias, b["A_log"], S, groups=G, **opt)
    u = b["u"][:, 0]
    c, hwant, mag = ref.conv(u, b["w"], bias, b["hist"], [(i, i + 1) for i in range(n)])
    HP, GN = H * P, G * N
    want, Sw, ymag, Smag = ref.scan(c[:, :HP].unflatten(1, (H, P)), b["dt"][:, 0], b["A_log"],
                                    c[:, HP:HP + GN].unflatten(1, (G, N)), c[:, HP + GN:].unflatten(1, (G, N)),
                                    opt.get("D"), opt.get("z"), opt.get("dt_bias"), b["S0"],
                                    [(i, i + 1) for i in range(n)])
    # the convolution's error 2^-20 of its sum of magnitudes enters through three factors
    grow = 3 * 2.0 ** -20 * float((mag / c.abs().clamp(min=1e-3)).max())
    within(S, Sw, (16 * U32 + grow) * Smag + 2.0 ** -20 * float(mag.max()) ** 2, "S")
    tol = (96 * U32 + grow) * ymag + 2.0 ** -20 * N * float(mag.max()) ** 3 + (UBF * want.abs() if dtype == "bf16" else 0)
    within(y, want, tol, "y")
    assert torch.equal(hist.cpu().double(), hwant)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_tokens_through_the_block_and_its_norms(dtype):
    """The calls as a model uses them: pre-norm, projection, convolution, scan, post-norm with the
    gate and the residual scale, over packed prompts; then single tokens of the same sequences with
    the state and the history handed on.  Each stage is held to the fp64 form of its own inputs."""
    lens, H, P, G, N, Dm = [70, 1, 133], 4, 64, 2, 64, 256
    HP, GN, n = H * P, G * N, 3
    C = HP + 2 * GN
    g = torch.Generator().manual_seed(51)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std)
    dt = DT[dtype]
    win, wout = r(Dm, HP + C + H, std=Dm ** -0.5).to(dt).cuda(), r(HP, Dm, std=HP ** -0.5).to(dt).cuda()
    d = scan_inputs(1, n, H, P, G, N, dtype, seed=52)
    w, bias = r(C, 4, std=0.5).cuda(), r(C, std=0.1).cuda()
    w_pre, w_post, sc = (1 + r(Dm, std=0.1)).cuda(), (1 + r(Dm, std=0.1)).cuda(), (0.5 + r(Dm, std=0.1)).cuda()
    total = sum(lens)
    h = r(total, Dm).cuda()                                        # the residual in fp32
    x = gdn.block_norm(torch.zeros(total, Dm, device="cuda", dtype=dt), h, w_pre=w_pre)[1]
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)

    def split(p):
        return (p[..., :HP].unflatten(-1, (H, P)), p[..., HP:HP + C], p[..., HP + C:])

    z, u, dtr = split(x @ win)
    c, hist = gdn.ssm_conv_varlen(u, w, bias, cu.cuda(), max(lens), want_hist=True)
    want, hwant, mag = ref.conv(u, w, bias, None, ref.spans(total, cu=cu))
    check_conv(c, want, mag, dtype)
    assert torch.equal(hist.cpu().double(), hwant)
    xs, Bm, Cm = c[:, :HP].unflatten(1, (H, P)), c[:, HP:HP + GN].unflatten(1, (G, N)), c[:, HP + GN:].unflatten(1, (G, N))
    y, S = gdn.ssm_scan_varlen(xs, dtr, d["A_log"], Bm, Cm, cu.cuda(), max(lens), D=d["D"], z=z, dt_bias=d["dt_bias"])
    e = dict(d, x=xs, dt=dtr, Bm=Bm, Cm=Cm, z=z)
    check_scan(y, S, e, ref.spans(total, cu=cu), dtype, uses_tensor_cores(P, N, dtype), s0=False)
    o = y.flatten(1) @ wout
    h1, x1 = gdn.block_norm(o, h, w_post=w_post, w_pre=w_pre, res_scale=sc)
    hw, xw = ref.block_norm(ref.f64(o), ref.f64(h), ref.f64(w_post), ref.f64(w_pre), None, ref.f64(sc), 1e-5)
    within(h1, hw, 2.0 ** -20 * (hw.abs() + 8) + 1e-30, "h_out")
    within(x1, xw, 2.0 ** -19 * (xw.abs() + 8) + (UBF * xw.abs() if dtype == "bf16" else 0), "x")
    # three tokens a sequence: its last position's x goes on as the next token's input
    x_t = x1[cu[1:].long() - 1]
    for _ in range(3):
        z, u, dtr = split(x_t @ win)
        Sb = S.clone()
        y, nxt = gdn.ssm_step(u, dtr, hist, w, bias, d["A_log"], S, groups=G, D=d["D"], z=z, dt_bias=d["dt_bias"])
        cc, hwant, _ = ref.conv(u, w, bias, hist, [(i, i + 1) for i in range(n)])
        yw, Sw, ymag, Smag = ref.scan(cc[:, :HP].unflatten(1, (H, P)), dtr, d["A_log"],
                                      cc[:, HP:HP + GN].unflatten(1, (G, N)), cc[:, HP + GN:].unflatten(1, (G, N)),
                                      d["D"], z, d["dt_bias"], Sb, [(i, i + 1) for i in range(n)])
        within(S, Sw, 2.0 ** -17 * (Smag + 1), "S after a token")
        within(y, yw, 2.0 ** -15 * (ymag + 1) + (UBF * yw.abs() if dtype == "bf16" else 0), "y of a token")
        assert torch.equal(nxt.cpu().double(), hwant)
        hist = nxt
        x_t = gdn.block_norm(y.flatten(1) @ wout, torch.zeros(n, Dm, device="cuda"), w_post=w_post, w_pre=w_pre)[1]


def test_step_in_a_graph_with_swapped_histories():
    """Two captured steps that swap the two history buffers, replayed, equal eager steps."""
    n, H, P, G, N = 4, 4, 64, 2, 128
    b = block_inputs(n, 1, H, P, G, N, "bf16", seed=61)
    def steps(S, h0, h1, count):
        ys = []
        for _ in range(count):
            y, _ = gdn.ssm_step(b["u"][:, 0], b["dt"][:, 0], h0, b["w"], b["bias"], b["A_log"], S, groups=G, D=b["D"],
                                z=b["z"][:, 0], dt_bias=b["dt_bias"], hist_out=h1)
            h0, h1 = h1, h0
            ys.append(y)
        return ys
    Se, he = b["S0"].clone(), b["hist"].clone()
    want = steps(Se, he, torch.empty_like(he), 4)
    Sg, hg = b["S0"].clone(), b["hist"].clone()
    spare = torch.empty_like(hg)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = steps(Sg, hg, spare, 2)
    Sg.copy_(b["S0"])
    hg.copy_(b["hist"])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[2]) and torch.equal(got[1], want[3]) and torch.equal(Sg, Se)


def test_scans_of_two_threads_at_once():
    """Scans that fill the GPU each, on streams and workspaces of their own: what each gets alone."""
    import threading
    cases = []
    for i, (P, N, T, H) in enumerate([(64, 128, 1500, 6), (128, 64, 700, 5), (64, 64, 2100, 40)]):
        d = scan_inputs(T, 1, H, P, 1, N, "bf16", seed=110 + i)
        one = {k: t.unsqueeze(0) if k in ("x", "dt", "Bm", "Cm", "z") else t for k, t in d.items()}
        cases.append((one["x"], one["dt"], one["A_log"], one["Bm"], one["Cm"], dict(D=d["D"], z=one["z"], S0=d["S0"])))
    alone = [gdn.ssm_scan(*c[:5], **c[5]) for c in cases]
    torch.cuda.synchronize()
    got, errors = [None] * len(cases), []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got[i] = gdn.ssm_scan(*cases[i][:5], **cases[i][5])
                torch.cuda.current_stream().synchronize()
        except Exception as e:                               # noqa: BLE001 (told to the test's own thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    gdn.check_error()
    assert not errors, errors
    for (y, s), (y0, s0) in zip(got, alone):
        assert torch.equal(y, y0) and torch.equal(s, s0)
