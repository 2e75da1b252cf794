"""The scan's tensor-core kernel with its gate: the gate's rows here are 16-byte aligned and a multiple of 8 values apart
(each test makes sure of it), which a gate cut out of rows with an odd number of time steps is not.  Tolerances are those
of the tensor-core kernel in test_gpu_ssm."""
import pytest
import torch

import gated_deltanet_linear_18_b200 as gdn
import ssm_ref as ref
import test_gpu_ssm as base

pytestmark = pytest.mark.gpu


def inputs(rows, nseq, H, P, G, N, seed, **kw):
    d = base.scan_inputs(rows, nseq, H, P, G, N, "bf16", seed=seed, **kw)
    d["z"] = d["z"].contiguous()
    assert P in (64, 128) and N in (64, 128)
    for k in ("x", "Bm", "Cm", "z"):
        assert d[k].stride(0) % 8 == 0 and d[k].data_ptr() % 16 == 0
    return d


def packed(d, cu, most, **kw):
    opt = {**dict(D=d["D"], z=d["z"], dt_bias=d["dt_bias"], S0=d["S0"]), **kw}
    y, sT = gdn.ssm_scan_varlen(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], cu.cuda(), most, **opt)
    gdn.check_error()
    return y, sT


def dense(d, B, T, **kw):
    v = {k: t.unflatten(0, (B, T)) if k in ("x", "dt", "Bm", "Cm", "z") else t for k, t in d.items()}
    opt = {**dict(D=v["D"], z=v["z"], dt_bias=v["dt_bias"], S0=v["S0"]), **kw}
    y, sT = gdn.ssm_scan(v["x"], v["dt"], v["A_log"], v["Bm"], v["Cm"], **opt)
    gdn.check_error()
    return y.flatten(0, 1), sT


SHAPES = [(2, 64, 1, 128), (3, 64, 1, 64), (4, 64, 4, 128), (5, 64, 1, 128), (6, 64, 2, 64), (2, 128, 1, 64), (4, 128, 2, 128)]


@pytest.mark.parametrize("T", [1, 2, 31, 33, 64, 65, 127, 128, 129, 255, 257, 513])
@pytest.mark.parametrize("H,P,G,N", SHAPES, ids=str)
def test_dense(T, H, P, G, N):
    B = 2
    d = inputs(B * T, B, H, P, G, N, seed=T + H)
    y, sT = dense(d, B, T)
    base.check_scan(y, sT, d, ref.spans(B * T, B=B, T=T), "bf16", True)


@pytest.mark.parametrize("z,s0,D,bias", [(True, False, False, False), (True, True, False, True), (True, False, True, False),
                                         (False, True, True, True)])
@pytest.mark.parametrize("P,N", [(64, 64), (128, 128)])
def test_optional_arguments(z, s0, D, bias, P, N):
    T, H = 150, 4
    d = inputs(T, 1, H, P, 2, N, seed=12)
    y, sT = dense(d, 1, T, D=d["D"] if D else None, z=d["z"].unsqueeze(0) if z else None,
                  dt_bias=d["dt_bias"] if bias else None, S0=d["S0"] if s0 else None)
    base.check_scan(y, sT, d, ref.spans(T, B=1, T=T), "bf16", True, z, s0, D, bias)


@pytest.mark.parametrize("P,N", [(64, 128), (128, 64)])
@pytest.mark.parametrize("fast", [False, True], ids=["slow", "fast"])
def test_long_and_fast_decays(P, N, fast):
    T = 2100
    d = inputs(T, 1, 2, P, 1, N, seed=22, fast=fast)
    y, sT = dense(d, 1, T)
    base.check_scan(y, sT, d, ref.spans(T, B=1, T=T), "bf16", True)


@pytest.mark.parametrize("P,N", [(64, 128), (128, 64)])
@pytest.mark.parametrize("a_log", [2.7, 100.0])
def test_tokens_that_reset_the_state(P, N, a_log):
    """As test_gpu_ssm's test of the same calls, with its bound."""
    T = 300
    d = inputs(T, 1, 2, P, 1, N, seed=24)
    d["dt"] = d["dt"].clone()
    d["dt"][5::7] = 3e4
    d["dt"][6::14] = -200.0
    d["A_log"] = torch.tensor([a_log, 0.0], device="cuda")
    y, sT = dense(d, 1, T, dt_bias=None)
    base.check_scan(y, sT, d, ref.spans(T, B=1, T=T), "bf16", True, bias=False, extra=2.0 ** -11)


@pytest.mark.parametrize("H,P,G,N", [(4, 64, 2, 128), (3, 64, 1, 64), (4, 128, 2, 128), (2, 128, 1, 64)], ids=str)
@pytest.mark.parametrize("lens", base.RAGGED + [[40, 0, 0, 512, 1, 383, 385]], ids=str)
def test_packed(H, P, G, N, lens):
    """Ragged and empty sequences, rows behind the last one left as they were."""
    behind = 3
    total = sum(lens) + behind
    d = inputs(total, len(lens), H, P, G, N, seed=len(lens) + P)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    out = torch.full((total, H, P), 7.0, device="cuda", dtype=torch.bfloat16)
    y, sT = packed(d, cu, max(lens), out=out)
    assert y is out and (out[total - behind:] == 7.0).all()
    base.check_scan(y, sT, d, ref.spans(total, cu=cu), "bf16", True)
    for s, n in enumerate(lens):
        if n == 0:
            assert torch.equal(sT[s], d["S0"][s])


def test_sequences_longer_than_told_and_rows_before_the_first():
    lens, most, lead = [190, 40, 300], 130, 5
    total = lead + sum(lens)
    cu = torch.tensor([lead] + lens).cumsum(0).to(torch.int32)
    sp = ref.spans(total, cu=cu, max_len=most)
    inside = torch.zeros(total, dtype=torch.bool)
    for a, b in sp:
        inside[a:b] = True
    d = inputs(total, 3, 2, 64, 1, 64, seed=7)
    out = torch.full((total, 2, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    y, sT = packed(d, cu, most, out=out)
    base.check_scan(y, sT, d, sp, "bf16", True)
    assert (out.cpu()[~inside] == 7.0).all()


@pytest.mark.parametrize("P,N", [(64, 128), (128, 64)])
def test_packed_neighbours_stay_isolated(P, N):
    """NaN and infinities in one sequence, its gate included, and behind the last one reach no other sequence."""
    lens, H = [100, 90, 70, 200], 2
    total = sum(lens) + 5
    d = inputs(total, 4, H, P, 1, N, seed=5)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    y0, s0 = packed(d, cu, 200)
    for k in ("x", "Bm", "Cm", "dt", "z"):
        d[k] = d[k].clone()
        d[k][100:190] = float("nan") if k not in ("Bm", "z") else float("inf")
        d[k][460:] = float("nan")
    y, sT = packed(d, cu, 200)
    for a, b, s in ((0, 100, 0), (190, 260, 2), (260, 460, 3)):
        assert torch.equal(y[a:b], y0[a:b]) and torch.equal(sT[s], s0[s])
    assert torch.isnan(y[100:190].float()).all() and torch.isnan(sT[1]).all()


@pytest.mark.parametrize("P,N", [(64, 64), (128, 128)])
def test_many_short_sequences(P, N):
    """More items than SMs: the same CTA goes from sequence to sequence, empty and longer ones among them."""
    g = torch.Generator().manual_seed(73)
    lens = torch.randint(0, 40, (330,), generator=g).tolist()
    lens[::37] = [0] * len(lens[::37])
    lens[5], lens[200], lens[329] = 300, 129, 256
    total, H = sum(lens), 128 // P
    d = inputs(total, len(lens), H, P, 1, N, seed=74)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    y, sT = packed(d, cu, max(lens))
    base.check_scan(y, sT, d, ref.spans(total, cu=cu), "bf16", True)
    y2, s2 = packed(d, cu, max(lens))
    assert torch.equal(y, y2) and torch.equal(sT, s2)


def test_whole_and_cut_pairs_together():
    """150 pairs of (sequence, two heads): 148 run whole, two in segments."""
    B, T, H = 3, 1030, 100
    d = inputs(B * T, B, H, 64, 2, 64, seed=82)
    y, sT = dense(d, B, T)
    base.check_scan(y, sT, d, ref.spans(B * T, B=B, T=T), "bf16", True)


def test_cut_pairs_of_ragged_sequences():
    """Segments of the longest sequence's length: some sequences end in their first, some inside a later one, some are
    empty."""
    lens, H = [1500, 0, 700, 1, 513, 129], 2
    total = sum(lens)
    d = inputs(total, len(lens), H, 64, 1, 128, seed=83)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    y, sT = packed(d, cu, max(lens))
    base.check_scan(y, sT, d, ref.spans(total, cu=cu), "bf16", True)


@pytest.mark.parametrize("P,N", [(64, 128), (128, 64)])
def test_in_pieces_continues(P, N):
    T, cut = 390, 201
    d = inputs(T, 1, 2, P, 1, N, seed=32)
    sT, ys = d["S0"], []
    for a, b in ((0, cut), (cut, T)):
        piece = {k: t[a:b] if k in ("x", "dt", "Bm", "Cm", "z") else t for k, t in d.items()}
        y, sT = dense(piece, 1, b - a, S0=sT)
        ys.append(y)
    base.check_scan(torch.cat(ys), sT, d, ref.spans(T, B=1, T=T), "bf16", True)


def test_columns_of_projection_rows():
    """z, x, B, C and dt as columns of one projection's rows [z | x B C | dt] of eight heads, and y of one row."""
    H, P, G, N, B, T = 8, 64, 2, 64, 2, 140
    g = torch.Generator().manual_seed(91)
    rows = torch.randn(B * T, 2 * H * P + 2 * G * N + H, generator=g).to(torch.bfloat16).cuda()
    z, x, Bm, Cm, dt = rows.split([H * P, H * P, G * N, G * N, H], -1)
    d = dict(inputs(1, B, H, P, G, N, seed=92), z=z.unflatten(1, (H, P)), x=x.unflatten(1, (H, P)),
             Bm=Bm.unflatten(1, (G, N)), Cm=Cm.unflatten(1, (G, N)), dt=dt)
    assert rows.stride(0) % 8 == 0
    y, sT = dense(d, B, T)
    base.check_scan(y, sT, d, ref.spans(B * T, B=B, T=T), "bf16", True)
    one = {k: t[:1] if k in ("x", "dt", "Bm", "Cm", "z", "S0") else t for k, t in d.items()}
    y1, s1 = dense(one, 1, 1)
    base.check_scan(y1, s1, one, ref.spans(1, B=1, T=1), "bf16", True)
