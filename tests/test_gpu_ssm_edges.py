"""The state space block's calls at the edges of their ranges: decay vectors beyond the L2 cache, bounds on the
sequences' lengths that no sequence comes near, the most rows of a packed call, and what the token step keeps in fp32."""
import pytest
import torch

import gated_deltanet_linear_18_b200 as gdn
import ssm_ref as ref
import ssm_step_ref as step_ref
import test_gpu_ssm as base
import test_ssm_step_bounds as step_bounds

pytestmark = pytest.mark.gpu


def test_scan_results_do_not_depend_on_the_order_of_the_sequences():
    """24 sequences of 64 heads, none cut: chunks' vectors, B, C and x come from HBM or L2 as it happens, on whichever
    SM takes them.  The sequences in another order give every one the same bits."""
    H, P, G, N = 64, 64, 1, 128
    g = torch.Generator().manual_seed(131)
    lens = torch.randint(900, 2049, (24,), generator=g)
    total, most = int(lens.sum()), int(lens.max())
    cg = torch.Generator(device="cuda").manual_seed(132)
    rows = torch.randn(total, H * P + 2 * G * N + H, generator=cg, device="cuda").to(torch.bfloat16)
    A_log = torch.log(torch.rand(H, generator=g) * 15 + 1).cuda()
    order = torch.randperm(24, generator=g)

    def run(rows, lens):
        cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(torch.int32).cuda()
        x, Bm, Cm, dt = rows.split([H * P, G * N, G * N, H], -1)
        y, sT = gdn.ssm_scan_varlen(x.unflatten(1, (H, P)), dt, A_log, Bm.unflatten(1, (G, N)), Cm.unflatten(1, (G, N)),
                                    cu, most)
        return y, sT

    y0, s0 = run(rows, lens)
    at = [int(v) for v in lens.cumsum(0) - lens]
    index = torch.cat([torch.arange(at[s], at[s] + int(lens[s])) for s in order]).cuda()
    for _ in range(3):
        y1, s1 = run(rows[index], lens[order])
        assert torch.equal(y1, y0[index]) and torch.equal(s1, s0[order.cuda()])
    gdn.check_error()


def test_conv_over_the_most_packed_rows():
    """2^30 rows of one channel, the sequence behind them empty: it hands its history on, and the last rows are those
    of a short call."""
    T = 2 ** 30
    g = torch.Generator(device="cuda").manual_seed(141)
    x = torch.randn(T, 1, generator=g, device="cuda", dtype=torch.bfloat16)
    w, bias = torch.randn(1, 4, generator=g, device="cuda"), torch.randn(1, generator=g, device="cuda")
    hist = torch.randn(2, 3, 1, generator=g, device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0, T, T], dtype=torch.int32, device="cuda")
    tail = gdn.ssm_conv(x[None, -5000:], w, bias)[0, 3:]
    out = torch.empty_like(x)
    for most in (T, 2 ** 31 - 1):
        out.zero_()
        _, h = gdn.ssm_conv_varlen(x, w, bias, cu, most, hist=hist, want_hist=True, out=out)
        assert torch.equal(h[0], x[-3:]) and torch.equal(h[1], hist[1])
        assert torch.equal(out[-4997:], tail)


@pytest.mark.parametrize("P,N,dtype", [(64, 128, torch.bfloat16), (128, 64, torch.bfloat16), (32, 16, torch.float32)])
def test_packed_calls_with_a_bound_of_zero_over_rows_in_no_sequence(P, N, dtype):
    """Empty sequences only, in a padded batch: states and histories are handed on, the rows keep their outputs."""
    n, rows, H = 3, 5, 2
    g = torch.Generator(device="cuda").manual_seed(151)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    t = lambda *s: r(*s).to(dtype)
    S0, y = r(n, H, N, P), torch.full((rows, H, P), 7.0, dtype=dtype, device="cuda")
    assert gdn.ssm_scan_workspace_bytes(n, 0, H, 1, P, N, dtype) == 0
    _, sT = gdn.ssm_scan_varlen(t(rows, H, P), t(rows, H), r(H), t(rows, 1, N), t(rows, 1, N), cu, 0, S0=S0, out=y)
    assert torch.equal(sT, S0) and (y == 7.0).all()
    hist, out = t(n, 3, 24), torch.full((rows, 24), 7.0, dtype=dtype, device="cuda")
    _, h = gdn.ssm_conv_varlen(t(rows, 24), r(24, 4), None, cu, 0, hist=hist, want_hist=True, out=out)
    assert torch.equal(h, hist) and (out == 7.0).all()


RAGGED = {"ragged": [0, 1, 127, 128, 129, 0, 300, 2, 0], "short": [1] * 40 + [0, 3], "one of many": [0] * 60 + [200] + [0] * 9}


@pytest.mark.parametrize("lead,behind", [(0, 0), (3, 200)])
@pytest.mark.parametrize("P,N", [(64, 128), (128, 64)])
@pytest.mark.parametrize("lens", RAGGED.values(), ids=RAGGED)
def test_packed_scan_under_a_bound_far_above_every_length(lens, P, N, lead, behind):
    """Bounds up to 2^31 - 1: scratch as the rows make necessary, and no byte of it beyond what the query says is
    written; results as the fp64 form's."""
    H, G, n = 4, 2, len(lens)
    total = lead + sum(lens) + behind
    d = base.scan_inputs(total, n, H, P, G, N, "bf16", seed=160 + P)
    d["z"] = d["z"].contiguous()                                    # (16-byte rows: the tensor cores' kernel)
    cu = torch.tensor([lead] + lens).cumsum(0).to(torch.int32)
    for most in (max(lens), total + 1000, 2 ** 31 - 1):
        need = gdn.ssm_scan_workspace_bytes(n, most, H, G, P, N, torch.bfloat16, total=total)
        ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")         # (NaN where not written)
        out = torch.full((total, H, P), 7.0, device="cuda", dtype=torch.bfloat16)
        args = (d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], cu.cuda(), most)
        opt = dict(D=d["D"], z=d["z"], dt_bias=d["dt_bias"], S0=d["S0"])
        y, sT = gdn.ssm_scan_varlen(*args, **opt, out=out, workspace=ws[:need])
        gdn.check_error()
        assert (ws[need:] == 0xFF).all() and (out[:lead] == 7.0).all() and (out[total - behind:] == 7.0).all()
        base.check_scan(y, sT, d, ref.spans(total, cu=cu), "bf16", True)
        y2, s2 = gdn.ssm_scan_varlen(*args, **opt, out=torch.full_like(out, 7.0))       # scratch from the allocator
        assert torch.equal(y2, y) and torch.equal(s2, sT)


def test_scratch_of_many_short_requests_under_one_long_bound():
    """512 requests of a few tokens and one of 3000 under a bound of 16384: room as for the rows, and the call runs."""
    lens = [5 + i % 13 for i in range(512)]
    lens[300] = 3000
    H, P, G, N, total = 8, 64, 1, 64, sum(lens)
    d = base.scan_inputs(total, 512, H, P, G, N, "bf16", seed=171)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    y, sT = gdn.ssm_scan_varlen(d["x"], d["dt"], d["A_log"], d["Bm"], d["Cm"], cu, 16384, D=d["D"], S0=d["S0"])
    records = H // 2 * (total // 128 + 512) * (2 * 128 * 5 + 16) * 4
    assert torch.cuda.max_memory_allocated() - before < records + y.nbytes + sT.nbytes + (8 << 20)
    base.check_scan(y, sT, d, ref.spans(total, cu=cu), "bf16", True, z=False, bias=False)


@pytest.mark.parametrize("full", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n,H,P,G,N", step_bounds.SHAPES, ids=str)
def test_step_keeps_the_convolution_in_fp32(n, H, P, G, N, dtype, full):
    """One token, each value held to a bound of its own, which bf16 between convolution and state update would break."""
    b = step_ref.inputs(n, H, P, G, N, dtype, seed=n + H)
    y, S, ty, tS, hist = step_ref.step(b, G, dtype, full)
    d = {k: v.cuda() for k, v in b.items()}
    opt = dict(D=d["D"], z=d["z"], dt_bias=d["dt_bias"]) if full else {}
    got, nxt = gdn.ssm_step(d["u"], d["dt"], d["hist"], d["w"], d["bias"] if full else None, d["A_log"], d["S"], groups=G,
                            **opt)
    base.within(d["S"], S, tS, "S")
    base.within(got, y, ty, "y")
    assert torch.equal(nxt.cpu().double(), hist)
