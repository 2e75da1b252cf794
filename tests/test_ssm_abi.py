"""The state space block's and the block norms' calls without a GPU: the C ABI's argument checks (nothing is
enqueued for a rejected call), workspace sizes, and the Python calls' refusals."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
FAKE = P(0x100000)          # never dereferenced: validation fails or returns before any CUDA call
OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def g():
    from gated_deltanet_linear_18_b200 import _build
    _build.build()
    import gated_deltanet_linear_18_b200 as gdn
    gdn.lib()
    return gdn


def conv(L, x=FAKE, ldx=64, w=FAKE, bias=None, hin=None, out=P(0x200000), hout=None, B=1, T=4, C=64, dtype=1):
    return L.gdn_ssm_conv(x, ldx, w, bias, hin, out, hout, B, T, C, dtype, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(C=0), INVALID), (dict(dtype=3), INVALID),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(out=None), INVALID),
    (dict(ldx=63), INVALID),                                     # tokens would overlap
    (dict(x=P(0x100001)), INVALID), (dict(w=P(0x100002)), INVALID), (dict(bias=P(0x100002)), INVALID),
    (dict(out=FAKE), INVALID), (dict(hin=FAKE, hout=FAKE), INVALID),
    (dict(B=0), OK), (dict(T=0), OK),                            # no work, no history asked for
])
def test_conv_validation(g, kw, expect):
    assert conv(g.lib(), **kw) == expect


def test_varlen_calls_need_offsets(g):
    L = g.lib()
    assert L.gdn_ssm_conv_varlen(FAKE, 64, FAKE, None, None, 1, 4, None, P(0x200000), None, 4, 64, 1, None) == INVALID
    assert L.gdn_ssm_conv_varlen(FAKE, 64, FAKE, None, P(0x100002), 1, 4, None, P(0x200000), None, 4, 64, 1,
                                 None) == INVALID
    ptr = [FAKE, 128, FAKE, 2, FAKE, 64, FAKE, 64, None, 0, FAKE, None, None]
    assert L.gdn_ssm_scan_varlen(*ptr, None, 1, 4, None, P(0x200000), None, FAKE, 1 << 40, 4, 2, 1, 64, 64, 1,
                                 None) == INVALID
    many = (1 << 30) + 1                                         # a row and a length have to add up in 32 bits
    assert L.gdn_ssm_conv_varlen(FAKE, 64, FAKE, None, FAKE, 1, 4, None, P(0x200000), None, many, 64, 1,
                                 None) == UNSUPPORTED
    assert L.gdn_ssm_scan_varlen(*ptr, FAKE, 1, 4, None, P(0x200000), None, FAKE, 1 << 40, many, 2, 1, 64, 64, 1,
                                 None) == UNSUPPORTED


def scan(L, x=FAKE, ldx=256, dt=FAKE, lddt=4, Bm=FAKE, ldb=128, Cm=FAKE, ldc=128, z=None, ldz=0, A=FAKE, D=None,
         bias=None, S0=None, y=P(0x200000), S_T=None, ws=P(0x300000), wb=1 << 40, B=1, T=130, H=4, G=2, Pd=64, N=64,
         dtype=1):
    return L.gdn_ssm_scan(x, ldx, dt, lddt, Bm, ldb, Cm, ldc, z, ldz, A, D, bias, S0, y, S_T, ws, wb, B, T, H, G, Pd,
                          N, dtype, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(G=0), INVALID), (dict(G=3), INVALID),
    (dict(dtype=9), INVALID), (dict(Pd=48), UNSUPPORTED), (dict(N=256), UNSUPPORTED), (dict(H=70000, G=1), UNSUPPORTED),
    (dict(B=70000), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(dt=None), INVALID), (dict(Bm=None), INVALID), (dict(Cm=None), INVALID),
    (dict(A=None), INVALID), (dict(y=None), INVALID), (dict(y=P(0x200008)), INVALID),
    (dict(ldx=255), INVALID), (dict(lddt=3), INVALID), (dict(ldb=127), INVALID), (dict(ldc=127), INVALID),
    (dict(z=FAKE, ldz=255), INVALID), (dict(x=P(0x100001)), INVALID), (dict(S0=P(0x100004)), INVALID),
    (dict(S0=FAKE, S_T=FAKE), INVALID),                          # the state may not be written over S0
    (dict(y=FAKE), INVALID),                                     # nor y over x
    (dict(ws=None), INVALID), (dict(wb=100), INVALID), (dict(ws=P(0x300010)), INVALID),
    (dict(B=0), OK),
])
def test_scan_validation(g, kw, expect):
    assert scan(g.lib(), **kw) == expect


def test_scan_workspace(g):
    f = g.ssm_scan_workspace_bytes
    bf, f32 = torch.bfloat16, torch.float32
    assert f(2, 300, 4, 1, 64, 128, f32) == 0 and f(2, 300, 4, 1, 32, 128, bf) == 0       # CUDA cores: none
    assert f(0, 300, 4, 1, 64, 128, bf) == 0 and f(2, 0, 4, 1, 64, 128, bf) == 0
    rec = (2 * 128 * 5 + 16) * 4                                  # a chunk's decay vectors of two heads
    # 3 chunks of 2 sequences, 4 heads in pairs (an odd head of a group still takes a pair), nothing cut
    assert f(2, 300, 4, 1, 64, 128, bf) == 256 + 2 * 2 * 3 * rec
    assert f(2, 300, 3, 1, 64, 128, bf) == f(2, 300, 4, 1, 64, 128, bf)
    assert f(2, 300, 4, 1, 128, 64, bf) == 256 + 2 * 4 * 3 * rec
    # one sequence of 64 chunks, one pair: 16 segments of four chunks, 15 states in between
    states = (15 * (128 * 128 + 2) * 4 + 255) // 256 * 256
    assert f(1, 8192, 2, 1, 64, 128, bf) == 256 + states + 64 * rec


def step(L, u=FAKE, ldu=512, dt=FAKE, lddt=4, z=None, ldz=0, hin=FAKE, hout=P(0x200000), w=FAKE, A=FAKE, S=FAKE,
         y=P(0x300000), n=2, H=4, G=2, Pd=64, N=64, dtype=1):
    return L.gdn_ssm_step(u, ldu, dt, lddt, z, ldz, hin, hout, w, None, A, None, None, S, y, n, H, G, Pd, N, dtype, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(n=-1), INVALID), (dict(H=3), INVALID), (dict(dtype=5), INVALID), (dict(Pd=20), UNSUPPORTED),
    (dict(u=None), INVALID), (dict(hin=None), INVALID), (dict(hout=None), INVALID), (dict(hout=FAKE), INVALID),
    (dict(w=None), INVALID), (dict(A=None), INVALID), (dict(S=None), INVALID), (dict(S=P(0x100008)), INVALID),
    (dict(y=None), INVALID), (dict(y=FAKE), INVALID), (dict(y=P(0x200000)), INVALID),     # y over u, over a history
    (dict(ldu=511), INVALID), (dict(lddt=3), INVALID), (dict(z=FAKE, ldz=4), INVALID),
    (dict(u=P(0x100001)), INVALID), (dict(n=0), OK),
])
def test_step_validation(g, kw, expect):
    assert step(g.lib(), **kw) == expect


def norm(L, y=FAKE, h=P(0x200000), z=None, wpost=None, wpre=FAKE, s=None, ho=P(0x300000), x=P(0x400000), rows=2, D=64,
         eps=1e-5, dtype=1, hd=1):
    return L.gdn_block_norm(y, h, z, wpost, wpre, s, ho, x, rows, D, eps, dtype, hd, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(rows=-1), INVALID), (dict(D=0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(dtype=4), INVALID), (dict(dtype=0, hd=1), UNSUPPORTED),            # fp32 with a bf16 residual
    (dict(y=None), INVALID), (dict(h=None), INVALID), (dict(ho=None), INVALID), (dict(x=None), INVALID),
    (dict(wpre=None), INVALID),                                              # x without its weight
    (dict(ho=P(0x200000)), INVALID), (dict(x=FAKE), INVALID),                # outputs over inputs
    (dict(y=P(0x100001)), INVALID), (dict(wpost=P(0x100002)), INVALID),
    (dict(rows=0), OK),
])
def test_norm_validation(g, kw, expect):
    assert norm(g.lib(), **kw) == expect


def norm_bwd(L, y=FAKE, ho=P(0x200000), z=None, dho=P(0x300000), dx=P(0x400000), wpost=None, wpre=FAKE, s=None,
             dy=P(0x500000), dh=P(0x600000), dz=None, dwpost=None, dwpre=FAKE, ds=None, ws=P(0x700000), wb=1 << 40,
             rows=2, D=64, dtype=1, hd=1):
    return L.gdn_block_norm_bwd(y, ho, z, dho, dx, wpost, wpre, s, dy, dh, dz, dwpost, dwpre, ds, ws, wb, rows, D, 1e-5,
                                dtype, hd, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(rows=-1), INVALID), (dict(D=0), INVALID), (dict(dtype=0, hd=1), UNSUPPORTED),
    (dict(y=None), INVALID), (dict(ho=None), INVALID), (dict(dx=None), INVALID), (dict(dy=None), INVALID),
    (dict(dh=None), INVALID), (dict(dwpre=None), INVALID), (dict(dwpost=FAKE), INVALID), (dict(ds=FAKE), INVALID),
    (dict(z=FAKE), INVALID), (dict(dz=FAKE), INVALID),                       # a gate and its gradient come together
    (dict(wpre=None, dwpre=None, dx=None, dho=None), INVALID),               # no gradient at all
    (dict(dy=FAKE), INVALID), (dict(dh=P(0x300000)), INVALID),
    (dict(ws=None), INVALID), (dict(wb=8), INVALID), (dict(ws=P(0x700010)), INVALID),
])
def test_norm_bwd_validation(g, kw, expect):
    assert norm_bwd(g.lib(), **kw) == expect


def test_norm_bwd_workspace(g):
    f = g.block_norm_bwd_workspace_bytes
    assert f(0, 64) == 0 and f(-1, 64) == 0 and f(8, 0) == 0
    # every row, group or CTA that writes a part of the two column sums has its place
    for rows, D, groups in ((1, 8, 12), (160, 4096, 2), (8192, 6144, 1), (500, 1024, 6), (50, 333, 1), (9, 10000, 1)):
        parts = max(min(rows, 148) * groups if D % 8 == 0 and D <= 8192 else 0, min(rows, 592))
        assert f(rows, D) == parts * 2 * D * 4, (rows, D)


def test_python_calls_refuse(g):
    t = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d)
    f = lambda *s: torch.zeros(*s)
    cu = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        g.ssm_conv(t(1, 4, 8), f(8, 4))
    with pytest.raises(ValueError, match=r"\[C, 4\]"):
        g.ssm_conv(t(1, 4, 8), f(4, 8))
    with pytest.raises(ValueError, match="hist"):
        g.ssm_conv(t(2, 4, 8), f(8, 4), hist=t(1, 3, 8))
    with pytest.raises(ValueError, match="float32"):
        g.ssm_conv(t(1, 4, 8), t(8, 4))
    with pytest.raises(ValueError, match="dtype"):
        g.ssm_conv(torch.zeros(1, 4, 8, dtype=torch.float16), f(8, 4))
    with pytest.raises(ValueError, match="contiguous"):
        g.ssm_conv(t(1, 4, 16)[..., ::2], f(8, 4))
    with pytest.raises(ValueError, match="evenly"):
        g.ssm_conv(t(2, 5, 8)[:, :4], f(8, 4))
    with pytest.raises(ValueError, match="overlap"):
        g.ssm_conv_varlen(t(1, 8).expand(4, 8), f(8, 4), None, cu, 4)
    with pytest.raises(ValueError, match="int32"):
        g.ssm_conv_varlen(t(4, 8), f(8, 4), None, cu.long(), 4)
    a = dict(x=t(2, 4, 2, 64), dt=t(2, 4, 2), A_log=f(2), Bm=t(2, 4, 1, 64), Cm=t(2, 4, 1, 64))
    with pytest.raises(ValueError, match="CUDA"):
        g.ssm_scan(**a)
    for bad in (dict(dt=t(2, 4, 3)), dict(Cm=t(2, 4, 1, 32)), dict(z=t(2, 4, 2, 32)), dict(A_log=f(3)), dict(D=f(1)),
                dict(S0=f(2, 2, 64, 32)), dict(Bm=f(2, 4, 1, 64)), dict(A_log=t(2)), dict(out=t(2, 4, 2, 32)),
                dict(state_out=f(1, 2, 64, 64))):
        with pytest.raises(ValueError):
            g.ssm_scan(**{**a, **bad})
    s = dict(u=t(3, 256), dt=t(3, 2), hist=t(3, 3, 256), w=f(256, 4), bias=None, A_log=f(2), S=f(3, 2, 64, 64), groups=1)
    with pytest.raises(ValueError, match="CUDA"):
        g.ssm_step(**s)
    for bad in (dict(groups=2), dict(groups=0), dict(hist=t(3, 2, 256)), dict(dt=f(3, 2)), dict(S=f(2, 2, 64, 64)),
                dict(hist_out=t(3, 3, 255)), dict(out=f(3, 2, 64)), dict(z=t(3, 2, 32))):
        with pytest.raises(ValueError):
            g.ssm_step(**{**s, **bad})
    with pytest.raises(ValueError, match="CUDA"):
        g.block_norm(t(4, 64), t(4, 64))
    for bad in (dict(h=t(4, 32)), dict(z=f(4, 64)), dict(w_post=f(32)), dict(w_pre=t(64)), dict(y=t(4, 128)[:, ::2])):
        with pytest.raises(ValueError):
            g.block_norm(**{**dict(y=t(4, 64), h=t(4, 64)), **bad})
    with pytest.raises(ValueError, match="dx"):
        g.block_norm_bwd(t(4, 64), t(4, 64), t(4, 64), w_pre=f(64))
    with pytest.raises(ValueError, match="dh_out"):
        g.block_norm_bwd(t(4, 64), t(4, 64), None)
