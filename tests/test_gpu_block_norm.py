"""The norms around a block, forward and backward, against the plain fp64 forms (the gradients also
against differences), through the public Python calls.

Tolerances, per value, from counting roundings (u = 2^-24 for fp32, 2^-8 for bf16): a norm's mean of
D squares is off by at most (D / 8 + 12) u in the order that the kernels sum it (8 values a thread, then a
tree), half of which enters the norm; SiLU is within 2^-20 of |z|.  So n, h_out and x are within
(D / 8 + 64) u of the magnitudes that enter them, a bf16 result adds 2^-8 of itself.  A gradient is the sum
of up to three terms, each with the relative error of four such factors: 4 (D / 8 + 64) u of the terms'
magnitudes; a column sum over R rows adds R u of the sum of magnitudes.
"""
import pytest
import torch

import gated_deltanet_linear_18_b200 as gdn
import ssm_ref as ref

pytestmark = pytest.mark.gpu

U32, UBF = 2.0 ** -24, 2.0 ** -8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def inputs(rows, D, dtype, h, post, pre, z, scale, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0: torch.randn(*s, generator=g) * std
    vec = lambda on, mean: (mean + r(D, std=0.1)).cuda() if on else None
    return dict(y=r(rows, D, std=0.7).to(DT[dtype]).cuda(), h=r(rows, D, std=2.0).to(DT[h]).cuda(),
                z=r(rows, D).to(DT[dtype]).cuda() if z else None, w_post=vec(post, 1.0), w_pre=vec(pre, 1.0),
                res_scale=vec(scale, 0.5))


def opts(d):
    return {k: d[k] for k in ("w_post", "w_pre", "z", "res_scale")}


def close(got, want, scale, factor, name):
    tol = factor * scale + (UBF * want.abs() if got.dtype == torch.bfloat16 else 0) + 1e-30
    err = (got.detach().cpu().double() - want).abs()
    bad = (err > tol) | torch.isnan(err)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol).max())} of allowed"


def h_scale(f, hw):
    """The magnitudes that enter h_out: h and the update, whose gate alone can be off by 2^-20 of it."""
    return 16 * (hw - f["h"]).abs() + f["h"].abs()


def x_scale(f, hw, xw):
    """x = h_out (r w_pre): the factor r w_pre = xw / hw carries h_out's error (which is large against
    h_out where h and the update cancel), and the norm adds its own relative error of x."""
    return xw.abs() + h_scale(f, hw) * (xw / hw).abs().nan_to_num()


WIDTHS = [(1, 1), (3, 7), (2, 8), (5, 64), (4, 250), (300, 256), (7, 1001), (9, 2048), (3, 2056), (160, 4096),
          (2, 6144), (5, 6152), (3, 8192), (2, 8200), (2, 10001)]
KINDS = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


@pytest.mark.parametrize("dtype,h", KINDS)
@pytest.mark.parametrize("rows,D", WIDTHS, ids=str)
def test_forward(rows, D, dtype, h):
    d = inputs(rows, D, dtype, h, True, True, True, True, seed=D)
    ho, x = gdn.block_norm(d["y"], d["h"], eps=EPS, **opts(d))
    gdn.check_error()
    f = {k: ref.f64(t) for k, t in d.items()}
    hw, xw = ref.block_norm(f["y"], f["h"], f["w_post"], f["w_pre"], f["z"], f["res_scale"], EPS)
    k = (D / 8 + 64) * U32
    close(ho, hw, h_scale(f, hw), k, "h_out")
    close(x, xw, x_scale(f, hw, xw), 2 * k, "x")


@pytest.mark.parametrize("post,pre,z,scale", [(True, True, False, False), (False, True, True, False), (True, False, True, True),
                                              (False, False, False, False), (False, True, False, True)])
@pytest.mark.parametrize("rows,D", [(6, 320), (4, 77), (400, 1024)])
def test_forward_optional_parts(post, pre, z, scale, rows, D):
    d = inputs(rows, D, "bf16", "f32", post, pre, z, scale, seed=3)
    ho, x = gdn.block_norm(d["y"], d["h"], eps=EPS, **opts(d))
    f = {k: ref.f64(t) for k, t in d.items()}
    hw, xw = ref.block_norm(f["y"], f["h"], f["w_post"], f["w_pre"], f["z"], f["res_scale"], EPS)
    k = (D / 8 + 64) * U32
    close(ho, hw, h_scale(f, hw), k, "h_out")
    assert (x is None) == (not pre)
    if pre:
        close(x, xw, x_scale(f, hw, xw), 2 * k, "x")


def grads(d, dh, dx, rows, D):
    """fp64 gradients by autograd with respect to y, z, the vectors and the residual after the block
    (from which the call starts), and for each the sum of the magnitudes of its terms."""
    f = {k: None if t is None else ref.f64(t).requires_grad_() for k, t in d.items()}
    after = f["h"]
    a = torch.zeros_like(after) if dh is None else ref.f64(dh)
    out = {}
    if f["w_pre"] is not None:
        gx = torch.autograd.grad(ref.rms(after, EPS) * f["w_pre"], (after, f["w_pre"]), ref.f64(dx))
        a = a + gx[0]
        out["dw_pre"] = gx[1]
    out["dh"] = a
    names = [k for k in ("y", "z", "w_post", "res_scale") if f[k] is not None]
    upd, _ = ref.block_norm(f["y"], torch.zeros_like(after), f["w_post"], None, f["z"], f["res_scale"], EPS)
    for k, g in zip(names, torch.autograd.grad(upd, [f[k] for k in names], a)):
        out["d" + k] = g
    with torch.no_grad():
        y, one = f["y"], torch.ones(D, dtype=torch.float64)
        w, wn, s = (one if f[k] is None else f[k].abs() for k in ("w_post", "w_pre", "res_scale"))
        amag = torch.zeros_like(after) if dh is None else ref.f64(dh).abs()
        mag = {}
        if f["w_pre"] is not None:
            r = 1 / torch.sqrt((after ** 2).mean(1, keepdim=True) + EPS)
            v = ref.f64(dx).abs() * wn
            amag = amag + r * (v + after.abs() * r * r * (v * after.abs()).mean(1, keepdim=True))
            mag["dw_pre"] = (ref.f64(dx) * after * r).abs().sum(0)
        mag["dh"] = amag
        q = 1 / torch.sqrt((y ** 2).mean(1, keepdim=True) + EPS) if f["w_post"] is not None else torch.ones(rows, 1).double()
        gate = one if f["z"] is None else (f["z"] / (1 + torch.exp(-f["z"]))).abs()
        n = (y * q).abs() * w
        dn = amag * s * gate
        if f["z"] is not None:
            mag["dz"] = amag * s * n * (1 + f["z"].abs())
        if f["res_scale"] is not None:
            mag["dres_scale"] = (amag * gate * n).sum(0)
        if f["w_post"] is not None:
            mag["dw_post"] = (dn * (y * q).abs()).sum(0)
            mag["dy"] = q * (w * dn + y.abs() * q * q * (w * dn * y.abs()).mean(1, keepdim=True))
        else:
            mag["dy"] = dn
    return out, mag


def check_grads(g, d, dh, dx, rows, D):
    want, mag = grads(d, dh, dx, rows, D)
    k = 4 * (D / 8 + 64) * U32
    for name, ref_g in want.items():
        close(g[name], ref_g.detach(), mag[name], k + (rows * U32 if g[name].dim() == 1 else 0), name)
    for name, t in g.items():
        assert (t is None) == (name not in want), name


@pytest.mark.parametrize("dtype,h", KINDS)
@pytest.mark.parametrize("rows,D", WIDTHS, ids=str)
def test_backward(rows, D, dtype, h):
    d = inputs(rows, D, dtype, h, True, True, True, True, seed=D + 1)
    g = torch.Generator().manual_seed(7)
    dh, dx = torch.randn(rows, D, generator=g).to(DT[h]).cuda(), torch.randn(rows, D, generator=g).to(DT[dtype]).cuda()
    got = gdn.block_norm_bwd(d["y"], d["h"], dh, dx, eps=EPS, **opts(d))
    gdn.check_error()
    check_grads(got, d, dh, dx, rows, D)


@pytest.mark.parametrize("post,pre,z,scale,dh_given", [(True, True, False, False, True), (False, True, True, False, True),
                                                       (True, False, True, True, True), (False, False, False, False, True),
                                                       (False, True, False, True, False), (True, True, True, True, False)])
@pytest.mark.parametrize("rows,D", [(6, 320), (4, 77), (400, 1024)])
def test_backward_optional_parts(post, pre, z, scale, dh_given, rows, D):
    d = inputs(rows, D, "bf16", "f32", post, pre, z, scale, seed=5)
    g = torch.Generator().manual_seed(8)
    dh = torch.randn(rows, D, generator=g).cuda() if dh_given else None
    dx = torch.randn(rows, D, generator=g).to(torch.bfloat16).cuda() if pre else None
    got = gdn.block_norm_bwd(d["y"], d["h"], dh, dx, eps=EPS, **opts(d))
    gdn.check_error()
    check_grads(got, d, dh, dx, rows, D)


def test_backward_against_differences():
    """Directional central differences of the kernel's own forward (fp32): the loss <dh_out, h_out> +
    <dx, x> along a random direction of every input, step 2^-7.  The forward's rounding, 2^-22 of the
    loss's terms (a random sum of 2 * 640 of them of size 1: below 2^-16 in all), over the step, and the
    third derivative's share (step^2 times terms of the loss's size: 2^-14 * 40) bound the difference."""
    rows, D = 4, 160
    d = inputs(rows, D, "f32", "f32", True, True, True, True, seed=9)
    g = torch.Generator().manual_seed(10)
    dh, dx = torch.randn(rows, D, generator=g).cuda(), torch.randn(rows, D, generator=g).cuda()

    def loss(v):
        ho, x = gdn.block_norm(v["y"], v["h"], eps=EPS, **opts(v))
        return float((ho.double() * dh.double()).sum() + (x.double() * dx.double()).sum())

    ho, _ = gdn.block_norm(d["y"], d["h"], eps=EPS, **opts(d))
    got = gdn.block_norm_bwd(d["y"], ho, dh, dx, eps=EPS, **opts(d))
    step = 2.0 ** -7
    for key, grad in (("y", "dy"), ("h", "dh"), ("z", "dz"), ("w_post", "dw_post"), ("w_pre", "dw_pre"),
                      ("res_scale", "dres_scale")):
        v = torch.randn(d[key].shape, generator=g).cuda()
        v /= v.norm()
        up, dn = dict(d), dict(d)
        up[key], dn[key] = d[key] + step * v, d[key] - step * v
        numeric = (loss(up) - loss(dn)) / (2 * step)
        exact = float((got[grad].double() * v.double()).sum())
        assert abs(numeric - exact) <= 2.0 ** -16 / step + 2.0 ** -14 * 40, (key, numeric, exact)


@pytest.mark.parametrize("rows,D", [(700, 1024), (50, 333)])
def test_reproducible_captured_and_on_another_stream(rows, D):
    d = inputs(rows, D, "bf16", "bf16", True, True, True, True, seed=12)
    dh, dx = torch.randn_like(d["h"]), torch.randn_like(d["y"])
    call = lambda: (gdn.block_norm(d["y"], d["h"], **opts(d)), gdn.block_norm_bwd(d["y"], d["h"], dh, dx, **opts(d)))
    flat = lambda r: [*r[0], *(r[1][k] for k in sorted(r[1]))]
    a = flat(call())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = flat(call())
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    d["y"].mul_(0.5)
    want = flat(call())
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(flat(out), want))
    gdn.check_error()


def test_unaligned_tensors_and_leading_dimensions():
    """A view that starts one value into a buffer (2-byte alignment), and [B, T, D] tensors."""
    rows, D = 5, 64
    d = inputs(rows, D, "bf16", "bf16", True, True, True, True, seed=13)
    buf = torch.empty(rows * D + 1, dtype=torch.bfloat16, device="cuda")
    off = buf[1:].view(rows, D).copy_(d["y"])
    a, b = gdn.block_norm(d["y"], d["h"], **opts(d)), gdn.block_norm(off, d["h"], **opts(d))
    for p, q in zip(a, b):      # the two kernels sum in another order: at most one bf16 step apart
        assert ((p.double() - q.double()).abs() <= 2 * UBF * p.double().abs()).all()
    c = gdn.block_norm(*(d[k].view(1, rows, D) for k in ("y", "h")), w_post=d["w_post"], w_pre=d["w_pre"],
                       z=d["z"].view(1, rows, D), res_scale=d["res_scale"])
    assert c[0].shape == (1, rows, D) and torch.equal(c[1][0], a[1])


def test_zero_rows():
    e = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    ho, x = gdn.block_norm(e, e.clone(), w_post=w, w_pre=w)
    assert ho.shape == x.shape == (0, 64)
    g = gdn.block_norm_bwd(e, e, e, e, w_post=w, w_pre=w)
    assert (g["dw_post"] == 0).all() and (g["dw_pre"] == 0).all()


def test_threads_with_widths_of_their_own():
    """Calls of several threads at once, each on its own stream, whose kernels need different amounts of shared
    memory: what each gets alone."""
    import threading
    widths = [2056, 4096, 6144, 8192]
    ds = [inputs(3, D, "bf16", "bf16", True, True, True, True, seed=D) for D in widths]
    got, errors = [None] * len(ds), []
    torch.cuda.synchronize()

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    got[i] = gdn.block_norm(ds[i]["y"], ds[i]["h"], eps=EPS, **opts(ds[i]))
                torch.cuda.current_stream().synchronize()
        except Exception as e:                               # noqa: BLE001 (told to the test's own thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(ds))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for d, (ho, x) in zip(ds, got):
        h1, x1 = gdn.block_norm(d["y"], d["h"], eps=EPS, **opts(d))
        assert torch.equal(ho, h1) and torch.equal(x, x1)
