"""The operators around the product where their definitions are strained:
gradients in fp32, far pre-activations, long vocabularies, walks over several
tiles, sizes past a launch's limits. Tolerances are sums of the method's own
roundings, as in test_gpu_ops.py, whose helpers are used."""
import pytest
import torch

import dense_tiled_gemm_tgemm_amd as tg
from test_gpu_ops import (BF, F32, HF, U, act64, act_grad64, e_lse, forward64, half_step, rand, slope, tiny, within,
                          xent64, xent_case, y_tol)

pytestmark = pytest.mark.gpu


# ------------------------------------ fp32 gradients of an fp32 result --

def rounded(got, ref, tol, what):
    """within(), for results that their type may not hold: infinite where the value
    lies past the type's largest one, either where it may."""
    big = torch.finfo(got.dtype).max
    g = got.detach().double().cpu()
    past, near = ref.abs() - tol > big, ref.abs() + tol > big
    assert (g[past] == torch.copysign(torch.full_like(ref, float("inf")), ref)[past]).all(), what
    near = near & ((g.abs() == float("inf")) | past)
    within(torch.where(near, ref, g), ref, tol, what)


def check_f32_gradients(M, N, K, dtype, act, layout, bdt, sx, sw, sdy, seed=1):
    """dx, dw, db of an fp32 result against the formula: dY is not rounded before
    the activation's derivative and the column sums; dP is rounded once, in units
    of its largest value (binary16: a step of 2^-24 of 2^14 at least)."""
    print(f"f32 grad {M} {N} {K} {dtype} {act} {layout} {bdt} {sx} {sw} {sdy}", flush=True)
    x, w, b = rand((M, K), seed, dtype, sx), rand((N, K), seed + 1, dtype, sw * K ** -0.5), rand((N,), seed + 2, bdt)
    dy = rand((M, N), seed + 3, F32, sdy)
    p, y64, e = forward64(x, w, b, act, None)
    xd, wd = x.cuda().requires_grad_(), (w if layout == "NxK" else w.t().contiguous()).cuda().requires_grad_()
    bd = b.cuda().requires_grad_()
    y = tg.linear(xd, wd, bd, act, out_dtype=F32, w_layout=layout)
    gx, gw, gb = torch.autograd.grad(y, [xd, wd, bd], dy.cuda())
    h, d64 = half_step(dtype), dy.double()
    dp = d64 * act_grad64(p, act)
    ep = torch.zeros_like(dp)
    if act != "none":
        ep = d64.abs() * (slope(act) * (e + h * 1.01 * p.abs() + tiny(dtype)) + 2.0 ** -20)
    er = ep + h * 1.01 * dp.abs() + tiny(dtype) * 2.0 ** -13 * float(d64.abs().max())
    want = dp.sum(0)
    rounded(gb, want, ep.sum(0) + (M + 4) * U * dp.abs().sum(0) + half_step(bdt) * 1.01 * want.abs() + tiny(bdt), "db")
    want = dp @ w.double()
    rounded(gx, want, 1.01 * (er @ w.double().abs()) + (N + 4) * U * (dp.abs() @ w.double().abs())
           + h * 1.02 * want.abs() + tiny(dtype), "dx")
    want = dp.t() @ x.double()
    rounded(gw if layout == "NxK" else gw.t(), want, 1.01 * (er.t() @ x.double().abs())
           + (M + 4) * U * (dp.abs().t() @ x.double().abs()) + h * 1.02 * want.abs() + tiny(dtype), "dw")


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_f32_gradient_keeps_its_range(act, dtype):
    """Gradients below binary16's smallest step and above its largest value, and of mixed size."""
    for sx, sw, sdy in ((300.0, 1 / 300, 1e-8), (1e-3, 1e-2, 1e5), (1.0, 1.0, 1.0)):
        for M, N, K, lay in ((130, 300, 72, "NxK"), (5, 40, 24, "KxN"), (700, 136, 200, "KxN"), (64, 5, 3, "NxK"), (1, 1, 1, "NxK")):
            check_f32_gradients(M, N, K, dtype, act, lay, F32 if M != 5 else dtype, sx, sw, sdy)


def test_f32_gradient_of_a_mean():
    """The mean of a large result: every gradient is 2^-26, below half of binary16's smallest step."""
    M, N, K = 8192, 8192, 16
    x, w = rand((M, K), 1, HF, 64.0).cuda().requires_grad_(), rand((N, K), 2, HF, 64.0).cuda().requires_grad_()
    b = torch.zeros((N,), device="cuda", requires_grad=True)
    gx, gw, gb = torch.autograd.grad(tg.linear(x, w, b, out_dtype=F32).mean(), [x, w, b])
    assert torch.equal(gb, torch.full_like(gb, 2.0 ** -13))
    for got, other in ((gx, w), (gw, x)):
        s = other.detach().double()
        want = (s.sum(0) * 2.0 ** -26)[None, :].expand(8192, K)
        within(got, want.cpu(), (8196 * U * (s.abs().sum(0) * 2.0 ** -26)[None, :].cpu() + half_step(HF) * 1.01 * want.abs().cpu()
                                 + tiny(HF)), "mean")


def test_f32_gradient_special_values():
    """Zeros; infinities and NaN stay in their rows of dx and columns of db, and do not set the scale."""
    x, w = rand((70, 40), 1, HF).cuda().requires_grad_(), rand((50, 40), 2, HF).cuda().requires_grad_()
    b = torch.zeros((50,), device="cuda", requires_grad=True)
    y = tg.linear(x, w, b, act="silu", out_dtype=F32)
    g = torch.autograd.grad(y, [x, w, b], torch.zeros((70, 50), device="cuda"), retain_graph=True)
    assert all(t.abs().max() == 0 for t in g)
    dy = rand((70, 50), 3, F32, 1e-6).cuda()
    clean = torch.autograd.grad(y, [x, w, b], dy, retain_graph=True)
    assert clean[0].abs().max() > 0
    for bad in (float("inf"), float("nan")):
        d2 = dy.clone()
        d2[3, 7] = bad
        gx, gw, gb = torch.autograd.grad(y, [x, w, b], d2, retain_graph=True)
        keep = torch.arange(70) != 3
        assert torch.equal(gx.cpu()[keep], clean[0].cpu()[keep]) and not gx[3].isfinite().any()
        cols = torch.arange(50) != 7
        assert torch.equal(gb.cpu()[cols], clean[2].cpu()[cols]) and not gb[7].isfinite()
        assert torch.equal(gw.cpu()[cols], clean[1].cpu()[cols]) and not gw[7].isfinite().any()


def test_f32_gradient_layouts_and_empty_operands():
    """Broadcast, transposed and strided fp32 gradients; no rows; no columns; a residual's gradient."""
    x, w = rand((50, 64), 1, HF).cuda().requires_grad_(), rand((40, 64), 2, HF).cuda().requires_grad_()
    r = rand((50, 40), 3, HF).cuda().requires_grad_()
    for act in ("none", "gelu"):
        y = tg.linear(x, w, None, act, r, out_dtype=F32)
        g1 = torch.autograd.grad(y, [x, w, r], torch.full((50, 40), 1e-3, device="cuda"), retain_graph=True)
        g2 = torch.autograd.grad(y, [x, w, r], torch.full((40, 50), 1e-3, device="cuda").t(), retain_graph=True)
        g3 = torch.autograd.grad(y, [x, w, r], torch.full((), 1e-3, device="cuda").expand(50, 40), retain_graph=True)
        g4 = torch.autograd.grad(y, [x, w, r], torch.full((50, 47), 1e-3, device="cuda")[:, 3:43])
        for g in (g2, g3, g4):
            assert all(torch.equal(a, b) for a, b in zip(g1, g))
        assert torch.equal(g1[2], torch.full_like(r, 1e-3))
    b = torch.zeros((24,), device="cuda", requires_grad=True)
    w = rand((24, 16), 1, HF).cuda().requires_grad_()
    for act in ("none", "silu"):
        x = torch.empty((0, 16), dtype=HF, device="cuda", requires_grad=True)
        gx, gw, gb = torch.autograd.grad(tg.linear(x, w, b, act, out_dtype=F32), [x, w, b], torch.empty((0, 24), device="cuda"))
        assert gx.shape == (0, 16) and gw.abs().max() == 0 and gb.abs().max() == 0
        x = rand((5, 16), 3, HF).cuda().requires_grad_()
        e = torch.empty((0, 16), dtype=HF, device="cuda", requires_grad=True)
        gx, ge = torch.autograd.grad(tg.linear(x, e, act=act, out_dtype=F32), [x, e], torch.empty((5, 0), device="cuda"))
        assert gx.abs().max() == 0 and ge.shape == (0, 16)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_act_grad_f32_entry(dtype):
    """dP in units of *scale, the power of two that the largest |dY| sets in binary16;
    only the column sums; nothing around the outputs is written."""
    M, N = 133, 301
    name = "bf16" if dtype == BF else "f16"
    for size in (1e-30, 3e-9, 1.0, 7e8, 1e38):
        dy, pre = rand((M, N), 1, F32).clamp(-3, 3) * size, rand((M, N), 2, dtype)
        dyd, pd = dy.cuda(), pre.cuda()
        for act in ("none", "gelu"):
            dp = torch.full((M + 2, N + 7), 7.0, dtype=dtype, device="cuda")
            db = torch.full((N + 4,), 7.0, device="cuda")
            sc = torch.full((3,), 7.0, device="cuda")
            need = tg.tgemm_act_grad_f32_workspace(M, N)
            ws = torch.empty(need, dtype=torch.uint8, device="cuda")
            for only_db in (False, True):
                rc = tg.tgemm_act_grad_f32(M, N, name, dyd.data_ptr(), N, act, None if act == "none" else pd.data_ptr(), N,
                                           None if only_db else dp[1:].data_ptr(), N + 7,
                                           None if only_db else sc[1:].data_ptr(), "f32", db[2:].data_ptr(), ws.data_ptr(),
                                           need, torch.cuda.current_stream().cuda_stream)
                assert rc == tg.TGEMM_OK
                g = dy.double() * act_grad64(pre.double(), act)
                slack = dy.double().abs() * 2.0 ** -20 * (act != "none")
                want = g.sum(0)
                if g.abs().sum(0).max() < torch.finfo(F32).max:      # (fp32 sums: their partial sums may overflow past that)
                    within(db[2:2 + N], want, slack.sum(0) + (M + 4) * U * g.abs().sum(0) + 2 * U * want.abs(), "db")
            scale = float(sc[1])
            top = float(dy.abs().max())
            assert scale == 1.0 if dtype == BF else (2.0 ** 14 <= top / scale < 2.0 ** 15)
            assert torch.frexp(torch.tensor(scale))[0] == 0.5
            within(dp[1:1 + M, :N].double() * scale, g, slack + half_step(dtype) * 1.01 * g.abs() + tiny(dtype) * scale, "dp")
            dp[1:1 + M, :N] = 7.0
            db[2:2 + N] = 7.0
            sc[1] = 7.0
            assert (dp == 7.0).all() and (db == 7.0).all() and (sc == 7.0).all()


# ------------------------------------------- pre-activations far from zero --

@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_gradient_of_far_preactivations(act):
    """Derivatives are 0 far below zero and 1 far above, also where the kept
    pre-activation has become infinite (binary16 past 65504) or its square does."""
    for dtype, far in ((HF, (300.0, 6.5e4, 9e4, 2e5)), (BF, (300.0, 9e4, 1e19, 1e20, 1e38))):
        for M in (3, 40):
            x = torch.full((M, 1), 8.0, dtype=dtype)
            v = torch.tensor(far + tuple(-f for f in far))
            w = (v / 8).to(dtype)[:, None]
            xd, wd = x.cuda().requires_grad_(), w.cuda().requires_grad_()
            dy = torch.ones((M, len(v)), dtype=dtype, device="cuda")
            gx, gw = torch.autograd.grad(tg.linear(xd, wd, act=act), [xd, wd], dy)
            want = (w[:, 0].double() > 0).double()
            assert torch.equal(gw.cpu()[:, 0].double(), want * 8 * M), (dtype, gw)
            assert gx.isfinite().all()
        # the call by itself
        pre = torch.tensor([[float("inf"), -float("inf"), float("nan"), far[-1], -far[-1]]]).to(dtype).cuda()
        dp, db = tg.act_grad(torch.ones((1, 5), dtype=dtype, device="cuda"), act, pre, F32)
        assert dp[0, [0, 3]].eq(1).all() and dp[0, [1, 4]].eq(0).all() and dp[0, 2].isnan()
        assert db[[0, 3]].eq(1).all() and db[[1, 4]].eq(0).all() and db[2].isnan()


# --------------------------------------- few rows over a long vocabulary --

@pytest.mark.parametrize("R", [1, 5, 17, 32])
def test_xent_few_rows_equal_logits_do_not_drift(R):
    """All logits equal: lse = z + log V. A wave adds some twenty groups of columns,
    four terms each, to its running sum, and the join some thirty parts: 125
    roundings of 2^-24, those of the logarithm and of lse, and one rounding of
    log2(e) z, the same in every term."""
    V, D = 600_000, 8
    for c in (360.0, -360.0, 412.0):     # where log2(e) c rounds by nearly half a step
        h = torch.zeros((R, D), dtype=BF)
        h[:, 0] = c
        w = torch.zeros((V, D), dtype=BF)
        w[:, 0] = 1
        t = torch.full((R,), V - 1)
        loss, lse = tg.linear_cross_entropy(h.cuda(), w.cuda(), t.cuda(), reduction="none", return_lse=True)
        z = float(h[0, 0])
        want = torch.full((R,), z, dtype=torch.float64) + torch.log(torch.tensor(float(V), dtype=torch.float64))
        tol = 125 * U + 2 * U * want.abs() + U * 1.4427 * abs(z)
        within(lse, want, tol, "lse")
        within(loss, want - z, tol, "loss")


@pytest.mark.parametrize("R", [1, 5, 17, 32])
@pytest.mark.parametrize("V", [70_001, 150_000])
@pytest.mark.parametrize("order", ["any", "rising", "falling"])
def test_xent_few_rows_over_several_groups(R, V, order):
    """More groups of columns than waves: the running maximum stays, rises or
    falls from group to group, logits of hundreds; an infinite logit in a later group."""
    D = 16
    h, w, t = xent_case(R, V, D, BF, ignored=0.2, scale=40.0)
    if order != "any":
        z0 = (h[0].double() @ w.double().t())
        w = w[torch.argsort(z0, descending=order == "falling")]
    z, lse, loss, valid, ez = xent64(h, w, t)
    got, gl = tg.linear_cross_entropy(h.cuda(), w.cuda(), t.cuda(), reduction="none", return_lse=True)
    el = e_lse(lse, ez) + 2 * U * 1.4427 * z.abs().amax(1)
    within(gl, lse, el, "lse")
    within(got, loss, torch.where(valid, el + ez + U * loss.abs(), torch.zeros_like(el)), "loss")
    # column V - 3 (a wave's last group): -inf drops out, +inf makes lse infinite
    for v in (-float("inf"), float("inf")):
        wi = w.clone()
        hi = h.clone()
        wi[:, 0] = 0
        wi[V - 3, 0] = v
        hi[:, 0] = 1
        got = tg.linear_cross_entropy(hi.cuda(), wi.cuda(), t.cuda(), reduction="none", return_lse=True)[1]
        if v > 0:
            assert (got == float("inf")).all()
        else:
            z2 = hi[:, 1:].double() @ wi[:, 1:].double().t()
            z2[:, V - 3] = v
            l2 = torch.logsumexp(z2, 1)
            within(got, l2, e_lse(l2, ez) + 2 * U * 1.4427 * z.abs().amax(1), "lse without the column")


# ------------------------------------------------- forward-mode tangents --

def test_forward_mode_is_refused_and_not_dropped():
    """A tangent of any operand raises; none is lost without a word."""
    import torch.autograd.forward_ad as fw
    x, w, b, r = (rand(s, i, BF).cuda() for i, s in enumerate(((4, 16), (24, 16), (24,), (4, 24))))
    t = torch.tensor([1, 2, -100, 3]).cuda()
    calls = {"linear": lambda x, w, b, r: tg.linear(x, w, b, "silu", r),
             "xent": lambda x, w, b, r: tg.linear_cross_entropy(x, w, t),
             "tn": lambda x, w, b, r: tg.gemm_tn(x, r),
             "act_grad": lambda x, w, b, r: tg.act_grad(r, "silu", r)}
    uses = {"linear": (0, 1, 2, 3), "xent": (0, 1), "tn": (0, 3), "act_grad": (3,)}
    for name, call in calls.items():
        for i in uses[name]:
            for leaf in (False, True):
                ops = [q.clone().requires_grad_(leaf) for q in (x, w, b, r)]
                with fw.dual_level():
                    ops[i] = fw.make_dual(ops[i], torch.ones_like(ops[i]))
                    with pytest.raises(NotImplementedError, match="forward-mode"):
                        call(*ops)
    with fw.dual_level():                            # operands without tangents are served inside a level too
        a = tg.linear(x, w, b, "silu", r)
    assert torch.equal(a, tg.linear(x, w, b, "silu", r))


# ------------------------------------------ row strides and vocabularies --

@pytest.mark.parametrize("R", [4, 40])
def test_xent_long_strides_are_copied(R):
    """Rows further apart than the kernels' offsets reach give the same results as contiguous ones."""
    ld, D, V = 4_000_008, 64, 30
    h, w, t = xent_case(R, V, D, BF, ignored=0.0)
    buf = torch.empty(R * ld, dtype=BF, device="cuda")
    hl = buf.as_strided((R, D), (ld, 1))
    hl.copy_(h.cuda())
    if R > V:                                        # (the buffer holds as many rows)
        wl = buf.as_strided((V, D), (ld, 1), 1024)
        wl.copy_(w.cuda())
    for kw in ({"reduction": "none"}, {}, {"recompute": True}):
        def both(h, w):
            hd, wd = h.detach().requires_grad_(), w.detach().requires_grad_()
            out = tg.linear_cross_entropy(hd, wd, t.cuda(), **kw)
            return (out.detach(),) + torch.autograd.grad(out.sum(), [hd, wd])
        want = both(h.cuda(), w.cuda())
        for ops in ((hl, w.cuda()),) + (((h.cuda(), wl), (hl, wl)) if R > V else ()):
            got = both(*ops)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(tg.linear_cross_entropy(hl, w.cuda(), t.cuda(), reduction="none"),
                           tg.linear_cross_entropy(h.cuda(), w.cuda(), t.cuda(), reduction="none"))


@pytest.mark.parametrize("reduction", ["sum", "mean"])
def test_xent_reduction_over_no_rows(reduction):
    """A sum over no rows is 0 (a mean divides by one at least), its gradients are zeros."""
    w = rand((30, 16), 1, BF).cuda().requires_grad_()
    h = torch.empty((0, 16), dtype=BF, device="cuda", requires_grad=True)
    t = torch.empty((0,), dtype=torch.int64, device="cuda")
    for kw in ({}, {"recompute": True}, {"return_lse": True}):
        loss = tg.linear_cross_entropy(h, w, t, reduction=reduction, **kw)
        if kw.get("return_lse"):
            loss, lse = loss
            assert lse.shape == (0,)
        assert loss.shape == () and loss.dtype == F32 and loss.item() == 0
        gh, gw = torch.autograd.grad(loss, [h, w])
        assert gh.shape == (0, 16) and gw.shape == w.shape and gw.abs().max() == 0
    with torch.no_grad():
        assert tg.linear_cross_entropy(h, w, t, reduction=reduction).item() == 0


@pytest.mark.parametrize("R", [5, 40])
def test_xent_vocabulary_past_four_million(R):
    """More columns than an operand's row may have elements: the columns are rows of the weight."""
    V, D = 4_000_037, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    h = torch.randn((R, D), generator=g, device="cuda").to(BF).requires_grad_()
    w = (torch.randn((V, D), generator=g, device="cuda") * 0.5).to(BF).requires_grad_()
    t = torch.randint(0, V, (R,), generator=g, device="cuda")
    t[1], t[2], t[3] = V - 1, 4_000_000, -100
    loss, lse = tg.linear_cross_entropy(h, w, t, reduction="none", return_lse=True)
    gh, gw = torch.autograd.grad(loss.sum(), [h, w])
    hd, wd = h.detach().double(), w.detach().double()
    z = hd @ wd.t()
    l64 = torch.logsumexp(z, 1)
    zt = z.gather(1, t.clamp(min=0)[:, None])[:, 0]
    live = (t >= 0).double()
    ez = ((D + 4) * U * (hd.abs() @ wd.abs().t()).amax(1)).cpu()
    el = e_lse(l64.cpu(), ez)
    within(lse, l64.cpu(), el, "lse")
    within(loss, ((l64 - zt) * live).cpu(), (el + ez + U * (l64 - zt).abs().cpu()) * live.cpu() , "loss")
    # z becomes the coefficients
    z.sub_(l64[:, None]).exp_().mul_(live[:, None])
    z[torch.arange(R, device="cuda"), t.clamp(min=0)] -= live
    want = z @ wd
    rel = (half_step(BF) * 1.02 + (2 * ez + 2.0 ** -18).cuda())[:, None]
    tol = (rel * z.abs() + 4 * U * (z.abs() > 0.5)) @ wd.abs() + (V + 4) * U * (z.abs() @ wd.abs()) + half_step(BF) * 1.02 * want.abs()
    within(gh, want.cpu(), tol.cpu(), "dh")
    cols = torch.cat([torch.tensor([0, 1, 3_999_999, 4_000_000, 4_000_001, V - 2, V - 1], device="cuda"), t[t >= 0]])
    want = z[:, cols].t() @ hd
    tol = ((rel * z.abs() + 4 * U * (z.abs() > 0.5))[:, cols].t() @ hd.abs() + (R + 4) * U * (z[:, cols].abs().t() @ hd.abs())
           + half_step(BF) * 1.02 * want.abs())
    within(gw[cols], want.cpu(), tol.cpu(), "dw")


@pytest.mark.parametrize("M", [1, 3, 40])
def test_linear_of_more_than_four_million_columns(M):
    """A residual and a kept pre-activation whose rows are longer than the tiles'
    offsets reach: those sizes do not run on tiles."""
    N, K = 4_000_003, 8
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn((M, K), generator=g, device="cuda").to(BF).requires_grad_()
    w = (torch.randn((N, K), generator=g, device="cuda") * 0.4).to(BF).requires_grad_()
    r = torch.randn((M, N), generator=g, device="cuda").to(BF).requires_grad_()
    y = tg.linear(x, w, None, "silu", r)
    xs, ws, rs = x.detach().cpu(), w.detach().cpu(), r.detach().cpu()
    p, ref, e = forward64(xs, ws, None, "silu", rs)
    within(y, ref, y_tol(p, ref, e, BF, rs), "y")
    dy = torch.randn((M, N), generator=g, device="cuda").to(BF)
    gx, gw, gr = torch.autograd.grad(y, [x, w, r], dy)
    assert torch.equal(gr, dy)
    h, d64 = half_step(BF), dy.double().cpu()
    dp = d64 * act_grad64(p, "silu")
    er = 1.01 * h * dp.abs() + 1.01 * d64.abs() * (1.2 * (e + h * 1.01 * p.abs()) + 2.0 ** -20)
    want = dp.t() @ xs.double()
    within(gw, want, er.t() @ xs.double().abs() + (M + 4) * U * (dp.abs().t() @ xs.double().abs()) + h * 1.02 * want.abs(), "dw")
    want = dp @ ws.double()
    within(gx, want, er @ ws.double().abs() + (N + 4) * U * (dp.abs() @ ws.double().abs()) + h * 1.02 * want.abs(), "dx")


# --------------------------------------------- sizes past one launch's grid --

def test_few_rows_of_more_columns_than_one_grid():
    """2^27 columns and a ragged end: past 2^32 threads in one launch of 16 columns a workgroup."""
    N, K = 2 ** 27 + 5, 1
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randint(-8, 9, (N, K), generator=g, device="cuda", dtype=torch.int8).to(BF)
    b = torch.randint(-8, 9, (N,), generator=g, device="cuda", dtype=torch.int8).to(BF)
    for M in (1, 2):
        x = torch.full((M, K), 2.0, dtype=BF, device="cuda")
        y = tg.linear(x, w, b, "relu")
        for i in range(M):
            assert torch.equal(y[i], (w[:, 0] * 2 + b).clamp(min=0))     # small whole numbers: exact


def test_column_sums_of_more_columns_than_one_grid():
    N = 2 ** 30 + 3
    dy = torch.randint(-8, 9, (1, N), device="cuda", dtype=torch.int8).to(BF)
    dp, db = tg.act_grad(dy, "none", None, BF)
    assert torch.equal(db, dy[0])


def test_xent_of_more_rows_than_one_grid():
    """2^28 rows and a ragged end of a vocabulary of one: lse is the logit, the loss 0."""
    R = 2 ** 28 + 21
    h = torch.randint(-8, 9, (R, 8), device="cuda", dtype=torch.int8).to(BF)
    w = torch.zeros((1, 8), dtype=BF, device="cuda")
    w[0, 3] = 1
    t = torch.zeros((R,), dtype=torch.int64, device="cuda")
    loss, lse = tg.linear_cross_entropy(h, w, t, reduction="none", return_lse=True)
    # (the exponential against the maximum is one step of log2(e) z away from 1)
    z = h[:, 3].float()
    assert ((lse - z).abs() <= e_lse(z, 0.0)).all() and (loss.abs() <= e_lse(z, 0.0)).all()


# ------------------------------------- walks over several tiles, and pieces --

@pytest.mark.parametrize("K", [130, 515, 128])
@pytest.mark.parametrize("layout", ["NxK", "KxN"])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_linear_walk(dtype, layout, K):
    """More 256-row tiles than compute units (17 x 18), ragged in every axis: the
    load stream goes on from one tile to the next around each end of tile. With
    residual and pre-activation; bit for bit with tiles of 128 rows, and sampled
    rows and columns against 64 bits."""
    M, N = 4200, 4401
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn((M, K), generator=g, device="cuda").to(dtype)
    w = (torch.randn((N, K), generator=g, device="cuda") * K ** -0.5).to(dtype)
    b, r = torch.randn((N,), generator=g, device="cuda"), torch.randn((M, N), generator=g, device="cuda").to(dtype)
    wl = w if layout == "NxK" else w.t().contiguous()
    for out in (dtype, F32):
        y = tg.linear(x, wl, b, "silu", r, out_dtype=out, w_layout=layout, tile_m=256, k_step=64, splits=1)
        z = tg.linear(x, wl, b, "silu", r, out_dtype=out, w_layout=layout, tile_m=128, k_step=64, splits=1)
        assert torch.equal(y, z)
        plain = tg.linear(x, wl, b, "silu", None, out_dtype=out, w_layout=layout, tile_m=256, k_step=64, splits=1)
        for rows, cols in ((slice(None, None, 149), slice(None)), (slice(None), slice(None, None, 157)), (slice(-3, None), slice(None))):
            xs, ws, bs, rs = x[rows].cpu(), w[cols].cpu(), b[cols].cpu(), r[rows, cols].cpu()
            p, ref, e = forward64(xs, ws, bs, "silu", rs)
            within(y[rows, cols], ref, y_tol(p, ref, e, out, rs), "y")
            p, ref, e = forward64(xs, ws, bs, "silu", None)
            within(plain[rows, cols], ref, y_tol(p, ref, e, out, None), "plain")
    # through autograd: pre is kept; automatic choices
    xd, wd, bd, rd = (q.clone().requires_grad_() for q in (x, wl, b, r))
    y = tg.linear(xd, wd, bd, "silu", rd, w_layout=layout)
    dy = torch.randn((M, N), generator=g, device="cuda").to(dtype)
    gx, gw, gb = torch.autograd.grad(y, [xd, wd, bd], dy)
    p = x.double() @ w.double().t() + b.double()
    e = (K + 6) * U * (x.double().abs() @ w.double().abs().t()) + 2 * U * p.abs()
    h, d64 = half_step(dtype), dy.double()
    dp = d64 * act_grad64(p, "silu")
    ep = d64.abs() * (1.2 * (e + h * 1.01 * p.abs() + tiny(dtype)) + 2.0 ** -20)
    er = ep + h * 1.01 * dp.abs() + tiny(dtype)
    want = dp @ w.double()
    within(gx, want.cpu(), (1.01 * (er @ w.double().abs()) + (N + 4) * U * (dp.abs() @ w.double().abs()) + h * 1.02 * want.abs()
                            + tiny(dtype)).cpu(), "dx")
    want = dp.t() @ x.double()
    within(gw if layout == "NxK" else gw.t(), want.cpu(),
           (1.01 * (er.t() @ x.double().abs()) + (M + 4) * U * (dp.abs().t() @ x.double().abs()) + h * 1.02 * want.abs()
            + tiny(dtype)).cpu(), "dw")
    want = dp.sum(0)
    within(gb, want.cpu(), (ep.sum(0) + (M + 4) * U * dp.abs().sum(0) + 2 * U * want.abs()).cpu(), "db")


@pytest.mark.parametrize("K", [130, 515, 128])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_gemm_tn_walk(dtype, K):
    """The same for A^T B, into fp32 and 16 bits, with what C holds added."""
    M, N = 4200, 4401
    g = torch.Generator(device="cuda").manual_seed(K)
    a = torch.randn((K, M + 3), generator=g, device="cuda").to(dtype)[:, :M]
    b = torch.randn((K, N + 2), generator=g, device="cuda").to(dtype)[:, :N]
    ad, bd = a.double(), b.double()
    ref, s = ad.t() @ bd, ad.abs().t() @ bd.abs()
    for out in (dtype, F32):
        c0 = torch.randn((M, N), generator=g, device="cuda").to(out)
        got = [tg.gemm_tn(a, b, out_dtype=out, tile_m=tm, k_step=64, splits=1) for tm in (256, 128)]
        acc = [tg.gemm_tn(a, b, out=c0.clone(), accumulate=True, tile_m=tm, k_step=64, splits=1) for tm in (256, 128)]
        assert torch.equal(*got) and torch.equal(*acc)
        within(got[0], ref.cpu(), ((K + 4) * U * s + half_step(out) * 1.01 * ref.abs() + tiny(out)).cpu(), "c")
        want = ref + c0.double()
        within(acc[0], want.cpu(), ((K + 4) * U * s + 2 * U * (want.abs() + c0.double().abs()) + half_step(out) * 1.01 * want.abs()
                                    + tiny(out)).cpu(), "c + c0")


def check_xent_step(R, V, D, dtype, rows, cols, dlse=False, ignored=0.1, scale=2.0, **kw):
    """Loss, lse and the gradients of all rows and of the weight's rows `cols` against 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(R + V + D)
    h = torch.randn((R, D), generator=g, device="cuda").to(dtype).requires_grad_()
    w = (torch.randn((V, D), generator=g, device="cuda") * scale * D ** -0.5).to(dtype).requires_grad_()
    t = torch.randint(0, V, (R,), generator=g, device="cuda")
    t[torch.rand((R,), generator=g, device="cuda") < ignored] = -100
    cols = torch.tensor(cols, device="cuda")
    t[5:5 + len(cols)] = cols                        # targets at the sampled columns
    t[-1] = V - 1
    e = torch.randn((R,), generator=g, device="cuda") if dlse else torch.zeros(R, device="cuda")
    if dlse:
        loss, lse = tg.linear_cross_entropy(h, w, t, reduction="sum", return_lse=True, **kw)
        gh, gw = torch.autograd.grad([loss, lse], [h, w], [torch.ones_like(loss), e])
    else:
        loss = tg.linear_cross_entropy(h, w, t, reduction="sum", **kw)
        gh, gw = torch.autograd.grad(loss, [h, w])
    hd, wd = h.detach().double(), w.detach().double()
    idx = torch.arange(0, R, max(R // rows, 1), device="cuda")
    l64 = torch.cat([torch.logsumexp(hd[i:i + 512] @ wd.t(), 1) for i in range(0, R, 512)])
    valid = t >= 0
    zt = (hd * wd[t.clamp(min=0)]).sum(1)
    l = ((l64 - zt) * valid).sum()
    # (norms bound the sums of absolute values)
    ez = (D + 4) * U * float(hd.norm(dim=1).max() * wd.norm(dim=1).max())
    el = ez + 2.0 ** -20 + 4 * U * float(l64.abs().max())
    within(loss, l.cpu(), ((el + ez) * valid.sum() + 8 * U * l.abs()).cpu(), "loss")
    if dlse:
        within(lse, l64.cpu(), torch.full_like(l64, el).cpu(), "lse")
    hs = half_step(dtype)
    a, ge = valid.double(), e.double()
    top = float(torch.maximum((a + ge).abs(), ge.abs()).max().clamp(min=1))
    once = dtype == BF and not dlse and not kw.get("recompute") and R >= 33

    def coefs(i, c):
        p = torch.exp(hd[i] @ wd[c].t() - l64[i, None])
        hot = (t[i, None] == (torch.arange(V, device="cuda") if isinstance(c, slice) else c)[None, :]).double()
        pa = (a + ge)[i, None].abs() * p
        G = (a + ge)[i, None] * p - a[i, None] * hot
        eG = pa * (ez + el + 2.0 ** -20) + 4 * U * (pa + a[i, None] * hot)
        if once:
            eG = eG + hs * 1.01 * pa * (1 - hot)
        eG = eG + hs * 1.01 * (G.abs() + eG) + (2.0 ** -39 * top if dtype == HF else 0.0)
        return G, eG * ((a != 0) | (ge != 0))[i, None]

    G, eG = coefs(idx, slice(None))
    want = G @ wd
    within(gh[idx], want.cpu(), (1.01 * (eG @ wd.abs()) + (V + 4) * U * (G.abs() @ wd.abs()) + hs * 1.02 * want.abs()
                                 + tiny(dtype)).cpu(), "dh")
    G, eG = coefs(slice(None), cols)
    want = G.t() @ hd
    within(gw[cols], want.cpu(), (1.01 * (eG.t() @ hd.abs()) + (R + 4) * U * (G.abs().t() @ hd.abs()) + hs * 1.02 * want.abs()
                                  + tiny(dtype)).cpu(), "dw")


@pytest.mark.parametrize("dtype,kw", [(BF, {}), (BF, {"recompute": True}), (HF, {}), (BF, {"dlse": True})])
def test_xent_walk(dtype, kw):
    """Long rows over many tiles (17 x 79 of 256 rows: walks), ragged in every axis."""
    check_xent_step(4200, 20001, 1030, dtype, 40, [0, 255, 256, 1023, 12345, 19999, 20000], **kw)


def test_xent_streamed_exponentials():
    """More than 512 MiB of exponentials: stored past the caches."""
    check_xent_step(4100, 70001, 640, BF, 20, [0, 127, 128, 69887, 69888, 70000])


@pytest.mark.parametrize("dtype,kw", [(BF, {"recompute": True}), (HF, {"dlse": True}), (HF, {})])
def test_xent_seams_of_the_pieces(dtype, kw):
    """Three pieces of the vocabulary, 23552, 23552 and 22897 columns: the weight's
    rows and targets on both sides of each seam, running sums over the pieces."""
    check_xent_step(9000, 70001, 16, dtype, 20,
                    [0, 1, 23550, 23551, 23552, 23553, 47102, 47103, 47104, 47105, 69999, 70000], scale=0.5, **kw)


def test_xent_recompute_keeps_no_logits():
    """recompute=True: a step's memory is its gradients, 2^28 coefficients (512 MiB)
    and the sums of split products, and the forward pass alone keeps rows, where
    fp32 logits take 3.7 GB; with gradients at once it is 2 bytes a logit."""
    R, V, D = 8192, 114_688, 64
    h = torch.randn((R, D), device="cuda").to(BF).requires_grad_()
    w = torch.randn((V, D), device="cuda").to(BF).requires_grad_()
    t = torch.randint(0, V, (R,), device="cuda")

    def peak(fn):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        torch.cuda.reset_peak_memory_stats()
        base = torch.cuda.memory_allocated()
        fn()
        return torch.cuda.max_memory_allocated() - base

    loss = []
    forward = peak(lambda: loss.append(tg.linear_cross_entropy(h, w, t, recompute=True)))
    # parts of 128 columns (8 bytes), and a handful of fp32 rows
    assert forward <= R * (V // 128) * 8 + 64 * R + (1 << 20)
    backward = peak(lambda: torch.autograd.grad(loss[0], [h, w]))
    sums = 2 ** 28 * 2 * 1.05 + 65 * R * D * 4 + 64 * 4 * 2 ** 28 // R * D
    assert backward <= sums + 2 * (R + V) * D * 2, (backward, sums)
    del loss
    at_once = peak(lambda: torch.autograd.grad(tg.linear_cross_entropy(h, w, t), [h, w]))
    assert at_once <= R * (V + 128) * 2 + R * (V // 128) * 8 + 64 * 4 * (R + V) * D + 2 * (R + V) * D * 2 + (1 << 20)


def test_gemm_tn_into_a_tensor_that_autograd_keeps():
    """Writing out marks it as changed: a backward pass that had saved its old values says so."""
    a, b = rand((20, 16), 1, BF).cuda(), rand((20, 24), 2, BF).cuda()
    c = rand((16, 24), 3, F32).cuda()
    s = torch.ones((), device="cuda", requires_grad=True)
    y = (c * s).sum()                                # keeps c for s's gradient
    before = c._version
    tg.gemm_tn(a, b, out=c, accumulate=True)
    assert c._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    leaf = torch.zeros((16, 24), device="cuda", requires_grad=True)
    with pytest.raises(ValueError, match="requires a gradient"):
        tg.gemm_tn(a, b, out=leaf)
    with torch.no_grad():
        tg.gemm_tn(a, b, out=leaf)                   # as an optimizer would
    assert leaf.abs().max() > 0
    with torch.inference_mode():
        assert torch.equal(tg.gemm_tn(a, b, out=torch.zeros((16, 24), device="cuda"), accumulate=True), tg.gemm_tn(a, b, out_dtype=F32))


def test_captured_step_with_an_f32_result_replays():
    """A binary16 layer with an fp32 result, its gradients (whose scale is found on
    the device) and a few rows' loss in a graph: every replay equals the eager
    results, for gradients of any size, with eager work in between."""
    x, w = rand((96, 256), 1, HF).cuda(), rand((200, 256), 2, HF, 0.06).cuda()
    v, t = rand((1000, 200), 3, HF, 0.1).cuda(), torch.randint(0, 1000, (16,)).cuda()
    dy = rand((96, 200), 4, F32).cuda()

    def step():
        xs, ws = x.detach().requires_grad_(), w.detach().requires_grad_()
        b = torch.zeros((200,), device="cuda", requires_grad=True)
        y = tg.linear(xs, ws, b, "gelu", out_dtype=F32)
        loss = tg.linear_cross_entropy(y[:16].half(), v, t)
        return (y.detach(), loss.detach()) + torch.autograd.grad([y, loss], [xs, ws, b], [dy, torch.ones_like(loss)])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for i, size in enumerate((1.0, 1e-9, 1e7, 1.0)):
        x.copy_(rand((96, 256), 10 + i, HF))
        dy.copy_(rand((96, 200), 20 + i, F32) * size)
        g.replay()
        torch.cuda.synchronize()
        want = step()
        again = step()
        torch.cuda.synchronize()
        for a, b, c in zip(out, want, again):
            assert torch.equal(a, b) and torch.equal(b, c)
            assert b.abs().max() > 0
