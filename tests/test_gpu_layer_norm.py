"""det_layer_norm and its gradients against 64-bit statements.

Tolerances, u = 2^-24: a thread adds 4 pairs of columns one after the other, its two eights and the pairs' halves; then
trees over 32 lanes and 32 warps: an addend passes at most depth = 4 + 1 + 1 + 5 + 5 additions.  With s the standard deviation:
  mean   off by at most (depth + 2) u mean|x|
  rstd   relative (depth + 8) u / 2 for the tree, the squares and the root, plus what the mean's error adds to the squares,
         (error of the mean / s)^2 and the differences' roundings u
  xh     (error of the mean + u |x - mean|) rstd + |xh| (error of rstd + 2 u)
and a result in T is rounded by half a step, eps(T) / 2.  The gradients take mean and rstd as given.  A column's sum passes
rows / parts additions in a register, 8 of groups, parts / 32 of a strand and 5 of the join."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24
DEPTH = 16


@pytest.fixture(scope="module")
def det():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from deterministic_floating_point_gb300 import _build, det as d
    _build.build()
    return d


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def close(got, want, tol, what=""):
    got = got.double().cpu()
    assert got.shape == want.shape
    off = (got - want).abs()
    assert bool((off <= tol).all()), (what, float((off - tol).max()), float(off.max()))


def smallest(dtype):
    """What rounding to a subnormal may be off by."""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps


def stats(x, eps):
    x = x.double()
    mean = x.mean(-1)
    var = ((x - mean[..., None]) ** 2).mean(-1)
    return mean, 1 / torch.sqrt(var + eps), var


def check_forward(r, x, w, b, eps):
    mean, rstd, var = stats(x, eps)
    e_mean = (DEPTH + 2) * U * x.double().abs().mean(-1)
    close(r.mean, mean, e_mean + 1e-300, "mean")
    # of var + eps: the tree, the squares and differences, the mean's error and the last operations
    e_var = var * (DEPTH + 6) * U + e_mean ** 2 * 1.01 + 4 * U * (var + eps)
    e_rstd = rstd * (e_var / (var + eps) / 2 * 1.01 + 4 * U)
    close(r.rstd, rstd, e_rstd, "rstd")
    d = (x.double() - mean[..., None])
    xh = d * rstd[..., None]
    e_xh = (e_mean[..., None] + U * d.abs()) * rstd[..., None] + d.abs() * e_rstd[..., None] + 2 * U * xh.abs()
    wd = torch.ones(()).double() if w is None else w.double()
    bd = torch.zeros(()).double() if b is None else b.double()
    want = xh * wd + bd
    close(r.out, want, e_xh * wd.abs() * 1.01 + 2 * U * (xh * wd).abs() + half_step(x.dtype) * want.abs() * 1.01
          + smallest(x.dtype), "out")


def column_depth(rows, cols):
    """Additions on a column's way: a register's, the groups of a CTA, a strand of the join and its tree.  (A row takes the
    warps it needs, here rounded up to a power of two: 256 threads hold as many groups of 3 warps as of 4, of 5 as of 8.)"""
    eights = 2 if cols > 256 else 1
    threads = max(32, 1 << max(0, math.ceil(math.log2(cols / (8 * eights)))))
    at_a_time = max(1, 256 // threads)
    parts = max(1, min(-(-rows // at_a_time), 152 * (1 if threads > 256 else 3 if eights == 1 else 2)))
    return -(-rows // (parts * at_a_time)) + at_a_time + -(-parts // 32) + 6


def check_backward(r, g, x, mean, rstd, w, param_dtype):
    rows, cols = x.shape
    g, x, m, s = g.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    wd = torch.ones(cols).double() if w is None else w.double()
    xh = (x - m) * s
    e_xh = 2 * U * xh.abs() * 1.01
    gw = g * wd
    one, two = gw.mean(1, keepdim=True), (gw * xh).mean(1, keepdim=True)
    e_one = (DEPTH + 4) * U * gw.abs().mean(1, keepdim=True)
    e_two = (DEPTH + 8) * U * (gw * xh).abs().mean(1, keepdim=True)
    if r.x is not None:
        want = s * (gw - one - xh * two)
        big = gw.abs() + one.abs() + (xh * two).abs()
        tol = s * (e_one + xh.abs() * e_two + (e_xh * two.abs()) + 6 * U * big) * 1.01
        dt = r.x.dtype
        close(r.x, want, tol + half_step(dt) * want.abs() * 1.01 + smallest(dt), "x")
    depth = column_depth(rows, cols)
    for got, terms in ((r.weight, g * xh), (r.bias, g)):
        if got is not None:
            want = terms.sum(0)
            close(got, want, (depth + 4) * U * terms.abs().sum(0) * 1.01 + half_step(param_dtype) * want.abs() * 1.01
                  + smallest(param_dtype), "params")


def make(rows, cols, dtype, seed, offset=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=gen) * 1.5 + torch.randn(rows, 1, generator=gen) * offset
    g = torch.randn(rows, cols, generator=gen)
    w = torch.randn(cols, generator=gen) * 0.3 + 1
    b = torch.randn(cols, generator=gen) * 0.3
    return x.to(dtype), g.to(dtype), w, b


SIZES = [(0, 8), (1, 1), (3, 2), (5, 7), (8, 8), (9, 31), (33, 32), (2, 255), (3, 256), (3, 257), (700, 64), (17, 511),
         (4, 512), (5, 513), (1300, 100), (3, 1000), (3, 1024), (650, 1030), (2, 2048), (3, 4095), (310, 4096), (2, 4097),
         (3, 8192), (2, 8200), (160, 16376), (3, 16383), (2, 16384), (450, 1401), (700, 2500), (330, 6000), (200, 10300)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("kind", list(DTYPES))
def test_forward_and_gradients(det, rows, cols, kind):
    dtype = DTYPES[kind]
    x, g, w, b = make(rows, cols, dtype, rows + cols)
    for param in {torch.float32, dtype}:
        wp, bp = w.to(param), b.to(param)
        r = det.det_layer_norm(x.cuda(), wp.cuda(), bp.cuda(), eps=1e-5)
        check_forward(r, x, wp, bp, 1e-5)
        grads = det.det_layer_norm_backward(g.cuda(), x.cuda(), r.mean, r.rstd, wp.cuda())
        check_backward(grads, g, x, r.mean.cpu(), r.rstd.cpu(), wp, param)


def test_without_weight_or_bias_and_parts_of_the_gradients(det):
    x, g, w, b = make(70, 300, torch.bfloat16, 3)
    xc, gc = x.cuda(), g.cuda()
    check_forward(det.det_layer_norm(xc), x, None, None, 1e-5)
    check_forward(det.det_layer_norm(xc, w.cuda(), eps=0.1), x, w, None, 0.1)
    check_forward(det.det_layer_norm(xc, bias=b.cuda(), eps=0.0), x, None, b, 0.0)
    r = det.det_layer_norm(xc, w.cuda())
    whole = det.det_layer_norm_backward(gc, xc, r.mean, r.rstd, w.cuda())
    for want in ((True, False, False), (False, True, False), (False, False, True), (False, True, True), (True, False, True)):
        part = det.det_layer_norm_backward(gc, xc, r.mean, r.rstd, w.cuda(), want_x=want[0], want_weight=want[1],
                                           want_bias=want[2])
        for wanted, a, c in zip(want, part, whole):
            assert (torch.equal(a, c) if wanted else a is None)
    plain = det.det_layer_norm_backward(gc, xc, r.mean, r.rstd, dtype=torch.bfloat16)
    check_backward(plain, g, x, r.mean.cpu(), r.rstd.cpu(), None, torch.bfloat16)


@pytest.mark.parametrize("kind", list(DTYPES))
@pytest.mark.parametrize("cols", [7, 64, 264, 1000, 4100])
def test_strides_alignment_and_neighbours_do_not_change_bits(det, kind, cols):
    dtype = DTYPES[kind]
    x, g, w, b = make(40, cols, dtype, cols)
    w, b = w.cuda(), b.cuda()
    whole = det.det_layer_norm(x.cuda(), w, b)
    grads = det.det_layer_norm_backward(g.cuda(), x.cuda(), whole.mean, whole.rstd, w)
    for pad, off in ((8, 0), (16, 8), (3, 1), (9, 5)):
        wide = torch.full((40, cols + pad + off), float("nan"), dtype=dtype, device="cuda")
        wide[:, off:off + cols] = x.cuda()
        wg = torch.full_like(wide, float("nan"))
        wg[:, off:off + cols] = g.cuda()
        xs, gs = wide[:, off:off + cols], wg[:, off:off + cols]
        r = det.det_layer_norm(xs, w, b)
        assert all(torch.equal(p, q) for p, q in zip(r, whole))
        again = det.det_layer_norm_backward(gs, xs, r.mean, r.rstd, w)
        assert all(torch.equal(p, q) for p, q in zip(again, grads))
    for i in (0, 13, 39):
        one = det.det_layer_norm(x[i:i + 1].cuda(), w, b)
        assert all(torch.equal(p[0], q[i]) for p, q in zip(one, whole))
        alone = det.det_layer_norm_backward(g[i:i + 1].cuda(), x[i:i + 1].cuda(), one.mean, one.rstd, w)
        assert torch.equal(alone.x[0], grads.x[i])
    # in place, and more dimensions
    y, h = x.cuda(), x.cuda().view(4, 10, cols)
    assert torch.equal(det.det_layer_norm(y, w, b, out=y).out, whole.out) and torch.equal(y, whole.out)
    assert torch.equal(det.det_layer_norm(h, w, b).rstd, whole.rstd.view(4, 10))


def test_far_means_constants_and_special_values(det):
    # values far from 0: what the mean leaves, not a difference of large sums
    x, _, w, b = make(20, 700, torch.float32, 9, offset=3000.0)
    check_forward(det.det_layer_norm(x.cuda(), w.cuda(), b.cuda()), x, w, b, 1e-5)
    # a constant row: its mean may be off by the tree's roundings, its result stays near the bias
    c = torch.full((2, 1000), 0.1)
    r = det.det_layer_norm(c.cuda(), w[:1].expand(1000).contiguous().cuda(), b[:1].expand(1000).contiguous().cuda())
    check_forward(r, c, w[:1].expand(1000), b[:1].expand(1000), 1e-5)
    bad = torch.randn(6, 300, generator=torch.Generator().manual_seed(1))
    bad[1, 7], bad[2, 299], bad[3, 0] = float("nan"), float("inf"), -float("inf")
    r = det.det_layer_norm(bad.cuda())
    for i in (1, 2, 3):
        assert r.out[i].isnan().all() and not r.mean[i].isfinite()
    for i in (0, 4, 5):
        assert r.out[i].isfinite().all()


def test_rows_that_do_not_fit_the_grid_once(det):
    """More rows than CTAs stay resident, read with the next row on its way."""
    for cols, rows in ((40, 70_001), (600, 9000), (2050, 3001), (16384, 400)):
        x, g, w, b = make(rows, cols, torch.bfloat16, cols)
        r = det.det_layer_norm(x.cuda(), w.cuda(), b.cuda())
        check_forward(r, x, w, b, 1e-5)
        grads = det.det_layer_norm_backward(g.cuda(), x.cuda(), r.mean, r.rstd, w.cuda())
        check_backward(grads, g, x, r.mean.cpu(), r.rstd.cpu(), w, torch.float32)


def plain(x, w, b, eps=1e-5):
    m = x.mean(-1, keepdim=True)
    return (x - m) / torch.sqrt(((x - m) ** 2).mean(-1, keepdim=True) + eps) * w + b


def test_autograd_against_differentiation_and_differences(det):
    from deterministic_floating_point_gb300 import autograd
    x, g, w, b = make(24, 130, torch.float32, 4)
    leaves = [t.cuda().requires_grad_(True) for t in (x, w, b)]
    out = autograd.layer_norm(leaves[0].view(4, 6, 130), leaves[1], leaves[2])
    (out.view(24, 130) * g.cuda()).sum().backward()
    ref = [t.double().requires_grad_(True) for t in (x, w, b)]
    (plain(*ref) * g.double()).sum().backward()
    size = [float(t.grad.abs().max()) for t in ref]
    for got, want, top in zip(leaves, ref, size):
        # the sums pass 60 roundings or fewer; addends cancel to no less than a hundredth of the largest result here
        close(got.grad, want.grad, 100 * 60 * U * top)
    gen = torch.Generator().manual_seed(5)
    step = 1e-5
    for i, t in enumerate((x, w, b)):
        d = torch.randn(t.shape, generator=gen).double()
        args = [a.double() for a in (x, w, b)]
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + step * d, args[i] - step * d
        slope = ((plain(*up) * g.double()).sum() - (plain(*down) * g.double()).sum()) / (2 * step)
        got = (leaves[i].grad.double().cpu() * d).sum()
        # 32-bit gradients, and the differences' own second-order error (step^2) and roundings (2^-52 / step)
        assert abs(float(got - slope)) <= 100 * 60 * U * size[i] * float(d.abs().sum()) + 1e-6 * abs(float(slope)) + 1e-6
    # a gradient that is a scalar's expansion, and one whose rows are transposed
    y = autograd.layer_norm(leaves[0], leaves[1], leaves[2])
    y.sum().backward()
    xt = x.cuda().t().contiguous().t().requires_grad_(True)
    autograd.layer_norm(xt, leaves[1], leaves[2]).t().contiguous().sum().backward()
    assert xt.grad.isfinite().all()
