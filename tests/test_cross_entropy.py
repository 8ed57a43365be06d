"""Cross entropy with label smoothing, z-loss and capped logits, of logits and of hidden . W^T, against the definition in
64 bits.

Tolerances (u = 2^-24, h = half a step of the output's type, per row with g the upstream gradient):
  logits    a capped logit takes a rounded quotient, tanh (3e-7) and a rounded product: off by 8 u |z|; of hidden . W^T,
            a tensor-core step adds 16 products to the running sum and drops up to a step of 2 u of the largest, and the
            mean of that is given back, u / 4 a step: off by d = (D / 16 + 1) 2.25 u sum |h w|. A capped logit's own d is no larger, since |dz/dx| <= 1.
  p         the argument's rounding (|log p| + 2) u, two more of log S, the base-2 exponential 3 u, S's own relative
            error (at most 40 additions of a thread and 6 u of its terms): p (64 + 2 |log p|) u, and p 2 d
  loss      log S as S: 64 u; m, z_t: 2 u of themselves and d; the mean: 40 additions and two roundings of
            mean |z - m|; zeta lse^2 follows lse; h |loss|
  dx        g slope (dp (1 + 2 zeta |lse|) + 8 u (p (1 + 2 zeta |lse|) + [j = t] + e / V)) + 32 u |dx| (the slope:
            16 u absolute where it is over 2 / 3, 20 u relative elsewhere) + 6 u |x / c| |dx| + h |dx|: the slope is about
            4 e^a, a = -2 |x / c|, and a carries three roundings (1 / c, the product with x, that with log2(e)), which
            are 3 u |a| = 6 u |x / c| of e^a
  dhidden, dW: every term's dz off as dx without h, by 2^-16 of itself as a pair of bf16 values (2^-8 as one), and the
            sum over K terms by (K / 16 + 2) 2 u of the sum of magnitudes; h of the result. Mixed: a value over 1/16 of its
            row's scale is a pair for certain, one below may be single (and one at the border either: 1.01)
"""
import ctypes
import math

import pytest
import torch

import vocab_wide_logprobs_gb300 as vp
from vocab_wide_logprobs_gb300 import _lib

OK, ERR_NULL, ERR_SHAPE, ERR_DTYPE, ERR_LAYOUT, ERR_ALIGN, ERR_LAUNCH, ERR_ARG, ERR_DEVICE = range(9)
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def plain(x, targets, smooth=0.0, zeta=0.0, cap=0.0, start=0):
    """Losses of fp64 logits from the definition; differentiable."""
    z = cap * torch.tanh(x / cap) if cap else x
    lse = torch.logsumexp(z, 1)
    t = (targets - start).clamp(min=0)
    loss = lse - (1 - smooth) * z.gather(1, t[:, None])[:, 0] + zeta * lse ** 2
    if smooth:
        loss = loss - smooth * z.mean(1)
    return torch.where(targets >= 0, loss, 0.0)


def plain_grad(x, targets, g, smooth=0.0, zeta=0.0, cap=0.0, start=0, total=None):
    """dx of sum g loss by the formula, and what its tolerance is made of."""
    V = x.shape[1]
    z = cap * torch.tanh(x / cap) if cap else x
    slope = 1 / torch.cosh(x / cap) ** 2 if cap else torch.ones_like(x)
    lse = torch.logsumexp(z, 1, keepdim=True)
    lp = z - lse
    p = torch.exp(lp)
    onehot = torch.zeros_like(x).scatter_(1, (targets - start).clamp(min=0)[:, None], 1.0)
    gr = torch.where(targets >= 0, g.double(), 0.0)[:, None]
    share = smooth / (total or V)
    a = 1 + 2 * zeta * lse
    dz = gr * (p * a - (1 - smooth) * onehot - share)
    # without cancellation at a target that carries its row
    exact = gr * (torch.expm1(lp) + 2 * zeta * lse * p + smooth - share)
    dz = torch.where(onehot > 0, exact, dz)
    z, lp = z.clamp(-1e30, 1e30), lp.clamp(min=-1e4)
    off = gr.abs() * slope * (p * (64 + 2 * lp.abs()) * U * a.abs() + 8 * U * (p * a.abs() + onehot + share))
    far = 6 * U * (x / cap).abs().clamp(max=1e4) if cap else 0.0
    return dz * slope, off + (32 * U + far) * (dz * slope).abs(), gr.abs() * slope * p * a.abs() * 2, z, lse


def loss_tol(x, ref, targets, smooth, zeta, cap, d):
    z = cap * torch.tanh(x / cap) if cap else x
    fin = torch.where(torch.isfinite(z), z, 0.0)
    m, lse = z.amax(1), torch.logsumexp(z, 1).abs()
    d = d + (8 * U * fin.abs().amax(1) if cap else 0.0)
    zt = z.gather(1, targets.clamp(min=0)[:, None])[:, 0]
    zt = torch.where(torch.isfinite(zt), zt, 0.0)
    mean = torch.where(torch.isfinite(z), (z - m[:, None]).abs(), 0.0).mean(1)
    base = 64 * U + 3 * d + 4 * U * (m.abs() + (zt - m).abs()) + smooth * 48 * U * mean
    return base * (1 + 2 * zeta * lse) + 4 * U * zeta * lse ** 2 + U * ref.abs().nan_to_num(posinf=0.0)


def near(got, ref, tol, what):
    got = got.double().to(ref.device)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN elsewhere"
    assert torch.equal(torch.isinf(got), torch.isinf(ref)), f"{what}: inf elsewhere"
    fine = torch.isfinite(ref)
    over = torch.where(fine, (got - ref).abs() - tol, torch.zeros_like(ref))
    assert over.max() <= 0, f"{what}: {float(over.max()):.2e} over its tolerance"


def rows(N, V, dtype, seed, sigma=3.0, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(N, V, generator=g) * sigma + offset).to(dtype)
    targets = torch.randint(0, V, (N,), generator=g)
    targets[torch.rand(N, generator=g) < 0.15] = -1
    targets[0] = V - 1
    return x, targets, torch.randn(N, generator=g)


OPTIONS = [dict(), dict(smooth=0.1, zeta=1e-4), dict(cap=30.0), dict(smooth=1.0), dict(smooth=0.2, zeta=1e-2, cap=4.0)]


def kw(o):
    names = {"smooth": "label_smoothing", "zeta": "z_loss", "cap": "softcap", "start": "vocab_start"}
    return {names[k]: v for k, v in o.items()}


def check_logits(x, targets, g, o, xg=None, dtype=None):
    xg = x.cuda() if xg is None else xg
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, stats = vp.vp_cross_entropy_fwd(xg, targets.cuda(), err_word=err, **kw(o))
    dx = vp.vp_cross_entropy_bwd(xg, targets.cuda(), stats, g.cuda(), err_word=err, **kw(o))
    x64 = x.double()
    s, z, c = o.get("smooth", 0.0), o.get("zeta", 0.0), o.get("cap", 0.0)
    ref = plain(x64, targets, s, z, c, o.get("start", 0))
    near(loss, ref, loss_tol(x64, ref, targets - o.get("start", 0), s, z, c, 0.0), "loss")
    d, off, per_d, zz, _ = plain_grad(x64, targets, g, s, z, c, o.get("start", 0))
    if c:
        off = off + per_d * 8 * U * zz.abs().amax(1, keepdim=True)
    near(dx, d, off + torch.finfo(x.dtype).eps / 2 * d.abs(), "dx")
    assert int(err) == 0 and dx.dtype == x.dtype
    return loss, stats, dx


# --------------------------------------------------------------------------- the reference itself
@pytest.mark.parametrize("o", OPTIONS)
def test_formula_is_the_derivative(o):
    """The formula against autograd of the definition and against central differences."""
    x, targets, g = rows(5, 13, F32, 3)
    x = x.double().requires_grad_()
    s, z, c = o.get("smooth", 0.0), o.get("zeta", 0.0), o.get("cap", 0.0)
    (plain(x, targets, s, z, c) * g).sum().backward()
    d = plain_grad(x.detach(), targets, g, s, z, c)[0]
    assert torch.allclose(x.grad, d, rtol=1e-12, atol=1e-14)
    step = 1e-5
    for j in range(13):
        e = torch.zeros(13, dtype=torch.float64)
        e[j] = step
        diff = (plain(x.detach() + e, targets, s, z, c) - plain(x.detach() - e, targets, s, z, c)) / (2 * step) * g
        assert torch.allclose(diff, d[:, j], rtol=1e-6, atol=1e-9)


# --------------------------------------------------------------------------- logits
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("o", OPTIONS)
@pytest.mark.parametrize("shape", [(1, 1), (3, 5), (2, 31), (7, 4096), (5, 8192), (4, 8193), (3, 20011), (40, 1000)])
def test_logits(shape, o, dtype):
    check_logits(*rows(*shape, dtype, sum(shape)), o)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_logits_wide_values_and_offsets(dtype):
    """A common offset, near-certain rows, capped logits far out, values around the split of the tanh."""
    x, targets, g = rows(6, 9001, dtype, 5, offset=200.0)
    check_logits(x, targets, g, dict(smooth=0.1))
    x, targets, g = rows(6, 9001, dtype, 6)
    x[torch.arange(6), targets.clamp(min=0)] = 40.0
    check_logits(x, targets, g, dict())
    check_logits(x, targets, g, dict(zeta=1e-4, smooth=0.1))
    x, targets, g = rows(6, 9001, dtype, 7, sigma=60.0)
    check_logits(x, targets, g, dict(cap=15.0, smooth=0.1, zeta=1e-3))
    x = torch.linspace(-2, 2, 6 * 1024).reshape(6, 1024).to(dtype) * 15.0
    check_logits(x, torch.arange(6) * 100, g, dict(cap=15.0))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_logits_where_rows_begin(dtype):
    """Rows at any offset from a 16-byte boundary, [B, T, V] views with two strides, and dx in place."""
    x, targets, g = rows(12, 8231, dtype, 9)
    for offset, gap in ((1, 0), (3, 5), (4, 4), (8, 1), (0, 8)):
        room = torch.full((offset + 12 * (8231 + gap),), math.nan, dtype=dtype, device="cuda")
        view = room[offset:].view(12, 8231 + gap)[:, :8231]
        view.copy_(x)
        check_logits(x, targets, g, dict(smooth=0.1), xg=view)
    for V in (9, 17, 33, 8192 + 15):                                 # rows of a few vectors, and of a slice and some
        x2, t2, g2 = rows(9, V, dtype, V)
        for offset, gap in ((0, 1), (5, 2), (2, 3), (7, 8)):
            room = torch.full((offset + 9 * (V + gap),), math.nan, dtype=dtype, device="cuda")
            view = room[offset:].view(9, V + gap)[:, :V]
            view.copy_(x2)
            check_logits(x2, t2, g2, dict(cap=9.0, zeta=1e-3), xg=view)
            check_logits(x2, t2, g2, dict(smooth=0.2), xg=view)
    full = torch.full((3, 5, 8231), math.nan, dtype=dtype, device="cuda")
    full[:, :-1] = x.view(3, 4, 8231).cuda()
    _, stats, dx = check_logits(x, targets, g, dict(cap=20.0), xg=full[:, :-1])
    for first in (0, 1):                                             # a base on a 16-byte boundary and one off it
        room = torch.empty(12 * 8231 + 1, dtype=dtype, device="cuda")
        inplace = room[first:first + 12 * 8231].view(12, 8231)
        inplace.copy_(x)
        loss, stats = vp.vp_cross_entropy_fwd(inplace, targets.cuda(), softcap=20.0)
        ref = vp.vp_cross_entropy_bwd(inplace, targets.cuda(), stats, g.cuda(), softcap=20.0)
        got = vp.vp_cross_entropy_bwd(inplace, targets.cuda(), stats, g.cuda(), softcap=20.0, dx=inplace)
        assert got.data_ptr() == inplace.data_ptr() and torch.equal(got, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vectors", [128, 512, 1024])
def test_logits_at_the_ends_of_row_sizes(vectors, dtype):
    """Rows that just fill the threads of one, two and four warps, and rows of a column more; few rows and many."""
    full = vectors * (8 if dtype == BF16 else 4)
    for V in (full - 1, full, full + 1):
        for N in (3, 700):
            x, targets, g = rows(N, V, dtype, V + N)
            check_logits(x, targets, g, dict(cap=9.0, smooth=0.2) if V == full else dict(zeta=1e-3))
    x, targets, g = rows(9, full, dtype, full)
    for offset in (1, 6):
        room = torch.full((offset + 9 * (full + 3),), math.nan, dtype=dtype, device="cuda")
        view = room[offset:].view(9, full + 3)[:, :full]
        view.copy_(x)
        check_logits(x, targets, g, dict(smooth=0.1), xg=view)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_logits_of_many_short_rows(dtype):
    """More rows than CTAs run at once, with rows to ignore among them; each as in a batch of its own, where it lies as it
    does in the large one (a row's sums depend on its address modulo 16 bytes)."""
    N, V = 11000, 70
    x, targets, g = rows(N, V, dtype, 23, sigma=8.0)
    xg = x.cuda()
    loss, stats, dx = check_logits(x, targets, g, dict(smooth=0.1, zeta=1e-3), xg=xg)
    o = dict(label_smoothing=0.1, z_loss=1e-3)
    for i in (0, 4863, 4864, N - 5):
        k = slice(i, i + 5)
        one, st = vp.vp_cross_entropy_fwd(xg[k], targets[k].cuda(), **o)
        assert torch.equal(one, loss[k]) and torch.equal(st.nan_to_num(7), stats[k].nan_to_num(7))
        assert torch.equal(vp.vp_cross_entropy_bwd(xg[k], targets[k].cuda(), st, g[k].cuda(), **o), dx[k])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("fill", ["inf", "lowest"])
def test_masked_columns(dtype, fill):
    x, targets, g = rows(8, 9001, dtype, 11)
    low = -math.inf if fill == "inf" else torch.finfo(dtype).min
    keep = torch.rand(8, 9001, generator=torch.Generator().manual_seed(1)) < 0.5
    keep[torch.arange(8), targets.clamp(min=0)] = True
    keep[2, 1:] = False                                              # one column left
    keep[2, 0] = True
    targets[2], targets[3] = 0, 4500
    keep[3, :4500], keep[3, 4501:] = False, False                    # and in another slice
    keep[3, 4500] = True
    x = torch.where(keep, x, torch.tensor(low, dtype=dtype))
    check_logits(x, targets, g, dict())
    if fill == "inf":
        # smoothing wants some of every column: infinite losses, finite gradients
        loss, stats, _ = check_logits(x, targets, g, dict(smooth=0.1))
        assert torch.isinf(loss[targets.cuda() >= 0]).all()
        # a cap makes -inf the number -cap
        check_logits(x, targets, g, dict(cap=20.0, smooth=0.1))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [700, 20000])
def test_rows_of_a_types_ends(dtype, V):
    """Rows of nothing but the type's lowest value (uniform, as the definition has it), and one-hot rows that span the
    type: nothing overflows on the way."""
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    x = torch.full((4, V), low, dtype=dtype)
    x[1, V - 3], x[2, 5], x[3, ::2] = high, 0.0, high
    targets, g = torch.tensor([7, V - 3, 5, 0]), torch.tensor([1.0, -2.0, 0.5, 3.0])
    loss, stats = vp.vp_cross_entropy_fwd(x.cuda(), targets.cuda())
    ref = torch.tensor([math.log(V), 0.0, 0.0, math.log((V + 1) // 2)], dtype=torch.float64)
    assert torch.allclose(loss.double().cpu(), ref, rtol=1e-6, atol=1e-6)
    dx = vp.vp_cross_entropy_bwd(x.cuda(), targets.cuda(), stats, g.cuda()).double().cpu()
    d = torch.zeros(4, V, dtype=torch.float64)
    d[0], d[3, ::2] = 1.0 / V, 3.0 / ((V + 1) // 2)
    d[0, 7] -= 1.0
    d[3, 0] -= 3.0
    assert torch.allclose(dx, d, rtol=torch.finfo(dtype).eps, atol=1e-7)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sums_of_logits_past_the_largest_float(dtype):
    """Half of 2^25 columns at either end of the type, with smoothing: their mean is a float, their sum is not, nor is what
    2^24 of them add up to."""
    V = 1 << 25
    high = torch.finfo(dtype).max
    x = torch.full((1, V), -high, dtype=dtype, device="cuda")
    x[0, ::2] = high
    targets = torch.tensor([4], device="cuda")
    want = 0.1 * high + math.log(V // 2)                             # mean_j (m - z_j) is half of 2 high
    loss, _ = vp.vp_cross_entropy_fwd(x, targets, label_smoothing=0.1)
    assert abs(float(loss) - want) <= 1e-6 * want
    parts = torch.stack([vp.vp_cross_entropy_partial(x[:, a:a + V // 2], targets, vocab_start=a) for a in (0, V // 2)])
    loss, _ = vp.vp_cross_entropy_merge(parts, label_smoothing=0.1)
    assert abs(float(loss) - want) <= 1e-6 * want


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N, V", [(4, 700), (700, 1001), (6, 9001)])
def test_a_masked_target(N, V, dtype):
    """Its loss is infinite, its gradient what the formula says of p = 0; and a z-loss of 1."""
    x, targets, g = rows(N, V, dtype, 57)
    targets = targets.clamp(min=0)
    x[torch.arange(0, N, 2), targets[::2]] = -math.inf
    x[torch.arange(1, N, 4), targets[1::4]] = torch.finfo(dtype).min
    for s, z in ((0.0, 0.0), (0.1, 0.0), (0.0, 1.0), (1.0, 1.0)):
        loss, stats = vp.vp_cross_entropy_fwd(x.cuda(), targets.cuda(), label_smoothing=s, z_loss=z)
        assert torch.isinf(loss[::2]).all() and torch.isfinite(loss[3::4]).all()
        dx = vp.vp_cross_entropy_bwd(x.cuda(), targets.cuda(), stats, g.cuda(), label_smoothing=s, z_loss=z)
        d, off, *_ = plain_grad(x.double(), targets, g, s, z)
        r = torch.arange(N)
        p0 = torch.isinf(x[r, targets])
        d[r[p0], targets[p0]] = g.double()[p0] * -(1 - s + s / V)
        near(dx, d, off + torch.finfo(dtype).eps / 2 * d.abs(), f"smooth {s}, zeta {z}")


FAR = [1.2e4, -65504.0, 1e5, -1e6, 3e7, -1e8, -1e9, 2.0 ** 30, -2.0 ** 30, 2.0 ** 30 + 128, -3e9, 1e20, -1e30, 3e38]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [700, 20000])
def test_rows_far_from_zero(dtype, V):
    """Rows of one value (all that a mask of -1e9 leaves, say) are uniform, and rows that lie close together around a far
    value are what their differences say: z - m is exact, so neither the loss nor p knows the offset. Where the differences are of
    64 and more, p below 2^-62 may come out 0."""
    g = torch.linspace(-2, 3, len(FAR))
    x = torch.tensor(FAR)[:, None].expand(-1, V).to(dtype).contiguous()
    targets = torch.arange(len(FAR)) * 49 + 3
    for spread in (0.0, 3.0):
        if spread:
            x = (x.double() + spread * torch.randn(len(FAR), V, generator=torch.Generator().manual_seed(V), dtype=torch.float64)).to(dtype)
        for s in (0.0, 0.1):
            loss, stats = vp.vp_cross_entropy_fwd(x.cuda(), targets.cuda(), label_smoothing=s)
            dx = vp.vp_cross_entropy_bwd(x.cuda(), targets.cuda(), stats, g.cuda(), label_smoothing=s)
            z = x.double() - x.double().amax(1, keepdim=True)
            ref = plain(z, targets, s)
            size = z.gather(1, targets[:, None])[:, 0].abs() + s * 24 * z.abs().mean(1)
            near(loss, ref, 64 * U + 2 * U * size + U * ref.abs(), "loss")
            d, off, *_ = plain_grad(z, targets, g, s)
            near(dx, d, off + g.abs().double()[:, None] * 2.0 ** -62 + torch.finfo(dtype).eps / 2 * d.abs(), "dx")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_with_nothing_or_with_nan(dtype):
    x, _, g = rows(7, 5003, dtype, 13)
    x[1] = -math.inf
    x[2, 4000] = math.nan
    x[3, 17] = math.inf
    x[4, 5002] = math.nan
    targets = torch.tensor([5, 5, 5, 5, -1, 4000, 17])
    loss, stats = vp.vp_cross_entropy_fwd(x.cuda(), targets.cuda(), label_smoothing=0.1)
    dx = vp.vp_cross_entropy_bwd(x.cuda(), targets.cuda(), stats, g.cuda(), label_smoothing=0.1)
    assert torch.isnan(loss).tolist() == [False, True, True, True, False, False, False]
    assert loss[4] == 0 and (dx[4] == 0).all()
    assert torch.isnan(dx[1:4]).all() and torch.isfinite(dx[5:]).all() and torch.isfinite(dx[0]).all()
    flags = vp.decode_rowstats(stats)["flags"].tolist()
    assert flags == [0, vp.ROW_EMPTY, vp.ROW_NANINF, vp.ROW_NANINF, vp.ROW_NANINF, 0, 0]
    # under a cap an infinity is a number, a NaN is not
    loss, stats = vp.vp_cross_entropy_fwd(x.cuda(), targets.cuda(), softcap=10.0)
    dx = vp.vp_cross_entropy_bwd(x.cuda(), targets.cuda(), stats, g.cuda(), softcap=10.0)
    assert torch.isnan(loss).tolist() == [False, False, True, False, False, False, False]
    assert (dx[1] == 0).all() and dx[3, 17] == 0 and torch.isfinite(dx[3]).all() and torch.isnan(dx[2]).all()
    assert abs(float(loss[1]) - math.log(5003)) < 1e-4


@pytest.mark.gpu
def test_targets_outside_the_shard():
    x, _, g = rows(5, 700, BF16, 15)
    targets = torch.tensor([700, 1399, 1400, 699, -7])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, stats = vp.vp_cross_entropy_fwd(x.cuda(), targets.cuda(), vocab_start=700, err_word=err)
    assert int(err) == vp.ERRBIT_TARGET and torch.isnan(loss).tolist() == [False, False, True, True, False]
    err.zero_()
    dx = vp.vp_cross_entropy_bwd(x.cuda(), targets.cuda(), stats, g.cuda(), vocab_start=700, err_word=err)
    assert int(err) == vp.ERRBIT_TARGET and torch.isnan(dx[2:4]).all() and (dx[4] == 0).all()
    ref = plain_grad(x.double()[:2], targets[:2], g[:2], start=700)[0]
    assert torch.allclose(dx[:2].double().cpu(), ref, rtol=2.0 ** -7, atol=1e-6)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N, V", [(70, 25008), (700, 1000)])
def test_a_row_does_not_depend_on_the_batch(N, V, dtype):
    """Neither joined out of several slices nor finished where it is summed (few short rows) or not (many)."""
    x, targets, g = (t.cuda() for t in rows(N, V, dtype, 17, sigma=12.0))
    o = dict(label_smoothing=0.1, z_loss=1e-3, softcap=25.0)
    loss, stats = vp.vp_cross_entropy_fwd(x, targets, **o)
    dx = vp.vp_cross_entropy_bwd(x, targets, stats, g, **o)
    for i in (0, 1, 37, 69):
        k = slice(i, i + 1)
        one, st = vp.vp_cross_entropy_fwd(x[k], targets[k], **o)
        assert torch.equal(one, loss[k]) and torch.equal(st, stats[k])
        assert torch.equal(vp.vp_cross_entropy_bwd(x[k], targets[k], st, g[k], **o), dx[k])


@pytest.mark.gpu
@pytest.mark.parametrize("V", [1000, 9000])
def test_a_linear_row_does_not_depend_on_the_batch(V):
    """Its loss and record: few rows and many, of pieces for eight lanes and for all of a CTA."""
    h, w, targets, _ = (t.cuda() for t in model(1500, V, 64, 18))
    o = dict(label_smoothing=0.1, z_loss=1e-3, softcap=25.0)
    loss, stats = vp.vp_linear_cross_entropy_fwd(h, w, targets, **o)
    for k in (slice(0, 1), slice(3, 4), slice(700, 900), slice(1499, 1500), slice(100, 1400)):
        one, st = vp.vp_linear_cross_entropy_fwd(h[k], w, targets[k], **o)
        assert torch.equal(one, loss[k]) and torch.equal(st, stats[k])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("o", OPTIONS)
def test_shards_merge_to_the_whole(dtype, o):
    x, targets, g = rows(9, 6001, dtype, 19)
    cuts = [0, 1, 2500, 2531, 6001]
    s, z, c = o.get("smooth", 0.0), o.get("zeta", 0.0), o.get("cap", 0.0)
    shards = [x[:, a:b].contiguous().cuda() for a, b in zip(cuts, cuts[1:])]
    parts = torch.stack([vp.vp_cross_entropy_partial(p, targets.cuda(), softcap=c, vocab_start=a)
                         for p, a in zip(shards, cuts)])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, stats = vp.vp_cross_entropy_merge(parts, label_smoothing=s, z_loss=z, err_word=err)
    ref = plain(x.double(), targets, s, z, c)
    near(loss, ref, loss_tol(x.double(), ref, targets, s, z, c, 0.0), "merged loss")
    d, off, per_d, zz, _ = plain_grad(x.double(), targets, g, s, z, c)
    if c:
        off = off + per_d * 8 * U * zz.abs().amax(1, keepdim=True)
    dx = torch.cat([vp.vp_cross_entropy_bwd(p, targets.cuda(), stats, g.cuda(), vocab_start=a, vocab_total=6001,
                                            err_word=err, **kw(o)) for p, a in zip(shards, cuts)], 1)
    near(dx, d, off + torch.finfo(dtype).eps / 2 * d.abs(), "sharded dx")
    assert int(err) == 0
    # a target that no shard holds
    loss, _ = vp.vp_cross_entropy_merge(parts[:2], label_smoothing=s, z_loss=z, err_word=err)
    held = (targets < 2500).cuda()
    assert torch.equal(torch.isnan(loss), ~held) and int(err) == vp.ERRBIT_TARGET


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_merged_masked_shards(dtype):
    """A shard of nothing but -inf, and a row of nothing at all."""
    x, targets, g = rows(4, 900, dtype, 21)
    x[1, 300:600] = -math.inf
    x[2] = -math.inf
    targets[:] = torch.tensor([5, 700, 3, -1])
    parts = torch.stack([vp.vp_cross_entropy_partial(x[:, a:a + 300].cuda(), targets.cuda(), vocab_start=a)
                         for a in (0, 300, 600)])
    for s in (0.0, 0.1):
        loss, stats = vp.vp_cross_entropy_merge(parts, label_smoothing=s)
        ref = plain(x.double(), targets, s)
        ref[2] = math.nan
        near(loss, ref, loss_tol(x.double(), ref, targets, s, 0.0, 0.0, 0.0).nan_to_num(), f"smooth {s}")


# --------------------------------------------------------------------------- hidden . W^T
def model(N, V, D, seed, sigma=2.5):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(N, D, generator=g).to(BF16)
    w = (torch.randn(V, D, generator=g) * sigma / math.sqrt(D)).to(BF16)
    targets = torch.randint(0, V, (N,), generator=g)
    targets[torch.rand(N, generator=g) < 0.1] = -1
    targets[0] = V - 1
    return h, w, targets, torch.randn(N, generator=g)


def pair_error(dz, x, targets, g, o, precision):
    """What carrying dz as bf16 values takes away, relative."""
    if precision != vp.GRAD_MIXED:
        return 2.0 ** -16 if precision == vp.GRAD_EXACT else 2.0 ** -8
    cap = o.get("cap", 0.0)
    z = cap * torch.tanh(x / cap) if cap else x
    lpt = (z - torch.logsumexp(z, 1, keepdim=True)).gather(1, targets.clamp(min=0)[:, None])
    scale = g.double().abs()[:, None] * (o.get("smooth", 0.0) - torch.expm1(lpt)).clamp(min=2.0 ** -20)
    if cap:
        zt = z.gather(1, targets.clamp(min=0)[:, None])
        scale = scale * (1 - (zt / cap) ** 2).clamp(min=2.0 ** -20)
    return torch.where(dz.abs() > 1.01 / 16 * scale, 2.0 ** -16, 2.0 ** -8)


def gradients(h64, w64, targets, g, o, precision):
    """[(dhidden, its tolerance without the output's rounding), (dW, ..)] in 64 bits."""
    s, z, c = o.get("smooth", 0.0), o.get("zeta", 0.0), o.get("cap", 0.0)
    (N, D), V = h64.shape, w64.shape[0]
    x, size = h64 @ w64.t(), h64.abs() @ w64.abs().t()
    dz, off, per_d, zz, _ = plain_grad(x, targets, g, s, z, c)
    d = (D / 16 + 1) * 2.25 * U * size.amax(1, keepdim=True) + (8 * U * zz.abs().amax(1, keepdim=True) if c else 0.0)
    # a logit off by d moves the cap's slope by at most |slope'| d <= d / c of itself
    off = off + per_d * d + (dz.abs() * d / c if c else 0.0)
    off = off + pair_error(dz, x, targets, g, o, precision) * dz.abs()
    return [(dz @ w64, off @ w64.abs() + (V / 16 + 2) * 2 * U * (dz.abs() @ w64.abs())),
            (dz.t() @ h64, off.t() @ h64.abs() + (N / 16 + 2) * 2 * U * (dz.abs().t() @ h64.abs()))]


def check_linear(h, w, targets, g, o, precision=None, where="cpu"):
    """where: the device of the reference's arithmetic."""
    precision = vp.GRAD_MIXED if precision is None else precision
    D, (N, V) = h.shape[1], (h.shape[0], w.shape[0])
    s, z, c = o.get("smooth", 0.0), o.get("zeta", 0.0), o.get("cap", 0.0)
    hg, wg, tg = h.cuda(), w.cuda(), targets.cuda()
    loss, stats = vp.vp_linear_cross_entropy_fwd(hg, wg, tg, **kw(o))
    dh, dw = vp.vp_linear_cross_entropy_bwd(hg, wg, tg, stats, g.cuda(), precision=precision, **kw(o))
    h, w, targets, g = (t.to(where) for t in (h, w, targets, g))
    loss, dh, dw = (t.to(where) for t in (loss, dh, dw))
    h64, w64 = h.double(), w.double()
    x, size = h64 @ w64.t(), h64.abs() @ w64.abs().t()
    d = (D / 16 + 1) * 2.25 * U * size.amax(1)
    ref = plain(x, targets, s, z, c, o.get("start", 0))
    near(loss, ref, loss_tol(x, ref, targets - o.get("start", 0), s, z, c, d), "loss")
    half = torch.finfo(BF16).eps / 2
    for got, (ref, tol), what in zip((dh, dw), gradients(h64, w64, targets, g, o, precision), ("dhidden", "dW")):
        near(got, ref, tol + half * ref.abs(), what)
    return loss, stats, dh, dw


@pytest.mark.gpu
@pytest.mark.parametrize("o", OPTIONS)
@pytest.mark.parametrize("shape", [(1, 1, 64), (3, 200, 64), (130, 700, 128), (257, 1025, 192), (64, 5003, 512)])
def test_linear(shape, o):
    check_linear(*model(*shape, sum(shape)), o)


@pytest.mark.gpu
@pytest.mark.parametrize("o", OPTIONS)
@pytest.mark.parametrize("shape", [(3, 70001, 64), (130, 20000, 256), (257, 8200, 576), (1500, 6000, 128)])
def test_linear_larger_tables(shape, o):
    """Tables and products from where on only the blocks of dz that count are summed as pairs."""
    check_linear(*model(*shape, sum(shape)), o, where="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(300, 1500, 256), (700, 9000, 64), (17, 9000, 1024)])
def test_linear_precisions_and_single_outputs(shape):
    h, w, targets, g = model(*shape, 31)
    o = dict(smooth=0.1, zeta=1e-4, cap=10.0)
    for precision in (vp.GRAD_FAST, vp.GRAD_EXACT):
        check_linear(h, w, targets, g, o, precision=precision)
    _, stats, dh, dw = check_linear(h, w, targets, g, o)
    args = (h.cuda(), w.cuda(), targets.cuda(), stats, g.cuda())
    a, none = vp.vp_linear_cross_entropy_bwd(*args, want_dW=False, **kw(o))
    assert none is None and torch.equal(a.cpu(), dh)
    none, b = vp.vp_linear_cross_entropy_bwd(*args, want_dhidden=False, **kw(o))
    assert none is None and torch.equal(b.cpu(), dw)


@pytest.mark.gpu
@pytest.mark.parametrize("precision", [vp.GRAD_MIXED, vp.GRAD_EXACT])
@pytest.mark.parametrize("N, V", [(4, 40000), (8200, 300), (16000, 16700), (33000, 8193)])
def test_linear_several_pieces(N, V, precision):
    """The vocabulary in one piece and in several (of 2^28 / N columns, and of 8192), the last one a column long."""
    check_linear(*model(N, V, 64, 33), dict(smooth=0.1, zeta=1e-4), precision=precision, where="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("precision", [vp.GRAD_MIXED, vp.GRAD_EXACT, vp.GRAD_FAST])
@pytest.mark.parametrize("N, V, D", [(1023, 256, 64), (1024, 257, 192), (5000, 1100, 256), (20000, 50, 64)])
def test_linear_small_vocabularies(N, V, D, precision):
    """dW's few tiles, their rows shared out over many pairs of SMs, and just not."""
    check_linear(*model(N, V, D, 37), dict(smooth=0.1, cap=20.0), precision=precision, where="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("N, V, D", [(1100, 33000, 1024), (8200, 32800, 1024), (1030, 8201, 4160)])
def test_linear_many_rows_of_large_tables(N, V, D):
    """What dhidden's rows add of dz's second halves by themselves, in one piece of the vocabulary and in two; a row
    without statistics takes no other row's part."""
    h, w, targets, g = model(N, V, D, 39)
    g[7] = 0.0
    _, stats, dh, _ = check_linear(h, w, targets, g, dict(smooth=0.1, zeta=1e-4), where="cuda")
    h[N - 3] = math.nan
    o = dict(label_smoothing=0.1, z_loss=1e-4)
    _, stats = vp.vp_linear_cross_entropy_fwd(h.cuda(), w.cuda(), targets.cuda(), **o)
    got, _ = vp.vp_linear_cross_entropy_bwd(h.cuda(), w.cuda(), targets.cuda(), stats, g.cuda(), want_dW=False, **o)
    rest = torch.arange(N, device="cuda") != N - 3
    assert torch.equal(got[rest], dh.cuda()[rest])
    assert targets[N - 3] < 0 or torch.isnan(got[N - 3]).all()


@pytest.mark.gpu
def test_dhidden_of_a_large_table_does_not_depend_on_the_rows_beside_it():
    """A row with 16 values whose bf16 rounding crosses the row's limit for pairs: they are pairs whether or not a row of the
    same block has one there. 17 equal logits of 18 among zeros and their target among them: p = (1 - m) / 17 with
    m = 32751 e^-18 / 17 = 2.9e-5, the limit (1 + m / 16) / 17 for |g| = 1, so the 16 lie 3.1e-5 of themselves below it, and
    with g / 17 = 1 + 0.75 2^-7 they round up over it."""
    N, V, D = 1024, 32768, 1024
    gen = torch.Generator().manual_seed(50)
    heavy = torch.arange(17) * 1024 + 5
    w = torch.randn(V, D, generator=gen).to(BF16)
    w[:, 0] = 0.0
    w[heavy, 0] = 18.0
    h = torch.zeros(N, D, dtype=BF16)
    h[:, 0] = 1.0
    g = torch.ones(N)
    g[5] = 17 * (1 + 0.75 / 128)
    rest = []
    for beside in (False, True):
        targets = torch.full((N,), -1)
        targets[5] = heavy[0]
        if beside:
            targets[6:22] = heavy[1:]
        args = h.cuda(), w.cuda(), targets.cuda()
        _, stats = vp.vp_linear_cross_entropy_fwd(*args)
        rest.append(vp.vp_linear_cross_entropy_bwd(*args, stats, g.cuda(), want_dW=False)[0][5])
    assert torch.equal(*rest)


@pytest.mark.gpu
@pytest.mark.parametrize("N, V, D, zeta", [(1100, 33000, 1024, 1.0), (1100, 33000, 1024, 1e3), (300, 20000, 256, 1.0)])
def test_linear_large_z_loss(N, V, D, zeta):
    """A z-loss whose gradient, 1 + 2 zeta lse of the softmax, is most of the row's: against 64 bits, with the row's scale
    times a quarter of that factor, and in about the time of a small one (the values over the limit stay a few a row)."""
    h, w, targets, g = (t.cuda() for t in model(N, V, D, 52))
    loss, stats = vp.vp_linear_cross_entropy_fwd(h, w, targets, z_loss=zeta)
    dh, dw = vp.vp_linear_cross_entropy_bwd(h, w, targets, stats, g, z_loss=zeta)
    h64, w64 = h.double(), w.double()
    x, size = h64 @ w64.t(), h64.abs() @ w64.abs().t()
    d = (D / 16 + 1) * 2.25 * U * size.amax(1, keepdim=True)
    ref = plain(x, targets, zeta=zeta)
    near(loss, ref, loss_tol(x, ref, targets, 0.0, zeta, 0.0, d[:, 0]), "loss")
    dz, off, per_d, _, lse = plain_grad(x, targets, g, zeta=zeta)
    a = 1 + 2 * zeta * lse
    # lse is off by d and its own rounding, and 2 zeta lse with it
    off = off + per_d * d + g.double().abs()[:, None] * torch.exp(x - lse) * 2 * zeta * (d + 64 * U + 4 * U * lse.abs())
    lpt = (x - lse).gather(1, targets.clamp(min=0)[:, None])
    scale = g.double().abs()[:, None] * (-torch.expm1(lpt)).clamp(min=2.0 ** -20) * (a.abs() / 4).clamp(min=1.0)
    off = off + torch.where(dz.abs() > 1.01 / 16 * scale, 2.0 ** -16, 2.0 ** -8) * dz.abs()
    half = torch.finfo(BF16).eps / 2
    for got, ref, tol in ((dh, dz @ w64, off @ w64.abs() + (V / 16 + 2) * 2 * U * (dz.abs() @ w64.abs())),
                          (dw, dz.t() @ h64, off.t() @ h64.abs() + (N / 16 + 2) * 2 * U * (dz.abs().t() @ h64.abs()))):
        near(got, ref, tol + half * ref.abs(), f"zeta {zeta}")

    def took(z):
        times = []
        for _ in range(4):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            vp.vp_linear_cross_entropy_bwd(h, w, targets, stats, g, z_loss=z)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    assert took(zeta) < 4 * took(0.0)


@pytest.mark.gpu
@pytest.mark.parametrize("precision", [vp.GRAD_MIXED, vp.GRAD_FAST, vp.GRAD_EXACT])
def test_linear_dW_of_columns_without_a_target(precision):
    """Row by row of dW where no value need be a pair: roundings of dz to bf16 and of the result are spread over half a step
    each, 2^-8 of the value at most and 2^-8 / sqrt(3) in the mean square, so the rows' squared errors add up to
    2^-16 / 3 (sum dz^2 |h|^2 + |dW|^2), without the first term where dz is a pair; no row alone is off by four times that."""
    h, w, targets, g = (t.cuda() for t in model(1100, 20000, 256, 56))
    o = dict(label_smoothing=0.1, z_loss=1e-4)
    _, stats = vp.vp_linear_cross_entropy_fwd(h, w, targets, **o)
    _, dw = vp.vp_linear_cross_entropy_bwd(h, w, targets, stats, g, want_dhidden=False, precision=precision, **o)
    h64 = h.double()
    dz = plain_grad(h64 @ w.double().t(), targets, g, 0.1, 1e-4)[0]
    ref = dz.t() @ h64
    free = torch.ones(20000, dtype=torch.bool, device="cuda")
    free[targets[targets >= 0]] = False
    error = (dw.double() - ref).square().sum(1)[free]
    allowed = ref.square().sum(1)
    if precision != vp.GRAD_EXACT:
        allowed = allowed + (dz.square() * h64.square().sum(1, keepdim=True)).sum(0)
    allowed = 2.0 ** -16 / 3 * allowed[free]
    assert error.sum() <= 1.1 * allowed.sum() and (error <= 16 * allowed).all()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [512, 4096])
def test_linear_losses_are_not_short(D):
    """The tensor cores' sums come out short, 2.4e-5 of a log-sum-exp at D = 4096; what is given back leaves the losses
    of Gaussian rows within 1e-6 of themselves, and sums without a rounding (one product each) within d."""
    h, w, targets, _ = model(200, 3000, D, 45)
    loss, _ = vp.vp_linear_cross_entropy_fwd(h.cuda(), w.cuda(), targets.cuda())
    ref = plain(h.double() @ w.double().t(), targets)
    assert float((loss.double().cpu() - ref).norm() / ref.norm()) < 1e-6
    h = torch.zeros_like(h)
    h[torch.arange(200), torch.arange(200) * 7 % D] = 8.0
    check_linear(h, w, targets, torch.ones(200), dict())


@pytest.mark.gpu
def test_linear_sums_of_logits_past_the_largest_float():
    """Logits of +-2^124, with smoothing: 128 of them add up to more than a float holds, their mean does not."""
    h, w = torch.zeros(3, 64, dtype=BF16), torch.zeros(1000, 64, dtype=BF16)
    h[:, 5] = torch.tensor([2.0 ** 60, -2.0 ** 60, 2.0 ** 10])
    w[:, 5] = 2.0 ** 64
    w[1::4, 5] = -2.0 ** 64
    targets = torch.tensor([4, 5, 0])
    loss, _ = vp.vp_linear_cross_entropy_fwd(h.cuda(), w.cuda(), targets.cuda(), label_smoothing=0.1)
    ref = plain(h.double() @ w.double().t(), targets, 0.1)
    assert torch.allclose(loss.double().cpu(), ref, rtol=1e-6)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [1024, 4096, 32768])
def test_linear_logits_whose_sums_are_exact(D):
    """One product each, of which nothing is cut off: what is given back all the same is D / 16 steps of 2^-26 of the logit,
    of 16384 columns at most, to a quarter of itself and the rounding of the factor and the product (2 u)."""
    h, w = torch.zeros(64, D, dtype=BF16), torch.zeros(1, D, dtype=BF16)
    at = torch.arange(64) * (D // 64) + 3
    h[torch.arange(64), at] = torch.randn(64, generator=torch.Generator().manual_seed(54)).to(BF16) * 30
    w[0, at] = torch.randn(64, generator=torch.Generator().manual_seed(55)).to(BF16)
    _, stats = vp.vp_linear_cross_entropy_fwd(h.cuda(), w.cuda(), torch.zeros(64, dtype=torch.int64, device="cuda"))
    got = vp.decode_rowstats(stats)["m"].double().cpu()              # of one column, the logit
    z = (h.double() @ w.double().t())[:, 0]
    back = min(D, 16384) / 16 * 2.0 ** -26
    assert ((got - z * (1 + back)).abs() <= (back / 4 + 2 * U) * z.abs()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("V", [1000, 70001])
def test_linear_rows_far_from_zero(V):
    """Rows of one far value: uniform, whatever the value. Row n takes column n of hidden and weight alone, so dW there is
    dz times the hidden value, rounded (dz twice, as a pair or as one value: 2^-8 each)."""
    N = 12
    scale = torch.tensor([1.0, -1.0]).repeat(6) * 2.0 ** torch.arange(12, 36, 2)
    h, w = torch.zeros(N, 64, dtype=BF16), torch.zeros(V, 64, dtype=BF16)
    h[torch.arange(N), torch.arange(N)] = scale.to(BF16)
    w[:, :N] = 1.3
    targets, g = torch.arange(N) * 30 + 1, torch.linspace(1, 2, N)
    loss, stats = vp.vp_linear_cross_entropy_fwd(h.cuda(), w.cuda(), targets.cuda())
    assert torch.allclose(loss.double().cpu(), torch.full((N,), math.log(V), dtype=torch.float64), rtol=0, atol=64 * U + U * math.log(V))
    _, dw = vp.vp_linear_cross_entropy_bwd(h.cuda(), w.cuda(), targets.cuda(), stats, g.cuda())
    dz = (dw[:, :N].double().cpu() / scale).t()
    ref = (g.double() / V)[:, None].repeat(1, V)
    ref[torch.arange(N), targets] -= g.double()
    assert ((dz - ref).abs() <= 2.1 * 2.0 ** -8 * ref.abs()).all()


@pytest.mark.gpu
def test_linear_near_certain_rows():
    h, w, targets, g = model(40, 900, 128, 35, sigma=1.0)
    used = targets >= 0
    w[targets[used]] = (h[used].float() * 0.3).to(BF16)              # logits of about 38 at the targets
    check_linear(h, w, targets, g, dict())
    check_linear(h, w, targets, g, dict(cap=30.0, smooth=0.1))


@pytest.mark.gpu
def test_linear_bad_rows():
    h, w, targets, g = model(6, 300, 64, 37)
    h[1, 3] = math.nan
    targets[:] = torch.tensor([5, 5, -1, 300, 7, 299])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (h.cuda(), w.cuda(), targets.cuda())
    loss, stats = vp.vp_linear_cross_entropy_fwd(*args, err_word=err, label_smoothing=0.1)
    assert torch.isnan(loss).tolist() == [False, True, False, True, False, False] and int(err) == vp.ERRBIT_TARGET
    err.zero_()
    dh, dw = vp.vp_linear_cross_entropy_bwd(*args, stats, g.cuda(), err_word=err, label_smoothing=0.1)
    assert int(err) == vp.ERRBIT_TARGET and torch.isnan(dw).all()
    assert torch.isnan(dh[[1, 3]]).all() and torch.isfinite(dh[[0, 4, 5]]).all() and (dh[2] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("o", OPTIONS)
def test_linear_shards(o):
    h, w, targets, g = model(150, 1000, 128, 39)
    s, z, c = o.get("smooth", 0.0), o.get("zeta", 0.0), o.get("cap", 0.0)
    cuts = [0, 300, 301, 1000]
    hg, tg = h.cuda(), targets.cuda()
    ws = [w[a:b].contiguous().cuda() for a, b in zip(cuts, cuts[1:])]
    parts = torch.stack([vp.vp_linear_cross_entropy_partial(hg, p, tg, softcap=c, vocab_start=a)
                         for p, a in zip(ws, cuts)])
    loss, stats = vp.vp_cross_entropy_merge(parts, label_smoothing=s, z_loss=z)

    x = h.double() @ w.double().t()
    ref = plain(x, targets, s, z, c)
    near(loss, ref, loss_tol(x, ref, targets, s, z, c, (128 / 16 + 1) * 2.25 * U * (h.double().abs() @ w.double().abs().t()).amax(1)),
         "merged")
    got = [vp.vp_linear_cross_entropy_bwd(hg, p, tg, stats, g.cuda(), vocab_start=a, vocab_total=1000, **kw(o))
           for p, a in zip(ws, cuts)]
    # each shard's dhidden is rounded, then their sum is taken in 64 bits
    half = torch.finfo(BF16).eps / 2
    (dh, dh_tol), (dw, dw_tol) = gradients(h.double(), w.double(), targets, g, o, vp.GRAD_MIXED)
    near(torch.cat([b for _, b in got]), dw, dw_tol + half * dw.abs(), "sharded dW")
    near(sum(a.double() for a, _ in got), dh, (1 + half) * dh_tol + half * sum(a.double().abs() for a, _ in got).cpu(),
         "sharded dhidden")


# --------------------------------------------------------------------------- streams, graphs, buffers
@pytest.mark.gpu
def test_another_stream_and_a_captured_step():
    h, w, targets, g = (t.cuda() for t in model(96, 1300, 128, 41))
    x = (h.float() @ w.float().t()).to(BF16)
    o = dict(label_smoothing=0.1, z_loss=1e-4, softcap=12.0)

    def step():
        a, st = vp.vp_cross_entropy_fwd(x, targets, **o)
        b, sl = vp.vp_linear_cross_entropy_fwd(h, w, targets, **o)
        return (a, vp.vp_cross_entropy_bwd(x, targets, st, g, **o), b,
                *vp.vp_linear_cross_entropy_bwd(h, w, targets, sl, g, **o))

    ref = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    h.mul_(0.5)
    x.copy_((h.float() @ w.float().t()).to(BF16))
    targets.copy_(targets.roll(1))
    for _ in range(2):
        graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, step()))
    assert vp.vp_fault_status() == 0


@pytest.mark.gpu
def test_two_streams_at_once():
    a, b = (tuple(t.cuda() for t in model(200, 3000, 256, s)) for s in (46, 47))

    def step(h, w, targets, g):
        loss, st = vp.vp_linear_cross_entropy_fwd(h, w, targets, softcap=9.0)
        dh, dw = vp.vp_linear_cross_entropy_bwd(h, w, targets, st, g, softcap=9.0)
        return loss, dh, vp.vp_embedding_bwd(dh, targets, 3000, dW=dw, accumulate=True)

    ref = step(*a), step(*b)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[], []]
    for _ in range(5):
        for i, (stream, args) in enumerate(zip(streams, (a, b))):
            with torch.cuda.stream(stream):
                got[i].append(step(*args))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for i in (0, 1) for out in got[i] for x, y in zip(out, ref[i]))


@pytest.mark.gpu
def test_callers_buffers_and_nothing_behind_them():
    x, targets, g = (t.cuda() for t in rows(10, 9001, F32, 43))
    loss, stats = torch.full((11,), 7.0, device="cuda"), torch.full((11, 8), 7.0, device="cuda")
    need = vp.vp_cross_entropy_workspace_size(10, 9001)
    work = torch.full((need + 64,), 99, dtype=torch.uint8, device="cuda")
    ref, rst = vp.vp_cross_entropy_fwd(x, targets, label_smoothing=0.1)
    vp.vp_cross_entropy_fwd(x, targets, label_smoothing=0.1, loss=loss[:10], stats=stats[:10], workspace=work[:-64])
    assert torch.equal(loss[:10], ref) and torch.equal(stats[:10], rst)
    assert need and (loss[10:] == 7).all() and (stats[10:] == 7).all() and (work[-64:] == 99).all()
    dx = torch.full((11, 9001), 7.0, device="cuda")
    vp.vp_cross_entropy_bwd(x, targets, stats[:10], g, label_smoothing=0.1, dx=dx[:10])
    assert (dx[10:] == 7).all()
    h, w, t, gg = (v.cuda() for v in model(20, 600, 64, 44))
    loss, st = vp.vp_linear_cross_entropy_fwd(h, w, t)
    dh, dw = torch.full((21, 64), 7.0, dtype=BF16, device="cuda"), torch.full((601, 64), 7.0, dtype=BF16, device="cuda")
    vp.vp_linear_cross_entropy_bwd(h, w, t, st, gg, dhidden=dh[:20], dW=dw[:600])
    assert (dh[20:] == 7).all() and (dw[600:] == 7).all() and not (dw[:600] == 7).all()


@pytest.mark.gpu
def test_buffers_at_their_least_alignment():
    """Workspaces of the loss on any 16-byte boundary, of the fused forms on any of 256, records on any of 8."""
    x, targets, g = (t.cuda() for t in rows(700, 9001, F32, 51))
    ref, rst = vp.vp_cross_entropy_fwd(x, targets)
    need = vp.vp_cross_entropy_workspace_size(700, 9001)
    work = torch.empty(need + 16, dtype=torch.uint8, device="cuda")[16:]
    assert work.data_ptr() % 32 == 16
    loss, stats = vp.vp_cross_entropy_fwd(x, targets, workspace=work)
    assert torch.equal(loss, ref) and torch.equal(stats, rst)
    parts = vp.partials(701, "cuda")[1:]
    assert parts.data_ptr() % 16 == 8
    vp.vp_cross_entropy_partial(x, targets, parts=parts, workspace=work)
    merged, _ = vp.vp_cross_entropy_merge(parts[None])
    assert torch.allclose(merged, ref, rtol=1e-6)
    h, w, t, gg = (v.cuda() for v in model(300, 9000, 128, 52))
    ref, st = vp.vp_linear_cross_entropy_fwd(h, w, t)
    dh, dw = vp.vp_linear_cross_entropy_bwd(h, w, t, st, gg)
    for size, call, want in ((vp.vp_linear_cross_entropy_workspace_size(300, 9000, 128),
                              lambda work: vp.vp_linear_cross_entropy_fwd(h, w, t, workspace=work), (ref, st)),
                             (vp.vp_linear_cross_entropy_bwd_workspace_size(300, 9000, 128),
                              lambda work: vp.vp_linear_cross_entropy_bwd(h, w, t, st, gg, workspace=work), (dh, dw))):
        work = torch.empty(size + 256, dtype=torch.uint8, device="cuda")[256:]
        assert work.data_ptr() % 512 == 256
        assert all(torch.equal(a, b) for a, b in zip(call(work), want))


@pytest.mark.gpu
def test_no_rows():
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    loss, stats = vp.vp_cross_entropy_fwd(torch.empty(0, 50, device="cuda"), none)
    assert loss.shape == (0,) and vp.vp_cross_entropy_bwd(torch.empty(0, 50, device="cuda"), none, stats, loss).shape == (0, 50)
    h, w = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.ones(50, 64, dtype=BF16, device="cuda")
    loss, stats = vp.vp_linear_cross_entropy_fwd(h, w, none)
    dh, dw = vp.vp_linear_cross_entropy_bwd(h, w, none, stats, loss)
    assert dh.shape == (0, 64) and (dw == 0).all()                   # a sum over no rows


# --------------------------------------------------------------------------- refusals (no GPU needed)
FAKE, ODD = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100001)
BIG = ctypes.c_size_t(1 << 40)


# wide enough to take a workspace: with one missing or short, nothing may be launched
def fwd(dtype=1, N=4, V=20000, smooth=0.0, z=0.0, cap=0.0, targets=FAKE, loss=FAKE, stats=FAKE, work=FAKE, size=BIG):
    return _lib.lib().vp_cross_entropy_fwd(FAKE, dtype, N, V, 4, 0, V, 0, smooth, z, cap, targets, loss, stats, work, size,
                                           None, None)


def test_refusals_of_the_library():
    lib = _lib.lib()
    nan, inf = math.nan, math.inf
    for bad in (dict(smooth=-0.1), dict(smooth=1.1), dict(smooth=nan), dict(z=-1.0), dict(z=nan), dict(z=inf),
                dict(cap=-1.0), dict(cap=nan), dict(cap=inf), dict(cap=1e-40), dict(size=ctypes.c_size_t(16))):
        assert fwd(**bad) == ERR_ARG, bad
    assert fwd(dtype=2) == ERR_DTYPE and fwd(V=0) == ERR_SHAPE and fwd(N=-1) == ERR_SHAPE
    for name in ("targets", "loss", "stats", "work"):
        assert fwd(**{name: None}) == ERR_NULL and fwd(**{name: ODD}) == ERR_ALIGN
    assert fwd(N=0, targets=None, loss=None, stats=None, work=None) == OK
    bwd = lambda total=0, dx=FAKE, smooth=0.0: lib.vp_cross_entropy_bwd(
        FAKE, 1, 4, 16, 4, 0, 16, 0, total, smooth, 0.0, 0.0, FAKE, FAKE, FAKE, dx, None, None)
    assert bwd(total=15) == ERR_SHAPE and bwd(dx=None) == ERR_NULL and bwd(dx=ODD) == ERR_ALIGN and bwd(smooth=2.0) == ERR_ARG
    part = lambda parts=FAKE, cap=0.0, work=FAKE: lib.vp_cross_entropy_partial(
        FAKE, 1, 4, 20000, 4, 0, 20000, 0, cap, FAKE, parts, work, BIG, None)
    assert part(parts=None) == ERR_NULL and part(work=None) == ERR_NULL and part(parts=ODD) == ERR_ALIGN and part(cap=-1.0) == ERR_ARG
    merge = lambda K=2, smooth=0.0, loss=FAKE: lib.vp_cross_entropy_merge(FAKE, K, 4, smooth, 0.0, loss, FAKE, None, None)
    assert merge(K=0) == ERR_SHAPE and merge(smooth=-1.0) == ERR_ARG and merge(loss=None) == ERR_NULL
    lin = lambda D=64, loss=FAKE, work=FAKE, size=BIG, cap=0.0: lib.vp_linear_cross_entropy_fwd(
        FAKE, FAKE, 4, 16, D, 0, 0.0, 0.0, cap, FAKE, loss, FAKE, work, size, None, None)
    assert lin(D=96) == ERR_SHAPE and lin(loss=None) == ERR_NULL and lin(cap=nan) == ERR_ARG
    assert lin(work=ctypes.c_void_p(0x100010)) == ERR_ALIGN and lin(size=ctypes.c_size_t(8)) == ERR_ARG
    back = lambda dh=FAKE, dw=FAKE, p=0, total=0, N=4, size=BIG: lib.vp_linear_cross_entropy_bwd(
        FAKE, FAKE, N, 16, 64, 0, total, 0.0, 0.0, 0.0, FAKE, FAKE, FAKE, dh, dw, p, FAKE, size, None, None)
    assert back(dh=None, dw=None) == ERR_ARG and back(p=3) == ERR_ARG and back(p=-1) == ERR_ARG and back(total=3) == ERR_SHAPE
    assert back(dw=ODD) == ERR_ALIGN and back(N=0, dw=None) == OK and back(size=ctypes.c_size_t(8)) == ERR_ARG
    assert lib.vp_linear_cross_entropy_partial(FAKE, FAKE, 4, 16, 64, 0, 0.0, FAKE, None, FAKE, BIG, None) == ERR_NULL
    assert lib.vp_cross_entropy_workspace_size(-1, 5) == 0 and lib.vp_linear_cross_entropy_workspace_size(4, 5, 65) == 0


def test_a_workspace_off_a_16_byte_boundary_is_refused():
    """The slices' records are written and read 16 bytes at a time."""
    eight = ctypes.c_void_p(0x100008)
    assert fwd(work=eight) == ERR_ALIGN
    assert _lib.lib().vp_cross_entropy_partial(FAKE, 1, 4, 20000, 4, 0, 20000, 0, 0.0, FAKE, FAKE, eight, BIG,
                                               None) == ERR_ALIGN


def test_refusals_of_the_binding():
    def status(fn):
        with pytest.raises(vp.VPError) as e:
            fn()
        return e.value.status

    N, V = 6, 40
    x, t, g, st = torch.zeros(N, V), torch.zeros(N, dtype=torch.int64), torch.zeros(N), vp.rowstats(N, "cpu")
    assert status(lambda: vp.vp_cross_entropy_fwd(x, t.int())) == 3
    assert status(lambda: vp.vp_cross_entropy_fwd(x, t[:-1])) == 2
    assert status(lambda: vp.vp_cross_entropy_fwd(x, t, loss=torch.empty(N + 1))) == 2
    assert status(lambda: vp.vp_cross_entropy_fwd(x.half(), t)) == 3
    assert status(lambda: vp.vp_cross_entropy_fwd(x.t(), torch.zeros(V, dtype=torch.int64))) == 4
    assert status(lambda: vp.vp_cross_entropy_fwd(x, t)) == 8                                # not on a GPU
    assert status(lambda: vp.vp_cross_entropy_bwd(x, t, st, g, dx=torch.empty(N, V, dtype=BF16))) == 3
    assert status(lambda: vp.vp_cross_entropy_bwd(x, t, st, torch.zeros(2 * N)[::2])) == 4
    assert status(lambda: vp.vp_cross_entropy_partial(x, t, parts=vp.partials(N - 1, "cpu"))) == 2
    assert status(lambda: vp.vp_cross_entropy_merge(vp.partials(N, "cpu"))) == 2
    h, w = torch.zeros(N, 64, dtype=BF16), torch.zeros(V, 64, dtype=BF16)
    assert status(lambda: vp.vp_linear_cross_entropy_fwd(h.float(), w, t)) == 3
    assert status(lambda: vp.vp_linear_cross_entropy_fwd(h, w[:, :32], t)) in (2, 4)
    assert status(lambda: vp.vp_linear_cross_entropy_bwd(h, w, t, st, g, dW=torch.empty(V, 65, dtype=BF16))) == 2
    assert status(lambda: vp.vp_linear_cross_entropy_bwd(h, w, t, st, g, dhidden=h.float())) == 3
