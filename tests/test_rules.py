"""Rules on logits (penalties, biases, masks, temperature), their gradient, and the ruled logprobs.

Every GPU result is compared with a plain implementation in 64 bits, row by
row. Tolerances count roundings (u = 2^-24, the fp32 half step; h = 2^-8 for
bf16 outputs, u for fp32 ones):

  * forward: at most 8 fp32 operations, each off by u of the largest magnitude
    M = (|x f| + |freq c| + |pres| + |bias|) / T it can meet, then the output's
    rounding: 8 u M + h |y|;
  * gradient of the rules: 4 operations and the rounding: (4 u + h) |dx|;
  * logp: the errors of z (8 u M, the row's largest M) enter z_t and the
    log-sum; an exponential is off by at most 4 u + 2 |t| u relative, weighted
    by p (E_p|t| < log V + 1 < 13); 32 fp32 additions per thread; the output:
    u (16 M + 26 + 4 + 32 + |logp|);
  * its gradient: d = log p is off by the same, so p by that share, and 6 more
    operations: |g f p| (e_logp + 8 u) + (6 u + h) |dx|, and 2^-126 for
    probabilities that flush to 0.
"""
import ctypes
import math

import pytest
import torch

import vocab_wide_logprobs_gb300 as vp
from vocab_wide_logprobs_gb300 import _lib

U = 2.0 ** -24
OK, ERR_NULL, ERR_SHAPE, ERR_DTYPE, ERR_LAYOUT, ERR_ALIGN, ERR_LAUNCH, ERR_ARG, ERR_DEVICE = range(9)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ---------------------------------------------------------------------------
# plain implementation, 64 bits, one row at a time
# ---------------------------------------------------------------------------
def plain_row(x, r, q, start):
    """(y, f, M) of one row: ruled logits, dy/dx, and the largest magnitude each column's operations meet."""
    x = x.double()
    V = x.numel()

    def per_row(name, default):
        return default if q.get(name) is None else float(q[name][r].double())

    rep, freq = per_row("repetition", 1.0), per_row("frequency", 0.0)
    pres, T = per_row("presence", 0.0), per_row("temperature", 1.0)
    prompt, output = {}, {}
    if q.get("spans") is not None:
        first, n_prompt, n_total = q["spans"][r].tolist()
        for i, v in enumerate(q["ids"][first:first + n_total].tolist()):
            if v >= 0 and 0 <= v - start < V:
                d = prompt if i < n_prompt else output
                d[v - start] = d.get(v - start, 0) + 1
    bias = {}
    if q.get("bias_spans") is not None:
        first, n = q["bias_spans"][r].tolist()
        for v, b in zip(q["bias_ids"][first:first + n].tolist(), q["bias_values"][first:first + n].tolist()):
            if v >= 0 and 0 <= v - start < V:
                bias[v - start] = b
    z, f, M = x.clone(), torch.ones(V, dtype=torch.float64), x.abs()
    for j in set(prompt) | set(output):
        f[j] = 1 / rep if z[j] > 0 else rep
        z[j] = z[j] / rep if z[j] > 0 else z[j] * rep
        M[j] = z[j].abs()
        if j in output:
            z[j] = z[j] - freq * output[j] - pres
            M[j] += abs(freq) * output[j] + abs(pres)
    for j, b in bias.items():
        z[j] += b
        M[j] += abs(b)
    z, f, M = z / T, f / T, M / T
    if q.get("mask") is not None:
        m = r if q.get("mask_rows") is None else int(q["mask_rows"][r])
        if m >= 0:
            words = q["mask"][m].tolist()
            allowed = torch.tensor([bool(words[j // 32] >> (j % 32) & 1) for j in range(V)])
            z[~allowed], f[~allowed] = -math.inf, 0.0
    return z, f, torch.where(torch.isfinite(M), M, 0.0)


def plain_logprob(z, t):
    lse = torch.logsumexp(z, 0)
    p = torch.exp(z - lse)
    g = -p
    g[t] = -torch.expm1(z[t] - lse)
    return z[t] - lse, p, g


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def make(N, V, dtype, seed, L=40, nb=0, masks=0, start=0, shared=False, drop=()):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(N, V, generator=g) * 3).to(dtype)
    total = start + V + 7
    ids = torch.randint(0, total, (N * L + 3,), generator=g)
    ids[torch.rand(ids.shape, generator=g) < 0.3] = start + V // 2      # one id many times
    ids[torch.rand(ids.shape, generator=g) < 0.05] = -1                 # padding
    if shared:                                                          # prefixes of one sequence
        spans = torch.stack((torch.zeros(N, dtype=torch.int64), torch.full((N,), min(2, L)),
                             torch.arange(N) % L + min(2, L)), 1)
    else:
        n = torch.randint(0, L + 1, (N,), generator=g)
        n[0] = L
        spans = torch.stack((torch.arange(N) * L, (n * torch.rand(N, generator=g)).long(), n), 1)
        if N > 2:
            spans[1] = torch.tensor([N * L, 0, 0])                      # an empty history
            spans[2, 1] = spans[2, 2]                                   # nothing but a prompt
    q = dict(ids=ids, spans=spans, repetition=0.7 + torch.rand(N, generator=g),
             frequency=torch.rand(N, generator=g) - 0.2, presence=torch.rand(N, generator=g) - 0.2,
             temperature=0.5 + torch.rand(N, generator=g))
    if nb:
        b = torch.randint(0, total, (N * nb,), generator=g)
        b[::5] = start + V // 3                                         # the same id again: the last one counts
        q.update(bias_ids=b, bias_values=torch.randn(N * nb, generator=g) * 4,
                 bias_spans=torch.stack((torch.arange(N) * nb, torch.randint(0, nb + 1, (N,), generator=g)), 1))
        q["bias_values"][::11] = -math.inf
    if masks:
        words = torch.randint(-2 ** 31, 2 ** 31, (masks, -(-V // 32)), generator=g, dtype=torch.int64)
        q.update(mask=words.to(torch.int32), mask_rows=torch.randint(-1, masks, (N,), generator=g))
    for name in drop:
        q[name] = None
    targets = torch.randint(0, V, (N,), generator=g) + start
    return x, q, targets, torch.randn(N, generator=g)


def to_gpu(q):
    return vp.logits_rules(**{k: None if t is None else t.cuda() for k, t in q.items()})


def check(got, ref, tol, what):
    got = got.double().cpu()
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    assert torch.equal(got[~fine & ~torch.isnan(ref)], ref[~fine & ~torch.isnan(ref)]), f"{what}: infinities"
    off = (got - ref).abs()[fine] - tol[fine]
    assert off.numel() == 0 or off.max() <= 0, f"{what}: {float(off.max())} over its tolerance"


CASES = [
    # N, V, dtype, options
    (1, 1, torch.float32, dict(L=3)),
    (3, 7, torch.bfloat16, dict(L=5, nb=3, masks=1)),
    (5, 130, torch.float32, dict(L=200, nb=9, masks=2, start=50)),
    (6, 1000, torch.bfloat16, dict(L=33, masks=3, shared=True)),
    (4, 8192, torch.bfloat16, dict(L=300, nb=40)),
    (3, 8193, torch.float32, dict(L=300, nb=40, masks=2)),
    (3, 8200, torch.bfloat16, dict(L=0)),
    (3, 20011, torch.bfloat16, dict(L=1500, nb=100, masks=2, start=1000)),
    (2, 24576, torch.float32, dict(L=700, masks=1, drop=("frequency", "presence"))),
    (2, 9000, torch.float32, dict(L=700, nb=5, drop=("repetition", "temperature"))),
    (3, 500, torch.bfloat16, dict(L=9, nb=4, masks=2,
                                  drop=("ids", "spans", "repetition", "frequency", "presence"))),
]
IDS = [f"{n}x{v}-{'bf16' if d == torch.bfloat16 else 'f32'}" for n, v, d, _ in CASES]


def views(x, kind):
    """The same rows, contiguous or inside a wider tensor at an odd offset."""
    x = x.cuda()
    if kind == "contiguous":
        return x
    wide = torch.full((x.shape[0] + 1, x.shape[1] + 5), float("nan"), dtype=x.dtype, device="cuda")
    wide[1:, 3:3 + x.shape[1]] = x
    return wide[1:, 3:3 + x.shape[1]]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["contiguous", "view"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_process_against_64_bits(case, kind):
    N, V, dtype, opt = case
    x, q, _, _ = make(N, V, dtype, 11 + V, **opt)
    start, h = opt.get("start", 0), half_step(dtype)
    rules, xg = to_gpu(q), views(x, kind)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dy = torch.randn(N, V).to(dtype)
    y = vp.vp_logits_process_fwd(xg, rules, vocab_start=start, err_word=err)
    dx = vp.vp_logits_process_bwd(xg, rules, dy.cuda(), vocab_start=start, err_word=err)
    held = xg.clone()
    again = vp.vp_logits_process_fwd(xg, rules, vocab_start=start, y=xg)       # in place
    torch.cuda.synchronize()
    assert int(err) == 0
    assert again.data_ptr() == xg.data_ptr() and torch.equal(again, y)
    assert torch.equal(held.cpu(), x)
    for r in range(N):
        z, f, M = plain_row(x[r], r, q, start)
        check(y[r], z, 8 * U * M + h * z.abs(), f"row {r}")
        ref = torch.where(f == 0, 0.0, dy[r].double() * f)
        check(dx[r], ref, (4 * U + h) * ref.abs() + 2.0 ** -133, f"gradient of row {r}")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["contiguous", "view"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_processed_logprobs_against_64_bits(case, kind):
    N, V, dtype, opt = case
    x, q, targets, grad = make(N, V, dtype, 23 + V, **opt)
    start, h = opt.get("start", 0), half_step(dtype)
    if N > 2:
        targets[1] = -5                                                        # ignored
    rules, xg, tg = to_gpu(q), views(x, kind), targets.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    logp, stats = vp.vp_processed_logprobs_fwd(xg, rules, tg, vocab_start=start, err_word=err)
    dx = vp.vp_processed_logprobs_bwd(xg, rules, tg, stats, grad.cuda(), vocab_start=start, err_word=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    for r in range(N):
        z, f, M = plain_row(x[r], r, q, start)
        if targets[r] < 0:
            assert float(logp[r]) == 0 and not dx[r].any()
            continue
        if not torch.isfinite(z).any():                                        # nothing is left
            assert torch.isnan(logp[r]) and torch.isnan(dx[r]).all()
            continue
        lp, p, g = plain_logprob(z, int(targets[r]) - start)
        tol = U * (16 * float(M.max()) + 62 + (abs(float(lp)) if torch.isfinite(lp) else 0.0))
        check(logp[r:r + 1], lp[None], torch.tensor([tol]), f"logp of row {r}")
        scale = (float(grad[r]) * f).abs()
        ref = torch.where(f == 0, 0.0, float(grad[r]) * f * g)
        check(dx[r], ref, scale * p * (tol + 8 * U) + (6 * U + h) * ref.abs() + scale * 2.0 ** -126 + 2.0 ** -133,
              f"gradient of row {r}")


@pytest.mark.gpu
def test_gradients_against_differences():
    """Central differences of the 64-bit forward: their error is step^2 / 6 of a third derivative below 8 g / T^3."""
    N, V, step = 3, 67, 2.0 ** -14
    x, q, targets, grad = make(N, V, torch.float32, 5, L=30, nb=6, masks=1)
    q["mask_rows"] = torch.tensor([-1, 0, 0])
    q["bias_values"] = q["bias_values"].clamp(min=-5)
    for r in range(N):                                                         # the targets are allowed
        word, bit = int(targets[r]) // 32, int(targets[r]) % 32
        q["mask"][0, word] = int(torch.tensor(int(q["mask"][0, word]) | (1 << bit)).to(torch.int32)) if bit < 31 else -1
    x[x.abs() < 2 * step] = 0.5                                                # away from the kink of the penalty
    rules, xg, tg = to_gpu(q), x.cuda(), targets.cuda()
    _, stats = vp.vp_processed_logprobs_fwd(xg, rules, tg)
    dx = vp.vp_processed_logprobs_bwd(xg, rules, tg, stats, grad.cuda()).double().cpu()
    dy = torch.randn(N, V)
    dz = vp.vp_logits_process_bwd(xg, rules, dy.cuda()).double().cpu()
    for r in range(N):
        for j in range(V):
            ends, rows = [], []
            for s in (step, -step):
                moved = x[r].double()
                moved[j] += s
                z = plain_row(moved, r, q, 0)[0]
                rows.append(z)
                ends.append(float(plain_logprob(z, int(targets[r]))[0]))
            T = float(q["temperature"][r])
            num = float(grad[r]) * (ends[0] - ends[1]) / (2 * step)
            tol = 8 * abs(float(grad[r])) / T ** 3 * step ** 2 + 1e-10
            assert abs(float(dx[r, j]) - num) <= tol + 1e-5 * abs(float(grad[r])) / T
            both = torch.isfinite(rows[0])
            num = float((dy[r].double()[both] * (rows[0] - rows[1])[both]).sum()) / (2 * step)
            assert abs(float(dz[r, j]) - num) <= 1e-9 + 1e-6 * abs(num)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [5003, 12288])
def test_a_common_offset_does_not_reach_the_logprob(dtype, V):
    """Peaked rows of logits around 10^4, temperatures that are no powers of two: the target's ruled logit is rounded
    where the maximum's is, and what either rounding takes away has to come back.

    Without penalties a column's value before the temperature is exact, so is its distance t to the row's largest, and
    what is left of the offset is the relative rounding of 1 / T and of the product, twice u of the distances: as in the
    tolerance above with E_p |t| < log V + 1 < 11, a logprob is off by u (2 (|logp| + 11) + 22 + 4 + 32 + |logp|)."""
    N = 64
    g = torch.Generator(device="cuda").manual_seed(V)
    row = torch.arange(N, device="cuda")
    x = torch.randn(N, V, generator=g, device="cuda") + 1e4 * (1 - 2 * (row % 2))[:, None]
    best = torch.randint(0, V, (N,), generator=g, device="cuda")
    x[row, best] += 30 * torch.rand(N, generator=g, device="cuda")
    x = x.to(dtype)
    T = 0.3 + torch.rand(N, generator=g, device="cuda")
    T[0] = 0.7
    rules = vp.logits_rules(temperature=T)
    z = x.double() / T.double()[:, None]
    lse = torch.logsumexp(z, 1)
    for targets in (best, torch.randint(0, V, (N,), generator=g, device="cuda"), x.float().argmax(1)):
        logp, stats = vp.vp_processed_logprobs_fwd(x, rules, targets)
        lp = z.gather(1, targets[:, None])[:, 0] - lse
        tol = U * (3 * lp.abs() + 80)
        assert ((logp.double() - lp).abs() - tol).max() <= 0
        # the gradient's p of the target is the logprob's
        dx = vp.vp_processed_logprobs_bwd(x, rules, targets, stats, torch.ones(N, device="cuda")).double()
        got = dx.gather(1, targets[:, None])[:, 0] * T.double()
        want = -torch.expm1(lp)
        tol = torch.exp(lp) * (tol + 8 * U) + (6 * U + half_step(dtype)) * want.abs() + 2.0 ** -126
        assert ((got - want).abs() - tol).max() <= 0


@pytest.mark.gpu
def test_masked_places_hide_what_they_hold():
    """NaN, infinities and the type's lowest value under the mask change nothing; a row left empty is NaN."""
    N, V = 4, 300
    x, q, targets, grad = make(N, V, torch.float32, 3, L=10)
    bits = torch.ones(2, 320, dtype=torch.int64)
    banned = torch.tensor([3, 31, 32, 64, 299])
    bits[0, banned] = 0
    bits[1] = 0
    words = (bits.view(2, 10, 32) << torch.arange(32)).sum(-1)
    q.update(mask=torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32),
             mask_rows=torch.tensor([0, 0, 0, 1]))
    targets[:] = 7
    targets[2] = 3                                                             # a masked target
    rules = to_gpu(q)
    clean = vp.vp_processed_logprobs_fwd(x.cuda(), rules, targets.cuda())
    dirty = x.clone()
    dirty[:, banned] = torch.tensor([math.nan, math.inf, -math.inf, torch.finfo(torch.float32).min, 3e38])
    logp, stats = vp.vp_processed_logprobs_fwd(dirty.cuda(), rules, targets.cuda())
    assert torch.equal(logp[:3], clean[0][:3]) and torch.equal(stats[:3], clean[1][:3])
    assert logp[2] == -math.inf and torch.isnan(logp[3])
    dx = vp.vp_processed_logprobs_bwd(dirty.cuda(), rules, targets.cuda(), stats, grad.cuda()).cpu()
    assert torch.isfinite(dx[:3]).all() and not dx[:3, banned].any() and torch.isnan(dx[3]).all()
    y = vp.vp_logits_process_fwd(dirty.cuda(), rules).cpu()
    assert (y[:3, banned] == -math.inf).all() and (y[3] == -math.inf).all()
    dy = torch.full((N, V), math.nan)
    assert not vp.vp_logits_process_bwd(dirty.cuda(), rules, dy.cuda()).cpu()[:, banned].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_out_of_range_are_data_errors(dtype):
    """A row whose rules point outside their arrays is NaN with the error bit; the other rows are not touched by it."""
    N, V = 9, 200
    x, q, targets, grad = make(N, V, dtype, 7, L=12, nb=4, masks=2)
    q["bias_values"] = q["bias_values"].clamp(min=-5)
    q["mask_rows"][:] = -1
    good = to_gpu(q)
    ref = vp.vp_logits_process_fwd(x.cuda(), good)
    n_ids = q["ids"].numel()
    big = 2 ** 62
    bad = {0: ("spans", [-1, 0, 2]), 1: ("spans", [n_ids - 1, 0, 2]), 2: ("spans", [0, 3, 2]),
           3: ("spans", [big, 0, big]), 4: ("bias_spans", [N * 4 - 1, 2]), 5: ("mask_rows", 2),
           6: ("repetition", 0.0), 7: ("temperature", math.nan)}
    for r, (name, value) in bad.items():
        q[name][r] = torch.tensor(value, dtype=q[name].dtype)
    rules, xg, tg = to_gpu(q), x.cuda(), targets.cuda()

    def run(call):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = call(err)
        assert int(err) == vp.ERRBIT_RULES
        return out

    y = run(lambda e: vp.vp_logits_process_fwd(xg, rules, err_word=e))
    assert torch.isnan(y[:8]).all() and torch.equal(y[8], ref[8])
    logp, stats = run(lambda e: vp.vp_processed_logprobs_fwd(xg, rules, tg, err_word=e))
    assert torch.isnan(logp[:8]).all() and torch.isfinite(logp[8])
    dx = run(lambda e: vp.vp_processed_logprobs_bwd(xg, rules, tg, stats, grad.cuda(), err_word=e))
    assert torch.isnan(dx[:8]).all() and torch.isfinite(dx[8]).all()
    dx = run(lambda e: vp.vp_logits_process_bwd(xg, rules, torch.ones(N, V, dtype=dtype, device="cuda"), err_word=e))
    assert torch.isnan(dx[:8]).all() and torch.isfinite(dx[8]).all()
    # a target outside the columns is the logprobs' own data error
    tg[8] = V
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    logp, stats = vp.vp_processed_logprobs_fwd(xg, good, tg, err_word=err)
    assert int(err) == vp.ERRBIT_TARGET and torch.isnan(logp[8]) and torch.isfinite(logp[:8]).all()
    assert torch.isnan(vp.vp_processed_logprobs_bwd(xg, good, tg, stats, grad.cuda())[8]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("name", ["temperature", "repetition"])
def test_divisors_whose_reciprocals_do_not_fit_are_data_errors(name, dtype):
    """The kernels multiply by reciprocals: below 2^-127 these have no room, and 0 times infinity is not 0."""
    V, least = 200, 2.0 ** -127
    fine = [least, 2.0 ** -126, 1e-30, 1.0, torch.finfo(torch.float32).max]
    bad = [least - 2.0 ** -149, 2.0 ** -128, 1e-39, 2.0 ** -149, 0.0, -1.0, math.inf, math.nan]
    N = len(fine) + len(bad)
    value = torch.tensor(fine + bad, dtype=torch.float64).float()
    x = torch.zeros(N, V, dtype=dtype)                                        # all of it is seen: 0 / anything is 0
    q = dict(ids=torch.arange(V), spans=torch.tensor([[0, 0, V]]).repeat(N, 1), repetition=torch.ones(N))
    q[name] = value
    rules, xg, tg = to_gpu(q), x.cuda(), torch.full((N,), 3, device="cuda")
    seen = []

    def run(call):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = call(err)
        seen.append(int(err))
        return out

    ok = torch.tensor([True] * len(fine) + [False] * len(bad), device="cuda")
    y = run(lambda e: vp.vp_logits_process_fwd(xg, rules, err_word=e))
    assert torch.isnan(y[~ok]).all() and not y[ok].any()
    logp, stats = run(lambda e: vp.vp_processed_logprobs_fwd(xg, rules, tg, err_word=e))
    assert torch.isnan(logp[~ok]).all() and (logp[ok] + math.log(V)).abs().max() <= U * 80
    run(lambda e: vp.vp_logits_process_bwd(xg, rules, torch.ones_like(xg), err_word=e))
    # gradients: a small upstream one, so that its product with the reciprocal fits
    dx = run(lambda e: vp.vp_processed_logprobs_bwd(xg, rules, tg, stats, torch.full((N,), 2.0 ** -20, device="cuda"),
                                                    err_word=e))
    assert torch.isnan(dx[~ok]).all() and torch.isfinite(dx[ok]).all()
    assert seen == [vp.ERRBIT_RULES] * 4


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_spans_are_checked_without_penalties_too(dtype):
    """Spans that no penalty reads change nothing, but one that is out of range is a data error all the same."""
    N, V = 5, 9000
    x, q, targets, grad = make(N, V, dtype, 41, L=12, drop=("repetition", "frequency", "presence"))
    xg, tg, gg, dy = x.cuda(), targets.cuda(), grad.cuda(), torch.randn(N, V).to(dtype).cuda()

    def run(rules):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        logp, stats = vp.vp_processed_logprobs_fwd(xg, rules, tg, err_word=err)
        errs, outs = [int(err)], [logp]
        for call in (lambda e: vp.vp_logits_process_fwd(xg, rules, err_word=e),
                     lambda e: vp.vp_logits_process_bwd(xg, rules, dy, err_word=e),
                     lambda e: vp.vp_processed_logprobs_bwd(xg, rules, tg, stats, gg, err_word=e)):
            err.zero_()
            outs.append(call(err))
            errs.append(int(err))
        return outs, errs

    ref, errs = run(vp.logits_rules(temperature=q["temperature"].cuda()))
    assert errs == [0] * 4
    got, errs = run(to_gpu(q))
    assert errs == [0] * 4 and all(torch.equal(a, b) for a, b in zip(got, ref))
    q["spans"][1] = torch.tensor([q["ids"].numel() - 1, 0, 2])
    q["spans"][3] = torch.tensor([0, 3, 2])
    got, errs = run(to_gpu(q))
    assert errs == [vp.ERRBIT_RULES] * 4
    for a, b in zip(got, ref):
        assert torch.isnan(a[[1, 3]]).all() and torch.equal(a[[0, 2, 4]], b[[0, 2, 4]])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_without_a_target_are_zero_whatever_their_rules(dtype):
    """Padding: a negative target with NaN logits or rules out of range gives 0 and a zero row, as in the plain logprobs."""
    N, V = 6, 5000
    x, q, targets, grad = make(N, V, dtype, 43, L=12)
    targets[1:5] = -1
    q["temperature"][1], q["repetition"][2], q["spans"][3, 0] = 0.0, math.nan, -4
    x[4, 17] = math.nan
    rules, xg, tg = to_gpu(q), x.cuda(), targets.cuda()
    for call, bit in ((lambda e: vp.vp_processed_logprobs_fwd(xg, rules, tg, err_word=e), vp.ERRBIT_RULES),
                      (lambda e: vp.vp_logprobs_fwd(xg, tg, err_word=e), 0)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        logp, stats = call(err)
        assert int(err) == bit and not logp[1:5].any() and torch.isfinite(logp[[0, 5]]).all()
        if bit:
            err.zero_()
            dx = vp.vp_processed_logprobs_bwd(xg, rules, tg, stats, grad.cuda(), err_word=err)
            assert int(err) == bit
        else:
            dx = vp.vp_logprobs_bwd(xg, tg, stats, grad.cuda())
        assert not dx[1:5].any() and torch.isfinite(dx[[0, 5]]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_do_not_depend_on_the_batch(dtype):
    N, V = 37, 20000
    x, q, targets, grad = make(N, V, dtype, 9, L=60, nb=5, masks=3)
    xg, tg, gg = x.cuda(), targets.cuda(), grad.cuda()
    rules = to_gpu(q)
    logp, stats = vp.vp_processed_logprobs_fwd(xg, rules, tg)
    dx = vp.vp_processed_logprobs_bwd(xg, rules, tg, stats, gg)
    for r in (0, 17, 36):
        one = {k: v if k in ("ids", "bias_ids", "bias_values", "mask") else v[r:r + 1].contiguous() for k, v in q.items()}
        lp, st = vp.vp_processed_logprobs_fwd(xg[r:r + 1], to_gpu(one), tg[r:r + 1])
        d = vp.vp_processed_logprobs_bwd(xg[r:r + 1], to_gpu(one), tg[r:r + 1], st, gg[r:r + 1])
        assert torch.equal(lp.view(torch.int32), logp[r:r + 1].view(torch.int32))
        assert torch.equal(st.view(torch.int32), stats[r:r + 1].view(torch.int32))
        assert torch.equal(d.view(torch.int16), dx[r:r + 1].contiguous().view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [9000, 9001])
def test_rows_do_not_depend_on_where_they_begin(dtype, V):
    N = 6
    x, q, targets, grad = make(N, V, dtype, 12, L=60, nb=5, masks=3)
    rules, tg, gg = to_gpu(q), targets.cuda(), grad.cuda()
    bits = torch.int32 if dtype == torch.float32 else torch.int16
    first = None
    for offset in (0, 1, 3, 8):
        for gap in (0, 1, 4, 16):
            room = torch.full((offset + N * (V + gap),), float("nan"), dtype=dtype, device="cuda")
            xg = room[offset:].view(N, V + gap)[:, :V]
            xg.copy_(x)
            y = vp.vp_logits_process_fwd(xg, rules)
            logp, stats = vp.vp_processed_logprobs_fwd(xg, rules, tg)
            dx = vp.vp_processed_logprobs_bwd(xg, rules, tg, stats, gg)
            dy = vp.vp_logits_process_bwd(xg, rules, dx)
            got = [y.view(bits), logp.view(torch.int32), stats.view(torch.int32), dx.view(bits), dy.view(bits)]
            if first is None:
                first = got
            assert all(torch.equal(a, b) for a, b in zip(got, first)), (offset, gap)


@pytest.mark.gpu
def test_no_rules_are_the_plain_logprobs():
    N, V = 5, 9001
    x, _, targets, grad = make(N, V, torch.bfloat16, 2)
    xg, tg = x.cuda(), targets.cuda()
    none = vp.logits_rules()
    assert torch.equal(vp.vp_logits_process_fwd(xg, none), xg)
    logp, _ = vp.vp_processed_logprobs_fwd(xg, none, tg)
    ref, _ = vp.vp_logprobs_fwd(xg, tg)
    tol = U * (16 * 20 + 62 + 40)
    assert (logp - ref).abs().max() <= 2 * tol


@pytest.mark.gpu
def test_ruled_logits_through_the_other_ops():
    """process_fwd, then the library's own logprobs, then process_bwd: the fused call's results, in fp32."""
    N, V = 6, 5003
    x, q, targets, grad = make(N, V, torch.float32, 13, L=80, nb=6, masks=2)
    rules, xg, tg, gg = to_gpu(q), x.cuda(), targets.cuda(), grad.cuda()
    y = vp.vp_logits_process_fwd(xg, rules)
    ref, st = vp.vp_logprobs_fwd(y, tg)
    logp, stats = vp.vp_processed_logprobs_fwd(xg, rules, tg)
    fine = torch.isfinite(ref)
    assert torch.equal(fine, torch.isfinite(logp)) and (ref - logp)[fine].abs().max() < 1e-4
    dz = vp.vp_logprobs_bwd(y, tg, st, gg)
    dx = vp.vp_processed_logprobs_bwd(xg, rules, tg, stats, gg)
    chained = vp.vp_logits_process_bwd(xg, rules, dz)
    assert (chained - dx)[fine].abs().max() < 1e-4


@pytest.mark.gpu
def test_streams_and_graphs():
    """On a stream of its own, and captured once and replayed on new inputs."""
    N, V = 4, 10000
    x, q, targets, grad = make(N, V, torch.bfloat16, 17, L=50, nb=3, masks=1)
    rules, tg, gg = to_gpu(q), targets.cuda(), grad.cuda()
    xs = [x.cuda(), (x.float() * 0.5 + 1).to(torch.bfloat16).cuda()]

    def step(xg):
        logp, stats = vp.vp_processed_logprobs_fwd(xg, rules, tg)
        return logp, vp.vp_processed_logprobs_bwd(xg, rules, tg, stats, gg), vp.vp_logits_process_fwd(xg, rules)

    refs = [step(v) for v in xs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step(xs[1])
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, refs[1]))
    held = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(held)
    for v, ref in zip(xs[::-1], refs[::-1]):
        held.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


@pytest.mark.gpu
@pytest.mark.parametrize("n_ids", [20000, 100000, 3000000, 9000000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_rows_of_few_ids(dtype, n_ids):
    """More tiles than run at once, rows with and without a history in turn, ids far apart in a long list."""
    N, V = 1500, 8200
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(N, V, generator=g, device="cuda").to(dtype)
    ids = torch.full((n_ids,), -1, dtype=torch.int64, device="cuda")
    at = torch.arange(0, N, 7, device="cuda")
    first = at * (n_ids // N)
    for k, v in enumerate((5, 5, 8199)):
        ids[first + k] = v
    spans = torch.zeros(N, 3, dtype=torch.int64, device="cuda")
    spans[at, 0], spans[at, 2] = first, 3
    two = torch.full((N,), 2.0, device="cuda")
    rules = vp.logits_rules(ids=ids, spans=spans, frequency=two, temperature=two)
    z = x.float().clone()
    z[at, 5] -= 4
    z[at, 8199] -= 2
    z /= 2                                                        # exact: a power of two
    assert torch.equal(vp.vp_logits_process_fwd(x, rules), z.to(dtype))
    targets = torch.full((N,), 5, dtype=torch.int64, device="cuda")
    logp, stats = vp.vp_processed_logprobs_fwd(x, rules, targets)
    ref = torch.log_softmax(z.double(), 1)
    assert (logp.double() - ref[:, 5]).abs().max() < U * (16 * 8 + 62 + 16)
    one = torch.ones(N, device="cuda")
    dx = vp.vp_processed_logprobs_bwd(x, rules, targets, stats, one).double()
    g64 = -ref.exp()
    g64[:, 5] = -torch.expm1(ref[:, 5])
    g64 /= 2
    assert ((dx - g64).abs() - (half_step(dtype) + U * 220) * g64.abs() - 2.0 ** -126).max() <= 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("uniform", [True, False])
def test_long_shared_histories(dtype, uniform):
    """Several slices of a row for one CTA, more ids and listed columns than its lists hold, all four calls."""
    N, V, L, start = 400, 20001, 6000, 3
    g = torch.Generator(device="cuda").manual_seed(2)
    x = (torch.randn(N, V, generator=g, device="cuda") * 3).to(dtype)
    u = torch.rand(L + N, generator=g, device="cuda")
    ids = ((u if uniform else u ** 4) * (V + 9)).long()                       # a few outside the columns
    r = torch.arange(N, device="cuda")
    n_prompt, n_total = torch.full_like(r, 2500), L + r // 2
    n_total[::9] = 0
    n_prompt[::9] = 0
    spans = torch.stack((torch.zeros_like(r), n_prompt, n_total), 1)
    at = torch.arange(L + N, device="cuda")
    local = ids - start
    ok = (local >= 0) & (local < V)

    def counts(first, last):                                                  # of ids[first[r]:last[r]] in each row
        use = ok[None, :] & (at[None, :] >= first[:, None]) & (at[None, :] < last[:, None])
        return torch.zeros(N, V, dtype=torch.float64, device="cuda").scatter_add_(
            1, local.clamp(0, V - 1).expand(N, -1), use.double())

    c_p, c_o = counts(torch.zeros_like(r), n_prompt), counts(n_prompt, n_total)
    # powers of two: every product and quotient is exact, a count's product too
    rules = vp.logits_rules(ids=ids, spans=spans.contiguous(), repetition=torch.full((N,), 2.0, device="cuda"),
                            frequency=torch.full((N,), 2.0 ** -6, device="cuda"),
                            presence=torch.full((N,), 0.25, device="cuda"), temperature=torch.full((N,), 0.5, device="cuda"))
    f = torch.where(c_p + c_o > 0, torch.where(x > 0, 0.5, 2.0), 1.0).double()
    z = 2 * (x.double() * f - c_o * 2.0 ** -6 - 0.25 * (c_o > 0))
    M = 2 * ((x.double() * f).abs() + c_o * 2.0 ** -6 + 0.25)
    y = vp.vp_logits_process_fwd(x, rules, vocab_start=start)
    assert ((y.double() - z).abs() - 8 * U * M - half_step(dtype) * z.abs()).max() <= 0
    dy = torch.randn(N, V, generator=g, device="cuda").to(dtype)
    dx = vp.vp_logits_process_bwd(x, rules, dy, vocab_start=start)
    assert torch.equal(dx, (dy.double() * f * 2).to(dtype))
    t = torch.randint(0, V, (N,), generator=g, device="cuda")
    logp, stats = vp.vp_processed_logprobs_fwd(x, rules, t + start, vocab_start=start)
    again = vp.vp_processed_logprobs_fwd(x, rules, t + start, vocab_start=start)
    assert torch.equal(logp, again[0]) and torch.equal(stats, again[1])       # whoever finds a column first
    ref = torch.log_softmax(z, 1)
    lp = ref.gather(1, t[:, None])[:, 0]
    tol = U * (16 * M.amax(1) + 62 + lp.abs())
    assert ((logp.double() - lp).abs() - tol).max() <= 0
    grad = torch.randn(N, generator=g, device="cuda")
    dx = vp.vp_processed_logprobs_bwd(x, rules, t + start, stats, grad, vocab_start=start)
    p = ref.exp()
    e = (-p).scatter_(1, t[:, None], -torch.expm1(lp)[:, None])
    scale = 2 * f * grad.double()[:, None]
    off = (dx.double() - scale * e).abs()
    assert (off - scale.abs() * p * (tol[:, None] + 8 * U) - (6 * U + half_step(dtype)) * (scale * e).abs()
            - scale.abs() * 2.0 ** -126).max() <= 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [20000, 20001])
@pytest.mark.parametrize("N", [3, 60])
def test_long_histories_of_their_own(N, V, dtype):
    """Rows of up to 9000 ids, most of them in the first slices: a few rows, and more tiles than run at once."""
    L = 9000
    g = torch.Generator(device="cuda").manual_seed(3)
    x = (torch.randn(N, V, generator=g, device="cuda") * 3).to(dtype)
    ids = (torch.rand(N, L, generator=g, device="cuda") ** 4 * (V + 9)).long()   # a few outside the columns
    n_total = torch.randint(0, L + 1, (N,), generator=g, device="cuda")
    n_total[0], n_total[1] = L, 0
    n_prompt = n_total // 3
    row = torch.arange(N, device="cuda")
    spans = torch.stack((row * L, n_prompt, n_total), 1)
    at = torch.arange(L, device="cuda")[None, :]

    def counts(first, last):
        use = (at >= first[:, None]) & (at < last[:, None]) & (ids < V)
        return torch.zeros(N, V, dtype=torch.float64, device="cuda").scatter_add_(1, ids.clamp(max=V - 1), use.double())

    c_p, c_o = counts(torch.zeros_like(n_prompt), n_prompt), counts(n_prompt, n_total)
    assert int((c_o[0, :4096] > 0).sum()) > 512                               # a tile with more of them than its list holds
    rules = vp.logits_rules(ids=ids.view(-1), spans=spans, repetition=torch.full((N,), 2.0, device="cuda"),
                            frequency=torch.full((N,), 2.0 ** -6, device="cuda"),
                            presence=torch.full((N,), 0.25, device="cuda"), temperature=torch.full((N,), 0.5, device="cuda"))
    f = torch.where(c_p + c_o > 0, torch.where(x > 0, 0.5, 2.0), 1.0).double()
    z = 2 * (x.double() * f - c_o * 2.0 ** -6 - 0.25 * (c_o > 0))
    M = 2 * ((x.double() * f).abs() + c_o * 2.0 ** -6 + 0.25)
    y = vp.vp_logits_process_fwd(x, rules)
    assert ((y.double() - z).abs() - 8 * U * M - half_step(dtype) * z.abs()).max() <= 0
    assert torch.equal(y, vp.vp_logits_process_fwd(x, rules))


def by_row(q, name, default):
    return default if q.get(name) is None else q[name].double()[:, None]


def ruled_rows(x, q, rows):
    """(z, f, M) of some rows as plain_row has them, on x's device; vocab_start 0 and no repeated bias ids."""
    V = x.shape[1]
    q = {k: t if k in ("ids", "bias_ids", "bias_values", "mask") else t[rows] for k, t in q.items() if t is not None}
    x = x[rows].double()
    rep, T = by_row(q, "repetition", 1.0), by_row(q, "temperature", 1.0)
    freq, pres = by_row(q, "frequency", 0.0), by_row(q, "presence", 0.0)
    c_p, c_o, bias = (torch.zeros_like(x) for _ in range(3))
    for i, (first, n_prompt, n_total) in enumerate(q["spans"].tolist()):
        ids = q["ids"][first:first + n_total]
        for counts, part in ((c_p, ids[:n_prompt]), (c_o, ids[n_prompt:])):
            part = part[(part >= 0) & (part < V)]
            counts[i].scatter_add_(0, part, torch.ones_like(part, dtype=torch.float64))
    if "bias_spans" in q:
        for i, (first, n) in enumerate(q["bias_spans"].tolist()):
            ids, values = q["bias_ids"][first:first + n], q["bias_values"][first:first + n].double()
            bias[i, ids] = values
    f = torch.where(c_p + c_o > 0, torch.where(x > 0, 1 / rep, rep), torch.ones_like(x))
    z = x * f
    M = z.abs() + freq.abs() * c_o + pres.abs() * (c_o > 0) + bias.abs()
    z = (z - freq * c_o - pres * (c_o > 0) + bias) / T
    f, M = f / T, M / T
    if "mask" in q:
        bits = torch.arange(V, device=x.device)
        for i, m in enumerate(q["mask_rows"].tolist()):
            if m >= 0:
                banned = (q["mask"][m].long()[bits // 32] >> (bits % 32) & 1) == 0
                z[i, banned], f[i, banned], M[i, banned] = -math.inf, 0.0, 0.0
    return z, f, M


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N, V", [(3, 140003), (1000, 151936), (1200, 262208)])
def test_rows_of_many_slices(N, V, dtype):
    """More slices than the join has lanes (a few rows), more than 32 and more than 64 of a row for one CTA.

    The tolerances are those above with log V + 1 < 14: u (16 M + 64 + |logp|) for a logprob."""
    L, nb = 500, 20
    g = torch.Generator(device="cuda").manual_seed(V + N)
    x = (torch.randn(N, V, generator=g, device="cuda") * 3).to(dtype)
    u = torch.rand(N * L, generator=g, device="cuda")
    row = torch.arange(N, device="cuda")
    n_total = torch.randint(0, L + 1, (N,), generator=g, device="cuda")
    words = torch.randint(-2 ** 31, 2 ** 31, (2, -(-V // 32)), generator=g, device="cuda").to(torch.int32)
    q = dict(ids=(torch.where(u < 0.5, u * 2, (u - 0.5) ** 3 * 8) * V).long().clamp(max=V - 1),
             spans=torch.stack((row * L, n_total // 3, n_total), 1),
             repetition=1 + torch.rand(N, generator=g, device="cuda"),
             frequency=torch.rand(N, generator=g, device="cuda"), presence=torch.rand(N, generator=g, device="cuda"),
             temperature=0.5 + torch.rand(N, generator=g, device="cuda"),
             bias_ids=(row[:, None] * 17 + torch.arange(nb, device="cuda") * (V // nb)).view(-1) % V,
             bias_values=torch.randn(N * nb, generator=g, device="cuda"),
             bias_spans=torch.stack((row * nb, torch.full_like(row, nb)), 1),
             mask=words, mask_rows=torch.randint(-1, 2, (N,), generator=g, device="cuda"))
    targets = torch.randint(0, V, (N,), generator=g, device="cuda")
    targets[::3] = q["ids"].view(N, L)[::3, 0]                                # some of them listed
    grad = torch.randn(N, generator=g, device="cuda")
    dy = torch.randn(N, V, generator=g, device="cuda").to(dtype)
    rules, h = vp.logits_rules(**q), half_step(dtype)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = vp.vp_logits_process_fwd(x, rules, err_word=err)
    dz = vp.vp_logits_process_bwd(x, rules, dy, err_word=err)
    logp, stats = vp.vp_processed_logprobs_fwd(x, rules, targets, err_word=err)
    dx = vp.vp_processed_logprobs_bwd(x, rules, targets, stats, grad, err_word=err)
    assert int(err) == 0 and vp.vp_fault_status() == 0
    for r0 in range(0, N, 50):
        rows = slice(r0, r0 + 50)
        z, f, M = ruled_rows(x, q, rows)
        kept = torch.isfinite(z)
        assert torch.equal(y[rows].isneginf(), ~kept) and not y[rows].isnan().any()
        off = (y[rows].double() - z).abs() - 8 * U * M - h * z.abs()
        assert off[kept].max() <= 0
        ref = dy[rows].double() * f
        assert ((dz[rows].double() - ref).abs() - (4 * U + h) * ref.abs()).max() <= 2.0 ** -133
        lse = torch.logsumexp(z, 1)
        t = targets[rows, None]
        lp = z.gather(1, t)[:, 0] - lse
        fine = torch.isfinite(lp)                                             # a masked target's is -inf
        tol = U * (16 * M.amax(1) + 64 + torch.where(fine, lp.abs(), 0.0))
        got = logp[rows].double()
        assert (got[~fine] == -math.inf).all() and ((got - lp).abs() - tol)[fine].max() <= 0
        p = torch.exp(z - lse[:, None])
        e = (-p).scatter_(1, t, -torch.expm1(lp)[:, None])
        scale = f * grad[rows].double()[:, None]
        ref = torch.where(f == 0, 0.0, scale * e)
        off = (dx[rows].double() - ref).abs() - scale.abs() * (p * (tol[:, None] + 8 * U) + 2.0 ** -126)
        assert (off - (6 * U + h) * ref.abs()).max() <= 2.0 ** -133


@pytest.mark.gpu
@pytest.mark.parametrize("n", [32766, 32767, 32768, 70001])
def test_one_id_many_times(n):
    """Occurrences around the widths they are counted in."""
    x = torch.zeros(2, 5000, device="cuda")
    ids = torch.full((n,), 4321, dtype=torch.int64, device="cuda")
    spans = torch.tensor([[0, 0, n], [0, n, n]], device="cuda")               # all output; all prompt
    rules = vp.logits_rules(ids=ids, spans=spans, frequency=torch.full((2,), 2.0 ** -4, device="cuda"),
                            presence=torch.full((2,), 8.0, device="cuda"))
    y = vp.vp_logits_process_fwd(x, rules)
    assert float(y[0, 4321]) == -n / 16 - 8 and int((y != 0).sum()) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_a_batch(dtype):
    """[B, T, V] views with two strides, odd V, outputs with strides of their own."""
    B, T, V = 3, 4, 2051
    full = torch.randn(B, T + 1, V + 2, device="cuda").to(dtype)
    x = full[:, :-1, 1:V + 1]
    flat = x.reshape(B * T, V)
    cpu, q, targets, grad = make(B * T, V, dtype, 31, L=40, nb=4, masks=3)
    rules = to_gpu(q)
    ref = vp.vp_logits_process_fwd(flat, rules)
    assert torch.equal(vp.vp_logits_process_fwd(x, rules).view(B * T, V), ref)
    out = torch.full((T, B, V + 7), 9.0, device="cuda").to(dtype)             # rows of another order
    y = out.transpose(0, 1)[:, :, 3:V + 3]
    vp.vp_logits_process_fwd(x, rules, y=y)
    assert torch.equal(y.reshape(B * T, V), ref) and (out[:, :, :3] == 9).all() and (out[:, :, V + 3:] == 9).all()
    tg, gg = targets.cuda(), grad.cuda()
    logp, st = vp.vp_processed_logprobs_fwd(x, rules, tg)
    one, st1 = vp.vp_processed_logprobs_fwd(flat, rules, tg)
    assert torch.equal(logp.view(torch.int32), one.view(torch.int32))
    assert torch.equal(vp.vp_processed_logprobs_bwd(x, rules, tg, st, gg).view(torch.int16),
                       vp.vp_processed_logprobs_bwd(flat, rules, tg, st1, gg).view(torch.int16))
    dy = torch.randn(B * T, V, device="cuda").to(dtype)
    assert torch.equal(vp.vp_logits_process_bwd(x, rules, dy), vp.vp_logits_process_bwd(flat, rules, dy))
    buf = dy.clone()
    assert torch.equal(vp.vp_logits_process_bwd(x, rules, buf, dx=buf), vp.vp_logits_process_bwd(flat, rules, dy))
    held = flat.clone()
    assert torch.equal(vp.vp_processed_logprobs_bwd(held, rules, tg, st1, gg, dx=held).view(torch.int16),
                       vp.vp_processed_logprobs_bwd(flat, rules, tg, st1, gg).view(torch.int16))


@pytest.mark.gpu
@pytest.mark.slow
def test_offsets_past_32_bits():
    """Rows that begin past 2^31 elements, and a history list whose last ids do."""
    V, N = 8192, 270000                                                        # 2.2e9 elements
    x = torch.zeros(N, V, dtype=torch.bfloat16, device="cuda")
    row = torch.linspace(-2, 2, V).to(torch.bfloat16)
    x[-1] = row.cuda()
    n_ids = 2 ** 31 + 100
    ids = torch.full((n_ids,), -1, dtype=torch.int64, device="cuda")
    ids[-3:] = torch.tensor([5, 5, 8191], device="cuda")
    spans = torch.zeros(N, 3, dtype=torch.int64, device="cuda")
    spans[-1] = torch.tensor([n_ids - 3, 0, 3], device="cuda")
    rules = vp.logits_rules(ids=ids, spans=spans, frequency=torch.full((N,), 2.0, device="cuda"))
    y = vp.vp_logits_process_fwd(x, rules, y=x)
    row = row.float()
    row[5] -= 4
    row[8191] -= 2
    assert torch.equal(y[-1].cpu().float(), row.to(torch.bfloat16).float()) and not y[-2].any()


# ---------------------------------------------------------------------------
# refusals (CPU)
# ---------------------------------------------------------------------------
FAKE, FAKE_ODD = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100001)      # never dereferenced


def rules_struct(**kw):
    s = _lib.LogitsRulesStruct()
    for k, v in kw.items():
        setattr(s, k, v)
    return ctypes.byref(s)


def test_entry_points_check_arguments_on_the_host():
    L = _lib.lib()
    row, none = (FAKE, 1, 4, 16, 4, 0, 16, 0), rules_struct()
    P = 0x100000

    def fwd(rules=none, y=FAKE, y_s_i=16, row=row, err=None):
        return L.vp_logits_process_fwd(*row, rules, y, 0, y_s_i, err, None)

    assert fwd(row=(FAKE, 7, 4, 16, 4, 0, 16, 0)) == ERR_DTYPE
    assert fwd(row=(FAKE, 1, 4, 0, 4, 0, 16, 0)) == ERR_SHAPE
    assert fwd(row=(FAKE, 1, 4, 16, 4, 0, -1, 0)) == ERR_LAYOUT
    assert fwd(y_s_i=-16) == ERR_LAYOUT
    assert fwd(rules=None) == ERR_NULL and fwd(y=None) == ERR_NULL
    assert fwd(row=(FAKE, 1, 4, 16, 4, 0, 16, -1)) == ERR_ARG                        # vocab_start
    assert fwd(y=FAKE_ODD) == ERR_ALIGN and fwd(err=FAKE_ODD) == ERR_ALIGN
    assert fwd(row=(None, 1, 0, 16, 4, 0, 16, 0), rules=None, y=None) == OK          # N = 0
    assert fwd(rules_struct(spans=P, n_ids=3)) == ERR_NULL                           # spans without ids
    assert fwd(rules_struct(spans=P, ids=P, n_ids=-1)) == ERR_SHAPE
    assert fwd(rules_struct(spans=P + 4, ids=P, n_ids=3)) == ERR_ALIGN
    assert fwd(rules_struct(temperature=P + 2)) == ERR_ALIGN
    assert fwd(rules_struct(bias_spans=P, n_bias=2, bias_ids=P)) == ERR_NULL
    assert fwd(rules_struct(mask=P, n_masks=0)) == ERR_SHAPE
    assert fwd(rules_struct(mask=P, n_masks=3, mask_stride=1)) == ERR_SHAPE          # fewer than N without mask_rows
    assert fwd(rules_struct(mask=P, n_masks=4, mask_stride=0)) == ERR_SHAPE
    assert fwd(rules_struct(mask=P, n_masks=4, mask_stride=-1)) == ERR_LAYOUT
    assert fwd(rules_struct(mask=P + 1, n_masks=4, mask_stride=1)) == ERR_ALIGN
    assert L.vp_logits_process_bwd(*row, none, None, FAKE, None, None) == ERR_NULL
    assert L.vp_logits_process_bwd(*row, none, FAKE, FAKE_ODD, None, None) == ERR_ALIGN
    ws = ctypes.c_size_t(1 << 20)
    assert L.vp_processed_logprobs_fwd(*row, none, None, FAKE, FAKE, FAKE, ws, None, None) == ERR_NULL
    assert L.vp_processed_logprobs_fwd(*row, none, FAKE, FAKE, FAKE_ODD, FAKE, ws, None, None) == ERR_ALIGN
    assert L.vp_processed_logprobs_fwd(*row, none, FAKE, FAKE, FAKE, FAKE, ctypes.c_size_t(8), None, None) == ERR_ARG
    assert L.vp_processed_logprobs_bwd(*row, none, FAKE, FAKE, None, FAKE, None, None) == ERR_NULL
    assert L.vp_processed_logprobs_bwd(*row, None, FAKE, FAKE, FAKE, FAKE, None, None) == ERR_NULL
    assert vp.vp_processed_logprobs_workspace_size(3, 4096) == 3 * 40
    assert vp.vp_processed_logprobs_workspace_size(3, 4097) == 2 * 3 * 40
    assert vp.vp_processed_logprobs_workspace_size(3, 0) == 0


def status(fn):
    with pytest.raises(vp.VPError) as e:
        fn()
    return e.value.status


def test_rules_are_checked_when_they_are_made():
    i64, f32 = torch.int64, torch.float32
    ids, spans, pen = torch.zeros(5, dtype=i64), torch.zeros(4, 3, dtype=i64), torch.ones(4)
    mask = torch.zeros(4, 2, dtype=torch.int32)
    R = vp.logits_rules
    assert R(ids=ids, spans=spans, repetition=pen, mask=mask).rows == 4
    assert status(lambda: R(ids=ids.int(), spans=spans)) == ERR_DTYPE
    assert status(lambda: R(ids=ids, spans=spans.to(f32))) == ERR_DTYPE
    assert status(lambda: R(ids=ids, spans=spans[:, :2].contiguous())) == ERR_SHAPE
    assert status(lambda: R(ids=ids, spans=spans, presence=torch.ones(5))) == ERR_SHAPE
    assert status(lambda: R(ids=ids, spans=spans, frequency=torch.ones(8)[::2])) == ERR_LAYOUT
    assert status(lambda: R(ids=ids)) == ERR_NULL
    assert status(lambda: R(spans=spans)) == ERR_NULL
    assert status(lambda: R(repetition=pen)) == ERR_NULL
    assert status(lambda: R(bias_spans=torch.zeros(4, 2, dtype=i64), bias_ids=ids)) == ERR_NULL
    assert status(lambda: R(bias_spans=torch.zeros(4, 2, dtype=i64), bias_ids=ids, bias_values=torch.ones(4))) == ERR_SHAPE
    assert status(lambda: R(mask=mask.long())) == ERR_DTYPE
    assert status(lambda: R(mask=mask.t())) == ERR_LAYOUT
    assert status(lambda: R(mask_rows=torch.zeros(4, dtype=i64))) == ERR_NULL


def test_rules_reach_the_fields_of_the_struct():
    f, i = torch.float32, torch.int64
    t = {k: torch.zeros(n, dtype=d) for k, n, d in (
        ("ids", 5, i), ("spans", (2, 3), i), ("repetition", 2, f), ("frequency", 2, f), ("presence", 2, f), ("bias_ids", 4, i),
        ("bias_values", 4, f), ("bias_spans", (2, 2), i), ("mask", (3, 7), torch.int32), ("mask_rows", 2, i),
        ("temperature", 2, f))}
    q = vp.logits_rules(**t).struct
    assert all(getattr(q, k) == v.data_ptr() for k, v in t.items())
    assert (q.n_ids, q.n_bias, q.n_masks, q.mask_stride) == (5, 4, 3, 7)
    q = vp.logits_rules().struct
    assert not any(getattr(q, k) for k, _ in q._fields_)


def test_calls_check_the_rules_and_tensors():
    x = torch.zeros(4, 64)
    t, g, st = torch.zeros(4, dtype=torch.int64), torch.zeros(4), vp.rowstats(4, "cpu")
    ok = vp.logits_rules(temperature=torch.ones(4))
    assert status(lambda: vp.vp_logits_process_fwd(x[:3], ok)) == ERR_SHAPE                    # rules of 4 rows
    assert status(lambda: vp.vp_logits_process_fwd(x, vp.logits_rules(mask=torch.zeros(4, 1, dtype=torch.int32)))) == ERR_SHAPE
    assert status(lambda: vp.vp_logits_process_fwd(x, vp.logits_rules(mask=torch.zeros(3, 2, dtype=torch.int32)))) == ERR_SHAPE
    assert status(lambda: vp.vp_logits_process_fwd(x, ok, y=torch.zeros(4, 65))) == ERR_SHAPE
    assert status(lambda: vp.vp_logits_process_fwd(x, ok, y=x.to(torch.bfloat16))) == ERR_DTYPE
    assert status(lambda: vp.vp_logits_process_fwd(x, ok, y=torch.zeros(1, 64).expand(4, 64))) == ERR_LAYOUT
    assert status(lambda: vp.vp_logits_process_fwd(x.t(), ok)) in (ERR_LAYOUT, ERR_SHAPE)
    assert status(lambda: vp.vp_logits_process_bwd(x, ok, torch.zeros(4, 63))) == ERR_SHAPE
    assert status(lambda: vp.vp_logits_process_bwd(x, ok, x.to(torch.bfloat16))) == ERR_DTYPE
    assert status(lambda: vp.vp_processed_logprobs_fwd(x, ok, t.int())) == ERR_DTYPE
    assert status(lambda: vp.vp_processed_logprobs_bwd(x, ok, t, st, g, dx=torch.zeros(4, 63))) == ERR_SHAPE
    assert status(lambda: vp.vp_processed_logprobs_bwd(x, ok, t, st, g.double())) == ERR_DTYPE
    # what fits, but is not on a GPU, is refused before the library is called
    for call in (lambda: vp.vp_logits_process_fwd(x, ok), lambda: vp.vp_logits_process_bwd(x, ok, x),
                 lambda: vp.vp_processed_logprobs_fwd(x, ok, t),
                 lambda: vp.vp_processed_logprobs_bwd(x, ok, t, st, g)):
        assert status(call) == ERR_DEVICE


def test_plain_gradient_against_differences():
    """The reference's own factor and gradient, against central differences of its forward."""
    x, q, targets, _ = make(2, 40, torch.float32, 1, L=20, nb=4)
    q["bias_values"] = q["bias_values"].clamp(min=-5)
    step = 2.0 ** -16
    for r in range(2):
        row = x[r].double()
        z, f, _ = plain_row(row, r, q, 0)
        _, _, g = plain_logprob(z, int(targets[r]))
        for j in range(40):
            ends = []
            for s in (step, -step):
                moved = row.clone()
                moved[j] += s
                ends.append(plain_logprob(plain_row(moved, r, q, 0)[0], int(targets[r]))[0])
            assert abs(float(ends[0] - ends[1]) / (2 * step) - float(g[j] * f[j])) < 1e-7
