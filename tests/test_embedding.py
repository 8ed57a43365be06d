"""The vocabulary's table as an embedding: the lookup (bit for bit) and the gradient by sorted tokens.

Tolerance of the gradient, u = 2^-24: a sum of n values in fp32 in any order is off by (n - 1) u of the sum of
magnitudes, the scale and its product by 2 u, what is added to by another, and the output's rounding by half a step h:
(n + 3) u (s sum |dy| + |before|) + h |result|.
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
TYPES = [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)]


def make_ids(N, V, seed, kind="zipf"):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        return torch.full((N,), V // 2)
    if kind == "sorted":
        return torch.arange(N) * V // max(N, 1)
    ids = (torch.rand(N, generator=g, dtype=torch.float64) ** (4 if kind == "zipf" else 1) * V).long().clamp(max=V - 1)
    ids[torch.rand(N, generator=g) < 0.05] = -1
    return ids


def plain_lookup(w, ids, scale, dtype, start=0):
    local = ids - start
    here = (ids >= 0) & (local >= 0) & (local < w.shape[0])
    y = w[torch.where(here, local, 0).reshape(-1)].reshape(*ids.shape, w.shape[1]).float() * torch.tensor(scale, dtype=F32)
    return torch.where(here[..., None], y, 0.0).to(dtype)


def check_grad(dy, ids, V, scale=1.0, start=0, sharded=False, dtype=None, before=None, dyg=None, **kwargs):
    """dy and ids on the CPU ([N, D] and [N]); dyg: the tensor that the call gets."""
    dyg = dy.cuda() if dyg is None else dyg
    dtype = dtype or dy.dtype
    dW = None if before is None else before.to(dtype).cuda()
    got = vp.vp_embedding_bwd(dyg, ids.cuda(), V, scale=scale, vocab_start=start, sharded=sharded, dtype=dtype, dW=dW,
                              accumulate=before is not None, **kwargs)
    local = ids - start
    here = (ids >= 0) & (local >= 0) & (local < V)
    d64 = dy.double()[here] * float(torch.tensor(scale, dtype=F32))
    add = lambda v: torch.zeros(V, dy.shape[1], dtype=torch.float64).index_add_(0, local[here], v)
    ref, size = add(d64), add(d64.abs())
    n = torch.zeros(V, dtype=torch.float64).index_add_(0, local[here], torch.ones_like(local[here]).double())[:, None]
    if before is not None:
        old = before.to(dtype).double()
        assert torch.equal(got.cpu()[n[:, 0] == 0], before.to(dtype)[n[:, 0] == 0])      # left as they were
        ref, size = ref + old, size + old.abs()
    tol = (n + 3) * U * size + torch.finfo(dtype).eps / 2 * ref.abs()
    assert got.dtype == dtype and got.shape == ref.shape
    over = (got.double().cpu() - ref).abs() - tol
    assert over.max() <= 0, f"{float(over.max()):.2e} over its tolerance"
    return got


def rand(N, D, dtype, seed=0):
    return torch.randn(N, D, generator=torch.Generator().manual_seed(seed + N + D)).to(dtype)


# --------------------------------------------------------------------------- lookup
@pytest.mark.gpu
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("D", [1, 5, 8, 64, 517, 520, 1032, 4096])
def test_lookup(D, types):
    V = 1000
    w, ids = rand(V, D, types[0]), make_ids(300, V, D)
    for scale in (1.0, math.sqrt(D) + 0.3):
        got = vp.vp_embedding_fwd(w.cuda(), ids.cuda(), scale=scale, dtype=types[1])
        assert got.dtype == types[1] and torch.equal(got.cpu(), plain_lookup(w, ids, scale, types[1]))
    # a table out of a wider one, a batch of sequences, a caller's buffer off a 16-byte boundary
    for gap in (3, 8):
        wide = torch.full((V, D + gap), math.nan, dtype=types[0], device="cuda")
        wide[:, gap:] = w.cuda()
        got = vp.vp_embedding_fwd(wide[:, gap:], ids.view(20, 15).cuda(), scale=2.5, dtype=types[1])
        assert got.shape == (20, 15, D)
        assert torch.equal(got.view(-1, D).cpu(), plain_lookup(w, ids, 2.5, types[1]))
    room = torch.full((1 + 300 * D + 1,), 7.0, dtype=types[1], device="cuda")
    vp.vp_embedding_fwd(w.cuda(), ids.cuda(), dtype=types[1], out=room[1:-1])
    assert torch.equal(room[1:-1].view(300, D).cpu(), plain_lookup(w, ids, 1.0, types[1])) and room[0] == 7 == room[-1]


@pytest.mark.gpu
def test_lookup_of_one_token_and_of_none():
    w = rand(151936, 64, BF16).cuda()
    for t in (0, 151935):
        assert torch.equal(vp.vp_embedding_fwd(w, torch.tensor([t], device="cuda")), w[t:t + 1])
    assert vp.vp_embedding_fwd(w, torch.empty(0, 3, dtype=torch.int64, device="cuda")).shape == (0, 3, 64)


@pytest.mark.gpu
def test_lookup_of_shards_and_of_wrong_ids():
    w = rand(1000, 72, F32)
    ids = torch.tensor([0, 499, 500, 999, -1, -5, 250])
    halves = [vp.vp_embedding_fwd(w[a:a + 500].cuda(), ids.cuda(), scale=3.0, vocab_start=a, sharded=True) for a in (0, 500)]
    assert torch.equal((halves[0] + halves[1]).cpu(), plain_lookup(w, ids, 3.0, F32))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = vp.vp_embedding_fwd(w[:500].cuda(), ids.cuda(), err_word=err)
    assert int(err) == vp.ERRBIT_TARGET
    assert torch.isnan(got).all(1).tolist() == [False, False, True, True, False, False, False]
    assert torch.equal(got[[0, 1, 4, 5, 6]].cpu(), plain_lookup(w[:500], ids, 1.0, F32)[[0, 1, 4, 5, 6]])
    err.zero_()
    vp.vp_embedding_fwd(w.cuda(), ids.cuda(), err_word=err)
    assert int(err) == 0


@pytest.mark.gpu
def test_lookup_past_32_bits():
    """Rows that lie more than 2^31 elements into the table."""
    w = torch.zeros(300000, 8192, dtype=BF16, device="cuda")
    ids = torch.tensor([299999, 1, 262144, 270000], device="cuda")
    w[ids] = torch.randn(4, 8192, device="cuda").to(BF16)
    assert torch.equal(vp.vp_embedding_fwd(w, ids), w[ids])
    dy = torch.randn(4, 8192, device="cuda").to(BF16)
    got = vp.vp_embedding_bwd(dy, ids, 300000, dW=w)
    assert torch.equal(got[ids], dy) and int((got != 0).any(1).sum()) == 4


# --------------------------------------------------------------------------- gradient
@pytest.mark.gpu
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("D", [1, 5, 8, 64, 517, 520, 2056, 4096])
def test_gradient_widths(D, types):
    for N, kind in ((1, "flat"), (37, "zipf"), (128, "one"), (700, "zipf")):
        ids = make_ids(N, 600, D + N, kind)
        check_grad(rand(N, D, types[0]), ids, 600, scale=1.7, dtype=types[1])
        check_grad(rand(N, D, types[0]), ids, 600, scale=1.7, dtype=types[1], before=rand(600, D, F32, 5))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["zipf", "flat", "one", "sorted"])
@pytest.mark.parametrize("N, V", [(2, 1), (8, 9), (128, 5003), (129, 77), (100, 90), (9, 8), (250, 33), (500, 5003), (2049, 5003), (5000, 160000),
                                  (20000, 300), (70000, 40)])
def test_gradient_runs(N, V, kind):
    """Runs of one id within a window of tokens, at its ends, and over many windows; tables of more rows than the SMs have
    counters for, and of fewer than there are SMs."""
    ids = make_ids(N, V, N, kind)
    got = check_grad(rand(N, 24, BF16), ids, V, dtype=F32)
    again = vp.vp_embedding_bwd(rand(N, 24, BF16).cuda(), ids.cuda(), V, dtype=F32)
    assert torch.equal(got, again)                                   # the same sums every time
    check_grad(rand(N, 24, BF16), ids, V, before=rand(V, 24, BF16, 1))


@pytest.mark.gpu
@pytest.mark.parametrize("N, D", [(600, 517), (600, 1032), (2600, 130), (2600, 2056), (30000, 13), (32767, 16), (32768, 16), (100001, 11)])
def test_gradient_of_long_runs(N, D):
    """Runs over windows by the dozen, in narrow, wide and odd tables, beside short ones; warps of the sort that have more
    tokens of one CTA than they note, batches just below and above those that are dealt out first."""
    V = 700
    ids = make_ids(N, V, D)
    ids[torch.rand(N, generator=torch.Generator().manual_seed(N)) < 0.4] = 7
    ids[N // 3:N // 3 + N // 4] = 8
    dy = rand(N, D, BF16)
    check_grad(dy, ids, V, scale=0.7, dtype=F32)
    check_grad(dy, ids, V, before=rand(V, D, BF16, 3))
    whole = vp.vp_embedding_bwd(dy.cuda(), ids.cuda(), V)
    assert torch.equal(whole, vp.vp_embedding_bwd(dy.cuda(), ids.cuda(), V))


@pytest.mark.gpu
@pytest.mark.parametrize("V", [1, 5, 300, 131077, 1100000])
def test_gradient_of_large_batches(V):
    """Tables of fewer rows than the sort has CTAs, and of more than it can deal to: sums and order as of any other."""
    N = 50000
    ids, dy = make_ids(N, V, V, "flat"), rand(N, 8, BF16)
    ids[::7] = V // 2
    got = check_grad(dy, ids, V, dtype=F32)
    assert torch.equal(got, vp.vp_embedding_bwd(dy.cuda(), ids.cuda(), V, dtype=F32))


@pytest.mark.gpu
@pytest.mark.parametrize("N", [300, 40000])
def test_sorted_ids_of_every_size(N):
    """Ids at the ends of 64 and of 32 bits, and shards that begin anywhere, in a batch that is sorted."""
    V, D = 77, 16
    dy = rand(N, D, F32)
    for start in (0, 5, 2 ** 32 - 30, 2 ** 62, 2 ** 63 - 1 - V):
        ids = torch.full((N,), -1)
        near = torch.arange(start - 40, min(start + V + 40, 2 ** 63 - 1))
        ids[:len(near)] = near
        ends = [-2 ** 63, -2 ** 63 + 1, -2, 0, 1, 2 ** 31, 2 ** 32, 2 ** 32 + 3, 2 ** 62, 2 ** 63 - 1]
        ids[len(near):len(near) + len(ends)] = torch.tensor(ends)
        ids = ids[torch.randperm(N, generator=torch.Generator().manual_seed(N))]
        check_grad(dy, ids, V, start=start, sharded=True)


@pytest.mark.gpu
def test_gradient_of_batches_and_views():
    V, D = 400, 136
    ids = make_ids(60, V, 3)
    dy = rand(60, D, BF16)
    full = torch.full((4, 16, D), math.nan, dtype=BF16, device="cuda")
    full[:, :-1] = dy.view(4, 15, D).cuda()
    check_grad(dy, ids, V, dyg=full[:, :-1])
    for gap in (1, 8):
        wide = torch.full((60, D + gap), math.nan, dtype=BF16, device="cuda")
        wide[:, gap:] = dy.cuda()
        check_grad(dy, ids, V, dyg=wide[:, gap:])
    # one gradient for every token, expanded
    one = rand(1, D, BF16)
    check_grad(one.expand(60, D), ids, V, dyg=one.cuda().expand(60, D), dtype=F32)
    # an output off a 16-byte boundary, and what lies around it
    room = torch.full((V * D + 2,), 7.0, dtype=BF16, device="cuda")
    vp.vp_embedding_bwd(dy.cuda(), ids.cuda(), V, dW=room[1:-1])
    assert torch.equal(room[1:-1].view(V, D), vp.vp_embedding_bwd(dy.cuda(), ids.cuda(), V))
    assert room[0] == 7 and room[-1] == 7


@pytest.mark.gpu
def test_gradient_of_shards_and_of_wrong_ids():
    V, D = 1000, 40
    ids = make_ids(500, V, 9)
    dy = rand(500, D, F32)
    for a in (0, 500):
        check_grad(dy, ids, 500, start=a, sharded=True, scale=0.5)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    check_grad(dy, ids, V, err_word=err)
    assert int(err) == 0
    check_grad(dy, ids, 500, start=500, sharded=True, err_word=err)
    assert int(err) == 0
    check_grad(dy, ids, 500, start=500, err_word=err)                # their tokens count nowhere
    assert int(err) == vp.ERRBIT_TARGET
    huge = torch.tensor([2 ** 62, -2 ** 62, 5, 2 ** 40, -1])
    check_grad(dy[:5], huge, V, err_word=err)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [5, 900])
def test_gradient_without_tokens(N):
    dy = rand(N, 64, BF16)
    for ids in (torch.full((N,), -1), torch.full((N,), 2000)):
        check_grad(dy, ids, 1000, sharded=True)
        check_grad(dy, ids, 1000, sharded=True, before=rand(1000, 64, BF16, 2))
    none = torch.empty(0, dtype=torch.int64)
    check_grad(dy[:0], none, 1000)
    check_grad(dy[:0], none, 1000, before=rand(1000, 64, BF16, 2))


@pytest.mark.gpu
@pytest.mark.parametrize("N", [3, 3000])
def test_nan_stays_with_its_token(N):
    dy, ids = rand(N, 64, BF16), make_ids(N, 5000, N, "sorted")
    dy[1, 7], dy[2, 9] = math.nan, math.inf
    got = vp.vp_embedding_bwd(dy.cuda(), ids.cuda(), 5000, dtype=F32).cpu()
    assert torch.isnan(got).nonzero().tolist() == [[int(ids[1]), 7]] and torch.isinf(got).nonzero().tolist() == [[int(ids[2]), 9]]


@pytest.mark.gpu
@pytest.mark.parametrize("D", [40, 37])
@pytest.mark.parametrize("N, V, share", [(3000, 100, 0.0), (3000, 50, 0.6), (100, 50, 0.5)])
def test_infinities_of_runs_over_windows(N, V, share, D):
    """Infinite sums as plain additions have them, whether an id's tokens lie in a few windows (30 of them), in many (1800) or
    in a single launch (50): inf from one infinity or from finite values that overflow, NaN from two of opposite signs."""
    hot = 20
    ids = torch.arange(N) % V
    ids[torch.rand(N, generator=torch.Generator().manual_seed(N)) < share] = hot
    dy = rand(N, D, F32)
    mine = (ids == hot).nonzero()[:, 0]
    first, middle, last = int(mine[0]), int(mine[len(mine) // 2]), int(mine[-1])
    dy[first, 0], dy[middle, 1], dy[last, 2] = math.inf, -math.inf, math.inf
    dy[first, 3], dy[last, 3] = math.inf, -math.inf
    dy[middle, 4] = math.nan
    dy[mine, 5], dy[mine, 6] = 3e38, -3e38                           # two of them overflow
    dy[first, 7], dy[last, 7] = math.inf, math.inf
    dy[mine, 8] = 3e37                                               # twelve do, more than a window of eight has
    for before in (None, rand(V, D, F32, 1)):
        dW = None if before is None else before.cuda()
        got = vp.vp_embedding_bwd(dy.cuda(), ids.cuda(), V, dW=dW, accumulate=before is not None).cpu()
        inf = math.inf
        assert got[hot, [0, 1, 2, 5, 6, 7, 8]].tolist() == [inf, -inf, inf, inf, -inf, inf, inf]
        assert torch.isnan(got[hot, 3:5]).all() and torch.isfinite(got[hot, 9:]).all()
        assert torch.isfinite(got[torch.arange(V) != hot]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("N", [40, 3000])
def test_streams_graphs_and_workspaces(N):
    V, D = 3000, 256
    ids, dy = make_ids(N, V, 4).cuda(), rand(N, D, BF16).cuda()
    w = rand(V, D, BF16).cuda()
    work = torch.empty(vp.vp_embedding_bwd_workspace_size(N, V, D), dtype=torch.uint8, device="cuda")

    def step():
        return (vp.vp_embedding_fwd(w, ids, scale=2.0), vp.vp_embedding_bwd(dy, ids, V, workspace=work),
                vp.vp_embedding_bwd(dy, ids, V, dW=w.clone(), accumulate=True, workspace=work))

    ref = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    graphs = []
    for _ in range(2):                                               # two graphs with one workspace, one after the other
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out))
    ids.copy_(make_ids(N, V, 5).cuda())
    dy.mul_(-2)
    for graph, _ in graphs * 2:
        graph.replay()
    ref = step()
    assert all(torch.equal(a, b) for _, out in graphs for a, b in zip(out, ref))


# --------------------------------------------------------------------------- together
def tied_step(w, ids, targets, scale, grad, **rules):
    """Gradient of the table of a model that is nothing but its table: looked up, and as the head."""
    h = vp.vp_embedding_fwd(w, ids, scale=scale)
    loss, stats = vp.vp_linear_cross_entropy_fwd(h, w, targets, **rules)
    dh, dw = vp.vp_linear_cross_entropy_bwd(h, w, targets, stats, grad, **rules)
    vp.vp_embedding_bwd(dh, ids, w.shape[0], scale=scale, dW=dw, accumulate=True)
    return loss, dw


@pytest.mark.gpu
def test_a_tied_model_learns_from_both_ends():
    V, D, N, scale = 700, 128, 150, 8.0
    w = (rand(V, D, F32) * 0.02).to(BF16)
    ids, targets = make_ids(N, V, 1), make_ids(N, V, 2, "flat")
    grad = torch.full((N,), 1.0 / N)
    rules = dict(label_smoothing=0.1, z_loss=1e-3, softcap=5.0)
    loss, dw = tied_step(w.cuda(), ids.cuda(), targets.cuda(), scale, grad.cuda(), **rules)

    w64 = w.double().requires_grad_()
    h = w64[ids.clamp(min=0)] * scale * (ids >= 0)[:, None]
    z = 5.0 * torch.tanh(h @ w64.t() / 5.0)
    lse = torch.logsumexp(z, 1)
    ref = lse - 0.9 * z.gather(1, targets.clamp(min=0)[:, None])[:, 0] - 0.1 * z.mean(1) + 1e-3 * lse ** 2
    ref = torch.where(targets >= 0, ref, 0.0)
    (ref * grad).sum().backward()
    assert torch.allclose(loss.double().cpu(), ref.detach(), rtol=2e-5, atol=2e-5)
    # three roundings to bf16 (dhidden, the head's part, the sum), each half a step of magnitudes that may cancel
    lim = 3 * 2.0 ** -8 * (w64.grad.abs() + w64.grad.abs().amax(1, keepdim=True) / 4)
    over = (dw.double().cpu() - w64.grad).abs() - lim - 2e-7
    assert over.max() <= 0, float(over.max())
    # the same step captured, and replayed on new tokens
    wg, ig, tg, gg = w.cuda(), ids.cuda(), targets.cuda(), grad.cuda()
    tied_step(wg, ig, tg, scale, gg, **rules)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tied_step(wg, ig, tg, scale, gg, **rules)
    ig.copy_(make_ids(N, V, 3))
    tg.copy_(make_ids(N, V, 4))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, tied_step(wg, ig, tg, scale, gg, **rules)))


@pytest.mark.gpu
def test_the_example_learns():
    """The example's rollout, learnt from: its loss and its table's gradient against the definition in 64 bits."""
    from examples import decode_and_score
    out = decode_and_score.run(B=3, prompt=9, steps=8, V=1003, D=128)
    w64 = out["table"].double().cpu().requires_grad_()
    seen, targets = out["seen"].cpu(), out["targets"].cpu()
    z = 30 * torch.tanh((w64[seen] * 128 ** -0.5) @ w64.t() / 30)
    lse = torch.logsumexp(z, 1)
    loss = (lse - 0.9 * z.gather(1, targets[:, None])[:, 0] - 0.1 * z.mean(1) + 1e-4 * lse ** 2).mean()
    loss.backward()
    loss = float(loss.detach())
    assert abs(float(out["loss"]) - loss) < 2e-5 * loss and out["fault"] == 0
    # three roundings to bf16 (dhidden, the head's part, the sum), each half a step of magnitudes that may cancel
    lim = 3 * 2.0 ** -8 * (w64.grad.abs() + w64.grad.abs().amax(1, keepdim=True) / 4)
    assert ((out["dtable"].double().cpu() - w64.grad).abs() - lim - 2e-7).max() <= 0


# --------------------------------------------------------------------------- refusals (no GPU needed)
FAKE, ODD = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100001)
BIG = ctypes.c_size_t(1 << 40)


def test_refusals_of_the_library():
    lib = _lib.lib()

    def fwd(table=FAKE, dtype=1, V=16, D=64, stride=64, ids=FAKE, N=4, out=FAKE, out_dtype=1):
        return lib.vp_embedding_fwd(table, dtype, V, D, stride, ids, N, 0, 0, 1.0, out, out_dtype, None, None)

    assert fwd(dtype=2) == ERR_DTYPE and fwd(out_dtype=-1) == ERR_DTYPE
    assert fwd(V=0) == ERR_SHAPE and fwd(D=0) == ERR_SHAPE and fwd(N=-1) == ERR_SHAPE and fwd(V=2 ** 31) == ERR_SHAPE
    assert fwd(stride=-1) == ERR_LAYOUT
    for name in ("table", "ids", "out"):
        assert fwd(**{name: None}) == ERR_NULL and fwd(**{name: ODD}) == ERR_ALIGN
    assert fwd(N=0, table=None, ids=None, out=None) == OK

    # more tokens than take no workspace: with one missing or short, nothing may be launched
    def bwd(dy=FAKE, dtype=1, N=400, D=64, R=400, s_i=64, ids=FAKE, V=16, dW=FAKE, out_dtype=1, add=0, work=FAKE, size=BIG):
        return lib.vp_embedding_bwd(dy, dtype, N, D, R, 0, s_i, ids, V, 0, 0, 1.0, dW, out_dtype, add, work, size, None, None)

    assert bwd(dtype=2) == ERR_DTYPE and bwd(out_dtype=5) == ERR_DTYPE
    assert bwd(V=0) == ERR_SHAPE and bwd(D=0) == ERR_SHAPE and bwd(R=0) == ERR_SHAPE and bwd(s_i=-1) == ERR_LAYOUT
    for name in ("dy", "ids", "dW", "work"):
        assert bwd(**{name: None}) == ERR_NULL and bwd(**{name: ODD}) == ERR_ALIGN
    assert bwd(size=ctypes.c_size_t(8)) == ERR_ARG
    assert bwd(N=0, add=1, dy=None, dW=None, ids=None, work=None) == OK and bwd(N=0, dW=None) == ERR_NULL
    assert lib.vp_embedding_bwd_workspace_size(4, 0, 64) == 0 and lib.vp_embedding_bwd_workspace_size(400, 16, 64) > 0


def test_refusals_of_the_binding():
    def status(fn):
        with pytest.raises(vp.VPError) as e:
            fn()
        return e.value.status

    w, ids, dy = torch.zeros(20, 8), torch.zeros(6, dtype=torch.int64), torch.zeros(6, 8)
    assert status(lambda: vp.vp_embedding_fwd(w, ids.int())) == 3
    assert status(lambda: vp.vp_embedding_fwd(w, torch.zeros(12, dtype=torch.int64)[::2])) == 4
    assert status(lambda: vp.vp_embedding_fwd(w.t(), ids)) == 4
    assert status(lambda: vp.vp_embedding_fwd(w[0], ids)) == 2
    assert status(lambda: vp.vp_embedding_fwd(w.half(), ids, dtype=F32)) == 3
    assert status(lambda: vp.vp_embedding_fwd(w, ids, dtype=torch.float16)) == 3
    assert status(lambda: vp.vp_embedding_fwd(w, ids, out=torch.empty(6, 7))) == 2
    assert status(lambda: vp.vp_embedding_fwd(w, ids, out=torch.empty(6, 8, dtype=BF16))) == 3
    assert status(lambda: vp.vp_embedding_fwd(w, ids.to("meta"))) == 4
    assert status(lambda: vp.vp_embedding_fwd(w, ids)) == 8                                  # not on a GPU
    assert status(lambda: vp.vp_embedding_bwd(dy, ids[:-1], 20)) == 2
    assert status(lambda: vp.vp_embedding_bwd(dy, ids, 20, accumulate=True)) == 1
    assert status(lambda: vp.vp_embedding_bwd(dy, ids, 20, dW=torch.empty(19, 8))) == 2
    assert status(lambda: vp.vp_embedding_bwd(dy, ids, 20, dW=torch.empty(20, 8), dtype=BF16)) == 3
    assert status(lambda: vp.vp_embedding_bwd(dy, ids, 20, err_word=torch.zeros(1))) == 3
    assert status(lambda: vp.vp_embedding_bwd(dy, ids, 20, workspace=torch.zeros(4, 4).t())) == 4


@pytest.mark.parametrize("V", [0, -1, -20, 2 ** 31])
def test_a_table_of_no_rows_is_refused(V):
    dy, ids = torch.zeros(6, 8), torch.zeros(6, dtype=torch.int64)
    with pytest.raises(vp.VPError) as e:
        vp.vp_embedding_bwd(dy, ids, V)
    assert e.value.status == ERR_SHAPE
