"""Cases of the vocabulary table's operators, in their plain form and through the library: the embedding lookup and
its gradient, and the cross entropy of logits or of a hidden state times the table.

Operators ("op" of a case):
  lookup       rows of the table for token ids, scaled
  table_grad   the gradient of the table from the gradients of the rows that were looked up
  loss         softmax cross entropy of logits with label smoothing, z-loss and soft-capped logits: the loss of each row
               and the gradient of the logits
  linear_loss  the same of hidden . W^T without keeping the logits: losses, and the gradients of the hidden states and
               of the table; with "tied", the lookup's gradient is added to the table's
"""
import math

import torch

own = False

DEV = "cuda"
VOCAB = 75968            # this library's benchmark vocabulary shard; 151936 is both halves of it


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one sequence decoded: one row of the whole vocabulary's table
        dict(name="lookup_1", op="lookup", N=1, V=2 * VOCAB, D=4096, dtype="bf16", out="bf16", scaled=1, shard=-1, wide=0),
        # a training batch of the benchmark's rows, an fp32 master table read out as bf16
        dict(name="lookup_8192", op="lookup", N=8192, V=VOCAB, D=4096, dtype="f32", out="bf16", scaled=1, shard=-1, wide=0),
        # the benchmark's rows: a dense bf16 gradient of the table
        dict(name="table_grad_8192", op="table_grad", N=8192, V=VOCAB, D=4096, dtype="bf16", out="bf16", scaled=1,
             shard=-1, wide=0, hot=4),
        # a long batch on a narrow table, with fp32 gradients; its ids are spread over both halves of the vocabulary
        dict(name="table_grad_65536", op="table_grad", N=65536, V=VOCAB, D=1024, dtype="f32", out="f32", scaled=0,
             shard=1, wide=0, hot=2),
        # a few tokens of a small table with an odd width, out of a padded gradient
        dict(name="table_grad_5", op="table_grad", N=5, V=5003, D=517, dtype="bf16", out="f32", scaled=1, shard=-1,
             wide=3, hot=1),
        # the benchmark's rows: pretraining with label smoothing and z-loss
        dict(name="loss_8192", op="loss", N=8192, V=VOCAB, dtype="bf16", smooth=0.1, z=1e-4, cap=0.0, shard=0, wide=0),
        # a short batch of soft-capped logits, fp32, the whole vocabulary
        dict(name="loss_512_cap", op="loss", N=512, V=2 * VOCAB, dtype="f32", smooth=0.0, z=1e-4, cap=30.0, shard=0, wide=0),
        # the last tokens of three sequences out of a padded tensor, an odd vocabulary
        dict(name="loss_3", op="loss", N=3, V=5003, dtype="f32", smooth=0.05, z=0.0, cap=0.0, shard=0, wide=5),
        # a training step of the benchmark's head
        dict(name="linear_loss_8192", op="linear_loss", N=8192, V=VOCAB, D=4096, smooth=0.0, z=1e-4, cap=0.0, shard=0,
             tied=0),
        # a ragged batch, soft-capped and smoothed
        dict(name="linear_loss_1000_cap", op="linear_loss", N=1000, V=VOCAB, D=2048, smooth=0.1, z=1e-4, cap=30.0, shard=0,
             tied=0),
        # a small tied model: one gradient for the table from both of its ends
        dict(name="linear_loss_64_tied", op="linear_loss", N=64, V=5003, D=512, smooth=0.0, z=0.0, cap=0.0, shard=0, tied=1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lookup", "table_grad", "loss", "linear_loss"])
    if op in ("lookup", "table_grad"):
        D = rng.choice([_log_int(rng, 16, 8192), 8 * _log_int(rng, 2, 1024)])
        V = _log_int(rng, 1000, max(1000, min(2 * VOCAB, VOCAB * 4096 // D)))
        N = _log_int(rng, 1, max(1, min(65536, (1 << 26) // D)))
        case = dict(op=op, N=N, V=V, D=D, dtype=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "f32"]),
                    scaled=rng.choice([0, 1]), shard=rng.choice([-1, -1, 0, 1]), wide=rng.choice([0, 0, 3, 8]))
        if op == "table_grad":
            case["hot"] = rng.choice([1, 2, 4, 8])
        return case
    rules = dict(smooth=rng.choice([0.0, 0.1, 0.3]), z=rng.choice([0.0, 1e-4, 1e-2]),
                 cap=rng.choice([0.0, 0.0, 15.0, 30.0, 50.0]), shard=rng.choice([0, 0, 1]))
    V = _log_int(rng, 1000, 2 * VOCAB)
    if op == "loss":
        dtype = rng.choice(["bf16", "f32"])
        N = _log_int(rng, 1, max(1, min(8192, 8192 * VOCAB // V // (2 if dtype == "f32" else 1))))
        return dict(op=op, N=N, V=V, dtype=dtype, wide=rng.choice([0, 0, 3, 8]), **rules)
    D = 64 * _log_int(rng, 2, 64)
    N = _log_int(rng, 1, max(1, min(8192, 8192 * VOCAB * 4096 // (V * D), 8192 * VOCAB // V)))
    return dict(op=op, N=N, V=V, D=D, tied=rng.choice([0, 1]), **rules)


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, shape, sigma=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype).mul_(sigma)


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _ids(g, n, V, hot=4):
    """Token ids, a few far more often than the others: hot 1 is uniform."""
    return (torch.rand(n, generator=g, device=DEV, dtype=torch.float64) ** hot * V).long().clamp_(max=V - 1)


def _some(g, ids, share):
    """A share of the rows without an id (padding)."""
    return torch.where(torch.rand(ids.shape, generator=g, device=DEV) < share, -1, ids)


def prepare(case, seed):
    g = _gen(seed)
    op, N, V = case["op"], case["N"], case["V"]
    if op in ("lookup", "table_grad"):
        D, half = case["D"], case["shard"]                       # half -1: the table holds the whole vocabulary
        ids = _ids(g, N, V if half < 0 else 2 * V, case.get("hot", 4))
        if half >= 0:                                            # the halves alternate, so both are asked for alike
            ids = ids // 2 + ids % 2 * V
        s = dict(op=op, ids=_some(g, ids, 0.02) if N > 1 else ids, V=V, start=max(half, 0) * V, sharded=half >= 0,
                 scale=math.sqrt(D) if case["scaled"] else 1.0, out=_dtype(case["out"]))
        rows = V if op == "lookup" else N
        s["x"] = _randn(g, (rows, D + case["wide"]), 0.02 if op == "lookup" else 1e-3, _dtype(case["dtype"]))[:, :D]
        return s
    start = case["shard"] * V
    s = dict(op=op, start=start, targets=_some(g, _ids(g, N, V) + start, 0.03) if N > 1 else _ids(g, N, V) + start,
             grad=torch.full((N,), 1.0 / N, device=DEV) * (0.5 + torch.rand(N, generator=g, device=DEV)),
             rules=dict(label_smoothing=case["smooth"], z_loss=case["z"], softcap=case["cap"]))
    if op == "loss":
        s["x"] = _randn(g, (N, V + case["wide"]), 3.0, _dtype(case["dtype"]))[:, :V]
        return s
    s["h"] = _randn(g, (N, case["D"]), 1.0, torch.bfloat16)
    # logits with a standard deviation of 2.5 whatever D
    s["w"] = _randn(g, (V, case["D"]), 2.5 / math.sqrt(case["D"]), torch.bfloat16)
    s["tied"] = case["tied"]
    if case["tied"]:
        s["ids"] = _some(g, _ids(g, N, V) + start, 0.02)
        s["dy"] = _randn(g, (N, case["D"]), 1e-2 / N, torch.bfloat16)
        s["scale"] = math.sqrt(case["D"])
    return s


# --------------------------------------------------------------------------- plain forms
def _plain_places(ids, start, V):
    local = ids - start
    here = (ids >= 0) & (local >= 0) & (local < V)
    return torch.where(here, local, 0), here


def _plain_table_grad(dy, ids, start, V, scale):
    local, here = _plain_places(ids, start, V)
    rows = torch.where(here[:, None], dy.float() * scale, 0.0)
    return torch.zeros(V, dy.shape[1], device=DEV).index_add_(0, local, rows)


def _plain_loss(x, s):
    """(losses, gradient of x), both fp32, of fp32 logits x."""
    q, V = s["rules"], x.shape[1]
    cap, smooth, zeta = q["softcap"], q["label_smoothing"], q["z_loss"]
    z = cap * torch.tanh(x / cap) if cap else x
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True, dtype=torch.float64)
    lse = m.double() + torch.log(total)
    t, used = _plain_places(s["targets"], s["start"], V)
    zt = z.gather(1, t[:, None]).double()
    loss = lse - (1 - smooth) * zt + zeta * lse * lse
    if smooth:
        loss = loss - smooth * z.mean(1, keepdim=True, dtype=torch.float64)
    d = e.mul_(((1 + 2 * zeta * lse) / total).float())
    if smooth:
        d -= smooth / V
    d.scatter_add_(1, t[:, None], torch.full_like(m, -(1 - smooth)))
    d *= torch.where(used, s["grad"], 0.0)[:, None]
    if cap:
        d *= 1 - (z / cap) ** 2
    return torch.where(used, loss[:, 0], 0.0).float(), d


def _plain(s):
    op = s["op"]
    if op == "lookup":
        local, here = _plain_places(s["ids"], s["start"], s["V"])
        return torch.where(here[:, None], s["x"][local].float() * s["scale"], 0.0).to(s["out"])
    if op == "table_grad":
        return _plain_table_grad(s["x"], s["ids"], s["start"], s["V"], s["scale"]).to(s["out"])
    if op == "loss":
        loss, dx = _plain_loss(s["x"].float(), s)
        return {"loss": loss, "dx": dx.to(s["x"].dtype)}
    h, w = s["h"].float(), s["w"].float()
    loss, dz = _plain_loss(h @ w.t(), s)
    dh, dw = dz @ w, dz.t() @ h
    if s["tied"]:
        dw = dw + _plain_table_grad(s["dy"], s["ids"], s["start"], w.shape[0], s["scale"])
    return {"loss": loss, "dhidden": dh.to(s["h"].dtype), "dW": dw.to(s["w"].dtype)}


# --------------------------------------------------------------------------- the library's calls
def run(s):
    if not own:
        return _plain(s)
    import vocab_wide_logprobs_gb300 as vp
    op = s["op"]
    if op == "lookup":
        return vp.vp_embedding_fwd(s["x"], s["ids"], scale=s["scale"], vocab_start=s["start"], sharded=s["sharded"],
                                   dtype=s["out"])
    if op == "table_grad":
        return vp.vp_embedding_bwd(s["x"], s["ids"], s["V"], scale=s["scale"], vocab_start=s["start"],
                                   sharded=s["sharded"], dtype=s["out"])
    if op == "loss":
        loss, stats = vp.vp_cross_entropy_fwd(s["x"], s["targets"], vocab_start=s["start"], **s["rules"])
        return {"loss": loss, "dx": vp.vp_cross_entropy_bwd(s["x"], s["targets"], stats, s["grad"],
                                                            vocab_start=s["start"], **s["rules"])}
    loss, stats = vp.vp_linear_cross_entropy_fwd(s["h"], s["w"], s["targets"], vocab_start=s["start"], **s["rules"])
    dh, dw = vp.vp_linear_cross_entropy_bwd(s["h"], s["w"], s["targets"], stats, s["grad"], vocab_start=s["start"],
                                            **s["rules"])
    if s["tied"]:
        vp.vp_embedding_bwd(s["dy"], s["ids"], dw.shape[0], scale=s["scale"], vocab_start=s["start"], dW=dw,
                            accumulate=True)
    return {"loss": loss, "dhidden": dh, "dW": dw}


# --------------------------------------------------------------------------- work and exact values
def work(case):
    op, N, V = case["op"], case["N"], case["V"]
    size = {"bf16": 2, "f32": 4}
    if op == "lookup":
        # half of a split vocabulary's ids are looked up here; a row asked for again need not be read again
        D, here = case["D"], N if case["shard"] < 0 else N // 2
        return {"bytes": min(here, V) * D * size[case["dtype"]] + N * (D * size[case["out"]] + 8), "flops": N * D}
    if op == "table_grad":
        D, here = case["D"], N if case["shard"] < 0 else N // 2
        return {"bytes": here * D * size[case["dtype"]] + 8 * N + V * D * size[case["out"]], "flops": here * D}
    if op == "loss":
        # a read, then a read and a write
        return {"bytes": 3 * N * V * size[case["dtype"]] + 56 * N, "flops": (40 if case["cap"] else 12) * N * V}
    D = case["D"]
    return {"bytes": 4 * (N + V) * D + 56 * N + (2 * N * D if case["tied"] else 0), "flops": 6 * N * V * D}


def _exact_table_grad(dy, ids, start, V, scale):
    """Sums over the tokens in the order of their ids: differences of running sums at the ends of each id's tokens."""
    place = torch.where((ids >= start) & (ids < start + V), ids - start, V)
    order = torch.argsort(place, stable=True)
    ends = torch.searchsorted(place[order], torch.arange(V, device=DEV), right=True)
    out = torch.empty(V, dy.shape[1], dtype=torch.float64, device=DEV)
    for c in range(0, dy.shape[1], 512):
        sums = torch.cumsum(dy[:, c:c + 512][order].double(), 0)
        sums = torch.cat((torch.zeros_like(sums[:1]), sums))[ends]
        out[:, c:c + 512] = scale * torch.diff(sums, dim=0, prepend=torch.zeros_like(sums[:1]))
    return out


def _exact_loss(x, targets, grad, rules, out_loss):
    """The gradient of one block of rows (fp64 logits, local targets); their losses go to out_loss."""
    cap, smooth, zeta = rules["softcap"], rules["label_smoothing"], rules["z_loss"]
    V = x.shape[1]
    slope = None
    if cap:
        ex = torch.exp(-2 / cap * x.abs())                       # tanh by its exponential
        slope = 4 * ex / (1 + ex) ** 2
        x = torch.sign(x) * cap * (1 - ex) / (1 + ex)
    lse = torch.logsumexp(x, 1)
    logp = x - lse[:, None]
    used = targets >= 0
    t = targets.clamp(min=0)
    r = torch.arange(x.shape[0], device=DEV)
    nll = -logp[r, t]
    out_loss[:] = torch.where(used, (1 - smooth) * nll - smooth * logp.mean(1) + zeta * lse ** 2, 0.0)
    want = torch.full_like(x, smooth / V)
    want[r, t] += 1 - smooth
    # softmax minus what the target distribution wants, and the derivative of zeta lse^2
    d = torch.exp(logp)
    d = d - want + 2 * zeta * lse[:, None] * d
    if slope is not None:
        d = d * slope
    return d * torch.where(used, grad.double(), 0.0)[:, None]


def exact(case, seed):
    op, N, V = case["op"], case["N"], case["V"]
    if op == "linear_loss" and N * V * case["D"] > 1 << 40:      # some 10 seconds of fp64 products
        return None
    s = prepare(case, seed)
    if op == "lookup":
        table = torch.cat((s["x"].double(), torch.zeros(1, case["D"], dtype=torch.float64, device=DEV)))
        ids = s["ids"]
        return s["scale"] * table[torch.where((ids >= s["start"]) & (ids < s["start"] + V), ids - s["start"], V)]
    if op == "table_grad":
        return _exact_table_grad(s["x"], s["ids"], s["start"], V, s["scale"])
    targets = torch.where(s["targets"] < 0, -1, s["targets"] - s["start"])
    loss = torch.empty(N, dtype=torch.float64, device=DEV)
    step = max(1, (1 << 27) // V)
    if op == "loss":
        dx = torch.empty(N, V, dtype=torch.float64, device=DEV)
        for i in range(0, N, step):
            k = slice(i, i + step)
            dx[k] = _exact_loss(s["x"][k].double(), targets[k], s["grad"][k], s["rules"], loss[k])
        return {"loss": loss, "dx": dx}
    h, w = s["h"].double(), s["w"].double()
    dh, dw = torch.empty_like(h), torch.zeros_like(w)
    for i in range(0, N, step):
        k = slice(i, i + step)
        dz = _exact_loss(h[k] @ w.t(), targets[k], s["grad"][k], s["rules"], loss[k])
        dh[k] = dz @ w
        dw.addmm_(dz.t(), h[k])
    if s["tied"]:
        dw += _exact_table_grad(s["dy"], s["ids"], s["start"], V, s["scale"])
    return {"loss": loss, "dhidden": dh, "dW": dw}
