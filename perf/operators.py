"""Cases of the ruled-logits and the 4-bit head operators, in their plain form and through the library.

Operators ("op" of a case):
  quantize       MXFP4 quantisation of a matrix, and back to the values that the codes stand for
  linear         a hidden state quantised to MXFP4, times a head that is kept in MXFP4: logits
  process_fwd    penalties for repeated tokens, biases, temperature and a grammar mask put on logits
  process_bwd    the gradient of that with respect to the logits
  logprobs       logprobs of one target per row under the ruled distribution, with the gradient of the logits
"""
import math

import torch

own = False

DEV = "cuda"
VOCAB = 75968            # this library's benchmark vocabulary shard; 151936 is both halves of it
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)     # between neighbouring magnitudes of E2M1


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # the head's weight matrix, quantised once when a model is loaded
        dict(name="quantize_head", op="quantize", rows=VOCAB, D=4096, dtype="bf16"),
        # a few tokens' hidden states between two decode steps
        dict(name="quantize_few", op="quantize", rows=3, D=2112, dtype="f32"),
        # one sequence decoded: the head's bytes are all there is
        dict(name="linear_1", op="linear", N=1, V=VOCAB, D=4096, out="bf16"),
        # a decode batch of odd size over the whole vocabulary, fp32 logits for the sampler
        dict(name="linear_37", op="linear", N=37, V=2 * VOCAB, D=2048, out="f32"),
        # a prefill or a scoring chunk
        dict(name="linear_1000", op="linear", N=1000, V=VOCAB, D=4096, out="bf16"),
        # scoring of whole rollouts
        dict(name="linear_8192", op="linear", N=8192, V=VOCAB, D=4096, out="bf16"),
        # one sequence decoded with every rule on
        dict(name="process_1", op="process_fwd", N=1, V=VOCAB, dtype="bf16", form="decode", L=700, bias=20, masks=1,
             shard=0, wide=0),
        # a decode batch with long histories, fp32 logits
        dict(name="process_64", op="process_fwd", N=64, V=2 * VOCAB, dtype="f32", form="decode", L=16384, bias=300,
             masks=8, shard=0, wide=0),
        # the gradient of a training batch's ruled logits, second half of a split vocabulary
        dict(name="process_bwd_1024", op="process_bwd", N=1024, V=VOCAB, dtype="bf16", form="prefix", L=512, bias=0,
             masks=0, shard=1, wide=0),
        # rollouts scored and trained on: the benchmark's rows, each with its own prefix as history
        dict(name="logprobs_8192", op="logprobs", N=8192, V=VOCAB, dtype="bf16", form="prefix", L=512, bias=0, masks=4,
             shard=0, wide=0),
        # the same in fp32 with an odd vocabulary, read out of a padded tensor
        dict(name="logprobs_24", op="logprobs", N=24, V=5003, dtype="f32", form="prefix", L=40, bias=7, masks=2, shard=0,
             wide=5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "process_fwd", "process_bwd", "logprobs"])
    if op == "quantize":
        D = 64 * _log_int(rng, 1, 128)
        return dict(op=op, rows=_log_int(rng, 1, max(1, min(200000, VOCAB * 4096 // D))), D=D,
                    dtype=rng.choice(["bf16", "f32"]))
    if op == "linear":
        V, D = _log_int(rng, 1000, 2 * VOCAB), 64 * _log_int(rng, 2, 64)
        top = min(8192, 8192 * VOCAB * 4096 // (V * D), 8192 * VOCAB // V)
        out = rng.choice(["bf16", "f32"])
        return dict(op=op, N=_log_int(rng, 1, top // 2 if out == "f32" else top), V=V, D=D, out=out)
    V, dtype = _log_int(rng, 1000, 2 * VOCAB), rng.choice(["bf16", "f32"])
    N = _log_int(rng, 1, max(1, min(8192, 8192 * VOCAB // V // (2 if dtype == "f32" else 1))))
    form = "decode" if op == "process_fwd" else rng.choice(["decode", "prefix"])
    L = _log_int(rng, 1, min(32768 if form == "decode" else 2048, max(1, (8 << 20) // N)))
    return dict(op=op, N=N, V=V, dtype=dtype, form=form, L=L, bias=rng.choice([0, 0, _log_int(rng, 1, 1000)]),
                masks=rng.choice([0, 1, _log_int(rng, 1, 16)]), shard=rng.choice([0, 0, 1]), wide=rng.choice([0, 0, 3, 8]))


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, shape, sigma=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype).mul_(sigma)


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def scale_bytes(N, D):
    """Bytes of a matrix's scales: tiles of 128 rows x 4 blocks of 32 columns, 512 bytes each, row tiles outermost."""
    return -(-N // 128) * -(-D // 128) * 512


def _scale_places(N, D):
    """Where the scale of (row, block) lies: its tile, then 16 bytes for each row % 32, 4 for each (row % 128) // 32."""
    r = torch.arange(N, device=DEV)[:, None]
    b = torch.arange(D // 32, device=DEV)[None, :]
    return ((r // 128) * -(-D // 128) + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4


def plain_quantize(x):
    """(magnitude index with sign in bit 3, biased exponent of the scale) of each element and block of x [N, D]."""
    N, D = x.shape
    blocks = x.float().reshape(N, D // 32, 32)
    amax = blocks.abs().amax(-1)
    bad = ~torch.isfinite(amax)
    exp = (torch.frexp(torch.where(bad, 1.0, amax))[1] - 1 - 2).clamp(-127, 127)      # frexp: amax = m 2^e, m in [1/2, 1)
    exp = torch.where(amax == 0, -127, exp)
    v = torch.ldexp(blocks, -exp[..., None])
    a = v.abs()
    # nearest magnitude: how many borders lie below; a tie goes to the even index, so the borders with an odd
    # index below them are taken one fp32 step lower
    borders = torch.tensor(BORDERS, device=DEV)
    borders[1::2] = torch.nextafter(borders[1::2], torch.zeros(3, device=DEV))
    code = torch.bucketize(a, borders, out_int32=True)
    code = torch.where(bad[..., None], 0, code + 8 * torch.signbit(blocks))
    return code.to(torch.uint8).reshape(N, D), torch.where(bad, 255, exp + 127).to(torch.uint8)


def plain_pack(code, exp):
    """The public layout: two codes to a byte, the even column in the low bits; scales in tiles."""
    N, D = code.shape
    scales = torch.zeros(scale_bytes(N, D), dtype=torch.uint8, device=DEV)
    scales[_scale_places(N, D).reshape(-1)] = exp.reshape(-1)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous(), scales


def plain_values(code, exp):
    """What codes [N, D] and scales [N, D / 32] stand for, in fp32."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    v = table[code.int()].reshape(code.shape[0], -1, 32)
    e = exp.int()[..., None]
    return torch.where(e == 255, math.nan, torch.ldexp(v, e - 127)).reshape(code.shape)


def plain_unpack(packed, scales):
    N, D = packed.shape[0], 2 * packed.shape[1]
    code = torch.stack((packed & 15, packed >> 4), dim=-1).reshape(N, D)
    return code, scales[_scale_places(N, D)]


def _rule_inputs(case, g, x, train):
    """Histories, penalties, biases and masks of N rows over V columns, and the rows' targets where `train`."""
    N, V, L = case["N"], case["V"], case["L"]
    start = case["shard"] * V                                  # the call's columns are ids start .. start + V - 1
    total_V = V * (1 + case["shard"])

    def ids(n):                                                # a few ids far more often than the others
        u = torch.rand(n, generator=g, device=DEV)
        return (u ** 4 * total_V).long().clamp_(max=total_V - 1)

    targets = None
    if case["form"] == "decode":                               # rows of L ids, each filled to a length of its own
        hist = ids(N * L)
        n_total = torch.randint(0 if N > 1 else L, L + 1, (N,), generator=g, device=DEV)
        n_prompt = (n_total * torch.rand(N, generator=g, device=DEV)).long()
        spans = torch.stack((torch.arange(N, device=DEV) * L, n_prompt, n_total), 1)
    else:                                                      # sequences of a prompt of L and T answers; row t sees t of them
        T = min(N, 1024)
        B = -(-N // T)
        hist = ids(B * (L + T))
        r = torch.arange(N, device=DEV)
        spans = torch.stack((r // T * (L + T), torch.full_like(r, L), L + r % T), 1)
        targets = hist[spans[:, 0] + spans[:, 2]]
    if train:
        # targets in this shard, but for a few rows that are ignored
        local = targets % V if targets is not None else ids(N) % V
        targets = torch.where(torch.rand(N, generator=g, device=DEV) < 0.03, -1, local + start)
    rules = dict(ids=hist, spans=spans.contiguous(),
                 repetition=1.0 + 0.3 * torch.rand(N, generator=g, device=DEV),
                 frequency=0.5 * torch.rand(N, generator=g, device=DEV),
                 presence=0.5 * torch.rand(N, generator=g, device=DEV),
                 temperature=0.6 + 0.8 * torch.rand(N, generator=g, device=DEV))
    if case["bias"]:
        nb = case["bias"]
        rules.update(bias_ids=torch.randint(0, total_V, (N * nb,), generator=g, device=DEV),
                     bias_values=4 * torch.randn(N * nb, generator=g, device=DEV),
                     bias_spans=torch.stack((torch.arange(N, device=DEV) * nb, torch.full((N,), nb, device=DEV)), 1))
    if case["masks"]:
        M = case["masks"]
        words = -(-V // 32)
        allowed = torch.rand(M, words * 32, generator=g, device=DEV) < torch.linspace(0.9, 0.2, M, device=DEV)[:, None]
        rows = torch.randint(-1 if N > 1 else 0, M, (N,), generator=g, device=DEV)
        if train:                                              # a token that was sampled had been allowed
            allowed[rows.clamp(min=0), (targets - start).clamp(min=0)] = True
        bits = (allowed.view(M, words, 32).long() << torch.arange(32, device=DEV)).sum(-1)
        rules.update(mask=torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32), mask_rows=rows)
    return rules, targets, start


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "quantize":
        return dict(op=op, x=_randn(g, (case["rows"], case["D"]), 0.02, _dtype(case["dtype"])))
    if op == "linear":
        w = _randn(g, (case["V"], case["D"]), 0.02, torch.bfloat16)
        codes = torch.empty(case["V"], case["D"] // 2, dtype=torch.uint8, device=DEV)
        exps = torch.empty(case["V"], case["D"] // 32, dtype=torch.uint8, device=DEV)
        for i in range(0, case["V"], 16384):
            c, e = plain_quantize(w[i:i + 16384])
            codes[i:i + 16384] = c[:, 0::2] | (c[:, 1::2] << 4)
            exps[i:i + 16384] = e
        scales = torch.zeros(scale_bytes(case["V"], case["D"]), dtype=torch.uint8, device=DEV)
        scales[_scale_places(case["V"], case["D"]).reshape(-1)] = exps.reshape(-1)
        return dict(op=op, h=_randn(g, (case["N"], case["D"]), 1.0, torch.bfloat16), codes=codes, scales=scales,
                    out=_dtype(case["out"]))
    N, V = case["N"], case["V"]
    x = _randn(g, (N, V + case["wide"]), 3.0, _dtype(case["dtype"]))[:, :V]
    rules, targets, start = _rule_inputs(case, g, x, op == "logprobs")
    # the number of (row, id) pairs: known on the host to whoever wrote the spans
    s = dict(op=op, x=x, rules=rules, start=start, pairs=int(rules["spans"][:, 2].sum()))
    if op == "process_bwd":
        s["dy"] = _randn(g, (N, V), 1e-3, _dtype(case["dtype"]))
    if op == "logprobs":
        s.update(targets=targets, grad=torch.randn(N, generator=g, device=DEV))
    return s


# --------------------------------------------------------------------------- plain forms
def _plain_rules(s):
    """(seen, occurrences among the outputs, bias, allowed) as [N, V] tensors, None where there is no such rule."""
    x, q = s["x"], s["rules"]
    N, V = x.shape
    spans = q["spans"]
    row = torch.repeat_interleave(torch.arange(N, device=DEV), spans[:, 2], output_size=s["pairs"])
    first = torch.cumsum(spans[:, 2], 0) - spans[:, 2]
    at = torch.arange(row.numel(), device=DEV) - first[row]
    local = q["ids"][spans[row, 0] + at] - s["start"]
    inside = (local >= 0) & (local < V)
    place = row * V + local.clamp(0, V - 1)
    is_output = (at >= spans[row, 1]) & inside
    count = torch.zeros(N * V, dtype=torch.int32, device=DEV).scatter_add_(0, place, is_output.int()).view(N, V)
    seen = torch.zeros(N * V, dtype=torch.int32, device=DEV).scatter_add_(0, place, inside.int()).view(N, V) > 0
    bias = allowed = None
    if "bias_ids" in q:
        nb = q["bias_ids"].numel() // N
        local = q["bias_ids"].view(N, nb) - s["start"]
        inside = (local >= 0) & (local < V)
        entry = torch.where(inside, torch.arange(nb, device=DEV)[None, :] + 1, 0)
        last = torch.zeros(N, V, dtype=torch.int64, device=DEV).scatter_reduce_(1, local.clamp(0, V - 1), entry, "amax")
        bias = torch.where(last > 0, q["bias_values"].view(N, nb).gather(1, (last - 1).clamp(min=0)), 0.0)
    if "mask" in q:
        bits = (q["mask"][:, :, None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1
        bits = bits.view(q["mask"].shape[0], -1)[:, :V] > 0
        allowed = bits[q["mask_rows"].clamp(min=0)] | (q["mask_rows"] < 0)[:, None]
    return seen, count, bias, allowed


def _plain_process(s, rules):
    seen, count, bias, allowed = rules
    x, q = s["x"].float(), s["rules"]
    rep, T = q["repetition"][:, None], q["temperature"][:, None]
    z = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    z = z - q["frequency"][:, None] * count - q["presence"][:, None] * (count > 0)
    if bias is not None:
        z = z + bias
    z = z / T
    return z if allowed is None else torch.where(allowed, z, -math.inf)


def _plain_factor(s, rules):
    seen, _, _, allowed = rules
    rep, T = s["rules"]["repetition"][:, None], s["rules"]["temperature"][:, None]
    f = torch.where(seen, torch.where(s["x"] > 0, 1 / rep, rep), 1.0) / T
    return f if allowed is None else torch.where(allowed, f, 0.0)


def _plain_logprobs(s):
    rules = _plain_rules(s)
    z = _plain_process(s, rules)
    N, V = z.shape
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True, dtype=torch.float64)
    used = s["targets"] >= 0
    t = torch.where(used, s["targets"] - s["start"], 0)[:, None]
    logp = (z.gather(1, t).double() - m.double() - torch.log(total))[:, 0]
    p = e / total.float()
    p.scatter_add_(1, t, torch.full((N, 1), -1.0, device=DEV))      # p - onehot
    dx = torch.where(used, -s["grad"], 0.0)[:, None] * p * _plain_factor(s, rules)
    return {"logp": torch.where(used, logp, 0.0).float(), "dx": dx.to(s["x"].dtype)}


def _plain(s):
    op = s["op"]
    if op == "quantize":
        return torch.cat([plain_values(*plain_quantize(part)).to(s["x"].dtype) for part in s["x"].split(16384)])
    if op == "linear":
        h = plain_values(*plain_quantize(s["h"]))
        w = plain_values(*plain_unpack(s["codes"], s["scales"]))
        return (h @ w.t()).to(s["out"])
    if op == "process_fwd":
        return _plain_process(s, _plain_rules(s)).to(s["x"].dtype)
    if op == "process_bwd":
        return (s["dy"].float() * _plain_factor(s, _plain_rules(s))).to(s["x"].dtype)
    return _plain_logprobs(s)


# --------------------------------------------------------------------------- the library's calls
def run(s):
    if not own:
        return _plain(s)
    import vocab_wide_logprobs_gb300 as vp
    op = s["op"]
    if op == "quantize":
        return vp.vp_mxfp4_dequantize(*vp.vp_mxfp4_quantize(s["x"]), dtype=s["x"].dtype)
    if op == "linear":
        return vp.vp_linear_mxfp4_fwd(*vp.vp_mxfp4_quantize(s["h"]), s["codes"], s["scales"], dtype=s["out"])
    rules = vp.logits_rules(**s["rules"])
    if op == "process_fwd":
        return vp.vp_logits_process_fwd(s["x"], rules, vocab_start=s["start"])
    if op == "process_bwd":
        return vp.vp_logits_process_bwd(s["x"], rules, s["dy"], vocab_start=s["start"])
    logp, stats = vp.vp_processed_logprobs_fwd(s["x"], rules, s["targets"], vocab_start=s["start"])
    return {"logp": logp,
            "dx": vp.vp_processed_logprobs_bwd(s["x"], rules, s["targets"], stats, s["grad"], vocab_start=s["start"])}


# --------------------------------------------------------------------------- work and exact values
def work(case):
    op = case["op"]
    if op == "quantize":
        n, es = case["rows"] * case["D"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * n * es + n // 2 + n // 32, "flops": 4 * n}
    if op == "linear":
        N, V, D = case["N"], case["V"], case["D"]
        return {"bytes": N * D * 2 + V * (D // 2 + D // 32) + N * V * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * N * V * D}
    N, V, es = case["N"], case["V"], 2 if case["dtype"] == "bf16" else 4
    if case["form"] == "decode":
        ids = N * case["L"] // 2
    else:
        ids = -(-N // 1024) * (case["L"] + min(N, 1024))
    small = 8 * ids + N * case["bias"] * 12 + case["masks"] * V // 8 + N * 48
    # process: one read and one write; logprobs: a read, then a read and a write
    moves = 3 if op == "logprobs" else 2
    return {"bytes": moves * N * V * es + small, "flops": (12 if op == "logprobs" else 3) * N * V}


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "quantize":
        if case["rows"] * case["D"] > 1 << 28:
            return torch.cat([_exact_quantize(p) for p in s["x"].split(4096)])
        return _exact_quantize(s["x"])
    if op == "linear":
        h = _exact_quantize(s["h"])
        V, D = case["V"], case["D"]
        y = torch.empty(case["N"], V, dtype=torch.float64, device=DEV)
        values = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=DEV)
        tiles = s["scales"].view(-1, -(-D // 128), 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, -(-D // 128) * 4)
        for i in range(0, V, 8192):
            c = s["codes"][i:i + 8192].long()
            w = torch.stack((values[c % 16], values[c // 16]), 2).reshape(c.shape[0], D // 32, 32)
            w = w * torch.exp2(tiles[i:i + c.shape[0], :D // 32].double() - 127)[..., None]
            y[:, i:i + 8192] = h @ w.reshape(-1, D).t()
        return y
    N, V = case["N"], case["V"]
    q = s["rules"]
    res = torch.empty(N, V, dtype=torch.float64, device=DEV)
    logp = torch.zeros(N, dtype=torch.float64, device=DEV)
    words = q["mask"].cpu().numpy().view("uint32") if "mask" in q else None
    mask = None
    if words is not None:
        import numpy as np
        mask = torch.from_numpy(np.unpackbits(words.view("uint8"), axis=1, bitorder="little")[:, :V].astype(bool)).to(DEV)
    host = {k: v.cpu() for k, v in q.items() if k != "mask"}
    per_row = {k: q[k].double().tolist() for k in ("repetition", "frequency", "presence", "temperature")}
    mask_rows = q["mask_rows"].tolist() if mask is not None else None
    targets = s["targets"].tolist() if op == "logprobs" else None
    grads = s["grad"].double().tolist() if op == "logprobs" else None
    for r in range(N):
        # the row's distinct ids, how often each is among the outputs, and its biases by column
        first, n_prompt, n_total = host["spans"][r].tolist()
        ids = host["ids"][first:first + n_total] - s["start"]
        inside = (ids >= 0) & (ids < V)
        uniq, inv = torch.unique(ids[inside], return_inverse=True)
        is_output = (torch.arange(n_total) >= n_prompt)[inside]
        count = torch.zeros(uniq.numel(), dtype=torch.float64).index_add_(0, inv, is_output.double())
        bias = {}
        if case["bias"]:
            b0, nb = host["bias_spans"][r].tolist()
            columns = (host["bias_ids"][b0:b0 + nb] - s["start"]).tolist()
            bias = {c: v for c, v in zip(columns, host["bias_values"][b0:b0 + nb].tolist()) if 0 <= c < V}
        x = s["x"][r].double()
        rep, freq, pres, T = (per_row[k][r] for k in ("repetition", "frequency", "presence", "temperature"))
        factor = torch.full((V,), 1 / T, dtype=torch.float64, device=DEV)
        z = x.clone()
        if uniq.numel():
            u, c = uniq.to(DEV), count.to(DEV)
            f = torch.where(x[u] > 0, 1 / rep, rep)
            z[u] = x[u] * f - freq * c - pres * (c > 0)
            factor[u] *= f
        if bias:
            z[torch.tensor(list(bias), device=DEV)] += torch.tensor(list(bias.values()), dtype=torch.float64, device=DEV)
        z /= T
        if mask is not None and mask_rows[r] >= 0:
            banned = ~mask[mask_rows[r]]
            z[banned] = -math.inf
            factor[banned] = 0.0
        if op == "process_fwd":
            res[r] = z
        elif op == "process_bwd":
            res[r] = s["dy"][r].double() * factor
        elif targets[r] < 0:
            res[r] = 0
        else:
            t = targets[r] - s["start"]
            lse = torch.logsumexp(z, 0)
            p = torch.exp(z - lse)
            logp[r] = z[t] - lse
            g = -p
            g[t] = -torch.expm1(z[t] - lse)
            res[r] = grads[r] * factor * g
    return res if op != "logprobs" else {"logp": logp, "dx": res}


def _exact_quantize(x):
    x = x.double()
    b = x.reshape(x.shape[0], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    X = torch.exp2((torch.floor(torch.log2(amax.clamp(min=2.0 ** -126))) - 2).clamp(-127, 127))
    v = (b / X).abs()
    # E2M1: steps of 1/2 below 2, of 1 below 4, of 2 up to 6; torch.round ties to even multiples of the step
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0))
    return (torch.sign(b) * (torch.round(v / step) * step).clamp(max=6.0) * X).reshape(x.shape)
