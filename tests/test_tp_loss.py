"""The cross entropy and the embedding with the vocabulary split across ranks: the host's side on two CPU ranks (gloo), with
stand-ins for the calls that need a GPU, and the calls themselves in a group of one."""
import math
import os
import socket

import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

N, V, CUT, D = 12, 70, 31, 8      # rank 0 has columns (rows of the table) [0, 31), rank 1 [31, 70)


def _data():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(N, V, generator=g, dtype=torch.float64)
    targets = torch.randint(0, V, (N,), generator=g)
    targets[:3] = torch.tensor([CUT - 1, CUT, -1])
    return x, targets, torch.randn(V, D, generator=g), torch.randint(-1, V, (3, 4), generator=g)


def _loss(x, targets, smooth, zeta, cap):
    z = cap * torch.tanh(x / cap)
    lse = torch.logsumexp(z, 1)
    loss = lse - (1 - smooth) * z.gather(1, targets.clamp(min=0)[:, None])[:, 0] - smooth * z.mean(1) + zeta * lse ** 2
    return torch.where(targets >= 0, loss, 0.0)


def _stand_ins(api):
    """Records of five numbers: log sum exp, sum, the target's logit or 0, columns, whether the target is here."""
    def partial(x, targets, softcap=0.0, vocab_start=0):
        z = softcap * torch.tanh(x / softcap)
        local = targets - vocab_start
        here = (targets >= 0) & (local >= 0) & (local < x.shape[1])
        zt = torch.where(here, z.gather(1, torch.where(here, local, 0)[:, None])[:, 0], 0.0)
        n = torch.full_like(zt, x.shape[1])
        return torch.stack((torch.logsumexp(z, 1), z.sum(1), zt, n, here.double()), 1)

    def linear_partial(hidden, weight, targets, softcap=0.0, vocab_start=0):
        return partial(hidden @ weight.t(), targets, softcap, vocab_start)

    def merge(parts, label_smoothing=0.0, z_loss=0.0, err_word=None):
        lse, n = torch.logsumexp(parts[..., 0], 0), parts[..., 3].sum(0)
        loss = lse - (1 - label_smoothing) * parts[..., 2].sum(0) - label_smoothing * parts[..., 1].sum(0) / n + z_loss * lse ** 2
        return torch.where(parts[..., 4].sum(0) > 0, loss, 0.0), parts

    def lookup(weight, ids, scale=1.0, vocab_start=0, sharded=False, dtype=None):
        local = ids - vocab_start
        here = (ids >= 0) & (local >= 0) & (local < weight.shape[0])
        assert sharded
        return torch.where(here[..., None], scale * weight[torch.where(here, local, 0)], 0.0).to(dtype or weight.dtype)

    api.vp_cross_entropy_partial, api.vp_linear_cross_entropy_partial = partial, linear_partial
    api.vp_cross_entropy_merge, api.vp_embedding_fwd = merge, lookup


def _rank(rank, world, port, q):
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=world)
    try:
        from vocab_wide_logprobs_gb300 import api, tp
        _stand_ins(api)
        x, targets, table, ids = _data()
        own, start = (slice(0, CUT), 0) if rank == 0 else (slice(CUT, V), CUT)
        rules = dict(label_smoothing=0.1, z_loss=0.01, softcap=5.0)
        loss, parts = tp.tp_cross_entropy_fwd(x[:, own], targets, start, **rules)
        h = x[:, :D]
        linear, _ = tp.tp_linear_cross_entropy_fwd(h, table.double()[own], targets, start, **rules)
        rows = tp.tp_embedding_fwd(table[own], ids, start, scale=2.0, dtype=torch.bfloat16)
        q.put((rank, loss.numpy(), linear.numpy(), rows.float().numpy(), tuple(parts.shape)))
    finally:
        dist.destroy_process_group()


@pytest.mark.timeout(180)
def test_two_ranks_have_the_whole_vocabularys_results():
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    procs = [ctx.Process(target=_rank, args=(r, 2, port, q)) for r in range(2)]
    for p in procs:
        p.start()
    results = [q.get(timeout=150) for _ in procs]
    for p in procs:
        p.join(timeout=30)
        assert p.exitcode == 0
    x, targets, table, ids = _data()
    rows = torch.where((ids >= 0)[..., None], 2.0 * table[ids.clamp(min=0)], 0.0).to(torch.bfloat16).float()
    for _, loss, linear, got, shape in results:
        assert shape == (2, N, 5)
        assert torch.allclose(torch.from_numpy(loss), _loss(x, targets, 0.1, 0.01, 5.0), rtol=1e-12)
        assert torch.allclose(torch.from_numpy(linear), _loss(x[:, :D] @ table.double().t(), targets, 0.1, 0.01, 5.0), rtol=1e-12)
        assert torch.equal(torch.from_numpy(got), rows)


@pytest.mark.gpu
def test_a_group_of_one_has_the_unsharded_results(tmp_path):
    import vocab_wide_logprobs_gb300 as vp
    from vocab_wide_logprobs_gb300 import tp
    dist.init_process_group("gloo", init_method=f"file://{tmp_path}/store", rank=0, world_size=1)
    try:
        g = torch.Generator(device="cuda").manual_seed(4)
        h = torch.randn(50, 64, generator=g, device="cuda").to(torch.bfloat16)
        table = torch.randn(900, 64, generator=g, device="cuda").to(torch.bfloat16)
        ids = torch.randint(-1, 900, (50,), generator=g, device="cuda")
        x, rules = (h.float() @ table.float().t()), dict(label_smoothing=0.1, z_loss=1e-3, softcap=20.0)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        for (got, _), (want, _) in ((tp.tp_cross_entropy_fwd(x, ids, 0, err_word=err, **rules), vp.vp_cross_entropy_fwd(x, ids, **rules)),
                                    (tp.tp_linear_cross_entropy_fwd(h, table, ids, 0, err_word=err, **rules),
                                     vp.vp_linear_cross_entropy_fwd(h, table, ids, **rules))):
            assert torch.allclose(got, want, rtol=1e-6)
        assert int(err) == 0
        got = tp.tp_embedding_fwd(table, ids, 0, scale=math.sqrt(64), dtype=torch.float32)
        assert torch.equal(got, vp.vp_embedding_fwd(table, ids, scale=math.sqrt(64), dtype=torch.float32))
    finally:
        dist.destroy_process_group()
