"""Decode with a 4-bit head and rules on the logits, score the rollout under the same rules, then learn from it.

A stand-in model (the hidden state of a token is its embedding) drives the calls as a rollout worker and a
trainer make them:

  decode, one token for each sequence a step
      vp_embedding_fwd        the tokens' rows of the embedding
      vp_mxfp4_quantize       the hidden states
      vp_linear_mxfp4_fwd     times the head, kept in MXFP4: logits
      vp_logits_process_fwd   penalties for repeated tokens, biases, a grammar mask, a temperature (in place)
      Gumbel-max              the next token
  score, all tokens of all sequences at once
      vp_mxfp4_quantize, vp_linear_mxfp4_fwd    the same logits, row (b, t) of sequence b's prefix
      vp_processed_logprobs_fwd / _bwd          logprobs of the drawn tokens and the gradient of their sum
  learn, all tokens at once, with the embedding as the head (a tied model)
      vp_embedding_fwd                          hidden states
      vp_linear_cross_entropy_fwd / _bwd        the loss and its gradients, the logits never stored
      vp_embedding_bwd                          the lookup's gradient, added to the head's

    python examples/decode_and_score.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import vocab_wide_logprobs_gb300 as vp  # noqa: E402


def grammar(V, words, device, generator):
    """Two mask rows: every second token, and a random four fifths."""
    allowed = torch.zeros(2, 32 * words, dtype=torch.bool, device=device)
    allowed[0, :V:2] = True
    allowed[1, :V] = torch.rand(V, generator=generator, device=device) < 0.8
    bits = (allowed.view(2, words, 32).long() << torch.arange(32, device=device)).sum(-1)
    return torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)


def learn(table, ids, targets, scale, label_smoothing=0.1, z_loss=1e-4, softcap=30.0):
    """The mean loss of a tied model, scale * table[ids] . table^T, that is to predict the targets, and the gradient of its table."""
    rules = dict(label_smoothing=label_smoothing, z_loss=z_loss, softcap=softcap)
    hidden = vp.vp_embedding_fwd(table, ids, scale=scale)
    loss, stats = vp.vp_linear_cross_entropy_fwd(hidden, table, targets, **rules)
    grad = torch.full_like(loss, 1 / loss.numel())
    dhidden, dtable = vp.vp_linear_cross_entropy_bwd(hidden, table, targets, stats, grad, **rules)
    vp.vp_embedding_bwd(dhidden, ids, table.shape[0], scale=scale, dW=dtable, accumulate=True)
    return loss.mean(), dtable


def run(B=4, prompt=24, steps=16, V=5003, D=512, device="cuda", seed=0):
    g = torch.Generator(device=device).manual_seed(seed)
    embedding = torch.randn(V, D, generator=g, device=device).to(torch.bfloat16)
    head = vp.vp_mxfp4_quantize((torch.randn(V, D, generator=g, device=device) * 0.1).to(torch.bfloat16))
    T = prompt + steps
    ids = torch.randint(0, V, (B, T), generator=g, device=device)
    ids[:, prompt:] = -1                                          # not drawn yet
    row = torch.arange(B, device=device)
    per_sequence = dict(repetition=torch.full((B,), 1.2, device=device), frequency=torch.full((B,), 0.3, device=device),
                        presence=torch.full((B,), 0.1, device=device), temperature=torch.full((B,), 0.8, device=device))
    bias_ids, bias_values = torch.tensor([7, 8, 9], device=device), torch.tensor([2.0, -2.0, float("-inf")], device=device)
    mask, mask_rows = grammar(V, (V + 31) // 32, device, g), row % 3 - 1      # -1: a sequence without a grammar

    def rules(sequence, n_output):
        """Of rows that see the prompt and the first n_output tokens of their sequences."""
        n = sequence.numel()
        spans = torch.stack((sequence * T, torch.full((n,), prompt, device=device), prompt + n_output), 1)
        biases = torch.zeros(n, 2, dtype=torch.int64, device=device)
        biases[:, 1] = bias_ids.numel()                           # all rows share one list
        return vp.logits_rules(ids=ids.view(-1), spans=spans.contiguous(), bias_ids=bias_ids, bias_values=bias_values,
                               bias_spans=biases, mask=mask, mask_rows=mask_rows[sequence],
                               **{k: v[sequence] for k, v in per_sequence.items()})

    def logits(tokens):
        hidden = vp.vp_embedding_fwd(embedding, tokens.contiguous())
        return vp.vp_linear_mxfp4_fwd(*vp.vp_mxfp4_quantize(hidden), *head, dtype=torch.float32)

    drawn_logp = torch.empty(B, steps, dtype=torch.float64, device=device)
    for t in range(steps):
        y = logits(ids[:, prompt + t - 1])
        vp.vp_logits_process_fwd(y, rules(row, torch.full((B,), t, device=device)), y=y)
        noise = -torch.log(-torch.log(torch.rand(B, V, generator=g, device=device).clamp_(1e-20, 1 - 1e-7)))
        token = (y + noise).argmax(1)
        drawn_logp[:, t] = torch.log_softmax(y.double(), 1).gather(1, token[:, None])[:, 0]
        ids[:, prompt + t] = token

    sequence = row.repeat_interleave(steps)
    step = torch.arange(steps, device=device).repeat(B)
    x = logits(ids[sequence, prompt + step - 1])
    err = torch.zeros(1, dtype=torch.int32, device=device)
    q, targets = rules(sequence, step), ids[sequence, prompt + step].contiguous()
    logp, stats = vp.vp_processed_logprobs_fwd(x, q, targets, err_word=err)
    dx = vp.vp_processed_logprobs_bwd(x, q, targets, stats, torch.ones_like(logp), err_word=err)
    seen = ids[sequence, prompt + step - 1].contiguous()
    loss, dtable = learn(embedding, seen, targets, D ** -0.5)
    return dict(ids=ids, drawn_logp=drawn_logp.view(-1), logp=logp, dx=dx, err=int(err), fault=vp.vp_fault_status(),
                table=embedding, seen=seen, targets=targets, loss=loss, dtable=dtable)


if __name__ == "__main__":
    out = run()
    print(f"drew {out['logp'].numel()} tokens: mean logprob {out['logp'].mean():.4f}, "
          f"largest difference to the logprobs at decode {(out['logp'] - out['drawn_logp']).abs().max():.1e}, "
          f"gradient rms {out['dx'].float().square().mean().sqrt():.3e}; "
          f"loss of the tied model {out['loss']:.4f}, its table's gradient rms {out['dtable'].float().square().mean().sqrt():.3e}")
