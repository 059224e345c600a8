"""Distil a student from a teacher whose output matrix is stored in 8 bits, and score the result.

    python examples/distill_from_8bit_teacher.py [--steps 30]

1. The teacher's output matrix is quantised once (e4m3, a scale per 128 x 128 block).
2. Its logits, one chunk of positions at a time, are read for the top K tokens of every position:
   the teacher cache, from logits instead of full-precision hidden states and weights.
3. The student trains on the KL loss against that cache plus, where a position has a known answer,
   the answer's log-likelihood and a small entropy bonus, both straight from its hidden states.
4. The student's held-out answers are scored, once as a batch and once position by position.

The data are random: hidden states stand for a frozen student body, the teacher for a rotation of it.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_kl_loss_gb300 as fckl  # noqa: E402


def teacher_cache(Ht, W8, scale, K, chunk):
    """Top-K cache (idx int32 [N, K], logp fp32 [N, K]) of an 8-bit teacher head; only one chunk's
    logits exist at a time."""
    N = Ht.shape[0]
    idx = torch.empty(N, K, dtype=torch.int32, device=Ht.device)
    logp = torch.empty(N, K, dtype=torch.float32, device=Ht.device)
    for a in range(0, N, chunk):
        logits = fckl.block_scaled_projection(Ht[a:a + chunk], W8, scale)
        no_tokens = torch.empty(logits.shape[0], 0, dtype=torch.int32, device=Ht.device)
        _, _, _, idx[a:a + chunk], logp[a:a + chunk] = fckl.token_logprobs(logits, no_tokens, top=K)
    fckl.check()
    return idx, logp


def run(N=1024, d=256, V=8000, K=50, chunk=512, steps=30, answers=0.25, alpha=0.1, beta=0.01, lr=0.01, seed=0, log=print):
    g = torch.Generator("cuda").manual_seed(seed)
    Ht = torch.randn(N, d, generator=g, device="cuda").bfloat16()
    Wt = (torch.randn(V, d, generator=g, device="cuda") * 3 / d ** 0.5).bfloat16()
    W8, scale = fckl.block_quantize(Wt, rows=128)
    idx, logp = teacher_cache(Ht, W8, scale, K, chunk)

    W = (torch.randn(V, d, generator=g, device="cuda") / d ** 0.5).bfloat16().requires_grad_()
    rot = torch.linalg.qr(torch.randn(d, d, generator=g, device="cuda"))[0]
    H = (Ht.float() @ rot).bfloat16()
    # one known answer for some positions, the teacher's most probable token; -1 elsewhere
    known = torch.rand(N, 1, generator=g, device="cuda") < answers
    tokens = torch.where(known, idx[:, :1], torch.full_like(idx[:, :1], -1))
    opt = torch.optim.Adam([W], lr=lr)
    history = []
    for step in range(steps):
        opt.zero_grad()
        kl = fckl.fused_chunked_kl(H, W, idx, logp, chunk, scale=1 / N)
        lp, entropy = fckl.fused_token_logprobs(H, W, tokens, chunk)
        loss = kl - alpha * lp.sum() / known.sum() - beta * entropy.mean()
        loss.backward()
        opt.step()
        history.append((float(kl.detach()), float(lp.detach().sum() / known.sum())))
        if step % 10 == 0 or step == steps - 1:
            log(f"step {step:3d}  KL {history[-1][0]:.4f}  log-likelihood of the answers {history[-1][1]:.4f}")
    fckl.check()
    # held out: the positions without an answer, scored on the teacher's choice
    rest = (~known[:, 0]).nonzero()[:8, 0]
    Hh, th = H[rest].contiguous(), idx[rest, :1].contiguous()
    batch, _, _ = fckl.projected_logprobs(Hh, W.detach(), th, chunk)
    single = torch.cat([fckl.projected_logprobs(Hh[i:i + 1], W.detach(), th[i:i + 1], chunk)[0] for i in range(len(rest))])
    fckl.check()
    log(f"held out: {batch.mean():.4f} per token, batched and single scores differ by at most "
        f"{(batch - single).abs().max():.1e}")
    return history, batch, single


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=30)
    run(steps=ap.parse_args().steps)
