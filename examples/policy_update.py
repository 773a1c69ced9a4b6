"""A policy trained on its own samples, with every vocabulary-sized step on the library's kernels.

The policy is one bf16 head over fixed features of a few contexts.  A step samples a token per row (`sample`),
takes the log-probabilities of the tokens under the sampling and the reference head straight from the features
(`lm_head_logprob`), forms the clipped policy loss and its gradient on the logits (`policy_loss`, written over the
logits), and updates the head with 8-bit states (`adamw_step`).  Each context rewards the tokens of one residue
class; a preference phase (`preference_loss`) then prefers single tokens of it.

    python examples/policy_update.py [--steps 60] [--vocab 4096] [--rows 2048]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import top_sampling_apply_gb300 as tsa  # noqa: E402

CLASSES = 8  # a context's rewarded tokens: those congruent to its number


def train(steps=60, vocab=4096, rows=2048, width=256, seed=0, device="cuda"):
    """Mean reward of the first and the last policy step, and the mean reward margin of the preference phase."""
    g = torch.Generator(device=device).manual_seed(seed)
    features = torch.randn(CLASSES, width, generator=g, device=device).to(torch.bfloat16)
    head = (torch.randn(vocab, width, generator=g, device=device) * 0.02).to(torch.bfloat16)
    reference = head.clone()
    grad = torch.zeros_like(head)
    plan = tsa.adamw_plan([head], [grad], *tsa.adamw_state([head], 8))
    context = torch.arange(rows, device=device) % CLASSES
    hidden = features[context]
    temperature, rewards, update = 0.9, [], 0
    rounding = seed + 1  # another key than the draws'
    for step in range(steps):
        logits = hidden @ head.t()
        tokens = tsa.sample(logits, temperature, top_p=0.99, seed=seed, offset=step)
        old = tsa.lm_head_logprob(hidden, head, tokens, temperature=temperature)
        ref = tsa.lm_head_logprob(hidden, reference, tokens, temperature=temperature)
        reward = (tokens % CLASSES == context).float()
        advantage = (reward - reward.mean()) / (reward.std() + 1e-4)
        for _ in range(2):  # two updates on the same samples: the second one needs the clipping
            logits = hidden @ head.t()
            loss = tsa.policy_loss(logits, tokens, old, advantage, ref_logprob=ref, kl_coef=1e-3, entropy_coef=1e-3,
                                   temperature=temperature, grad=logits)
            torch.mm(loss.grad.t(), hidden, out=grad)
            update += 1
            tsa.adamw_step(plan, update, 2e-3, weight_decay=0.0, seed=rounding, offset=update)
        rewards.append(reward.mean())
    # preference: of two one-token answers to a context, the rewarded one
    pairs = rows // 2
    hidden = torch.cat([features[context[:pairs]], features[context[:pairs]]])
    good = context[:pairs] + CLASSES * torch.randint(0, vocab // CLASSES, (pairs,), generator=g, device=device)
    tokens = torch.cat([good, (good + 1 + torch.arange(pairs, device=device) % (CLASSES - 1)) % vocab])
    start = torch.arange(2 * pairs + 1, device=device)
    reference = head.clone()
    ref = tsa.lm_head_logprob(hidden, reference, tokens)
    for _ in range(steps // 4):
        logits = hidden @ head.t()
        loss = tsa.preference_loss(logits, tokens, start, ref_logprob=ref, beta=0.5, grad=logits)
        torch.mm(loss.grad.t(), hidden, out=grad)
        update += 1
        tsa.adamw_step(plan, update, 2e-3, weight_decay=0.0, seed=rounding, offset=update)
    margin = (loss.reward[:pairs] - loss.reward[pairs:]).mean()
    return rewards[0].item(), rewards[-1].item(), margin.item()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--vocab", type=int, default=4096)
    ap.add_argument("--rows", type=int, default=2048)
    a = ap.parse_args()
    first, last, margin = train(a.steps, a.vocab, a.rows)
    print("mean reward %.3f -> %.3f, preference margin %.3f" % (first, last, margin))
