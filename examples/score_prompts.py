"""Conversations behind a key/value cache held in 4 bits, on random ternary weights: every
turn's prompts go through the layers together, packed, behind the turns before; their
tokens are scored (log probability, entropy, the likeliest alternatives); then each
conversation is continued token by token with the likeliest one.

    python examples/score_prompts.py [--batch 8] [--turns 2] [--longest 600] [--steps 16]

Sizes are one BitNet-shaped layer's (20 query heads over 5 key heads of 128) with a
smaller MLP and vocabulary.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_plane_select_gb300 as t  # noqa: E402
from bit_plane_select_gb300.stack import ServedStack  # noqa: E402
from draft_decode import D, HK, HQ, K, PAGE, VOCAB, weights  # noqa: E402,F401


def talk(batch=8, turns=2, longest=600, steps=16, layers=2, seed=0, top=5, dev="cuda"):
    """(scores, text, error flag): per turn the prompts' (logprob, entropy, top tokens, top
    logprobs) and lengths, the tokens of the continuation [steps, batch]."""
    g = torch.Generator().manual_seed(seed)
    room = turns * longest + steps + 1
    cols = -(-room // PAGE)
    table = torch.randperm(batch * cols, generator=g).to(torch.int32).view(batch, cols).to(dev)
    pos = torch.arange(room, dtype=torch.float64, device=dev)[:, None]
    ang = pos * 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device=dev) / D)
    stack = ServedStack(weights(seed, layers), D, t.Rope(ang.cos().float(), ang.sin().float()), batch * cols, PAGE,
                        cache_bits=4)
    embed = torch.randn(VOCAB, K, generator=g).to(dev)
    lens = torch.zeros(batch, dtype=torch.int32, device=dev)

    def logits(x):
        return (x / x.square().mean(-1, keepdim=True).sqrt()) @ embed.T * 0.1

    def scored(rows, given):
        n = rows.shape[0]
        out = [torch.empty(n, device=dev), torch.empty(n, device=dev), torch.empty(n, top, dtype=torch.int32, device=dev),
               torch.empty(n, top, device=dev)]
        t.trit_logprobs(t.LogprobJob(rows, given, *out), stack.err)
        return out

    def starts(n):
        return torch.cat((torch.zeros(1, dtype=torch.int64), torch.tensor(n).cumsum(0))).to(dev, torch.int32)

    scores, had = [], [0] * batch
    for _ in range(turns):
        n = torch.randint(1, longest + 1, (batch,), generator=g).tolist()
        had = [a + b for a, b in zip(had, n)]
        lens.copy_(torch.tensor(had, dtype=torch.int32))
        rows = sum(n)
        tokens = torch.randint(VOCAB, (rows,), generator=g, dtype=torch.int32)
        plan = stack.prompt_plan(t.KvBatch(table, lens, longest), rows, starts(n), sum(had), starts(had))
        x = stack.step(plan, embed[tokens.long().to(dev)].clone())
        # a row scores the token behind it; a prompt's last row has none yet
        given = torch.cat((tokens[1:], torch.full((1,), -1, dtype=torch.int32)))
        given[torch.tensor(n).cumsum(0) - 1] = -1
        score = scored(logits(x), given.to(dev))
        scores.append((n, score))
        last = score[2][(torch.tensor(n).cumsum(0) - 1).to(dev), 0]

    plan = stack.plan(t.KvBatch(table, lens, 1))
    text = []
    for _ in range(steps):
        text.append(last.clone())
        lens += 1
        last = scored(logits(stack.step(plan, embed[last.long()].clone())), torch.full((batch,), -1, dtype=torch.int32,
                                                                                       device=dev))[2][:, 0]
    torch.cuda.synchronize()
    return scores, torch.stack(text) if text else torch.empty(0, batch), int(stack.err.item())


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("batch", 8), ("turns", 2), ("longest", 600), ("steps", 16)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    scores, text, err = talk(a.batch, a.turns, a.longest, a.steps)
    for i, (n, (logprob, entropy, _, _)) in enumerate(scores):
        print(f"turn {i}: {sum(n)} tokens, mean log probability {float(logprob.sum()) / max(1, sum(n) - len(n)):.3f}, "
              f"mean entropy {float(entropy.mean()):.3f}")
    print(f"{text.numel()} tokens of {a.batch} conversations, error flag {err}")
