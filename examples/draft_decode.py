"""Drafted decoding of a batch behind a shared prompt, on random ternary weights:
the prompt goes through the layers once into pages that every sequence reads;
each step then appends every sequence's last token and its drafts, attends to the
prefix and the sequence's own pages, and keeps the drafts the target agrees
with plus one token drawn in their place.

    python examples/draft_decode.py [--batch 16] [--prompt 1000] [--steps 8] [--drafts 4]

The draft model is a stand-in: the target's own distribution of the step before,
flattened.  Sizes are one BitNet-shaped layer's (20 query heads over 5 key heads
of 128) with a smaller MLP and vocabulary.
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_plane_select_gb300 as t  # noqa: E402
import synth  # noqa: E402
from bit_plane_select_gb300.stack import ServedStack  # noqa: E402

K, F, D, HQ, HK, VOCAB, PAGE = 2560, 2048, 128, 20, 5, 4096, 64


def weights(seed, layers):
    out = []
    for i in range(layers):
        lw = {}
        for n, (rows, cols) in dict(q=(HQ * D, K), k=(HK * D, K), v=(HK * D, K), o=(K, HQ * D), gate=(F, K), up=(F, K),
                                    down=(K, F)).items():
            w = synth.ternary(synth.rng_for(seed, i, rows, cols), rows, cols, synth.P_ZERO)
            lw[n] = (torch.from_numpy(w), float(0.7 / np.sqrt(cols)))
        lw["attn_gain"] = lw["mlp_gain"] = torch.ones(K)
        out.append(lw)
    return out


def decode(batch=16, prompt=1000, steps=8, drafts=4, layers=2, seed=0, dev="cuda"):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    room = steps * (drafts + 1) + drafts + 1
    npre, own = -(-prompt // PAGE), -(-room // PAGE)
    pages = npre + batch * own
    ids = torch.arange(pages, dtype=torch.int32, device=dev)
    prefix, table = ids[:npre], ids[npre:].view(batch, own)

    pos = torch.arange(prompt + room, dtype=torch.float64, device=dev)[:, None]
    ang = pos * 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device=dev) / D)
    stack = ServedStack(weights(seed, layers), D, t.Rope(ang.cos().float(), ang.sin().float()), pages, PAGE)
    embed = torch.randn(VOCAB, K, generator=g, device=dev)

    # the prompt, once: one sequence whose own pages are the prefix's
    tokens = torch.randint(VOCAB, (prompt,), generator=g, device=dev)
    fill = t.KvBatch(prefix.view(1, -1), torch.tensor([prompt], dtype=torch.int32, device=dev), prompt)
    stack.step(stack.plan(fill), embed[tokens].clone())

    T = drafts + 1
    lens = torch.full((batch,), T, dtype=torch.int32, device=dev)
    who = t.KvBatch(table, lens, T, prefix_table=prefix, prefix_len=prompt)
    plan = stack.plan(who)
    draft = torch.zeros(batch, drafts, dtype=torch.int32, device=dev)
    p = torch.empty(batch, T, VOCAB, device=dev)
    q = torch.full((batch, drafts, VOCAB), 1.0 / VOCAB, device=dev)
    u, race = torch.empty(batch, drafts, device=dev), torch.empty(batch, VOCAB, device=dev)
    out = torch.empty(batch, T, dtype=torch.int32, device=dev)
    kept = torch.empty(batch, dtype=torch.int32, device=dev)
    verify = t.VerifyJob(p, q, draft, u, race, out, kept)

    last = torch.randint(VOCAB, (batch,), generator=g, device=dev, dtype=torch.int32)
    rows, text = torch.arange(batch, device=dev), []
    for _ in range(steps):
        draft.copy_(torch.multinomial(q.view(-1, VOCAB), 1, generator=g).view(batch, drafts))
        x = embed[torch.cat((last[:, None], draft), 1).long().view(-1)].clone()
        x = stack.step(plan, x)
        x = x / x.square().mean(-1, keepdim=True).sqrt()
        torch.softmax(x.view(batch, T, K) @ embed.T * 0.1, -1, out=p)
        u.uniform_(generator=g)
        race.exponential_(generator=g)
        t.trit_draft_verify(verify, stack.err)
        text.append((out.clone(), kept.clone()))
        last = out[rows, kept.long()]
        # the drafts that were not kept leave their slots to the next step's tokens
        lens += kept + 1
        q.copy_((0.7 * p[rows, kept.long()] + 0.3 / VOCAB)[:, None].expand_as(q))
    torch.cuda.synchronize()
    return text, int(stack.err.item())


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("batch", 16), ("prompt", 1000), ("steps", 8), ("drafts", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    text, err = decode(a.batch, a.prompt, a.steps, a.drafts)
    n = sum(int(k.sum()) + k.numel() for _, k in text)
    print(f"{n} tokens of {a.batch} sequences in {a.steps} steps, error flag {err}")
