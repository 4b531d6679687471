"""One speculative step after another with a drafted tree: correct, verify,
sample, commit, and train the drafter on what the target said.

A toy drafter and a toy two-layer target with random weights stand in for
trained ones; the calls are those of a serving loop:

  Corrector.correct        the drafter's block becomes a corrected chain
  (here) a tree of it      the anchor, the chain, and at each of its first
                           slots the runner-up candidate as a leaf
  TreeVerifier.attention   every target layer, over the paged cache and the tree
  TreeVerifier.sample      the target's token after every node
  TreeVerifier.commit      the accepted path's K/V into all layers' pages
  dcoco_distill_step       the drafter's loss against the target's top logits
                           along the drafted chain, and its gradient

Run:  python examples/tree_step.py
"""
from __future__ import annotations

import math
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import draft_correction_slot_gb300 as dc  # noqa: E402
import synth  # noqa: E402

V, D, LAYERS, HEADS, KV_HEADS, HEAD, PAGE, PAGES = 4096, 256, 2, 8, 2, 64, 16, 16
SLOTS, K, LEAVES = 16, 16, 4


def tree_of(chain: torch.Tensor, anchor: torch.Tensor, runner_up: torch.Tensor):
    """Tokens and parents [N, T]: node 0 the anchor, 1..B the chain, then a leaf beside each of the first nodes."""
    n, b = chain.shape
    parents = torch.cat([torch.arange(-1, b), torch.arange(LEAVES)]).to(torch.int32).cuda()
    tokens = torch.cat([anchor[:, None], chain, runner_up[:, :LEAVES]], 1)
    return tokens.contiguous(), parents.repeat(n, 1)


class Target:
    """Two attention layers and a tied output: enough for keys, values and logits that depend on the prefix."""

    def __init__(self, embed: torch.Tensor, g: torch.Generator):
        rows = (HEADS + 2 * KV_HEADS) * HEAD
        mk = lambda *s: (torch.randn(*s, generator=g, device="cuda") / math.sqrt(s[-1])).bfloat16()  # noqa: E731
        self.embed = embed
        self.qkv = [mk(rows, D) for _ in range(LAYERS)]
        self.out = [mk(D, HEADS * HEAD) for _ in range(LAYERS)]

    def forward(self, verifier, tokens, mask, cache, table, ctx_len):
        """-> logits [N, T, V], the nodes' K and V of every layer [L, N, T, KV_HEADS, HEAD]."""
        n, t = tokens.shape
        x = self.embed[tokens.long()] * 40
        k_new = torch.empty(LAYERS, n, t, KV_HEADS, HEAD, dtype=torch.bfloat16, device="cuda")
        v_new = torch.empty_like(k_new)
        for i in range(LAYERS):
            h = (torch.nn.functional.rms_norm(x.float(), (D,)).bfloat16() @ self.qkv[i].T).view(n, t, -1, HEAD)
            k_new[i], v_new[i] = h[:, :, HEADS:HEADS + KV_HEADS], h[:, :, HEADS + KV_HEADS:]
            a, _ = verifier.attention(h[:, :, :HEADS], k_new[i], v_new[i], cache[0][i], cache[1][i], table, ctx_len,
                                      tree_mask=mask)
            x = x + a.view(n, t, -1) @ self.out[i].T
        x = torch.nn.functional.rms_norm(x.float(), (D,)).bfloat16()
        return (x @ self.embed.T) * 1.2, k_new, v_new


def run(n: int = 4, steps: int = 6, seed: int = 0, verbose: bool = True) -> dict:
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    embed = (0.02 * torch.randn(V, D, generator=g, device="cuda")).bfloat16()
    weights = {k: torch.from_numpy(v) for k, v in synth.make_weights(rng, D).items()}
    corrector = dc.Corrector(weights, V, D, SLOTS, K, max_batch=n)
    verifier = dc.TreeVerifier(HEADS, KV_HEADS, HEAD, PAGE, PAGES, max_batch=n, max_tree=SLOTS + LEAVES)
    target = Target(embed, g)
    cache = [torch.zeros(LAYERS, n * PAGES, PAGE, KV_HEADS, HEAD, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = torch.randperm(n * PAGES, generator=g, device="cuda").view(n, PAGES).to(torch.int32)
    ctx_len = torch.zeros(n, dtype=torch.int32, device="cuda")
    anchor = torch.randint(0, V, (n,), generator=g, device="cuda", dtype=torch.int32)
    text = [[int(a)] for a in anchor]
    accepted, losses = [], []
    for _ in range(steps):
        # the drafter's block: hidden states around the anchor's embedding, logits around their products
        hidden = (embed[anchor.long()][:, None] * 40 + 0.7 * torch.randn(n, SLOTS, D, generator=g, device="cuda")).bfloat16()
        draft_logits = (hidden @ embed.T) * 3
        out = corrector.correct(draft_logits, hidden, embed)
        tokens, parents = tree_of(out["tokens"], anchor, out["topk_ids"][:, :, 1])
        mask = dc.tree_mask(parents)
        logits, k_new, v_new = target.forward(verifier, tokens, mask, cache, table, ctx_len)
        full = lambda x, dt=torch.float32: torch.full(tokens.shape, x, dtype=dt, device="cuda")  # noqa: E731
        sampled, _ = verifier.sample(logits, torch.rand(tokens.shape, generator=g, device="cuda"), temperature=full(0.6),
                                     top_k=full(50, torch.int32), top_p=full(0.9))
        done = verifier.commit(tokens, parents, sampled, k_new, v_new, cache[0], cache[1], table, ctx_len)
        # the drafter's slots against the target's top logits at the chain's nodes (node i predicts slot i + 1)
        top = logits[:, :SLOTS - 1].reshape(-1, V).float().topk(32, dim=1)
        student = draft_logits[:, 1:].reshape(-1, V).contiguous()
        rows = student.shape[0]
        loss, lse = (torch.empty(rows, device="cuda") for _ in range(2))
        grad = torch.empty_like(student)
        dc.dcoco_distill_step(student, top.indices.int(), top.values, torch.full((rows,), 1 / rows, device="cuda"),
                              loss=loss, lse=lse, grad=grad)
        accepted.append(done["accept_len"].float().mean().item())
        losses.append(loss.mean().item())
        for i in range(n):
            path = [int(t) for t in done["path"][i] if t >= 0][1:]
            text[i] += [int(tokens[i, t]) for t in path] + [int(done["next_token"][i])]
        anchor, ctx_len = done["next_token"], done["new_len"]
    assert corrector.status() == dc.DCOCO_OK and verifier.status() == dc.DCOCO_OK
    # the cache holds every committed token but the last anchor, in order
    assert [len(t) - 1 for t in text] == ctx_len.tolist()
    if verbose:
        print("accepted draft tokens a step:", [f"{a:.2f}" for a in accepted])
        print("distillation loss a step:    ", [f"{x:.3f}" for x in losses])
        print("tokens of request 0:", text[0])
    result = dict(text=text, accepted=accepted, losses=losses, target=target, cache=cache, table=table, ctx_len=ctx_len,
                  verifier=verifier, anchor=anchor)
    corrector.close()
    return result


if __name__ == "__main__":
    run()
