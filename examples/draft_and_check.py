"""Speculative decoding with a toy target model: the walk drafts, the tree operators check.

    python examples/draft_and_check.py [--rounds 8] [--requests 4] [--gamma 6] [--cache e4m3|e2m1|16] [--rotary]

The toy target's next-token logits are the walk's own bigram head plus a term from
one attention layer over all tokens so far, so most drafted tokens are right and
some are not.  A token's query, key and value rows depend on the token alone (one
table each), which keeps the model a few lines.  Every round, per request:

 1. two walks from the last token, one greedy and one sampled, are the two branches
    of a tree: node 0 is the last token, then gamma nodes a branch;
 2. the nodes' keys and values are written behind the context (Tree.write);
 3. every node attends to the context and its ancestors (Tree.attend);
 4. along each branch nodes are accepted while they are what the target says after
    their parent; the longer branch wins;
 5. its rows move to the front of the draft (Tree.keep), the context grows by them,
    and the target's answer after the last accepted node is the next round's node 0.

With --rotary the target norms its query and key heads and turns them by a node's depth,
and its pages come and go: Pages.grow gives a round's nodes their slots and positions,
Tree.place norms and turns them on the way into the cache (2.), and Pages.trim takes back
the pages of nodes that were not accepted.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
from serial_draft_head_gb300 import KVCache, Pages, Rotation, Tree, tree, walk  # noqa: E402

RANK = 256


class Target:
    """Random tables: the bigram head (W1, W2), a row of Q, K and V per token, and the
    attention term's way into the logits."""

    def __init__(self, vocab=4096, q_heads=8, kv_heads=2, head_dim=64, seed=0):
        g = torch.Generator("cpu").manual_seed(seed)

        def rand(*shape):
            return torch.randn(*shape, generator=g).to(torch.bfloat16).cuda()

        self.vocab, self.q_heads, self.kv_heads, self.head_dim = vocab, q_heads, kv_heads, head_dim
        self.W1, self.W2 = rand(vocab, RANK), rand(vocab, RANK) / 16
        self.q, self.k, self.v = (rand(vocab, h, head_dim) for h in (q_heads, kv_heads, kv_heads))
        self.out = rand(vocab, q_heads * head_dim) / 64

    def logits(self, tokens, attended):
        bigram = self.W1[tokens].float() @ self.W2.float().T
        return bigram + attended.reshape(len(tokens), -1).float() @ self.out.float().T


def decode(target, anchor, rounds, gamma, cache="e4m3", page=16, temperature=0.7, seed=1, rotary=False):
    """(texts, cache, pages, length): a list of tokens a request, anchor first, and the cache
    that holds the rows of all but the last of each."""
    B, T = len(anchor), 2 * gamma + 1
    H, D = target.kv_heads, target.head_dim
    most = rounds * (gamma + 1) + T
    width = -(-most // page)
    shape = (B * width, page, H, D)
    if cache == "e2m1":
        cached = KVCache.zeros(*shape, torch.uint8)
    elif cache == "e4m3":
        kv = [torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
        scales = [torch.empty(shape[:3], dtype=torch.uint8, device="cuda") for _ in range(2)]
        cached = KVCache(*kv, *scales)
    else:
        cached = KVCache(*[torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)])
    if rotary:
        pool = Pages(B * width, page, B, width)
        pages, count = pool.table, torch.full((B,), T, dtype=torch.int32, device="cuda")
        norm = torch.linspace(0.5, 1.5, D)
        rotation = Rotation(D, 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2)), norm, norm.flip(0))
    else:
        pages = torch.randperm(B * width).int().view(B, width).cuda()
    length = torch.zeros(B, dtype=torch.int32, device="cuda")
    first = torch.arange(B + 1, dtype=torch.int32, device="cuda") * T
    parent = torch.tensor(([-1] + list(range(gamma)) + [0] + list(range(gamma + 1, 2 * gamma))) * B,
                          dtype=torch.int32, device="cuda")
    mask = tree.ancestor_bits(parent, first)
    branches = torch.tensor([list(range(1, gamma + 1)), list(range(gamma + 1, T))], device="cuda")

    draft = walk.Walk(target.W1, target.W2, 2 * B, gamma)
    base = torch.zeros(2 * B, gamma, target.vocab, dtype=torch.bfloat16, device="cuda")
    heat = torch.tensor([0.0, temperature] * B, device="cuda")
    check = Tree(target.q_heads, H, D, max_requests=B, max_nodes=T)

    anchor = torch.tensor(anchor, dtype=torch.int32, device="cuda")
    texts = [[int(a)] for a in anchor]
    for r in range(rounds):
        drafted = draft.run(base, anchor.repeat_interleave(2), heat, seed + r)
        nodes = torch.cat([anchor[:, None], drafted.view(B, 2 * gamma)], 1)        # [B, T]
        flat = nodes.flatten().long()
        q = target.q[flat]
        if rotary:
            _, slot, position = pool.grow(length, count, B * T, mask=mask)
            q = check.place(cached, slot, q, target.k[flat], target.v[flat], position, rotation)
        else:
            check.write(cached, pages, length, first, target.k[flat], target.v[flat])
        attended, _ = check.attend(q, cached, pages, length, first, mask=mask)
        says = target.logits(flat, attended).argmax(-1).view(B, T)

        before = torch.cat([torch.zeros_like(branches[:, :1]), branches[:, :-1]], 1)
        right = nodes[:, branches] == says[:, before]                              # [B, 2, gamma]
        accepted = right.int().cumprod(-1).sum(-1)                                 # [B, 2]
        best = accepted.argmax(1)
        n = accepted.gather(1, best[:, None])[:, 0]
        path = torch.cat([torch.zeros(B, 1, device="cuda", dtype=torch.long), branches[best]], 1)
        kept = (n + 1).int()
        check.keep(cached, pages, length, path.int(), kept)
        anchor = says.gather(1, path.gather(1, n[:, None]))[:, 0].int()
        length = length + kept
        if rotary:
            pool.trim(length)
        for b in range(B):
            texts[b] += [int(nodes[b, path[b, i + 1]]) for i in range(int(n[b]))] + [int(anchor[b])]
    for status in (draft.status(), check.status()) + ((pool.status(),) if rotary else ()):
        if status != 0:
            raise RuntimeError(walk.dspark_walk_strerror(status))
    draft.close()
    check.close()
    return texts, cached, pages, length


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--rounds", type=int, default=8)
    p.add_argument("--requests", type=int, default=4)
    p.add_argument("--gamma", type=int, default=6)
    p.add_argument("--cache", choices=("e4m3", "e2m1", "16"), default="e4m3")
    p.add_argument("--rotary", action="store_true")
    a = p.parse_args()
    target = Target()
    texts, _, _, length = decode(target, list(range(1, a.requests + 1)), a.rounds, a.gamma, a.cache, rotary=a.rotary)
    for b, t in enumerate(texts):
        print("request %d: %d tokens in %d rounds: %s" % (b, len(t) - 1, a.rounds, t))
    print("tokens a round and request: %.2f" % (length.float().mean().item() / a.rounds))


if __name__ == "__main__":
    main()
