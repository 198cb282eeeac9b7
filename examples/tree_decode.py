"""Greedy decoding with candidate trees over a paged cache, every operator of
a step where a program would use it.

One attention layer with random weights stands in for the target model, and
plain decoding's own tokens, some of them replaced, stand in for the drafter.
The batch continues one prompt, held once.  A step:

    tree_mask     the tree's mask and position indices
    kv_append     the tree's keys and values behind each sequence's cache
    attn_shared   the nodes' attention to prompt, own cache and ancestors
    verify_tree   the longest accepted path and the token after it
    kv_append     with rows = the path: its nodes at consecutive positions

At the end kv_read gives the cache back, and the tokens are compared with
those of plain decoding (a token a step, the prompt in every sequence's own
table, attn_tree): greedy tree verification changes none.

    python examples/tree_decode.py [--e4m3]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

HQ, HKV, D, PAGE, VOCAB = 8, 2, 64, 16, 512
BRANCH, DEPTH = 3, 3


class Layer:
    """The stand-in for a target model: token -> q, k, v -> attention -> logits."""

    def __init__(self, device):
        import torch

        g = torch.Generator().manual_seed(0)

        def weights(*shape):
            return torch.randn(*shape, generator=g).to(device)

        self.embed = weights(VOCAB, 256)
        self.wq, self.wk, self.wv = (weights(256, h * D) / 16 for h in (HQ, HKV, HKV))
        self.head = weights(HQ * D + 256, VOCAB) / 16
        self.slopes = torch.tensor([2.0 ** -(h + 1) for h in range(HQ)], device=device)

    def qkv(self, tokens):
        import torch

        x = self.embed[tokens.long()]
        return [(x @ w).to(torch.bfloat16).view(*tokens.shape, -1, D).contiguous()
                for w in (self.wq, self.wk, self.wv)]

    def logits(self, tokens, out):
        import torch

        x = torch.cat((out.float().flatten(2), self.embed[tokens.long()]), -1)
        return (x @ self.head).contiguous()


def tree_parents():
    """A full tree: the root, then BRANCH children a node down to DEPTH."""
    parents, level = [-1], [0]
    for _ in range(DEPTH):
        last = len(parents)
        parents += [p for p in level for _ in range(BRANCH)]
        level = list(range(last, len(parents)))
    return parents


def plain(sv, layer, prompt, first, steps, e4m3):
    """A token a step; the prompt is part of every sequence's own cache."""
    import torch

    dev, B, P = prompt.device, first.shape[0], prompt.numel()
    width = -(-(P + steps) // PAGE)
    cache = sv.new_cache(B * width, HKV, PAGE, D, dev, e4m3)
    table = torch.arange(B * width, dtype=torch.int32, device=dev).view(B, width)
    _, k, v = layer.qkv(prompt.view(1, P).expand(B, P).contiguous())
    sv.kv_append(cache, table, torch.zeros(B, dtype=torch.int32, device=dev), k, v)
    at = torch.full((B,), P, dtype=torch.int32, device=dev)
    ws = sv.new_workspace(sv.spec_attn_workspace_size(B, 1, HQ, HKV, D), dev)
    token, tokens, margins = first.view(B, 1), [], []
    for _ in range(steps):
        q, k, v = layer.qkv(token)
        sv.kv_append(cache, table, at, k, v)
        at += 1
        out = sv.attn_tree(q, cache, table, at, slopes=layer.slopes, cap=30.0, workspace=ws)
        top = layer.logits(token, out)[:, 0].topk(2)
        token = top.indices[:, :1].int().contiguous()
        tokens.append(token)
        margins.append(top.values[:, :1] - top.values[:, 1:])
    assert sv.last_error(ws) == 0
    return torch.cat(tokens, 1), torch.cat(margins, 1)


def by_trees(sv, layer, prompt, first, steps, e4m3, guess):
    """Trees in which one branch holds the tokens of `guess`.  Returns the tokens,
    the passes taken, and the cache with its tables."""
    import torch

    dev, B, P = prompt.device, first.shape[0], prompt.numel()
    parents = tree_parents()
    N = len(parents)
    own, shared = -(-(steps + DEPTH + 1 + N) // PAGE), -(-P // PAGE)
    cache = sv.new_cache(shared + B * own, HKV, PAGE, D, dev, e4m3)
    prefix = torch.arange(shared, dtype=torch.int32, device=dev)
    table = (shared + torch.arange(B * own, dtype=torch.int32, device=dev)).view(B, own)
    _, k, v = layer.qkv(prompt.view(1, P))
    sv.kv_append(cache, prefix.view(1, shared), torch.zeros(1, dtype=torch.int32, device=dev), k, v)

    tree = torch.tensor(parents, dtype=torch.int32, device=dev)
    trees = tree.view(1, N).expand(B, N).contiguous()
    ws = sv.new_workspace(sv.spec_attn_workspace_size(B, N, HQ, HKV, D), dev)
    verify_ws = sv.new_workspace(sv.spec_verify_tree_workspace_size(B, N, VOCAB), dev)
    held = torch.zeros(B, dtype=torch.int32, device=dev)  # own positions, the root's not yet
    root, done, passes = first.clone(), [[] for _ in range(B)], 0
    g = torch.Generator().manual_seed(1)
    while min(map(len, done)) < steps:
        nodes = torch.randint(VOCAB, (B, N), generator=g)
        for b in range(B):  # the drafter: one branch may be right
            node = 0
            for d in range(DEPTH):
                node = parents.index(node) + int(torch.randint(BRANCH, (), generator=g))
                if len(done[b]) + d < steps:
                    nodes[b, node] = guess[b][len(done[b]) + d]
        nodes = nodes.int().to(dev)
        nodes[:, 0] = root
        mask, _, pos = sv.tree_mask(trees, (held + P).contiguous())
        q, k, v = layer.qkv(nodes)
        sv.kv_append(cache, table, held, k, v)
        out = sv.attn_shared(q, cache, prefix, P, table, (held + N).contiguous(), mask=mask, pos=pos,
                             slopes=layer.slopes, cap=30.0, workspace=ws)
        tokens, accepted, path, _ = sv.verify_tree(layer.logits(nodes, out), tree, nodes, DEPTH,
                                                   workspace=verify_ws)
        sv.kv_append(cache, table, held, k, v, rows=path)
        held += accepted + 1
        root = tokens.gather(1, accepted.long().view(B, 1)).view(B)
        passes += 1
        for b, (n, row) in enumerate(zip(accepted.tolist(), tokens.tolist())):
            done[b] += row[:n + 1]
            if len(done[b]) >= steps:  # a finished sequence starts over: its cache stays within its pages
                held[b], root[b], done[b] = 0, first[b], done[b][:steps]
    assert sv.last_error(ws) == 0 and sv.last_error(verify_ws) == 0
    return torch.tensor([d[:steps] for d in done], dtype=torch.int32), passes, cache, prefix.view(1, shared)


def run(steps=48, batch=4, prompt_len=75, e4m3=False):
    """Decodes both ways; returns what was compared."""
    import torch

    import speculative_decoding_verification_top_gb300 as sv

    dev = torch.device("cuda")
    g = torch.Generator().manual_seed(2)
    layer = Layer(dev)
    prompt = torch.randint(VOCAB, (prompt_len,), generator=g).int().to(dev)
    first = torch.randint(VOCAB, (batch,), generator=g).int().to(dev)
    want, margins = plain(sv, layer, prompt, first, steps, e4m3)
    want, margins = want.cpu(), margins.cpu()
    wrong = torch.rand(want.shape, generator=g) < 0.25
    guess = torch.where(wrong, torch.randint(VOCAB, want.shape, generator=g).int(), want)
    got, passes, cache, prefix_table = by_trees(sv, layer, prompt, first, steps, e4m3, guess.tolist())
    # Sums differ in order between the two; a token whose lead over the next
    # is within that rounding may differ, and what follows it.
    same = torch.cumprod((got == want).int(), 1).bool()
    for b in range(batch):
        n = int(same[b].sum())
        assert n == steps or margins[b, n] < 0.05, (b, n, margins[b, n])
    # The prompt's keys, read back, are the projection's to the storage's precision.
    back, _ = sv.kv_read(cache, prefix_table, torch.zeros(1, dtype=torch.int32, device=dev), prompt_len)
    keys = layer.qkv(prompt.view(1, prompt_len))[1]
    error = float(((back - keys).abs().amax(-1) / keys.abs().amax(-1)).max())
    assert error <= (2.0 ** -4 if e4m3 else 0.0), error
    return {"tokens": batch * steps, "alike": int(same.sum()), "passes": passes, "read back": error}


if __name__ == "__main__":
    args = argparse.ArgumentParser()
    args.add_argument("--e4m3", action="store_true", help="an e4m3 cache instead of bf16")
    args = args.parse_args()
    r = run(e4m3=args.e4m3)
    print("%(tokens)d tokens in %(passes)d passes over the batch, %(alike)d like plain decoding's" % r)
