"""Serving with drafted trees over a paged cache, from text to text.

A batch of prompts is encoded on the GPU; its ids and offsets stay there and
place the prompts in a paged key/value cache (`kv_plan`), whose rows are
stored by `KVCache.append` and read by `KVCache.attend`. Then each step drafts a
small tree of continuations per request, verifies it in one pass (ancestor
masks, positions by depth), keeps the path that the model itself would have
taken, and streams its bytes out. The model is a stand-in: one attention layer
with random weights.

    python examples/draft_tree_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import byte_level_bpe_gb300 as tk  # noqa: E402

Q_HEADS, KV_HEADS, DIM, BLOCK = 8, 2, 64, 16
# root, its two candidates, one more token under each
PARENTS = [-1, 0, 0, 1, 2]


class Model:
    """One attention layer over a paged cache, and the cheap draft without it."""

    def __init__(self, vocabulary, n_blocks, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        width = Q_HEADS * DIM

        def weights(*shape):
            return torch.randn(*shape, generator=gen, device="cuda").mul_(shape[0] ** -0.5).bfloat16()

        self.embedding = torch.randn(vocabulary, width, generator=gen, device="cuda").bfloat16()
        self.qkv = weights(width, (Q_HEADS + 2 * KV_HEADS) * DIM)
        self.out = weights(width, width)
        self.head = weights(width, vocabulary)
        self.gains = torch.rand(2, DIM, generator=gen, device="cuda") + 0.5
        self.rope = tk.rope_table(4096, DIM)
        pool = torch.empty(2, n_blocks, KV_HEADS, BLOCK, DIM, dtype=torch.bfloat16, device="cuda")
        self.cache, self.workspace = tk.KVCache(pool[0], pool[1]), tk.KVWorkspace()

    def logits(self, ids, offsets, plan, table, max_new):
        x = self.embedding[ids.long()]
        q = self.cache.append(x @ self.qkv, plan.positions, plan.slots, Q_HEADS, q_gain=self.gains[0],
                              k_gain=self.gains[1], rope=self.rope)
        o = self.cache.attend(q, offsets, plan.lengths, table, self.workspace, masks=plan.masks, max_new=max_new)
        return (x + 0.5 * (o.flatten(1) @ self.out)) @ self.head

    def draft(self, ids, k):
        return (self.embedding[ids.long()] @ self.head).topk(k, -1).indices.int()


class Batch:
    """The device state of a batch of requests: block tables, cached lengths, the free list's cursor."""

    def __init__(self, model, requests, width, n_blocks):
        self.model = model
        self.table = torch.zeros(requests, width, dtype=torch.int32, device="cuda")
        self.lengths = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.free = torch.arange(n_blocks, dtype=torch.int32, device="cuda")
        self.cursor = torch.zeros(1, dtype=torch.int64, device="cuda")

    def run(self, ids, offsets, max_new, parents=None, keep=True):
        """The logits of new tokens. keep=False leaves lengths and cursor as they were: the next
        call takes the same blocks again and overwrites the places."""
        plan = tk.kv_plan(offsets, self.lengths, self.table, self.free, BLOCK, ids.numel(), parents=parents,
                          cursor=self.cursor)
        logits = self.model.logits(ids, offsets, plan, self.table, max_new)
        if keep:
            self.lengths, self.cursor = plan.lengths, plan.info[:1]
        return logits


def _offsets(counts):
    return torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), device="cuda")


def prefill(model, tokenizer, prompts, width, n_blocks):
    """Encodes and stores the prompts, each a text or a list of (text, allow_special) segments; returns the batch
    and each request's first new token."""
    prompts = [[(p, False)] if isinstance(p, str) else p for p in prompts]
    ids, offsets = tokenizer.encode_segments([s for p in prompts for s in p])
    # the encode's offsets are its segments'; a request begins with its first one
    offsets = offsets[_offsets([len(p) for p in prompts])]
    batch = Batch(model, len(prompts), width, n_blocks)
    logits = batch.run(ids, offsets, ids.numel())
    return batch, logits[offsets[1:] - 1].argmax(-1).int()


def generate_drafted(batch, first, steps):
    """steps verification passes; returns the tokens of each request and the drafted ones kept."""
    model, R = batch.model, first.numel()
    parents = torch.tensor(PARENTS * R, dtype=torch.int32, device="cuda")
    pending = [[t] for t in first.tolist()]  # accepted, not yet stored
    done, kept = [[] for _ in range(R)], 0
    for _ in range(steps):
        # what was accepted goes into the cache as a chain; its last token is the tree's root
        if any(len(p) > 1 for p in pending):
            chain = [t for p in pending for t in p[:-1]]
            batch.run(torch.tensor(chain, dtype=torch.int32, device="cuda"), _offsets([len(p) - 1 for p in pending]),
                      max(len(p) - 1 for p in pending))
        root = torch.tensor([p[-1] for p in pending], dtype=torch.int32, device="cuda")
        pair = model.draft(root, 2)                    # [R, 2]
        under = model.draft(pair.flatten(), 1).view(R, 2)
        tree = torch.cat([root[:, None], pair, under], 1).flatten().contiguous()
        n = len(PARENTS)
        logits = batch.run(tree, torch.arange(0, (R + 1) * n, n, device="cuda"), n, parents=parents, keep=False)
        said, tree = logits.argmax(-1).view(R, n).tolist(), tree.view(R, n).tolist()
        for r in range(R):
            path, at = [tree[r][0]], 0
            while True:  # on to the child that holds what the model says
                nxt = next((c for c in range(n) if PARENTS[c] == at and tree[r][c] == said[r][at]), None)
                if nxt is None:
                    break
                path.append(tree[r][nxt])
                at = nxt
            kept += len(path) - 1
            done[r] += path
            pending[r] = path + [said[r][at]]
    return done, kept


def generate_plainly(batch, first, steps):
    """The same tokens one at a time."""
    R = first.numel()
    offsets = torch.arange(R + 1, device="cuda")
    done = [[] for _ in range(R)]
    for _ in range(steps):
        for r, t in enumerate(first.tolist()):
            done[r].append(t)
        first = batch.run(first, offsets, 1).argmax(-1).int()
    return done


def main():
    import workloads
    tokenizer = tk.Tokenizer(workloads.full_table(), workloads.SPECIALS)
    prompts = ["Shard the request over four ranks.", "def add(a, b):\n    return a + b\n", "1, 2, 3,", "x" * 300,
               [("What is a page?", False), ("<|endoftext|>", True), ("A block of", False)]]
    model = Model(tk.native.load().tk_max_id(tokenizer.handle) + 1, 256)
    batch, first = prefill(model, tokenizer, prompts, 40, 256)
    done, kept = generate_drafted(batch, first, 8)
    model.workspace.status()
    tokens = sum(len(d) for d in done)
    print(f"{tokens} tokens in 8 passes over {len(prompts)} requests, {kept} of them drafted")
    for prompt, ids in zip(prompts, done):
        stream = tokenizer.stream_decoder()
        text = prompt if isinstance(prompt, str) else "".join(t for t, _ in prompt)
        print(repr(text[:20]), "->", (stream.feed(ids) + stream.finish()).decode(errors="replace"))


if __name__ == "__main__":
    main()
