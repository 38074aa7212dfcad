"""One attention layer's decode step over drafted token trees, with the weights
pruned, a quantised paged cache and an adapter per sequence:

    qkv  = spmm_f16_lora(W_qkv, x)          projection, each column its adapter
    kv_append(cache, k, v, slots)           the drafted tokens enter the cache
    a    = attention_tree(q, cache, ...)    every drafted token over its branch
    y    = spmm_f16_lora(W_o, a)            output projection

and, once a branch is accepted, kv_gather and kv_append move its rows to where
the sequence goes on. The step is captured in a graph and replayed; the result
is compared with the same formulas in 64 bits.

    python examples/decode_step.py [--hidden 4096 --heads 32 --kv-heads 8 ...]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_unstructured_sparse_amd as bsp  # noqa: E402

KINDS = {"fp16": bsp.FP16, "int8": bsp.INT8, "int4": bsp.INT4}


def pruned(rng, M, K, density):
    """float16 M x K with the smallest entries of a normal draw set to zero."""
    W = (rng.standard_normal((M, K), dtype=np.float32) / np.sqrt(K * density)).astype(np.float16)
    W[np.abs(W) < np.quantile(np.abs(W[:64].astype(np.float32)), 1.0 - density)] = 0
    return W


def draft_tree(rng, T):
    """Parents of T drafted tokens (the first is the root) and, for each, the
    word of the tokens it sees: itself and its ancestors."""
    parent = [-1] + [int(rng.integers(0, i)) for i in range(1, T)]
    words = []
    for i in range(T):
        words.append((words[parent[i]] if i else 0) | (1 << i))
    return parent, words


class Layer:
    """Weights, adapters, cache and workspaces of the layer: made once."""

    def __init__(self, o, dev, rng):
        self.o, self.dev, d = o, dev, o.head_dim
        self.columns = o.batch * o.tree
        if self.columns > bsp.MAX_N:
            raise SystemExit(f"batch * tree is at most {bsp.MAX_N}")
        width = (o.heads + 2 * o.kv_heads) * d
        self.Wqkv, self.Wo = pruned(rng, width, o.hidden, o.density), pruned(rng, o.hidden, o.heads * d, o.density)
        self.qkv, self.out = bsp.encode(self.Wqkv).to_device(dev), bsp.encode(self.Wo).to_device(dev)
        self.lora_qkv, self.lora_out = self.adapters(rng, width, o.hidden), self.adapters(rng, o.hidden, o.heads * d)
        self.ws_qkv = bsp.new_lora_workspace(self.qkv, self.columns, self.lora_qkv, device=dev)
        self.ws_out = bsp.new_lora_workspace(self.out, self.columns, self.lora_out, device=dev)
        self.width = -(-(o.context + o.tree) // o.page)                 # pages of a sequence
        self.cache = bsp.new_kv_cache(KINDS[o.cache], o.batch * self.width, o.kv_heads, o.page, d, dev)
        self.table = torch.from_numpy(rng.permutation(o.batch * self.width).astype(np.int32)).to(dev)
        self.table = self.table.view(o.batch, self.width)
        self.ws_att = bsp.new_attention_workspace(self.cache, o.batch, o.tree, o.heads, self.width, dev)

    def adapters(self, rng, M, K):
        n, R = self.o.adapters, self.o.rank
        A = (rng.standard_normal((n, R, K)) / np.sqrt(K)).astype(np.float16)
        B = (0.2 * rng.standard_normal((n, M, R))).astype(np.float16)
        to = lambda x: torch.from_numpy(x).to(self.dev)
        return bsp.LoraAdapters(to(A), to(B), to(np.full(n, 0.5, np.float32)))

    def slots(self, b, first, n):
        """Cache slots of tokens first .. first + n - 1 of sequence b."""
        at = torch.arange(first, first + n, device=self.dev)
        return self.table[b, at // self.o.page].long() * self.o.page + at % self.o.page

    def step(self, x, index, slots, lens, q_start, words):
        o = self.o
        qkv = bsp.spmm_f16_lora(self.qkv, x, self.lora_qkv, index, workspace=self.ws_qkv)
        q, k, v = qkv.view(self.columns, -1, o.head_dim).split([o.heads, o.kv_heads, o.kv_heads], dim=1)
        bsp.kv_append(self.cache, k, v, slots)
        a = bsp.attention_tree(q, self.cache, self.table, lens, q_start, o.tree, tree_mask=words,
                               workspace=self.ws_att)
        return bsp.spmm_f16_lora(self.out, a.view(self.columns, -1), self.lora_out, index, workspace=self.ws_out)

    def accept(self, b, branch):
        """Move the rows of an accepted branch (drafted tokens, root first) to
        the places behind the context."""
        o = self.o
        at = torch.tensor(branch, device=self.dev)
        rows = bsp.kv_gather(self.cache, self.slots(b, o.context, o.tree)[at].contiguous())
        bsp.kv_append(self.cache, *rows, self.slots(b, o.context, len(branch)))
        return rows


def project(W, X, ad, index):
    """The projection with adapters in float64, rounded to float16 as stored."""
    Y = X @ W.astype(np.float64).T
    A, B = ad.A.cpu().numpy().astype(np.float64), ad.B.cpu().numpy().astype(np.float64)
    for n, a in enumerate(index):
        if a >= 0:
            Y[n] += float(ad.scale[a]) * (B[a] @ (A[a] @ X[n]))
    return Y.astype(np.float16).astype(np.float64)


def reference(layer, x, index, words):
    """The step in float64 over the cached rows as kv_gather returns them."""
    o, T, d = layer.o, layer.o.tree, layer.o.head_dim
    qkv = project(layer.Wqkv, x, layer.lora_qkv, index).reshape(layer.columns, -1, d)
    a = np.zeros((layer.columns, o.heads, d))
    for b in range(o.batch):
        K, V = bsp.kv_gather(layer.cache, layer.slots(b, 0, o.context + T))
        K, V = K.cpu().numpy().astype(np.float64), V.cpu().numpy().astype(np.float64)
        seen = np.ones((T, o.context + T), bool)
        for i in range(T):
            seen[i, o.context:] = [(int(words[b * T + i]) >> j) & 1 for j in range(T)]
        for h in range(o.heads):
            g = h // (o.heads // o.kv_heads)
            s = np.where(seen, qkv[b * T:(b + 1) * T, h] @ K[:, g].T * d ** -0.5, -np.inf)
            p = np.exp(s - s.max(1, keepdims=True))
            a[b * T:(b + 1) * T, h] = p / p.sum(1, keepdims=True) @ V[:, g]
    a = a.astype(np.float16).astype(np.float64)
    return project(layer.Wo, a.reshape(layer.columns, -1), layer.lora_out, index)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("hidden", 4096), ("heads", 32), ("kv-heads", 8), ("head-dim", 128), ("batch", 4),
                        ("tree", 8), ("context", 4096), ("page", 32), ("adapters", 3), ("rank", 16), ("steps", 200)):
        p.add_argument("--" + name, type=int, default=value)
    p.add_argument("--density", type=float, default=0.5)
    p.add_argument("--cache", choices=list(KINDS), default="int8")
    o = p.parse_args(argv)
    rng, dev = np.random.default_rng(0), torch.device("cuda:0")
    layer = Layer(o, dev, rng)
    i32 = dict(dtype=torch.int32, device=dev)

    # a prompt's keys and values, then the drafted tokens of every sequence
    for b in range(o.batch):
        k, v = (torch.randn(o.context, o.kv_heads, o.head_dim, device=dev).half() for _ in range(2))
        bsp.kv_append(layer.cache, k, v, layer.slots(b, 0, o.context))
    trees = [draft_tree(rng, o.tree) for _ in range(o.batch)]
    words = np.array([w for _, ws in trees for w in ws], np.uint64).view(np.int64)
    index = np.repeat(np.arange(o.batch) % (o.adapters + 1) - 1, o.tree)      # the first has no adapter
    x = rng.standard_normal((layer.columns, o.hidden)).astype(np.float16)
    args = (torch.from_numpy(x).to(dev), torch.tensor(index, **i32),
            torch.cat([layer.slots(b, o.context, o.tree) for b in range(o.batch)]),
            torch.full((o.batch,), o.context + o.tree, **i32),
            torch.arange(0, layer.columns + 1, o.tree, **i32), torch.from_numpy(words).to(dev))

    y = layer.step(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yg = layer.step(*args)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        if not torch.equal(y, yg):
            raise SystemExit("a replay differs from the eager step")
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(o.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()

    want = reference(layer, x.astype(np.float64), index, words)
    error = float(np.abs(y.cpu().numpy() - want).max() / np.abs(want).max())
    print(f"{o.batch} sequences x {o.tree} drafted tokens, {o.context} cached ({o.cache}): "
          f"{begin.elapsed_time(end) * 1e3 / o.steps:.1f} us a step, error {error:.1e} of the largest value")

    branch, leaf = [], o.tree - 1                                             # the last token's branch is accepted
    while leaf >= 0:
        branch, leaf = [leaf] + branch, trees[0][0][leaf]
    moved = layer.accept(0, branch)
    again = bsp.kv_gather(layer.cache, layer.slots(0, o.context, len(branch)))
    step = max(float((m.float() - g.float()).abs().max()) for m, g in zip(moved, again))
    print(f"branch {branch} accepted: {len(branch)} rows moved, read back within {step:.1e}")
    return error, step


if __name__ == "__main__":
    main()
