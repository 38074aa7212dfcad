"""The operators from a layer's hidden states to the cache, as workloads to time.

Four operators that a served step needs around the sparse projections, the
paged cache and the attention over it:

* ``pages``: the block tables, slots and positions of a step, made on the GPU
  from how many tokens each sequence keeps and appends;
* ``heads``: queries and keys normed head by head and rotated to their
  positions, the keys and values written to the cache in the same pass;
* ``tokens``: hidden states (with their residual sum and norm) quantised token
  by token to 8 or 4 bits, and read back;
* ``product``: 8-bit weights times 8-bit tokens with scales for each channel
  and token, for the layers left dense and for prompts.

With ``own`` false, ``run`` computes each of them in plain torch operations
in 32 bits (angles and codes in 64), rounded once at the end; with ``own`` true
it calls the library. ``exact`` gives the same outputs from the definitions in
64 bits.

pages. A sequence holds ``held`` pages of its row of the block table and
``lens`` tokens in them. A step keeps the first ``keep`` of them and appends
``new``; it then needs ceil((keep + new) / page) pages. Pages given back are
numbered sequence by sequence, pages taken likewise; the n-th page taken is the
n-th given back, or past those the free list's last, last but one, ... What
is given back and not taken goes onto the list's end, the first given back last.
A sequence whose pages do not all fit any more (nor any later one that takes
pages), whose rows pass the rows of the call or whose pages pass its row of the
table waits: it keeps its pages, its rows get slot -1 and its length for the
attention is 0. Token t of sequence b is in slot table[b][t / page] * page +
t % page. Position: keep + i for the i-th new token, with a mask of drafted
tokens (up to 64 of them) keep + the number of its ancestors.

heads. y = x / sqrt(mean(x^2) + eps) * weight over a head's channels, then pairs
(y1, y2) of the first ``rot`` channels become (y1 cos - y2 sin, y2 cos + y1 sin) at
the angle position * base^(-2 i / rot); the pairs are (i, i + rot / 2), or (2 i, 2 i
+ 1) where interleaved. Keys are rounded to float16 and then quantised as the
cache does: s = (max - min) / (2^bits - 1) rounded up to bfloat16, o the row's
minimum, u = round-half-even((x - o) / s), read back as s * u + o.

tokens. h = float16(x + residual); y = h * weight; with m = max |y| and L = 127 or
7, the codes are round-half-even(y * L / m) and the scale is m / sqrt(mean(h^2) +
eps) / L. Without a norm, y = x and the scale is m / L.

product. Y[n][m] = (sum_k W[m][k] X[n][k]) * scale_w[m] * scale_x[n].
"""
import math
import random

import numpy as np
import torch

own = False

KV_LEVELS = {"int8": 255, "int4": 15}
LEVELS = {"int8": 127, "int4": 7}
EPS = 1e-5
DEV = "cuda"


# ---------------------------------------------------------------- the cases

def _pages(name, B, page, ctx, most, prompt, short, tree):
    """B sequences of up to ctx tokens: most of them append up to `most` drafted tokens, every `prompt`-th one is
    replaced by a prompt or ends (0: none); short: the pool runs out before the last ones."""
    return dict(name=name, op="pages", B=B, page=page, ctx=ctx, most=most, prompt=prompt, short=short, tree=tree)


def _heads(name, n, hq, hkv, dim, rot, inter, norm, kind, page, ctx):
    """n tokens' heads; kind: the cache that takes the keys and values, or None for normed and rotated keys alone."""
    return dict(name=name, op="heads", n=n, hq=hq, hkv=hkv, dim=dim, rot=rot, inter=inter, norm=norm, kind=kind,
                page=page, ctx=ctx)


def _tokens(name, n, K, kind, norm, residual):
    """n tokens of K channels to codes of `kind`, and back."""
    return dict(name=name, op="tokens", n=n, K=K, kind=kind, norm=norm, residual=residual)


def _product(name, n, M, K):
    """n tokens through a dense M x K layer."""
    return dict(name=name, op="product", n=n, M=M, K=K)


def listed():
    return [
        # plain batched decoding: 32 requests append one token each, which is then taken back
        _pages("pages_step", 32, 64, 4096, 1, 0, False, False),
        # speculative decoding at a large batch: trees of up to 61 tokens, all rejected by the second call
        _pages("pages_trees", 256, 32, 8192, 61, 0, False, True),
        # a batch in which every 8th request ends or gives way to a prompt, and the pool is nearly full
        _pages("pages_prompts", 512, 16, 4096, 16, 8, True, False),
        # one new token, 32 heads of the 12288 x 4096 QKV projection, int8 cache
        _heads("heads_one_token", 1, 32, 32, 128, 128, False, True, "int8", 16, 500),
        # 8 trees of up to 16 drafted tokens, 64 query and 8 kv heads of the 10240 x 8192 fused QKV, int4 cache
        _heads("heads_trees_int4", 105, 64, 8, 128, 128, False, True, "int4", 32, 131072),
        # a batch of prompts, 32 heads, half of each head rotated in neighbouring pairs, keys kept as float16
        _heads("heads_prompts", 8192, 32, 32, 128, 64, True, False, None, 16, 8192),
        # the step of one request: residual sum, norm and int4 activations for the sparse QKV projection
        _tokens("tokens_one_int4", 1, 4096, "int4", True, True),
        # the FFN's inner activations of 32 requests to int8, ahead of the down projection
        _tokens("tokens_step_int8", 32, 11008, "int8", False, False),
        # a batch of prompts enters a layer: residual sum, norm, int8
        _tokens("tokens_prompts_int8", 8191, 8192, "int8", True, True),
        # one request on a dense 4096 x 4096 output projection
        _product("product_one", 1, 4096, 4096),
        # a step of 32 requests through the FFN's down projection
        _product("product_step", 32, 4096, 11008),
        # a batch of prompts through the QKV projection
        _product("product_prompts", 8192, 12288, 4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["pages", "heads", "tokens", "product", "product"])
    if op == "pages":
        # no more table entries than 512 sequences of 4096 tokens in pages of 16, four times over
        B, page = _log(rng, 1, 1024), rng.choice([16, 32, 64, 128])
        c = _pages(None, B, page, _log(rng, 1, min(131072, 524288 * page // B)), _log(rng, 1, 64),
                   rng.choice([0, 0, 2, 5, 8]), rng.random() < 0.3, rng.random() < 0.5)
    elif op == "heads":
        dim = rng.choice([64, 128, 128, 256])
        hkv = rng.choice([1, 2, 4, 8, 32])
        hq = hkv * (1 if hkv == 32 else rng.choice([1, 2, 3, 4, 5, 8]))
        n = _log(rng, 1, 8192 * 64 * 128 // ((hq + hkv) * dim))
        c = _heads(None, n, hq, hkv, dim, rng.choice([dim, dim, dim // 2, dim // 4]), rng.random() < 0.3,
                   rng.random() < 0.7, rng.choice([None, "fp16", "int8", "int4"]), rng.choice([16, 32, 64, 128]),
                   _log(rng, n, max(n, 1 << 20)))
    elif op == "tokens":
        K = _log(rng, 64, 16384)
        norm = rng.random() < 0.6
        c = _tokens(None, _log(rng, 1, 8191 * 8192 // K), K, rng.choice(["int8", "int4"]), norm,
                    norm and rng.random() < 0.6)
    else:
        K = _log(rng, 64, 11008)
        M = _log(rng, 64, 12288)
        c = _product(None, _log(rng, 1, min(8192, 8192 * 12288 * 4096 // (M * K))), M, K)
    del c["name"]
    return c


def _plan(case):
    """What is fixed by the case and not by the seed: a generator for lengths."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _steps(case):
    """(tokens held, kept, appended) of each sequence."""
    p, out = _plan(case), []
    for b in range(case["B"]):
        n = case["ctx"] if b == 0 else p.randint(case["ctx"] // 8, case["ctx"])
        if case["prompt"] and b % case["prompt"] == case["prompt"] - 1:
            out.append((n, 0, p.choice([0, p.randint(1, max(1, case["ctx"] // 4))])))
        else:
            out.append((n, n, case["most"] if b == 0 else p.randint(1, case["most"])))
    return out


def _pool(case):
    """(width of the table, free pages at the start)."""
    steps, page = _steps(case), case["page"]
    grow = sum(max(0, -(-(k + m) // page) - -(-n // page)) for n, k, m in steps)
    back = sum(max(0, -(-n // page) - -(-(k + m) // page)) for n, k, m in steps)
    free = max(0, (grow - back) * 3 // 4) if case["short"] else grow + 64
    return max(-(-max(n, k + m) // page) for n, k, m in steps), free


def _row_bytes(kind, dim):
    return {"fp16": 2 * dim, "int8": dim + 4, "int4": dim // 2 + 4}[kind]


def work(case):
    op = case["op"]
    if op == "pages":
        steps, page = _steps(case), case["page"]
        rows = sum(m for _, _, m in steps) + sum(n - k for n, k, _ in steps)
        moved = sum(abs(-(-(k + m) // page) - -(-n // page)) for n, k, m in steps)
        # rows: slot, position, sequence, and the drafted tokens' masks; sequences: lens and held read and written,
        # keep and new read, q_start and kv_lens written, by both calls; a page moved: its old place and its new one
        return dict(bytes=rows * (16 + (8 if case["tree"] else 0)) + 2 * case["B"] * 8 * 4 + 2 * 8 * moved,
                    flops=4 * rows)
    if op == "heads":
        n, hq, hkv, dim = (case[k] for k in ("n", "hq", "hkv", "dim"))
        data = 2 * 2 * n * hq * dim + 4 * n
        if case["kind"] is None:
            data += 2 * 2 * n * hkv * dim
        else:      # keys and values read and written, and read back
            data += n * (2 * 2 * hkv * dim * 2 + 2 * 2 * hkv * _row_bytes(case["kind"], dim) + 8)
        return dict(bytes=data, flops=10 * n * (hq + hkv) * dim)
    if op == "tokens":
        n, K = case["n"], case["K"]
        codes = K if case["kind"] == "int8" else (K + 1) // 2
        # read (with the residual) and written (with the sum), the codes written and read, the values written
        return dict(bytes=n * (K * (2 * (3 if case["residual"] else 1) + 2) + 2 * codes + 8), flops=8 * n * K)
    n, M, K = case["n"], case["M"], case["K"]
    return dict(bytes=M * K + n * K + 2 * n * M + 4 * (M + n), flops=2 * n * M * K)


# ---------------------------------------------------------------- inputs

def _gen(seed, *salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(random.Random(repr((seed,) + salt)).getrandbits(48))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _tree_words(p, steps, rows):
    """A word of ancestors for each row: the trees of the sequences' drafted tokens."""
    words = np.zeros(rows, np.uint64)
    at = 0
    for _, _, m in steps:
        row = []
        for i in range(m):
            parent = p.randint(-1, i - 1) if i else -1
            row.append((row[parent] if parent >= 0 else 0) | (1 << i if i < 64 else 0))
        words[at:at + m] = [w & (2 ** 64 - 1) for w in row]
        at += m
    return words.view(np.int64)


def _pages_inputs(case, seed):
    steps, page = _steps(case), case["page"]
    width, free = _pool(case)
    g = _gen(seed, "pages")
    held = [-(-n // page) for n, _, _ in steps]
    order = torch.randperm(sum(held) + free, generator=g, device=DEV).to(torch.int32)
    first = _i32(np.cumsum([0] + held[:-1]).tolist())
    p = torch.arange(width, device=DEV)
    inside = p[None, :] < _i32(held)[:, None]
    table = torch.where(inside, order[(first[:, None] + p).clamp(max=order.numel() - 1).long()], 0)
    pool = torch.full((order.numel(),), -1, dtype=torch.int32, device=DEV)
    pool[:free] = order[sum(held):]
    # the rows of a call are a multiple of 8, as a captured step's are: the last ones belong to no sequence
    rows = [-(-sum(m for _, _, m in steps) // 8) * 8, -(-sum(n - k for n, k, _ in steps) // 8) * 8]
    words = _tree_words(random.Random(repr((seed, "tree"))), steps, rows[0]) if case["tree"] else None
    return dict(page=page, table=table.contiguous(), lens=_i32([n for n, _, _ in steps]), held=_i32(held),
                free=torch.cat([_i32([free, 0]), pool]), keep=_i32([k for _, k, _ in steps]),
                new=_i32([m for _, _, m in steps]), back=_i32([n - k for n, k, _ in steps]), rows=rows,
                mask=torch.from_numpy(words).to(DEV) if case["tree"] else None,
                out=[_step_out(r, len(steps)) for r in rows])


def _step_out(rows, B):
    """slots, positions, sequences, q_start and kv_lens of a call."""
    i32 = torch.int32
    return [torch.zeros(rows, dtype=torch.int64, device=DEV), torch.zeros(rows, dtype=i32, device=DEV),
            torch.zeros(rows, dtype=i32, device=DEV), torch.zeros(B + 1, dtype=i32, device=DEV),
            torch.zeros(B, dtype=i32, device=DEV)]


def _heads_inputs(case, seed):
    n, hq, hkv, dim, page = (case[k] for k in ("n", "hq", "hkv", "dim", "page"))
    g = _gen(seed, "heads")
    # the fused projection's output: strong channels in the keys and queries, smaller values
    x = _normal(g, n, hq + 2 * hkv, dim)
    channel = _normal(g, 1, hq + hkv, dim)
    x[:, :hq + hkv] = x[:, :hq + hkv] * torch.where(channel.abs() > 2.0, 4.0, 1.0) + 0.5 * channel
    x[:, hq + hkv:] *= 0.5
    x = x.to(torch.float16)
    weight = [(1.0 + 0.2 * _normal(g, dim)).to(torch.float16) if case["norm"] else None for _ in "qk"]
    first = torch.randint(0, case["ctx"] - n + 1, (1,), generator=g, device=DEV)
    s = dict(Q=x[:, :hq], K=x[:, hq:hq + hkv], V=x[:, hq + hkv:], wq=weight[0], wk=weight[1], rot=case["rot"],
             inter=case["inter"], kind=case["kind"], page=page,
             positions=(first + torch.arange(n, device=DEV)).to(torch.int32))
    if case["kind"] is not None:
        pages = -(-n // page) + 1
        order = torch.randperm(pages, generator=g, device=DEV)
        t = torch.arange(n, device=DEV)
        s["slots"] = order[t // page] * page + t % page
        half = case["kind"] == "fp16"
        row = dim if half or case["kind"] == "int8" else dim // 2
        for name in ("ck", "cv"):
            s[name] = torch.zeros((pages, hkv, page, row), dtype=torch.float16 if half else torch.uint8, device=DEV)
            s[name + "s"] = None if half else torch.zeros((pages, hkv, page), dtype=torch.int32, device=DEV)
    return s


def _tokens_inputs(case, seed):
    n, K = case["n"], case["K"]
    g = _gen(seed, "tokens")
    channel = _normal(g, 1, K)                   # a few channels are far larger than the rest
    x = _normal(g, n, K) * torch.where(channel.abs() > 3.0, 20.0, 1.0)
    s = dict(X=x.to(torch.float16), K=K, kind=case["kind"], weight=None, residual=None)
    if case["norm"]:
        s["weight"] = (1.0 + 0.2 * _normal(g, K)).to(torch.float16)
    if case["residual"]:
        s["residual"] = (2.0 * _normal(g, n, K)).to(torch.float16)
    return s


def _product_inputs(case, seed):
    n, M, K = case["n"], case["M"], case["K"]
    g = _gen(seed, "product")
    W = torch.randint(-127, 128, (M, K), generator=g, device=DEV, dtype=torch.int8)
    # tokens as they come from the quantisation: rows of whole 16 bytes, the largest value 127
    pitch = -(-K // 16) * 16
    X = torch.zeros((n, pitch), dtype=torch.int8, device=DEV)
    x = _normal(g, n, K)
    top = x.abs().amax(-1, keepdim=True)
    X[:, :K] = torch.round(x / top * 127.0).to(torch.int8)
    return dict(W=W, X=X[:, :K], scale_w=0.0002 * (0.5 + torch.rand(M, generator=g, device=DEV)),
                scale_x=(top / 127.0)[:, 0].contiguous())


def prepare(case, seed):
    op = case["op"]
    s = {"pages": _pages_inputs, "heads": _heads_inputs, "tokens": _tokens_inputs, "product": _product_inputs}[op](
        case, seed)
    s["op"] = op
    if own:
        import bit_unstructured_sparse_amd as bsp
        if op == "pages":
            s["pages"] = bsp.KVPages(s["table"], s["lens"], s["held"], s["free"], s["page"])
            s["out"] = [bsp.KVStep(*o) for o in s["out"]]
        elif op == "heads":
            s["freq"] = bsp.rope_frequencies(s["rot"], 10000.0, device=DEV)
            if s["kind"] is not None:
                kind = {"fp16": bsp.FP16, "int8": bsp.INT8, "int4": bsp.INT4}[s["kind"]]
                s["cache"] = bsp.KVCache(kind, s["ck"], s["cv"], s["cks"], s["cvs"])
        elif op == "product":
            s["W"] = bsp.encode_int8(s["W"].cpu().numpy(), s["scale_w"].cpu().numpy()).to_device(DEV)
            s["workspace"] = bsp.new_gemm_workspace(s["W"], case["n"], device=DEV)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if op == "pages":
        # the step appends; the second call takes back what the first appended and restores what it gave away
        step = _pages_own if own else _pages_plain
        a = step(s, s["keep"], s["new"], 0, s["mask"])
        b = step(s, s["keep"], s["back"], 1, None)
        return a, b, s["table"], s["lens"], s["held"], s["free"]
    if op == "heads":
        return _heads_own(s) if own else _heads_plain(s)
    if op == "tokens":
        return _tokens_own(s) if own else _tokens_plain(s)
    if own:
        import bit_unstructured_sparse_amd as bsp
        return bsp.gemm_w8a8(s["W"], s["X"], s["scale_x"], workspace=s["workspace"])
    y = s["X"].float() @ s["W"].float().t()
    return (y * s["scale_w"][None, :] * s["scale_x"][:, None]).to(torch.float16)


def _pages_own(s, keep, new, call, mask):
    import bit_unstructured_sparse_amd as bsp
    return tuple(bsp.kv_step(s["pages"], keep, new, s["rows"][call], tree_mask=mask, out=s["out"][call]))


def _heads_own(s):
    import bit_unstructured_sparse_amd as bsp
    args = dict(q_weight=s["wq"], k_weight=s["wk"], eps=EPS, interleaved=s["inter"])
    if s["kind"] is None:
        return bsp.qk_norm_rope(s["Q"], s["K"], s["positions"], s["freq"], **args)
    Q = bsp.qk_norm_rope_append(s["Q"], s["K"], s["V"], s["positions"], s["freq"], s["cache"], s["slots"], **args)
    return (Q,) + tuple(bsp.kv_gather(s["cache"], s["slots"]))


def _tokens_own(s):
    import bit_unstructured_sparse_amd as bsp
    dtype = bsp.INT8 if s["kind"] == "int8" else bsp.INT4
    t = bsp.quantize_tokens(s["X"], dtype, weight=s["weight"], eps=EPS, residual=s["residual"])
    values = bsp.dequantize_tokens(t.codes, t.scale, dtype, s["K"])
    return (values, t.scale) + ((t.hidden,) if s["residual"] is not None else ())


def _pages_plain(s, keep, new, call, mask):
    P, rows, table, free = s["page"], s["rows"][call], s["table"], s["free"]
    B, width = table.shape
    lens, held, count, pool = s["lens"].long(), s["held"].long(), free[0].long(), free[2:]
    kept = torch.minimum(keep.long().clamp(min=0), lens)
    more = new.long().clamp(min=0)
    total = kept + more
    end = more.cumsum(0)
    start = end - more
    want = (total + P - 1) // P
    fits = (more == 0) | ((end <= rows) & (want <= width))
    change = torch.where(fits, want - held, 0)
    grow, shrink = change.clamp(min=0), (-change).clamp(min=0)
    given = shrink.sum()
    taken_end = grow.cumsum(0)
    fits = fits & ((grow == 0) | (taken_end <= count + given))
    taken = torch.where(fits, grow, 0)
    after = held + taken - shrink
    # pages given back, in order
    p = torch.arange(width, device=DEV)[None, :]
    number = (shrink.cumsum(0) - shrink)[:, None] + p - after[:, None]
    leaves = (p >= after[:, None]) & (p < held[:, None])
    freed = torch.zeros(B * width + 1, dtype=torch.int32, device=DEV)
    freed[torch.where(leaves, number, B * width)] = table
    # pages taken: those, then the end of the list
    number = (taken_end - grow)[:, None] + p - held[:, None]
    comes = (p >= held[:, None]) & (p < after[:, None])
    listed_at = (count - 1 - (number - given)).clamp(0, pool.numel() - 1)
    page = torch.where(number < given, freed[number.clamp(0, B * width)], pool[listed_at])
    table.copy_(torch.where(comes, page, table))
    left = given - taken.sum()
    i = torch.arange(pool.numel(), device=DEV)
    pushed = (i >= count) & (i < count + left)
    pool.copy_(torch.where(pushed, freed[(count + given - 1 - i).clamp(0, B * width)], pool))
    free[0] = (count + left).to(torch.int32)
    s["lens"].copy_(torch.where(fits, total, kept))
    s["held"].copy_(after)
    slots, positions, sequences, q_start, kv_lens = s["out"][call]
    q_start[0] = 0
    q_start[1:] = end.clamp(max=rows)
    kv_lens.copy_(torch.where(fits, total, 0))
    r = torch.arange(rows, device=DEV)
    b = torch.searchsorted(end, r, right=True)
    inside = b < B
    b = b.clamp(max=B - 1)
    i = r - start[b]
    t = kept[b] + i
    slot = table[b, (t // P).clamp(max=width - 1)].long() * P + t % P
    slots.copy_(torch.where(inside & fits[b], slot, -1))
    if mask is not None:
        bit = torch.arange(64, device=DEV)[None, :]
        depth = (((mask[:, None] >> bit) & 1) * (bit < i[:, None])).sum(-1)
        i = torch.where(more[b] <= 64, depth, i)
    positions.copy_(torch.where(inside, kept[b] + i, 0))
    sequences.copy_(torch.where(inside, b, -1))
    return tuple(s["out"][call])


def _rotate(x, weight, s):
    """float16 heads [n][heads][dim], normed (weight not None) and rotated, in 32 bits."""
    x = x.float()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    rot = s["rot"]
    omega = 10000.0 ** (-2.0 * torch.arange(rot // 2, device=DEV, dtype=torch.float64) / rot)
    angle = s["positions"].double()[:, None] * omega
    c, z = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    if s["inter"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * c - b * z, b * c + a * z), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * c - b * z, b * c + a * z), -1)
    return torch.cat((turned, x[..., rot:]), -1).to(torch.float16)


def _quantise_row(x, kind):
    """float16 rows [..., dim] -> (codes uint8, words int32), in 32 bits."""
    x = x.float()
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    levels = torch.full_like(lo, KV_LEVELS[kind])
    step = (((hi - lo) / levels).view(torch.int32) + 0xFFFF).bitwise_and(-65536).view(torch.float32)
    zero = step == 0
    u = torch.where(zero, 0.0, torch.round((x - lo) / torch.where(zero, 1.0, step)))
    u = torch.minimum(u, levels).to(torch.uint8)
    word = step.view(torch.int32) | (lo.to(torch.float16).view(torch.int16).to(torch.int32) & 0xFFFF)
    return (u[..., 0::2] | (u[..., 1::2] << 4) if kind == "int4" else u), word[..., 0]


def _cache_plain(s, name, x):
    """Rows to their slots, and back as float16."""
    page, off, kind = s["slots"] // s["page"], s["slots"] % s["page"], s["kind"]
    if kind == "fp16":
        s[name][page, :, off] = x
        return s[name][page, :, off]
    s[name][page, :, off], s[name + "s"][page, :, off] = _quantise_row(x, kind)
    u, word = s[name][page, :, off], s[name + "s"][page, :, off]
    if kind == "int4":
        u = torch.stack((u & 15, u >> 4), -1).flatten(-2)
    step = word.bitwise_and(-65536).view(torch.float32)
    lo = (word & 0xFFFF).to(torch.int16).view(torch.float16).float()
    return (step[..., None] * u.float() + lo[..., None]).to(torch.float16)


def _heads_plain(s):
    Q, K = _rotate(s["Q"], s["wq"], s), _rotate(s["K"], s["wk"], s)
    if s["kind"] is None:
        return Q, K
    return Q, _cache_plain(s, "ck", K), _cache_plain(s, "cv", s["V"])


def _tokens_plain(s):
    h = s["X"] if s["residual"] is None else (s["X"].float() + s["residual"].float()).to(torch.float16)
    x = h.float()
    y = x if s["weight"] is None else x * s["weight"].float()
    m = y.abs().amax(-1, keepdim=True)
    L = LEVELS[s["kind"]]
    # values next to a border between two codes: the quotient in 64 bits
    u = torch.round(y.double() * L / torch.where(m == 0, 1.0, m).double()).to(torch.int8)
    scale = m / L
    if s["weight"] is not None:
        scale = m / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) / L
    if s["kind"] == "int4":      # packed for the sparse product, two codes to a byte
        if u.shape[-1] % 2:
            u = torch.cat((u, torch.zeros_like(u[:, :1])), -1)
        packed = (u[:, 0::2] & 15) | (u[:, 1::2] << 4)
        u = torch.stack(((packed << 4) >> 4, packed >> 4), -1).flatten(-2)[:, :s["K"]]
    values = (u.float() * scale).to(torch.float16)
    return (values, scale[:, 0].contiguous()) + ((h,) if s["residual"] is not None else ())


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    op = case["op"]
    if op == "pages":
        return _exact_pages(case, _pages_inputs(case, seed))
    if op == "heads":
        return _exact_heads(_heads_inputs(case, seed))
    if op == "tokens":
        return _exact_tokens(_tokens_inputs(case, seed))
    s = _product_inputs(case, seed)
    Y = torch.matmul(s["X"].double(), s["W"].double().t().contiguous())
    return Y.mul_(s["scale_w"].double()).mul_(s["scale_x"].double()[:, None])


def _exact_pages(case, s):
    """The definition, page by page on the host."""
    P, width = s["page"], s["table"].shape[1]
    table, lens, held = s["table"].tolist(), s["lens"].tolist(), s["held"].tolist()
    count, pool = int(s["free"][0]), s["free"][2:].tolist()
    outs = []
    for call, (keep, new, mask) in enumerate(((s["keep"], s["new"], s["mask"]), (s["keep"], s["back"], None))):
        keep, new, rows = keep.tolist(), new.tolist(), s["rows"][call]
        words = None if mask is None else mask.cpu().numpy().view(np.uint64).tolist()
        start, todo, back = [0], [], []
        for b in range(len(lens)):
            start.append(start[-1] + new[b])
            want = -(-(keep[b] + new[b]) // P)
            todo.append(want if new[b] == 0 or (start[-1] <= rows and want <= width) else None)
            if todo[b] is not None and todo[b] < held[b]:
                back += table[b][todo[b]:held[b]]
        have, asked, handed = count + len(back), 0, 0
        slots, positions, sequences, kv_lens = [-1] * rows, [0] * rows, [-1] * rows, [0] * len(lens)
        for b in range(len(lens)):
            if todo[b] is not None and todo[b] > held[b]:
                asked += todo[b] - held[b]
                if asked > have:
                    todo[b] = None
                else:
                    for p in range(held[b], todo[b]):
                        if handed < len(back):
                            table[b][p] = back[handed]
                        else:
                            count -= 1
                            table[b][p] = pool[count]
                        handed += 1
            lens[b] = keep[b]
            if todo[b] is not None:
                held[b] = todo[b]
                lens[b] = kv_lens[b] = keep[b] + new[b]
            for i in range(new[b]):
                r, t = start[b] + i, keep[b] + i
                if r >= rows:
                    break
                sequences[r], positions[r] = b, t
                if words is not None and new[b] <= 64:
                    positions[r] = keep[b] + bin(words[r] & ((1 << i) - 1)).count("1")
                if todo[b] is not None:
                    slots[r] = table[b][t // P] * P + t % P
        for page in reversed(back[handed:]):
            pool[count] = page
            count += 1
        outs.append((torch.tensor(slots, dtype=torch.int64, device=DEV), _i32(positions), _i32(sequences),
                     _i32([min(x, rows) for x in start]), _i32(kv_lens)))
    return outs[0], outs[1], _i32(table), _i32(lens), _i32(held), _i32([count, 0] + pool)


def _exact_heads(s):
    def rotated(x, weight):
        x = x.double()
        if weight is not None:
            x = x * torch.rsqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()
        half = s["rot"] // 2
        y = x.clone()
        at = s["positions"].double()
        for i in range(half):
            angle = at * math.exp(-math.log(10000.0) * i / half)
            c, z = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
            j, k = (2 * i, 2 * i + 1) if s["inter"] else (i, i + half)
            y[..., j] = x[..., j] * c - x[..., k] * z
            y[..., k] = x[..., k] * c + x[..., j] * z
        return y

    def stored(x):
        if s["kind"] == "fp16":
            return x.double()
        x, L = x.to(torch.float16).double(), KV_LEVELS[s["kind"]]
        o = x.min(-1, keepdim=True).values
        step = ((x.max(-1, keepdim=True).values - o) / L).view(torch.int64)
        step = ((step + (1 << 45) - 1) & -(1 << 45)).view(torch.float64)    # bfloat16 keeps 7 of the 52 fraction bits
        return torch.round((x - o) / torch.where(step > 0, step, 1.0)).clamp(max=L) * step + o

    Q, K = rotated(s["Q"], s["wq"]), rotated(s["K"], s["wk"])
    return (Q, K) if s["kind"] is None else (Q, stored(K), stored(s["V"]))


def _exact_tokens(s):
    h = s["X"].double()
    if s["residual"] is not None:
        h = (h + s["residual"].double()).to(torch.float16).double()
    y = h if s["weight"] is None else h * s["weight"].double()
    L = LEVELS[s["kind"]]
    m = y.abs().max(-1, keepdim=True).values
    scale = m / L
    if s["weight"] is not None:
        scale = scale * torch.rsqrt(h.square().sum(-1, keepdim=True) / h.shape[-1] + EPS)
    values = torch.round(y * (L / 1.0) / torch.where(m > 0, m, 1.0)) * scale
    return (values, scale[:, 0].contiguous()) + ((h,) if s["residual"] is not None else ())
