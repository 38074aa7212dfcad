"""The decode-step operators of this library, as workloads to time.

Three operators of a served model's decode step, next to the sparse
projections: adapters of many requests beside one shared sparse projection,
a paged key/value cache quantised as it is written and read back, and the
attention of drafted token trees over that cache.

With ``own`` false, ``run`` computes each of them in plain torch operations
in 32 bits, rounded once at the end; with ``own`` true it calls the library.
``exact`` gives the same outputs from the definitions in 64 bits.

Cache layout (what ``prepare`` builds and both sides read): pages of
``page`` tokens, ``k`` and ``v`` [pages][kv_heads][page][row], a row being
head_dim float16 values, head_dim bytes (int8) or head_dim / 2 bytes (int4,
low nibble first). A quantised row stands for s * u + o, u its unsigned codes;
its 32-bit word ([pages][kv_heads][page]) holds s as bfloat16 in the high half
and o as float16 in the low half. s is (max - min) / (2^bits - 1) rounded up to
bfloat16, o the row's minimum, u = round-half-even((x - o) / s).
"""
import math
import random

import numpy as np
import torch

own = False

KINDS = ("fp16", "int8", "int4")
LEVELS = {"int8": 255, "int4": 15}
STALE_WORD = 0x7FC07E00          # a word of NaN scale and NaN minimum: what lies in unused slots
DEV = "cuda"


# ---------------------------------------------------------------- the cases

def _attention(name, B, T, hq, hkv, dim, ctx, kind, page, ragged, tree):
    """B sequences of up to ctx cached tokens, up to T drafted tokens each."""
    return dict(name=name, op="attention", B=B, T=T, hq=hq, hkv=hkv, dim=dim, ctx=ctx, kind=kind, page=page,
                ragged=ragged, tree=tree)


def _cache(name, op, n, hkv, dim, kind, page):
    """n tokens through the cache; op "write" (append, then read back) or "read"."""
    return dict(name=name, op=op, n=n, hkv=hkv, dim=dim, kind=kind, page=page)


def _lora(name, op, M, K, N, density, adapters, rank, mixed):
    """N tokens through an M x K sparse projection with `adapters` adapters of rank up to `rank`."""
    return dict(name=name, op=op, M=M, K=K, N=N, density=density, adapters=adapters, rank=rank, mixed=mixed)


def listed():
    return [
        # one user, one new token, a short conversation: 32 heads of the 12288 x 4096 QKV projection
        _attention("attention_one_token", 1, 1, 32, 32, 128, 500, "int8", 16, False, False),
        # plain batched decoding at mixed lengths: 64 query and 8 kv heads of the 10240 x 8192 fused QKV
        _attention("attention_batch_int4", 32, 1, 64, 8, 128, 4096, "int4", 64, True, False),
        # speculative decoding: a tree of up to 16 drafted tokens for each of 8 requests
        _attention("attention_trees_int8", 8, 16, 64, 8, 128, 8192, "int8", 32, True, True),
        # one very long document, a short chain of drafted tokens, an unquantised cache
        _attention("attention_long_fp16", 1, 8, 64, 8, 128, 131072, "fp16", 128, False, False),
        # wide trees (61 tokens) at an odd group of 5 query heads per kv head (40 heads of 5120 channels)
        _attention("attention_wide_trees", 4, 61, 40, 8, 128, 3001, "int4", 16, True, True),
        # the step of 32 requests writes one token each, 8 kv heads
        _cache("cache_write_step", "write", 32, 8, 128, "int4", 64),
        # a batch of prompts enters the cache, 32 kv heads
        _cache("cache_write_prompt", "write", 8192, 32, 128, "int8", 32),
        # a long shared prefix is read back as float16 (to move it, or to attend to it elsewhere)
        _cache("cache_read_prefix", "read", 65537, 8, 128, "int4", 16),
        # one request on the fp16 4096 x 4096 projection with its adapter of rank 8
        _lora("adapters_f16_one", "lora_f16", 4096, 4096, 1, 0.4, 4, 8, False),
        # 32 requests of 32 tenants, ranks 1 to 64, some without an adapter
        _lora("adapters_f16_many", "lora_f16", 4096, 4096, 32, 0.4, 32, 64, True),
        # the FFN's down projection (K past 4096: ranges of K and a workspace), rank 16
        _lora("adapters_f16_ffn_down", "lora_f16", 4096, 11008, 8, 0.3, 8, 16, False),
        # int4 weights and activations with the dequantised sum, float16 adapters beside them
        _lora("adapters_w4a4_qkv", "lora_w4a4", 12288, 4096, 8, 0.5, 8, 16, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "write", "read", "lora_f16", "lora_w4a4"])
    kind = rng.choice(KINDS)
    page = rng.choice([16, 32, 64, 128])
    dim = rng.choice([64, 128, 128, 256])
    if op == "attention":
        hkv = rng.choice([1, 2, 4, 8, 32])
        hq = hkv * (1 if hkv == 32 else rng.choice([1, 2, 3, 4, 5, 8]))
        B, T = _log(rng, 1, 32), _log(rng, 1, 64)
        # no more cached elements or products than the largest listed case
        most = min(131072 * 8 * 128 // (B * hkv * dim), 131072 * 8 * 64 * 128 // (B * T * hq * dim))
        ctx = _log(rng, min(T, most), max(T, most))
        c = _attention(None, B, T, hq, hkv, dim, ctx, kind, page, rng.random() < 0.7, rng.random() < 0.6)
    elif op in ("write", "read"):
        hkv = rng.choice([1, 2, 4, 8, 32])
        most = (8192 * 32 * 128 if op == "write" else 65537 * 8 * 128) // (hkv * dim)
        c = _cache(None, op, _log(rng, 1, most), hkv, dim, kind, page)
    else:
        K = 8 * _log(rng, 8, 1376)
        M = _log(rng, 64, min(16384, 12288 * 4096 // K))
        c = _lora(None, op, M, K, _log(rng, 1, 32), rng.choice([0.3, 0.4, 0.5, 0.7]), _log(rng, 1, 32),
                  8 * _log(rng, 1, 8), rng.random() < 0.5)
    del c["name"]
    return c


def _plan(case):
    """What is fixed by the case and not by the seed: a generator for lengths, ranks and indices."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case):
    """(drafted tokens, cached tokens with the drafted ones) per sequence."""
    p, out = _plan(case), []
    for b in range(case["B"]):
        t = case["T"] if not case["ragged"] or b == 0 else p.randint(1, case["T"])
        n = case["ctx"] if not case["ragged"] or b == 0 else p.randint(max(t, case["ctx"] // 8), max(t, case["ctx"]))
        out.append((t, max(t, n)))
    return out


def _adapter_use(case):
    """(rank of each adapter, adapter of each token or -1)."""
    p = _plan(case)
    rank = [p.randint(1, case["rank"]) if case["mixed"] else case["rank"] for _ in range(case["adapters"])]
    index = [-1 if case["mixed"] and p.random() < 0.125 else p.randrange(case["adapters"]) for _ in range(case["N"])]
    return rank, index


def _row_bytes(kind, dim):
    return {"fp16": 2 * dim, "int8": dim + 4, "int4": dim // 2 + 4}[kind]


def work(case):
    op = case["op"]
    if op == "attention":
        lens = _lengths(case)
        rows = sum(t for t, _ in lens) * case["hq"]
        return dict(bytes=2 * sum(n for _, n in lens) * case["hkv"] * _row_bytes(case["kind"], case["dim"])
                    + 2 * 2 * rows * case["dim"],
                    flops=4 * sum(t * n for t, n in lens) * case["hq"] * case["dim"])
    if op in ("write", "read"):
        rows = 2 * case["n"] * case["hkv"]
        codes, values = rows * _row_bytes(case["kind"], case["dim"]), rows * 2 * case["dim"]
        # write: values read, codes written, codes read back, values written
        return dict(bytes=(2 if op == "write" else 1) * (codes + values), flops=4 * rows * case["dim"])
    M, K, N = case["M"], case["K"], case["N"]
    rank, index = _adapter_use(case)
    nnz = case["density"] * M * K
    weights = M * ((K + 63) // 64) * 12 + (2 * nnz if op == "lora_f16" else nnz / 2)
    pairs = 2 * sum(rank[a] for a in set(index) if a >= 0) * (M + K)
    acts = N * (2 * K + 2 * M) + (0 if op == "lora_f16" else N * K // 2 + 4 * (N + M))
    return dict(bytes=int(weights + pairs + acts),
                flops=int(2 * nnz * N + 2 * sum(rank[a] for a in index if a >= 0) * (M + K)))


# ---------------------------------------------------------------- inputs

def _gen(seed, *salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(random.Random(repr((seed,) + salt)).getrandbits(48))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _kv_values(g, n, hkv, dim, key):
    """float16 rows [n][hkv][dim]: keys with strong channels and channel offsets, smaller values."""
    x = _normal(g, n, hkv, dim)
    if key:
        channel = _normal(g, 1, hkv, dim)
        x = x * torch.where(channel.abs() > 2.0, 4.0, 1.0) + 0.5 * channel
    else:
        x = 0.5 * x
    return x.to(torch.float16)


def _quantise(x, kind):
    """float16 rows [..., dim] -> (codes uint8, words int32), in 32 bits."""
    x = x.to(torch.float32)
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    levels = torch.full_like(lo, LEVELS[kind])
    step = ((hi - lo) / levels).view(torch.int32) + 0xFFFF           # rounded up to bfloat16
    step = step.bitwise_and(-65536).view(torch.float32)
    zero = step == 0
    u = torch.where(zero, 0.0, torch.round((x - lo) / torch.where(zero, 1.0, step)))
    u = torch.minimum(u, levels).to(torch.uint8)
    word = step.view(torch.int32) | (lo.to(torch.float16).view(torch.int16).to(torch.int32) & 0xFFFF)
    if kind == "int4":
        u = u[..., 0::2] | (u[..., 1::2] << 4)
    return u, word[..., 0]


def _dequantise(u, word, kind, dtype=torch.float32):
    if kind == "int4":
        u = torch.stack((u & 15, u >> 4), -1).flatten(-2)
    step = word.bitwise_and(-65536).view(torch.float32).to(dtype)
    lo = (word & 0xFFFF).to(torch.int16).view(torch.float16).to(dtype)
    return step[..., None] * u.to(dtype) + lo[..., None]


def _empty_cache(kind, pages, hkv, page, dim):
    """Cache tensors as an earlier owner of the pages left them: stale codes and NaN."""
    if kind == "fp16":
        k = torch.full((pages, hkv, page, dim), float("nan"), dtype=torch.float16, device=DEV)
        return dict(kind=kind, page=page, k=k, v=k.clone(), ks=None, vs=None)
    k = torch.full((pages, hkv, page, dim if kind == "int8" else dim // 2), 0xA7, dtype=torch.uint8, device=DEV)
    ks = torch.full((pages, hkv, page), STALE_WORD, dtype=torch.int32, device=DEV)
    return dict(kind=kind, page=page, k=k, v=k.clone(), ks=ks, vs=ks.clone())


def _store(cache, K, V, slots):
    """Plain write of rows [n][hkv][dim] to the slots (page * page_size + offset)."""
    p, o = slots // cache["page"], slots % cache["page"]
    for name, x in (("k", K), ("v", V)):
        if cache["kind"] == "fp16":
            cache[name][p, :, o] = x
        else:
            u, w = _quantise(x, cache["kind"])
            cache[name][p, :, o] = u
            cache[name + "s"][p, :, o] = w


def _load(cache, slots, dtype=torch.float32):
    """Plain read of the slots: K, V [n][hkv][dim]."""
    p, o = slots // cache["page"], slots % cache["page"]
    if cache["kind"] == "fp16":
        return cache["k"][p, :, o].to(dtype), cache["v"][p, :, o].to(dtype)
    return tuple(_dequantise(cache[n][p, :, o], cache[n + "s"][p, :, o], cache["kind"], dtype) for n in "kv")


def _cache_inputs(case, seed):
    n, hkv, dim, page = case["n"], case["hkv"], case["dim"], case["page"]
    g = _gen(seed, "cache")
    K, V = _kv_values(g, n, hkv, dim, True), _kv_values(g, n, hkv, dim, False)
    pages = -(-n // page) + 1
    order = torch.randperm(pages, generator=g, device=DEV)
    t = torch.arange(n, device=DEV)
    slots = order[t // page] * page + t % page
    cache = _empty_cache(case["kind"], pages, hkv, page, dim)
    if case["op"] == "read":
        _store(cache, K, V, slots)
    return cache, K, V, slots


def _attention_inputs(case, seed):
    lens = _lengths(case)
    B, hkv, dim, page = case["B"], case["hkv"], case["dim"], case["page"]
    g = _gen(seed, "attention")
    width = max(-(-n // page) for _, n in lens)
    need = sum(-(-n // page) for _, n in lens)
    cache = _empty_cache(case["kind"], need + 1, hkv, page, dim)
    order = torch.randperm(need + 1, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((B, width), dtype=torch.int32, device=DEV)
    used = 0
    for b, (_, n) in enumerate(lens):
        m = -(-n // page)
        table[b, :m] = order[used:used + m]
        used += m
        for first in range(0, n, 16384):
            t = torch.arange(first, min(n, first + 16384), device=DEV)
            rows = [_kv_values(g, t.numel(), hkv, dim, key) for key in (True, False)]
            _store(cache, *rows, table[b].long()[t // page] * page + t % page)
    total = sum(t for t, _ in lens)
    Q = (1.5 * _normal(g, total, case["hq"], dim)).to(torch.float16)
    masks, p = [], random.Random(repr((seed, "tree")))
    for t, _ in lens:
        row = []
        for i in range(t):
            parent = (p.randint(-1, i - 1) if i else -1) if case["tree"] else i - 1
            row.append((row[parent] if parent >= 0 else 0) | (1 << i))
        masks += row
    mask = torch.from_numpy(np.array(masks, np.uint64).view(np.int64)).to(DEV)
    starts = np.cumsum([0] + [t for t, _ in lens])
    return dict(cache=cache, table=table, Q=Q, mask=mask if case["tree"] else None,
                kv_lens=torch.tensor([n for _, n in lens], dtype=torch.int32, device=DEV),
                q_start=torch.tensor(starts, dtype=torch.int32, device=DEV), lens=lens,
                scale=1.0 / math.sqrt(dim))


def _lora_inputs(case, seed):
    M, K, N, R = case["M"], case["K"], case["N"], case["rank"]
    rank, index = _adapter_use(case)
    g = _gen(seed, "lora")
    keep = torch.rand(M, K, generator=g, device=DEV) < case["density"]
    X = _normal(g, N, K).to(torch.float16)
    s = dict(X=X, M=M, K=K, N=N)
    if case["op"] == "lora_f16":
        W = 0.02 * _normal(g, M, K)
        s["W"] = torch.where(keep, W, 0.0).to(torch.float16)
    else:
        u = torch.randint(0, 15, (M, K), generator=g, device=DEV, dtype=torch.int8)
        s["W"] = torch.where(keep, torch.where(u < 8, u - 8, u - 7), 0).to(torch.int8)
        s["scale_w"] = 0.004 * (0.5 + torch.rand(M, generator=g, device=DEV))
        s["scale_x"] = X.float().abs().amax(-1) / 7.0
        s["X4"] = torch.round(X.float() / s["scale_x"][:, None]).clamp(-8, 7).to(torch.int8)
    s["A"] = (_normal(g, case["adapters"], R, K) / math.sqrt(K)).to(torch.float16)
    s["B"] = (0.2 * _normal(g, case["adapters"], M, R)).to(torch.float16)
    s["scale"] = 0.5 + torch.rand(case["adapters"], generator=g, device=DEV)
    s["rank"] = torch.tensor(rank, dtype=torch.int32, device=DEV)
    s["index"] = torch.tensor(index, dtype=torch.int32, device=DEV)
    return s


def prepare(case, seed):
    op = case["op"]
    if op == "attention":
        s = _attention_inputs(case, seed)
        if own:
            import bit_unstructured_sparse_amd as bsp
            s["cache"] = _own_cache(bsp, s["cache"])
            s["max_q"] = max(t for t, _ in s["lens"])
            s["workspace"] = bsp.new_attention_workspace(s["cache"], case["B"], s["max_q"], case["hq"],
                                                         s["table"].shape[1], device=DEV)
    elif op in ("write", "read"):
        cache, K, V, slots = _cache_inputs(case, seed)
        s = dict(cache=cache, slots=slots)
        if op == "write":
            s.update(K=K, V=V)
        if own:
            import bit_unstructured_sparse_amd as bsp
            s["cache"] = _own_cache(bsp, cache)
    else:
        s = _lora_inputs(case, seed)
        if own:
            import bit_unstructured_sparse_amd as bsp
            W = bsp.encode(s.pop("W").cpu().numpy()).to_device(DEV)
            s["W"] = W
            s["adapters"] = bsp.LoraAdapters(s["A"], s["B"], s["scale"], s["rank"])
            if op == "lora_w4a4":
                s["X4"] = torch.from_numpy(bsp.pack_int4(s["X4"].cpu().numpy())).to(DEV)
            s["workspace"] = bsp.new_lora_workspace(W, s["N"], s["adapters"], device=DEV)
    s["op"] = op
    return s


def _own_cache(bsp, c):
    kind = {"fp16": bsp.FP16, "int8": bsp.INT8, "int4": bsp.INT4}[c["kind"]]
    return bsp.KVCache(kind, c["k"], c["v"], c["ks"], c["vs"])


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "attention":
        return _attend_plain(s)
    if op in ("write", "read"):
        if op == "write":
            _store(s["cache"], s["K"], s["V"], s["slots"])
        K, V = _load(s["cache"], s["slots"])
        return K.to(torch.float16), V.to(torch.float16)
    if op == "lora_f16":
        y = s["X"].float() @ s["W"].float().t()
    else:
        y = s["X4"].float() @ s["W"].float().t() * s["scale_w"][None, :] * s["scale_x"][:, None]
    a = s["index"].clamp(min=0).long()
    live = (torch.arange(s["A"].shape[1], device=DEV) < s["rank"][a][:, None]) & (s["index"] >= 0)[:, None]
    t = torch.bmm(s["A"][a].float(), s["X"].float()[:, :, None])[..., 0] * s["scale"][a][:, None]
    y = y + torch.bmm(s["B"][a].float(), torch.where(live, t, 0.0)[:, :, None])[..., 0]
    return y.to(torch.float16)


def _run_own(s):
    import bit_unstructured_sparse_amd as bsp
    op = s["op"]
    if op == "attention":
        return bsp.attention_tree(s["Q"], s["cache"], s["table"], s["kv_lens"], s["q_start"], s["max_q"],
                                  tree_mask=s["mask"], scale=s["scale"], workspace=s["workspace"])
    if op in ("write", "read"):
        if op == "write":
            bsp.kv_append(s["cache"], s["K"], s["V"], s["slots"])
        return bsp.kv_gather(s["cache"], s["slots"])
    if op == "lora_f16":
        return bsp.spmm_f16_lora(s["W"], s["X"], s["adapters"], s["index"], workspace=s["workspace"])
    return bsp.spmm_w4a4_dq_lora(s["W"], s["X4"], s["X"], s["scale_w"], s["scale_x"], s["adapters"], s["index"],
                                 workspace=s["workspace"])


def _attend_plain(s):
    Q, page = s["Q"], s["cache"]["page"]
    O = torch.empty_like(Q)
    first = 0
    for b, (t, n) in enumerate(s["lens"]):
        j = torch.arange(n, device=DEV)
        K, V = _load(s["cache"], s["table"][b].long()[j // page] * page + j % page)      # [n][hkv][dim]
        hkv, dim = K.shape[1:]
        G = Q.shape[1] // hkv
        q = Q[first:first + t].float().view(t, hkv, G, dim).permute(1, 0, 2, 3).reshape(hkv, t * G, dim)
        x = torch.bmm(q, K.permute(1, 2, 0).contiguous()) * s["scale"]                   # [hkv][t * G][n]
        d = j - (n - t)                                                                  # index among the drafted
        if s["mask"] is not None:
            bits = (s["mask"][first:first + t, None] >> d.clamp(min=0)[None, :]) & 1
            see = (d < 0)[None, :] | (bits == 1)
        else:
            see = d[None, :] <= torch.arange(t, device=DEV)[:, None]
        see = see[:, None, :].expand(t, G, n).reshape(t * G, n)
        x = torch.where(see[None], x, -math.inf)
        top = x.amax(-1, keepdim=True)
        e = torch.where(see[None], torch.exp(x - torch.where(top == -math.inf, 0.0, top)), 0.0)
        total = e.sum(-1, keepdim=True)
        y = torch.bmm(e, V.permute(1, 0, 2).contiguous()) / torch.where(total == 0, 1.0, total)
        O[first:first + t] = y.view(hkv, t, G, dim).permute(1, 0, 2, 3).reshape(t, hkv * G, dim).to(torch.float16)
        first += t
    return O


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    op = case["op"]
    if op == "attention":
        return _exact_attention(_attention_inputs(case, seed))
    if op in ("write", "read"):
        _, K, V, _ = _cache_inputs(case, seed)
        return _exact_rows(K, case["kind"]), _exact_rows(V, case["kind"])
    s = _lora_inputs(case, seed)
    X = s["X"].double()
    if op == "lora_f16":
        Y = torch.matmul(X, s["W"].double().t().contiguous())
    else:
        Y = torch.matmul(s["X4"].double(), s["W"].double().t().contiguous())
        Y = Y * s["scale_w"].double() * s["scale_x"].double()[:, None]
    rank, index = _adapter_use(case)
    for n, a in enumerate(index):
        if a >= 0:
            h = torch.mv(s["A"][a, :rank[a]].double(), X[n])
            Y[n] += s["scale"][a].double() * torch.mv(s["B"][a, :, :rank[a]].double(), h)
    return Y


def _exact_rows(x, kind):
    """What the quantised rows stand for, every step of the definition in 64 bits."""
    x = x.double()
    if kind == "fp16":
        return x
    o = x.min(-1, keepdim=True).values
    s = ((x.max(-1, keepdim=True).values - o) / LEVELS[kind]).view(torch.int64)
    s = ((s + (1 << 45) - 1) & -(1 << 45)).view(torch.float64)    # bfloat16 keeps 7 of the 52 fraction bits
    u = torch.round((x - o) / torch.where(s > 0, s, 1.0)).clamp(max=LEVELS[kind])
    return u * s + o


def _exact_attention(s):
    c, page = s["cache"], s["cache"]["page"]
    total, hq, dim = s["Q"].shape
    hkv = c["k"].shape[1]
    out = torch.zeros(total, hq, dim, dtype=torch.float64, device=DEV)
    first = 0
    for b, (t, n) in enumerate(s["lens"]):
        pages = s["table"][b, :-(-n // page)].long()
        past = n - t
        see = torch.ones(t, n, dtype=torch.bool)
        for i in range(t):
            bits = int(s["mask"][first + i]) if s["mask"] is not None else (2 << i) - 1
            see[i, past:] = torch.tensor([bool(bits >> j & 1) for j in range(t)])
        see = see.to(DEV)
        for h in range(hkv):
            if c["kind"] == "fp16":
                K, V = c["k"][pages, h].double(), c["v"][pages, h].double()
            else:
                K = _dequantise(c["k"][pages, h], c["ks"][pages, h], c["kind"], torch.float64)
                V = _dequantise(c["v"][pages, h], c["vs"][pages, h], c["kind"], torch.float64)
            K, V = K.reshape(-1, dim)[:n], V.reshape(-1, dim)[:n].contiguous()
            KT = K.t().contiguous()
            for i in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                x = torch.matmul(s["Q"][first:first + t, i].double(), KT) * s["scale"]
                x = x.masked_fill(~see, -math.inf)
                out[first:first + t, i] = torch.matmul(torch.softmax(x, -1), V)
        first += t
    return out
