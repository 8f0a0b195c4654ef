"""Cases of the operators behind many answers to one prompt: decode attention of requests that share a long
prefix, computed once for each group of them, and the choice of the next tokens from the logits by temperature,
top-k, top-p and min-p with given random numbers.  Each case runs either in a plain form (elementary torch
operations) or, with `own`, through the library's binding.

Head layouts are those of the library's Llama-shaped configurations (8B: 32 q and 8 kv heads of 128,
70B: 64 and 8, 405B-shaped: 128 and 8; vocabulary 128256) and a few generic ones.
"""
import math
import random

import torch

own = False

DEV = "cuda"
VOCAB = 128256
HEADS = [(32, 8, 128), (64, 8, 128), (128, 8, 128), (16, 16, 64), (8, 4, 256), (16, 2, 64), (24, 8, 128)]
PAGES = [16, 32, 64, 128, 256]
LARGEST_FLOPS = 2.7e11   # of a drawn attention case, and
LARGEST_BYTES = 4e8      # of its cache behind the prefixes, and
LARGEST_LOGITS = 1.3e8   # of a drawn choice of tokens: no more than the largest listed ones


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest call: four answers to a short prompt, a few tokens in, where latency counts
        dict(name="prefix-few", op="attn", M=4, groups=1, n_q=32, n_kv=8, hd=128, t=1, page=16, kv="bf16", prefix=1000,
             tail=20, mix=1),
        # an ordinary batch of the 70B heads over 8 shards behind one system prompt
        dict(name="prefix-batch", op="attn", M=64, groups=1, n_q=64, n_kv=8, hd=128, t=8, page=64, kv="bf16",
             prefix=8192, tail=500, mix=2),
        # several prompts of ragged lengths, a few answers each; three q heads per kv head
        dict(name="prefix-groups", op="attn", M=45, groups=7, n_q=24, n_kv=8, hd=128, t=2, page=32, kv="bf16",
             prefix=6001, tail=300, mix=3),
        # one very long document, read once for 16 questions: the cache's bytes count
        dict(name="prefix-long", op="attn", M=16, groups=1, n_q=64, n_kv=8, hd=128, t=8, page=64, kv="bf16",
             prefix=131072, tail=100, mix=4),
        # the 405B heads (16 q heads per kv head) over an e4m3 cache, two prompts
        dict(name="prefix-e4m3", op="attn", M=96, groups=2, n_q=128, n_kv=8, hd=128, t=4, page=32, kv="e4m3",
             prefix=15000, tail=400, mix=5),
        # heads of 256
        dict(name="prefix-256", op="attn", M=77, groups=3, n_q=8, n_kv=4, hd=256, t=1, page=128, kv="bf16",
             prefix=9000, tail=200, mix=6),
        # the largest: 256 answers behind 30 thousand positions: the tensor cores count
        dict(name="prefix-large", op="attn", M=256, groups=1, n_q=64, n_kv=8, hd=128, t=8, page=64, kv="bf16",
             prefix=30000, tail=250, mix=7),
        # one request's next token, nucleus sampling
        dict(name="sample-one", op="sample", M=1, V=VOCAB, pad=0, rows="nucleus", masked=0.0, mix=8),
        # a decode batch whose requests each bring their own settings, some greedy, some vocabulary masked out
        dict(name="sample-mixed", op="sample", M=32, V=VOCAB, pad=0, rows="mixed", masked=0.1, mix=9),
        # a large batch with a temperature only: every token of the vocabulary may be chosen
        dict(name="sample-plain", op="sample", M=256, V=VOCAB, pad=64, rows="plain", masked=0.0, mix=10),
        # a smaller vocabulary of odd size, top-k alone
        dict(name="sample-topk", op="sample", M=300, V=32003, pad=1, rows="topk", masked=0.0, mix=11),
        # the largest batch, nucleus sampling
        dict(name="sample-nucleus", op="sample", M=1000, V=VOCAB, pad=0, rows="nucleus", masked=0.0, mix=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    mix = rng.randrange(1 << 30)
    if rng.random() < 0.4:
        V = _log(rng, 300, VOCAB)
        return dict(op="sample", M=_log(rng, 1, min(2000, int(LARGEST_LOGITS / V))), V=V, pad=rng.choice([0, 1, 64]),
                    rows=rng.choice(["plain", "topk", "nucleus", "minp", "mixed"]), masked=rng.choice([0.0, 0.0, 0.5]),
                    mix=mix)
    n_q, n_kv, hd = rng.choice(HEADS)
    t = rng.choice([s for s in (1, 2, 4, 8) if n_kv % s == 0])
    kv = rng.choice(["bf16", "bf16", "e4m3"])
    M = _log(rng, 2, 256)
    prefix = _log(rng, 16, min(131072, int(LARGEST_FLOPS / (4.2 * n_q * hd * M))))
    return dict(op="attn", M=M, groups=_log(rng, 1, max(1, M // 2)), n_q=n_q, n_kv=n_kv, hd=hd, t=t, page=rng.choice(PAGES),
                kv=kv, prefix=prefix, tail=_log(rng, 1, max(2, min(1000, int(LARGEST_BYTES / (M * n_kv * hd * 4))))), mix=mix)


def _ceil(a, b):
    return -(-a // b)


def _groups(case):
    """First row of each group (and the end), the groups' prefixes, and each request's length, its new token
    included.  Several groups: their sizes and prefixes differ, the first keeps the longest."""
    r = random.Random(case["mix"])
    M, G = case["M"], case["groups"]
    cu = [0]
    for i in range(1, G):
        cu.append(min(M - G + i, max(cu[-1] + 1, round((i + r.uniform(-0.4, 0.4)) * M / G))))
    cu.append(M)
    prefix = [case["prefix"]] + [r.randint((case["prefix"] + 1) // 2, case["prefix"]) for _ in range(G - 1)]
    lens = [prefix[g] + r.randint(1, case["tail"]) for g in range(G) for _ in range(cu[g], cu[g + 1])]
    return cu, prefix, lens


def _shared(case, prefix):
    """Positions of the prefix that lie on whole pages: what requests can share."""
    return prefix // case["page"] * case["page"]


def work(case):
    M = case["M"]
    if case["op"] == "sample":
        return {"bytes": 4 * M * case["V"] + M * (4 * 5 + 8), "flops": 6 * M * case["V"]}
    n_q, n_kv, hd = case["n_q"], case["n_kv"], case["hd"]
    cu, prefix, lens = _groups(case)
    stored = 0  # positions that have to be read
    for g, p in enumerate(prefix):
        s = _shared(case, p)
        stored += s + sum(n - s for n in lens[cu[g]:cu[g + 1]])
    size = 2 if case["kv"] == "bf16" else 1
    return {"bytes": stored * n_kv * hd * 2 * size + M * n_q * (hd * 4 + 4), "flops": 4 * sum(lens) * n_q * hd}


# --------------------------------------------------------------------------------------- the inputs
def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + salt)
    return g


def _pool(g, case, n_pages):
    """Keys or values of a page pool [t][n_pages][n_kv/t][page][hd], and the heads' scales."""
    shape = (case["t"], n_pages, case["n_kv"] // case["t"], case["page"], case["hd"])
    pool = torch.empty(shape, device=DEV, dtype=torch.bfloat16 if case["kv"] == "bf16" else torch.float8_e4m3fn)
    std = 1.0 if case["kv"] == "bf16" else 70.0
    for s in range(shape[0]):
        pool[s] = (torch.randn(shape[1:], generator=g, device=DEV) * std).to(pool.dtype)
    scale = None
    if case["kv"] == "e4m3":
        scale = (torch.rand(case["n_kv"], generator=g, device=DEV) + 0.5) / 70.0
    return pool, scale


def _settings(case):
    """Temperature, top_k, top_p and min_p of each row."""
    r = random.Random(case["mix"])
    rows = []
    for _ in range(case["M"]):
        kind = case["rows"]
        if kind == "mixed":
            kind = r.choice(["greedy", "plain", "topk", "nucleus", "minp", "all"])
        t, k, p, q = 0.0 if kind == "greedy" else r.uniform(0.5, 1.3), 0, 1.0, 0.0
        if kind in ("topk", "all"):
            k = r.choice([1, 5, 20, 40, 50, 64, 200])
        if kind in ("nucleus", "all"):
            p = r.uniform(0.7, 0.98)
        if kind in ("minp", "all"):
            q = r.uniform(0.01, 0.1)
        rows.append((t, k, p, q))
    return rows


def prepare(case, seed):
    g, M = _gen(seed, 23), case["M"]
    s = dict(case=case)
    if own:
        from megatron_tensor_transformer_gb300 import tpx
        s["tpx"] = tpx
    i32, f32 = dict(dtype=torch.int32, device=DEV), dict(dtype=torch.float32, device=DEV)
    if case["op"] == "sample":
        V = case["V"]
        logits = torch.empty((M, V + case["pad"]), device=DEV)  # the rows lie apart where there is padding
        for a in range(0, M, 256):
            logits[a:a + 256] = torch.randn((min(256, M - a), V + case["pad"]), generator=g, device=DEV) * 2.5
        logits = logits[:, :V]
        # a few tokens well ahead of the others, as a trained model has them
        ahead = torch.randint(0, V, (M, 12), generator=g, device=DEV)
        logits.scatter_add_(1, ahead, torch.rand((M, 12), generator=g, device=DEV) * 9.0)
        if case["masked"]:
            keep = torch.rand(V, generator=g, device=DEV) >= case["masked"]
            keep[V // 2] = True
            logits.masked_fill_(~keep, float("-inf"))
        t, k, p, q = zip(*_settings(case))
        s |= dict(logits=logits, u=torch.rand(M, generator=g, device=DEV), temperature=torch.tensor(t, **f32),
                  top_k=torch.tensor(k, **i32), top_p=torch.tensor(p, **f32), min_p=torch.tensor(q, **f32),
                  ids=torch.zeros(M, **i32), logprob=torch.zeros(M, **f32))
        return s
    n_q, n_kv, hd, page = case["n_q"], case["n_kv"], case["hd"], case["page"]
    cu, prefix, lens = _groups(case)
    whole = [_shared(case, p) // page for p in prefix]  # pages of a group
    most = max(_ceil(n, page) for n in lens) + 1
    n_pages = sum(whole) + sum(_ceil(n, page) - whole[i] for i in range(len(whole)) for n in lens[cu[i]:cu[i + 1]]) + 3
    s["k_pages"], s["k_scale"] = _pool(g, case, n_pages)
    s["v_pages"], s["v_scale"] = _pool(g, case, n_pages)
    # the table: a group's rows begin with the same pages, then each has its own
    ids = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((M, most), -1, **i32)
    at = 0
    for i in range(len(whole)):
        rows = slice(cu[i], cu[i + 1])
        table[rows, : whole[i]] = ids[at: at + whole[i]]
        at += whole[i]
        held = torch.tensor([_ceil(n, page) for n in lens[rows]], device=DEV)
        col = torch.arange(most, device=DEV)[None, :]
        mine = (col >= whole[i]) & (col < held[:, None])
        n = int((held - whole[i]).sum())
        table[rows] = table[rows].masked_scatter(mine, ids[at: at + n])
        at += n
    s |= dict(table=table, lens=torch.tensor(lens, **i32), cu=torch.tensor(cu, **i32), prefix=torch.tensor(prefix, **i32),
              q=(torch.randn((M, n_q * hd), generator=g, device=DEV) * 1.5).to(torch.bfloat16),
              o=torch.zeros((M, n_q * hd), dtype=torch.bfloat16, device=DEV), lse=torch.zeros((M, n_q), **f32),
              # sizes of the padded batch, which the host knows
              most_rows=max(b - a for a, b in zip(cu, cu[1:])), most_pages=max(whole),
              most_own=max(n - w * page for i, w in enumerate(whole) for n in lens[cu[i]:cu[i + 1]]))
    if own:
        s["shape"] = tpx.make_shape(n_q * hd, n_q=n_q, n_kv=n_kv, hd=hd, t=case["t"])
        s["pages"] = tpx.make_pages(page, n_pages, most, tpx.TP_BF16 if case["kv"] == "bf16" else tpx.TP_FP8_E4M3)
        s["ws"] = tpx.new_prefix_attn_workspace(s["shape"], M, DEV)
    return s


# -------------------------------------------------------------------------------------- the passes
def run(s):
    if own:
        tpx = s["tpx"]
        if s["case"]["op"] == "sample":
            tpx.tp_sample_tokens(s["logits"], s["u"], s["ids"], temperature=s["temperature"], top_k=s["top_k"],
                                 top_p=s["top_p"], min_p=s["min_p"], logprob=s["logprob"])
            return {k: s[k] for k in ("ids", "logprob")}
        tpx.tp_prefix_attn_decode(s["shape"], s["pages"], s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                                  s["cu"], s["prefix"], s["o"], s["ws"], lse=s["lse"], k_scale=s["k_scale"],
                                  v_scale=s["v_scale"])
        return {k: s[k] for k in ("o", "lse")}
    return _plain_sample(s) if s["case"]["op"] == "sample" else _plain_attn(s)


def _pages_of(s, pool, scale, ids):
    """[B, n_kv, ids.shape[1] * page, hd] in 32 bits: the pages ids [B, n] one after another."""
    c = s["case"]
    raw = pool if pool.dtype == torch.bfloat16 else pool.view(torch.uint8)
    x = raw[:, ids.long().clamp(min=0)].view(pool.dtype).float()  # [t, B, n, n_kv/t, page, hd]
    x = x.permute(1, 0, 3, 2, 4, 5).reshape(ids.shape[0], c["n_kv"], ids.shape[1] * c["page"], c["hd"])
    return x if scale is None else x * scale[None, :, None, None]


def _plain_attn(s):
    c = s["case"]
    M, n_q, n_kv, hd, page = c["M"], c["n_q"], c["n_kv"], c["hd"], c["page"]
    per, dev = n_q // n_kv, s["q"].device
    cu, lens = s["cu"].long(), s["lens"].long()
    first, size, pages = cu[:-1], cu[1:] - cu[:-1], s["prefix"].long() // page
    q = s["q"].float().view(M, n_kv, per, hd) * (1.0 / math.sqrt(hd))
    # the groups' prefixes: a padded batch of groups, a group's rows and heads side by side
    i = torch.arange(s["most_rows"], device=dev)
    row = (first[:, None] + i).clamp(max=M - 1)  # [G, rows]
    qg = q[row].permute(0, 2, 1, 3, 4).reshape(len(size), n_kv, s["most_rows"] * per, hd)
    shared = s["table"][first][:, : s["most_pages"]]
    score = qg @ _pages_of(s, s["k_pages"], s["k_scale"], shared).transpose(2, 3)
    seen = torch.arange(score.shape[3], device=dev) < (pages * page)[:, None]
    score = score.masked_fill(~seen[:, None, None, :], float("-inf"))
    ref = score.amax(-1, keepdim=True) if score.shape[3] else score.new_full((*score.shape[:3], 1), float("-inf"))
    e = torch.exp(score - torch.where(torch.isfinite(ref), ref, 0.0))
    parts = e @ _pages_of(s, s["v_pages"], s["v_scale"], shared), ref, e.sum(-1, keepdim=True)
    # back to the requests' order
    g = torch.searchsorted(cu, torch.arange(M, device=dev), right=True) - 1
    at = torch.arange(M, device=dev) - first[g]
    o1, m1, l1 = (x.view(len(size), n_kv, s["most_rows"], per, -1)[g, :, at] for x in parts)
    # what each request has behind its group's pages
    n_own = _ceil(s["most_own"], page)
    col = pages[g][:, None] + torch.arange(n_own, device=dev)
    mine = s["table"].gather(1, col.clamp(max=s["table"].shape[1] - 1))
    score = q @ _pages_of(s, s["k_pages"], s["k_scale"], mine).transpose(2, 3)
    seen = torch.arange(score.shape[3], device=dev) < (lens - pages[g] * page)[:, None]
    score = score.masked_fill(~seen[:, None, None, :], float("-inf"))
    m2 = score.amax(-1, keepdim=True)
    top = torch.maximum(m1, m2)
    e = torch.exp(score - top)
    f = torch.exp(m1 - top)
    total = l1 * f + e.sum(-1, keepdim=True)
    o = (o1 * f + e @ _pages_of(s, s["v_pages"], s["v_scale"], mine)) / total
    s["o"].copy_(o.reshape(M, n_q * hd))
    s["lse"].copy_((top + total.log()).view(M, n_q))
    return {k: s[k] for k in ("o", "lse")}


def _plain_sample(s):
    # in 64 bits: which token is chosen may hang on the last bits of a sum over the vocabulary
    t = s["temperature"].double()[:, None]
    x, at = s["logits"].sort(dim=1, descending=True, stable=True)  # ranks: equal logits by id
    d = x.double() - x[:, :1].double()
    w = torch.exp(d / torch.where(t > 0, t, 1.0))
    rank = torch.arange(w.shape[1], device=w.device)
    k = s["top_k"].long()[:, None]
    keep = (k <= 0) | (rank < k)
    sums = torch.where(keep, w, 0.0).cumsum(1)
    p = s["top_p"].double()[:, None]
    before = torch.cat([torch.zeros_like(sums[:, :1]), sums[:, :-1]], 1)
    keep &= (p >= 1) | (before < p * sums[:, -1:])
    q = s["min_p"].double()[:, None]
    keep &= (q <= 0) | (w >= q)
    keep &= (t > 0) | (rank == 0)
    keep[:, 0] = True
    w = torch.where(keep, w, 0.0)
    by_id = torch.zeros_like(w).scatter_(1, at, w).cumsum(1)
    total = by_id[:, -1:]
    chosen = torch.searchsorted(by_id, s["u"].double()[:, None] * total, right=True).clamp(max=w.shape[1] - 1)
    s["ids"].copy_(chosen[:, 0])
    mine = torch.exp((s["logits"].gather(1, chosen).double() - x[:, :1].double()) / torch.where(t > 0, t, 1.0))
    s["logprob"].copy_((mine / total).log()[:, 0])
    return {k: s[k] for k in ("ids", "logprob")}


# ----------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    """What run() returns, request by request or row by row in 64 bits; None for whole numbers."""
    s = prepare(case, seed)
    M = case["M"]
    if case["op"] == "sample":
        out = []
        for m, (t, k, p, q) in enumerate(_settings(case)):
            z = s["logits"][m].double()
            # the settings as the 32-bit numbers that the call is given
            t, p, q = float(s["temperature"][m]), float(s["top_p"][m]), float(s["min_p"][m])
            if t <= 0:
                out.append(torch.zeros((), dtype=torch.float64, device=DEV))
                continue
            prob = torch.softmax(z / t, 0)
            order = torch.argsort(prob, descending=True, stable=True)[: k if k > 0 else len(z)]
            best = prob[order]
            mass = best.cumsum(0) - best
            n = int((mass < p * best.sum()).sum()) if p < 1 else len(best)
            live = order[:n][best[:n] >= q * best[0]]
            kept = live.sort().values
            edge = prob[kept].cumsum(0)
            i = int((edge <= float(s["u"][m]) * edge[-1]).sum())
            out.append((prob[kept[min(i, len(kept) - 1)]] / edge[-1]).log())
        return dict(ids=None, logprob=torch.stack(out))
    n_q, n_kv, hd, t, page = (case[k] for k in ("n_q", "n_kv", "hd", "t", "page"))
    cu, prefix, lens = _groups(case)
    o = torch.zeros((M, n_kv, n_q // n_kv, hd), dtype=torch.float64, device=DEV)
    lse = torch.zeros((M, n_kv, n_q // n_kv), dtype=torch.float64, device=DEV)

    def cached(m, lo, n, h):
        """k and v of positions lo .. n - 1 of request m's kv head h."""
        j = torch.arange(lo, n, device=DEV)
        at, sh, local = s["table"][m].long()[j // page], h // (n_kv // t), h % (n_kv // t)
        for name in ("k", "v"):
            pool = s[name + "_pages"]
            if case["kv"] == "e4m3":
                x = pool.view(torch.uint8)[sh, at, local, j % page].view(pool.dtype).double()
                yield x * s[name + "_scale"][h].double()
            else:
                yield pool[sh, at, local, j % page].double()

    for i in range(case["groups"]):
        rows = list(range(cu[i], cu[i + 1]))
        cut = _shared(case, prefix[i])
        for h in range(n_kv):
            qg = s["q"][rows[0]:rows[-1] + 1].double().view(len(rows), n_kv, -1, hd)[:, h] / math.sqrt(hd)
            k, v = cached(rows[0], 0, cut, h)
            w = qg @ k.t()
            for n, m in enumerate(rows):
                k2, v2 = cached(m, cut, lens[m], h)
                both = torch.cat([w[n], qg[n] @ k2.t()], 1)
                lse[m, h] = torch.logsumexp(both, 1)
                both = torch.softmax(both, 1)
                o[m, h] = both[:, :cut] @ v + both[:, cut:] @ v2
    return dict(o=o.view(M, n_q * hd), lse=lse.view(M, n_q))
