"""Cases of the paged decode operators: block tables and slots built from request lengths, rotary
positions with the append into a paged key-value cache, attention of one new token over that cache,
and log probabilities of given tokens.  Each case runs either in a plain form (elementary torch
operations in 32 bits) or, with `own`, through the library's binding.

Head layouts are those of the library's Llama-shaped configurations (8B: 32 q and 8 kv heads of 128,
70B: 64 and 8, 405B-shaped: 128 and 8; vocabulary 128256) and a few generic ones.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
VOCAB = 128256
HEADS = [(32, 8, 128), (64, 8, 128), (128, 8, 128), (16, 16, 64), (8, 4, 256), (16, 2, 64), (24, 8, 128)]
PAGES = [16, 32, 64, 128, 256]
LARGEST_BYTES = 1.0e9  # no drawn case touches more than the largest listed one


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one step of a decode server: every request gets one token, some cross into a new page
        dict(name="tables-decode", op="tables", M=256, page=64, old=8192, new=1, pad=0, mix=1),
        # a batch of prompts admitted at once, pages of 16, the rows padded to the captured size
        dict(name="tables-prefill", op="tables", M=37, page=16, old=300, new=6000, pad=1021, mix=2),
        # the decode step of the 70B heads over 8 shards; three padding rows with no slot
        dict(name="rope-decode", op="rope", M=32, n_q=64, n_kv=8, hd=128, t=8, page=64, kv="bf16", layout="half",
             rot=128, scaling="wavelength", far=131072, holes=3, mix=3),
        # a prefill chunk of the 70B heads
        dict(name="rope-prefill", op="rope", M=8192, n_q=64, n_kv=8, hd=128, t=8, page=16, kv="bf16", layout="half",
             rot=128, scaling="none", far=8192, holes=0, mix=4),
        # a ragged chunk into an e4m3 cache: interleaved pairs on part of the head, long context
        dict(name="rope-e4m3-part", op="rope", M=1003, n_q=32, n_kv=8, hd=128, t=2, page=32, kv="e4m3",
             layout="interleaved", rot=64, scaling="yarn", far=1000000, holes=5, mix=5),
        # the smallest call: one sequence of a few hundred tokens, where latency counts
        dict(name="attn-one-short", op="attn", M=1, n_q=32, n_kv=8, hd=128, t=1, page=16, kv="bf16", longest=519,
             spread="all", window=0, mix=6),
        # one sequence of 128 Ki tokens: all SMs share its length
        dict(name="attn-one-long", op="attn", M=1, n_q=64, n_kv=8, hd=128, t=8, page=64, kv="bf16", longest=131071,
             spread="all", window=0, mix=7),
        # an ordinary decode batch of the 70B heads, ragged, one request without tokens
        dict(name="attn-batch", op="attn", M=32, n_q=64, n_kv=8, hd=128, t=8, page=16, kv="bf16", longest=4096,
             spread="ragged", window=0, mix=8),
        # the 405B heads (16 q heads per kv head) over an e4m3 cache
        dict(name="attn-e4m3-batch", op="attn", M=48, n_q=128, n_kv=8, hd=128, t=4, page=32, kv="e4m3", longest=8192,
             spread="ragged", window=0, mix=9),
        # heads of 256 with a sliding window: the cache before the window is not read
        dict(name="attn-window", op="attn", M=61, n_q=8, n_kv=4, hd=256, t=1, page=128, kv="bf16", longest=6000,
             spread="ragged", window=1024, mix=10),
        # the sampled tokens of one decode step, some vocabulary masked out
        dict(name="logprobs-decode", op="logprobs", M=32, V=VOCAB, k=8, masked=0.2, mix=11),
        # the tokens of a prompt, 20 alternatives each
        dict(name="logprobs-prompt", op="logprobs", M=1900, V=VOCAB, k=20, masked=0.0, mix=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "rope", "rope", "attn", "attn", "attn", "logprobs"])
    mix = rng.randrange(1 << 30)
    if op == "tables":
        M = _log(rng, 1, 2000)
        new = 1 if rng.random() < 0.5 else _log(rng, 2, max(3, min(6000, 200000 // M)))
        return dict(op=op, M=M, page=rng.choice(PAGES), old=_log(rng, 1, 16384), new=new, pad=rng.choice([0, 3, 700]),
                    mix=mix)
    if op == "logprobs":
        V = _log(rng, 500, VOCAB)
        return dict(op=op, M=_log(rng, 1, min(4000, int(LARGEST_BYTES / 4 / V) - 1)), V=V, k=rng.choice([0, 1, 5, 20, 32]),
                    masked=rng.choice([0.0, 0.1, 0.9]), mix=mix)
    n_q, n_kv, hd = rng.choice(HEADS)
    t = rng.choice([s for s in (1, 2, 4, 8) if n_kv % s == 0])
    kv = rng.choice(["bf16", "e4m3"])
    if op == "rope":
        M = _log(rng, 1, 9000 * 8192 // ((n_q + 2 * n_kv) * hd + 8192))
        return dict(op=op, M=M, n_q=n_q, n_kv=n_kv, hd=hd, t=t, page=rng.choice(PAGES), kv=kv,
                    layout=rng.choice(["half", "interleaved"]), rot=rng.choice([hd, hd // 2, hd // 4]),
                    scaling=rng.choice(["none", "linear", "wavelength", "yarn"]), far=_log(rng, 2 * M, 1 << 22),
                    holes=rng.choice([0, M // 9]), mix=mix)
    M = _log(rng, 1, 200)
    longest = _log(rng, 1, min(100000, int(LARGEST_BYTES / 2.5 / (M * n_kv * hd * 2 * 2)) + 1))
    return dict(op=op, M=M, n_q=n_q, n_kv=n_kv, hd=hd, t=t, page=rng.choice(PAGES), kv=kv, longest=longest,
                spread=rng.choice(["ragged", "all"]), window=rng.choice([0, 0, max(1, longest // 3)]), mix=mix)


def _attn_lens(case):
    """Cached tokens of each request, the new one included; ragged batches hold a request without any."""
    if case["spread"] == "all":
        return [case["longest"]] * case["M"]
    r = random.Random(case["mix"])
    lens = [r.randint(1, case["longest"]) for _ in range(case["M"])]
    lens[r.randrange(case["M"])] = case["longest"]
    if case["M"] > 3:
        lens[r.randrange(case["M"])] = 0
    return lens


def _table_lens(case):
    """Tokens each request holds and is to get; now and then one that gets none."""
    r = random.Random(case["mix"])
    old = [r.randint(0, case["old"]) for _ in range(case["M"])]
    new = [1 if case["new"] == 1 else r.randint(0, case["new"]) for _ in range(case["M"])]
    return old, new


def _ceil(a, b):
    return -(-a // b)


def work(case):
    if case["op"] == "tables":
        old, new = _table_lens(case)
        rows, M = sum(new) + case["pad"], case["M"]
        fresh = sum(_ceil(o + n, case["page"]) - _ceil(o, case["page"]) for o, n in zip(old, new))
        return {"bytes": 4 * (2 * M + M + (M + 1) + 2 * rows + 2 * fresh + 3), "flops": 0}
    if case["op"] == "logprobs":
        M, V = case["M"], case["V"]
        return {"bytes": 4 * M * V + M * (16 + 8 * case["k"]), "flops": 6 * M * V}
    n_q, n_kv, hd, M = case["n_q"], case["n_kv"], case["hd"], case["M"]
    size = 2 if case["kv"] == "bf16" else 1
    if case["op"] == "rope":
        kept = M - case["holes"]
        return {"bytes": M * n_q * hd * 4 + kept * 2 * n_kv * hd * (2 + size) + 8 * M,
                "flops": 3 * (M * n_q + kept * n_kv) * case["rot"]}
    n = sum(min(x, case["window"]) if case["window"] else x for x in _attn_lens(case))
    return {"bytes": n * n_kv * hd * 2 * size + M * n_q * hd * 4 + M * n_q * 4, "flops": 4 * n * n_q * hd}


# --------------------------------------------------------------------------------------- the inputs
def _rope_args(case):
    """Rotation parameters as the library's tp_rope_params names them."""
    return dict(rot_dim=case["rot"], theta=500000.0, layout=case["layout"], scaling=case["scaling"], factor=8.0,
                original_len=8192, low_freq_factor=1.0, high_freq_factor=4.0, beta_fast=32.0, beta_slow=1.0)


def _rope_freqs(case):
    """Angle per position of each rotated pair, and the factor on cos and sin, in 64 bits."""
    a = _rope_args(case)
    i = np.arange(a["rot_dim"] // 2, dtype=np.float64)
    f = a["theta"] ** (-2.0 * i / a["rot_dim"])
    if a["scaling"] == "none":
        return f, 1.0
    if a["scaling"] == "linear":
        return f / a["factor"], 1.0
    if a["scaling"] == "wavelength":  # long wavelengths are stretched, short ones kept, a ramp between
        turns = a["original_len"] * f / (2 * math.pi)
        keep = np.clip((turns - a["low_freq_factor"]) / (a["high_freq_factor"] - a["low_freq_factor"]), 0.0, 1.0)
        return f * keep + f / a["factor"] * (1 - keep), 1.0
    def pair_of(turns):  # the (fractional) pair that turns so often over the original length
        return a["rot_dim"] * math.log(a["original_len"] / (turns * 2 * math.pi)) / (2 * math.log(a["theta"]))
    lo = max(0, math.floor(pair_of(a["beta_fast"])))
    hi = min(a["rot_dim"] - 1, math.ceil(pair_of(a["beta_slow"])))
    stretch = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
    return f / a["factor"] * stretch + f * (1 - stretch), 0.1 * math.log(a["factor"]) + 1.0


def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + salt)
    return g


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _pool(g, case, n_pages):
    """Keys or values of a page pool [t][n_pages][n_kv/t][page][hd], and the heads' scales."""
    shape = (case["t"], n_pages, case["n_kv"] // case["t"], case["page"], case["hd"])
    pool = torch.empty(shape, device=DEV, dtype=torch.bfloat16 if case["kv"] == "bf16" else torch.float8_e4m3fn)
    std = 1.0 if case["kv"] == "bf16" else 70.0
    for s in range(shape[0]):
        pool[s] = _normal(g, shape[1:], std, pool.dtype)
    scale = None
    if case["kv"] == "e4m3":
        scale = (torch.rand(case["n_kv"], generator=g, device=DEV) + 0.5) / 70.0
    return pool, scale


def prepare(case, seed):
    g, op, M = _gen(seed, 17), case["op"], case["M"]
    s = dict(case=case)
    if own:
        from megatron_tensor_transformer_gb300 import tpx
        s["tpx"] = tpx
    i32 = dict(dtype=torch.int32, device=DEV)
    if op == "tables":
        old, new = _table_lens(case)
        page, rows = case["page"], sum(new) + case["pad"]
        held = [_ceil(o, page) for o in old]
        most = max(_ceil(o + n, page) for o, n in zip(old, new)) + 2
        fresh = sum(_ceil(o + n, page) for o, n in zip(old, new)) - sum(held)
        n_pages = sum(held) + fresh + 7
        ids = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
        table = torch.full((M, most), -1, **i32)
        at = torch.arange(most, device=DEV)[None, :] < torch.tensor(held, device=DEV)[:, None]
        table[at] = ids[: sum(held)]
        s |= dict(lens=torch.tensor(old, **i32), add=torch.tensor(new, **i32), table=table, n_pages=n_pages,
                  free=ids[sum(held):].clone(), head=torch.tensor([2], **i32), lens_out=torch.zeros(M, **i32),
                  cu=torch.zeros(M + 1, **i32), positions=torch.zeros(rows, **i32), slots=torch.zeros(rows, **i32),
                  counts=torch.zeros(3, **i32))
        if own:
            s["pages"] = tpx.make_pages(page, n_pages, most)
        return s
    if op == "logprobs":
        V = case["V"]
        logits = torch.empty((M, V), device=DEV)
        for a in range(0, M, 256):
            logits[a:a + 256] = torch.randn((min(256, M - a), V), generator=g, device=DEV) * 2.5
        if case["masked"]:
            keep = torch.rand(V, generator=g, device=DEV) >= case["masked"]
            keep[V // 2] = True
            logits.masked_fill_(~keep, float("-inf"))
        # the token that was sampled: mostly among the likely ones
        noise = torch.rand((M, 64), generator=g, device=DEV)
        near = torch.randint(0, V, (M, 64), generator=g, device=DEV)
        ids = near.gather(1, (logits.gather(1, near) + noise).argmax(1, keepdim=True))[:, 0].to(torch.int32)
        f32 = dict(dtype=torch.float32, device=DEV)
        s |= dict(logits=logits, ids=ids, logprob=torch.zeros(M, **f32), entropy=torch.zeros(M, **f32),
                  rank=torch.zeros(M, **i32))
        s["top_logprob"] = torch.zeros((M, case["k"]), **f32) if case["k"] else None
        s["top_id"] = torch.zeros((M, case["k"]), **i32) if case["k"] else None
        return s
    n_q, n_kv, hd, page = case["n_q"], case["n_kv"], case["hd"], case["page"]
    if op == "rope":
        n_pages = _ceil(M, page) + 5
        s["k_pages"], s["k_scale"] = _pool(g, case, n_pages)
        s["v_pages"], s["v_scale"] = _pool(g, case, n_pages)
        s["qkv"] = _normal(g, (M, (n_q + 2 * n_kv) * hd))
        start = torch.randint(0, max(1, case["far"] - M), (1,), generator=g, device=DEV)
        # a run of positions for a chunk; for a decode batch one position of each request
        s["positions"] = ((start + torch.arange(M, device=DEV)) if M > 256 else
                          torch.randint(0, case["far"], (M,), generator=g, device=DEV)).to(torch.int32)
        order = torch.randperm(n_pages, generator=g, device=DEV)
        at = torch.arange(M, device=DEV)
        slots = order[at // page] * page + at % page
        if case["holes"]:
            slots[M - case["holes"]:] = -1
        s["slots"] = slots.to(torch.int32)
        f, m = _rope_freqs(case)
        s["freqs"], s["mscale"] = torch.from_numpy(f).to(DEV), m
        s["q"] = torch.zeros((M, n_q * hd), dtype=torch.bfloat16, device=DEV)
        if own:
            s["shape"] = tpx.make_shape(n_q * hd, n_q=n_q, n_kv=n_kv, hd=hd, t=case["t"])
            s["pages"] = tpx.make_pages(page, n_pages, n_pages, tpx.TP_BF16 if case["kv"] == "bf16" else tpx.TP_FP8_E4M3)
            args = _rope_args(case)
            for word in ("layout", "scaling"):
                args[word] = getattr(tpx, "TP_ROPE_" + args[word].upper())
            s["rope"] = tpx.make_rope(**args)
        return s
    lens = _attn_lens(case)
    held = [_ceil(n, page) for n in lens]
    most, n_pages = max(1, max(held)) + 1, sum(held) + 3
    s["k_pages"], s["k_scale"] = _pool(g, case, n_pages)
    s["v_pages"], s["v_scale"] = _pool(g, case, n_pages)
    table = torch.full((M, most), -1, **i32)
    at = torch.arange(most, device=DEV)[None, :] < torch.tensor(held, device=DEV)[:, None]
    table[at] = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)[: sum(held)]
    s |= dict(table=table, lens=torch.tensor(lens, **i32), q=_normal(g, (M, n_q * hd), 1.5),
              o=torch.zeros((M, n_q * hd), dtype=torch.bfloat16, device=DEV),
              lse=torch.zeros((M, n_q), dtype=torch.float32, device=DEV), longest=max(lens))
    if own:
        s["shape"] = tpx.make_shape(n_q * hd, n_q=n_q, n_kv=n_kv, hd=hd, t=case["t"])
        s["pages"] = tpx.make_pages(page, n_pages, most, tpx.TP_BF16 if case["kv"] == "bf16" else tpx.TP_FP8_E4M3)
        s["ws"] = tpx.new_paged_attn_workspace(s["shape"], DEV)
    return s


# -------------------------------------------------------------------------------------- the passes
def run(s):
    op = s["case"]["op"]
    if own:
        tpx = s["tpx"]
        if op == "tables":
            tpx.tp_paged_tables(s["pages"], s["lens"], s["add"], s["free"], s["table"], s["lens_out"], s["cu"],
                                s["positions"], s["slots"], s["counts"], head=s["head"])
            return {k: s[k] for k in ("table", "lens_out", "cu", "positions", "slots", "counts")}
        if op == "rope":
            tpx.tp_rope_append(s["shape"], s["rope"], s["pages"], s["qkv"], s["positions"], s["slots"], s["q"],
                               s["k_pages"], s["v_pages"], k_scale=s["k_scale"], v_scale=s["v_scale"])
            return {k: s[k] for k in ("q", "k_pages", "v_pages")}
        if op == "attn":
            tpx.tp_paged_attn_decode(s["shape"], s["pages"], s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                                     s["o"], s["ws"], lse=s["lse"], window=s["case"]["window"], k_scale=s["k_scale"],
                                     v_scale=s["v_scale"])
            return {k: s[k] for k in ("o", "lse")}
        tpx.tp_token_logprobs(s["logits"], s["ids"], s["logprob"], s["entropy"], s["rank"], s["top_logprob"], s["top_id"])
        return {k: s[k] for k in ("logprob", "entropy", "rank", "top_logprob", "top_id")}
    return {"tables": _plain_tables, "rope": _plain_rope, "attn": _plain_attn, "logprobs": _plain_logprobs}[op](s)


def _plain_tables(s):
    page, rows, table = s["case"]["page"], s["slots"].shape[0], s["table"]
    lens, add = s["lens"].long(), s["add"].long()
    most, n_free = table.shape[1], s["free"].shape[0]
    held = (lens + page - 1) // page
    ends = add.cumsum(0)
    first = ends - add
    fits = (lens + add <= most * page) & (ends <= rows)
    need = torch.where(fits, (lens + add + page - 1) // page - held, 0)
    taken = need.cumsum(0)
    fits &= (need == 0) | (s["head"] + taken <= n_free)
    row = torch.arange(rows, device=table.device)
    m = torch.searchsorted(ends, row, right=True)
    real = m < lens.shape[0]
    m = m.clamp(max=lens.shape[0] - 1)
    pos = lens[m] + row - first[m]
    fresh = pos // page - held[m]  # which of the request's new pages, negative in a page it holds
    got = s["free"][(s["head"] + (taken - need)[m] + fresh).clamp(0, n_free - 1)]
    page_id = torch.where(fresh >= 0, got, table[m, (pos // page).clamp(max=most - 1)]).long()
    live = real & fits[m]
    opens = live & (fresh >= 0) & (pos % page == 0)
    # every row writes: those that open no page write back what their last entry holds
    spot = torch.where(opens, m * most + pos // page, 0)
    value = torch.where(opens, page_id, table[0, 0].long()).to(torch.int32)
    grown = table.flatten().scatter_reduce(0, spot, value, "amax")
    table.copy_(grown.view_as(table))
    s["lens_out"].copy_(torch.where(fits, lens + add, lens))
    s["cu"].copy_(torch.cat([torch.zeros_like(ends[:1]), ends]))
    s["positions"].copy_(torch.where(real, pos, 0))
    s["slots"].copy_(torch.where(live, page_id * page + pos % page, -1))
    s["counts"].copy_(torch.stack([s["head"][0] + torch.where(fits, need, 0).sum(), ends[-1], (~fits).sum()]))
    return {k: s[k] for k in ("table", "lens_out", "cu", "positions", "slots", "counts")}


def _plain_rope(s):
    c = s["case"]
    M, n_q, n_kv, hd, t, rot = c["M"], c["n_q"], c["n_kv"], c["hd"], c["t"], c["rot"]
    x = s["qkv"].float().view(M, t, (n_q + 2 * n_kv) // t, hd)
    qk, v = x[:, :, : (n_q + n_kv) // t], x[:, :, (n_q + n_kv) // t:]
    angle = s["positions"].double()[:, None] * s["freqs"]
    cos, sin = ((f(angle) * s["mscale"]).float()[:, None, None, :] for f in (torch.cos, torch.sin))
    if c["layout"] == "half":
        a, b, rest = qk[..., : rot // 2], qk[..., rot // 2: rot], qk[..., rot:]
        qk = torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    else:
        a, b, rest = qk[..., 0:rot:2], qk[..., 1:rot:2], qk[..., rot:]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        qk = torch.cat([turned, rest], -1)
    s["q"].copy_(qk[:, :, : n_q // t].reshape(M, n_q * hd))
    k = qk[:, :, n_q // t:]
    kept = slice(0, M - c["holes"])  # the rows behind have no slot
    slot = s["slots"][kept].long()
    for new, pool, scale in ((k, s["k_pages"], s["k_scale"]), (v, s["v_pages"], s["v_scale"])):
        if scale is not None:
            new = (new / scale.view(t, n_kv // t, 1)).clamp(-448.0, 448.0)
        raw = pool if pool.dtype == torch.bfloat16 else pool.view(torch.uint8)
        raw[:, slot // c["page"], :, slot % c["page"]] = new[kept].to(pool.dtype).view(raw.dtype)
    return {k: s[k] for k in ("q", "k_pages", "v_pages")}


def _gathered(s, pool, scale):
    """[M, n_kv, longest, hd] in 32 bits: each request's tokens in order, whatever its pages are."""
    c = s["case"]
    held = _ceil(s["longest"], c["page"])
    ids = s["table"][:, :held].long().clamp(min=0)
    raw = pool if pool.dtype == torch.bfloat16 else pool.view(torch.uint8)
    x = raw[:, ids].view(pool.dtype).float()  # [t, M, held, n_kv/t, page, hd]
    x = x.permute(1, 0, 3, 2, 4, 5).reshape(c["M"], c["n_kv"], held * c["page"], c["hd"])[:, :, : s["longest"]]
    return x if scale is None else x * scale[None, :, None, None]


def _plain_attn(s):
    c = s["case"]
    M, n_q, n_kv, hd = c["M"], c["n_q"], c["n_kv"], c["hd"]
    q = s["q"].float().view(M, n_kv, n_q // n_kv, hd)
    score = q @ _gathered(s, s["k_pages"], s["k_scale"]).transpose(2, 3) * (1.0 / math.sqrt(hd))
    pos, n = torch.arange(s["longest"], device=q.device), s["lens"].long()[:, None]
    seen = pos < n
    if c["window"]:
        seen &= pos >= n - c["window"]
    score = score.masked_fill(~seen[:, None, None, :], float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isfinite(top), top, 0.0))
    total = p.sum(-1, keepdim=True)
    o = (p @ _gathered(s, s["v_pages"], s["v_scale"])) / torch.where(total > 0, total, 1.0)
    s["o"].copy_(o.reshape(M, n_q * hd))
    s["lse"].copy_((top + total.log())[..., 0].view(M, n_q))
    return {k: s[k] for k in ("o", "lse")}


def _plain_logprobs(s):
    x, ids, k = s["logits"], s["ids"].long()[:, None], s["case"]["k"]
    V = x.shape[1]
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    lse = top + total.log()
    own_logit = x.gather(1, ids)
    s["logprob"].copy_((own_logit - lse)[:, 0])
    s["entropy"].copy_((lse - (e * torch.where(e > 0, x, 0.0)).sum(1, keepdim=True) / total)[:, 0])
    col = torch.arange(V, device=x.device)
    ahead = (x > own_logit) | ((x == own_logit) & (col < ids))
    s["rank"].copy_(ahead.sum(1) + 1)
    if k:
        # a whole number that orders as (logit, then the lower index first)
        bits = x.view(torch.int32).long()
        key = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF)) * (1 << 20) + (V - col)
        at = key.topk(k, dim=1).indices
        s["top_id"].copy_(at)
        s["top_logprob"].copy_(x.gather(1, at) - lse)
    return {k: s[k] for k in ("logprob", "entropy", "rank", "top_logprob", "top_id")}


# ----------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    """What run() returns, request by request or row by row in 64 bits; None for whole numbers."""
    op = case["op"]
    if op == "tables":
        return None
    s = prepare(case, seed)
    if op == "logprobs":
        logprob, entropy, tops = [], [], []
        for a in range(0, case["M"], 64):
            x = s["logits"][a:a + 64].double()
            lp = x - torch.logsumexp(x, 1, keepdim=True)
            logprob.append(lp.gather(1, s["ids"][a:a + 64].long()[:, None])[:, 0])
            entropy.append(-(lp.exp() * lp.nan_to_num(neginf=0.0)).sum(1))
            if case["k"]:
                tops.append(lp.sort(1, descending=True).values[:, : case["k"]])
        return dict(logprob=torch.cat(logprob), entropy=torch.cat(entropy), rank=None,
                    top_logprob=torch.cat(tops) if tops else None, top_id=None)
    M, n_q, n_kv, hd, t, page = (case[k] for k in ("M", "n_q", "n_kv", "hd", "t", "page"))
    if op == "rope":
        f, mscale = _rope_freqs(case)
        turn = s["positions"].double()[:, None] * torch.from_numpy(f).to(DEV)
        z = torch.polar(torch.full_like(turn, mscale), turn)  # multiplying by z turns a pair
        pairs = torch.arange(case["rot"], device=DEV)
        pairs = pairs.view(2, -1).t() if case["layout"] == "half" else pairs.view(-1, 2)  # [rot/2, 2] dims
        cols = (n_q + 2 * n_kv) // t * hd
        q = torch.empty((M, n_q * hd), dtype=torch.float64, device=DEV)
        pools = [p.double() for p in (s["k_pages"], s["v_pages"])]
        kept = torch.nonzero(s["slots"] >= 0)[:, 0]
        at, off = s["slots"][kept].long() // page, s["slots"][kept].long() % page

        def turned(c0):
            x = s["qkv"][:, c0:c0 + hd].double()
            y = torch.complex(x[:, pairs[:, 0]], x[:, pairs[:, 1]]) * z
            x[:, pairs[:, 0]], x[:, pairs[:, 1]] = y.real, y.imag
            return x

        for h in range(n_q):
            sh, local = h // (n_q // t), h % (n_q // t)
            q[:, h * hd:(h + 1) * hd] = turned(sh * cols + local * hd)
        for h in range(n_kv):
            sh, local = h // (n_kv // t), h % (n_kv // t)
            c0 = sh * cols + (n_q // t + local) * hd
            for i, x in enumerate((turned(c0), s["qkv"][:, c0 + n_kv // t * hd:][:, :hd].double())):
                if case["kv"] == "e4m3":  # the nearest code
                    x = x / s["v_scale" if i else "k_scale"][h].double()
                    x = x.clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
                pools[i][sh, at, local, off] = x[kept]
        return dict(q=q, k_pages=pools[0], v_pages=pools[1])
    o = torch.zeros((M, n_kv, n_q // n_kv, hd), dtype=torch.float64, device=DEV)
    lse = torch.full((M, n_kv, n_q // n_kv), float("-inf"), dtype=torch.float64, device=DEV)
    for m, n in enumerate(_attn_lens(case)):
        j = torch.arange(max(0, n - case["window"]) if case["window"] else 0, n, device=DEV)
        if not len(j):
            continue
        at = s["table"][m].long()[j // page]
        for h in range(n_kv):
            sh, local = h // (n_kv // t), h % (n_kv // t)
            k, v = (s[p][sh].view(torch.uint8)[at, local, j % page].view(s[p].dtype).double()
                    if case["kv"] == "e4m3" else s[p][sh, at, local, j % page].double() for p in ("k_pages", "v_pages"))
            if case["kv"] == "e4m3":
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            w = s["q"][m].double().view(n_kv, -1, hd)[h] @ k.t() / math.sqrt(hd)
            lse[m, h] = torch.logsumexp(w, 1)
            o[m, h] = torch.softmax(w, 1) @ v
    return dict(o=o.view(M, n_q * hd), lse=lse.view(M, n_q))
