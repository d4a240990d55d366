"""Cases of the single-token serving operators: decode attention over the paged cache, eviction from the cache by
accumulated attention weight, and sampling with temperature, top-k, top-p and min-p.

With `own` false, run() computes an operator in its plain form with elementary torch operations; with `own` true it
calls the library.  Both see the same inputs; the cache's pools are plain tensors on one side and the library's own
memory, seen as tensors, on the other.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
INF = float("inf")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one request at the start of an answer, heads of the tiny configuration: the latency of one call
        dict(name="attend_first", op="attend", batch=1, n_q=4, n_kv=2, hd=64, lo=128, hi=128, window=0, score=False),
        # one request of the 0.5B-class shape at a 2048-token context, weights accumulated for a later eviction
        dict(name="attend_single", op="attend", batch=1, n_q=14, n_kv=2, hd=64, lo=2048, hi=2048, window=0, score=True),
        # the benchmark's 8 requests with contexts of 512 to 4096, weights accumulated
        dict(name="attend_mixed8", op="attend", batch=8, n_q=14, n_kv=2, hd=64, lo=512, hi=4096, window=0, score=True),
        # the concurrency workload's 32 requests with contexts of 1024 to 8192 over shuffled pages
        dict(name="attend_paged32", op="attend", batch=32, n_q=14, n_kv=2, hd=64, lo=1024, hi=8192, window=0, score=False),
        # the 7B-class shape, 16 requests at 4096, weights accumulated
        dict(name="attend_seven_b", op="attend", batch=16, n_q=32, n_kv=8, hd=128, lo=4096, hi=4096, window=0, score=True),
        # one long document at the 7B-class shape, an odd length
        dict(name="attend_long", op="attend", batch=1, n_q=32, n_kv=8, hd=128, lo=100003, hi=100003, window=0, score=True),
        # one request's cache over the 24 layers of the 0.5B-class shape cut from 2048 rows to 512
        dict(name="evict_single", op="evict", layers=24, batch=1, n_q=14, n_kv=2, hd=64, lo=2048, hi=2048, budget=512, sinks=4, recent=64),
        # the benchmark's 8 requests cut to 1001 rows (those below stay as they are)
        dict(name="evict_mixed8", op="evict", layers=24, batch=8, n_q=14, n_kv=2, hd=64, lo=512, hi=4096, budget=1001, sinks=4, recent=128),
        # 8 layers of the 7B-class shape, 16 requests at 4096 cut to 1024 rows
        dict(name="evict_seven_b", op="evict", layers=8, batch=16, n_q=32, n_kv=8, hd=128, lo=4096, hi=4096, budget=1024, sinks=4, recent=128),
        # one row of the 7B-class vocabulary, the usual chat settings
        dict(name="sample_one", op="sample", rows=1, vocab=32000, kind="top", masked=0.0),
        # 32 requests of the 0.5B-class vocabulary, each with its own settings, part of the vocabulary masked out
        dict(name="sample_mixed32", op="sample", rows=32, vocab=151936, kind="mixed", masked=0.3),
        # every row of a 32-request block (17 rows each) at a temperature alone
        dict(name="sample_block", op="sample", rows=544, vocab=151936, kind="plain", masked=0.0),
    ]


HEADS = [(4, 2, 64), (14, 2, 64), (32, 8, 128), (6, 6, 64), (10, 2, 128), (3, 1, 128)]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "evict", "sample"])
    if op == "sample":
        vocab = rng.choice([4096, 32000, 151936, log_int(rng, 50, 160001)])
        rows = log_int(rng, 1, max(1, min(544, 80_000_000 // vocab)))
        return dict(op=op, rows=rows, vocab=vocab, kind=rng.choice(["top", "mixed", "mixed", "plain"]), masked=rng.choice([0.0, 0.3, 0.9]))
    n_q, n_kv, hd = rng.choice(HEADS)
    batch = log_int(rng, 1, 32)
    if op == "attend":
        hi = log_int(rng, 1, max(1, min(100000, 60_000_000 // (batch * n_kv * hd))))
        lo = rng.choice([hi, rng.randint(0, hi)])
        return dict(op=op, batch=batch, n_q=n_q, n_kv=n_kv, hd=hd, lo=lo, hi=hi, window=rng.choice([0, 0, log_int(rng, 1, hi)]), score=rng.random() < 0.6)
    layers = log_int(rng, 1, 24)
    hi = log_int(rng, 40, max(40, min(16000, 60_000_000 // (layers * batch * n_kv * hd))))
    lo = rng.choice([hi, rng.randint(0, hi)])
    budget = rng.randint(17, hi)
    sinks = rng.choice([0, 1, 4])
    return dict(op=op, layers=layers, batch=batch, n_q=n_q, n_kv=n_kv, hd=hd, lo=lo, hi=hi, budget=budget, sinks=sinks, recent=rng.randint(0, min(200, budget - sinks)))


def work(case):
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": 4.0 * n + 28.0 * case["rows"], "flops": 4.0 * n}
    pairs = case["batch"] * case["n_kv"]
    mean = (case["lo"] + case["hi"]) / 2
    row = case["hd"] * 2
    if case["op"] == "attend":
        n = mean + 1
        if case["window"]:
            n = min(n, case["window"])
        b = pairs * (n * row * 2 + (8 * n if case["score"] else 0)) + case["batch"] * case["n_q"] * (2 * row + 4) + pairs * 2 * row
        return {"bytes": b, "flops": 4.0 * case["batch"] * case["n_q"] * n * case["hd"]}
    # the share of requests above the budget, and their mean length
    lo, hi, budget = case["lo"], case["hi"], case["budget"]
    cut = 1.0 if lo > budget else max(0.0, (hi - budget) / (hi - lo + 1))
    over = (max(lo, budget + 1) + hi) / 2
    per = 4 * over + 8 * budget + 4 * row * max(0, budget - case["sinks"])
    return {"bytes": case["layers"] * pairs * (cut * per + (1 - cut) * 4 * budget) + 8 * case["batch"], "flops": case["layers"] * pairs * mean}


# ------------------------------------------------------------------ inputs
def generator(seed, salt):
    return torch.Generator(device="cuda").manual_seed((seed * 1000003 + salt) & 0x7FFFFFFF)


def tokens_room(case):
    return max(case["hi"] + 1, 17)


def cache_inputs(case, seed, layers):
    """The page table (shuffled) and the lengths of one cache."""
    ppr = -(-tokens_room(case) // PAGE)
    pages = case["batch"] * ppr
    table = torch.randperm(pages, generator=generator(seed, 1), device="cuda").to(torch.int32).view(case["batch"], ppr)
    lens = torch.randint(case["lo"], case["hi"] + 1, (case["batch"],), generator=generator(seed, 2), device="cuda", dtype=torch.int32)
    return table, lens


MODELS = {}


def own_cache(case, layers, table):
    """The library's cache of this shape and its pools as tensors; the model is made once, as a program keeps it."""
    from speculative_decoding_block_gb300 import binding as B

    key = (layers, case["n_q"], case["n_kv"], case["hd"])
    if key not in MODELS:
        hidden, ffn, vocab = 64, 64, 64
        n = {"wq": case["n_q"] * case["hd"], "wk": case["n_kv"] * case["hd"], "wv": case["n_kv"] * case["hd"]}
        mats = [(n["wq"], hidden), (n["wk"], hidden), (n["wv"], hidden), (hidden, n["wq"]), (ffn, hidden), (ffn, hidden), (hidden, ffn)]
        weights = [torch.zeros(m, dtype=torch.bfloat16, device="cuda") for m in mats]
        cfg = B.ModelConfig(layers, hidden, case["n_q"], case["n_kv"], case["hd"], ffn, vocab, 1e4, 1e-6, 1, 0, 0, 131072)
        embed = torch.zeros((vocab, hidden), dtype=torch.bfloat16, device="cuda")
        MODELS[key] = B.vsd_model_create(cfg, embed, [B.weight_entry("bf16", w) for w in weights] * layers)
    model = MODELS[key]
    kv = B.vsd_kv_create(model, case["batch"], tokens_room(case))
    B.vsd_kv_set_page_table(kv, table)
    return (model, kv) + tuple(B.vsd_kv_pools(kv))


def prepare(case, seed):
    if case["op"] == "sample":
        return prepare_sample(case, seed)
    layers = case.get("layers", 1)
    table, lens = cache_inputs(case, seed, layers)
    s = {"case": case, "table": table, "lens": lens}
    shape = (layers, table.numel(), case["n_kv"], PAGE, case["hd"])
    if own:
        s["model"], s["kv"], s["k_pool"], s["v_pool"] = own_cache(case, layers, table)
    else:
        s["k_pool"], s["v_pool"] = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s["k_pool"].normal_(0.0, 1.0, generator=generator(seed, 3))
    s["v_pool"].normal_(0.0, 1.0, generator=generator(seed, 4))
    batch, n_q, n_kv, hd, room = case["batch"], case["n_q"], case["n_kv"], case["hd"], tokens_room(case)
    if case["op"] == "attend":
        # queries twice the keys' size give scores of a standard deviation of 2: a few heavy rows, a long tail
        s["q"] = (2.0 * torch.randn((batch, n_q, hd), generator=generator(seed, 5), device="cuda")).to(torch.bfloat16)
        s["k_new"] = torch.randn((batch, n_kv, hd), generator=generator(seed, 6), device="cuda").to(torch.bfloat16)
        s["v_new"] = torch.randn((batch, n_kv, hd), generator=generator(seed, 7), device="cuda").to(torch.bfloat16)
        s["out"] = torch.zeros((batch, n_q * hd), dtype=torch.float16, device="cuda")
        s["lse"] = torch.zeros((batch, n_q), dtype=torch.float32, device="cuda")
        # weights of earlier tokens: few rows hold most of the mass
        s["score"] = torch.rand((batch, n_kv, room), generator=generator(seed, 8), device="cuda").pow(8) if case["score"] else None
    else:
        x = torch.randn((layers, batch, n_kv, room), generator=generator(seed, 8), device="cuda")
        # heavy-tailed weights; a tenth of the rows were never attended to and tie at zero
        never = torch.rand((layers, batch, n_kv, room), generator=generator(seed, 9), device="cuda") < 0.1
        s["score"] = torch.where(never, torch.zeros_like(x), torch.exp(2.0 * x))
        s["new_lens"] = torch.zeros_like(lens)
        s["kept"] = torch.zeros((layers, batch, n_kv, case["budget"]), dtype=torch.int32, device="cuda")
    return s


def prepare_sample(case, seed):
    rows, vocab, kind = case["rows"], case["vocab"], case["kind"]
    # a bell of unlikely tokens and some twenty likely ones
    x = 2.0 * torch.randn((rows, vocab), generator=generator(seed, 11), device="cuda")
    likely = torch.randint(0, vocab, (rows, 20), generator=generator(seed, 12), device="cuda")
    x.scatter_add_(1, likely, 4.0 + 8.0 * torch.rand((rows, 20), generator=generator(seed, 13), device="cuda"))
    if case["masked"]:
        hidden = torch.rand((rows, vocab), generator=generator(seed, 14), device="cuda") < case["masked"]
        hidden[:, 7] = False
        x.masked_fill_(hidden, -INF)
    r = torch.rand((6, rows), generator=generator(seed, 15), device="cuda")
    one = torch.ones(rows, device="cuda")
    if kind == "plain":
        t, k, p, m = 0.7 * one, None, None, None
    elif kind == "top":
        t, k, p, m = 0.7 * one, torch.full((rows,), 50, dtype=torch.int32, device="cuda"), 0.9 * one, None
    else:
        # each row its own: a tenth greedy; top-k, top-p and min-p each on half of the rows
        t = torch.where(r[0] < 0.1, 0.0 * one, 0.2 + 1.3 * r[0])
        k = torch.where(r[1] < 0.5, 0.0 * one, torch.floor(10 + 400 * (r[1] - 0.5))).to(torch.int32)
        p = torch.where(r[2] < 0.5, one, 0.5 + 0.49 * r[2])
        m = torch.where(r[3] < 0.5, 0.0 * one, 0.2 * (r[3] - 0.5))
    u = r[4].clamp(1e-6, 1 - 1e-6)
    return {"case": case, "logits": x, "t": t, "k": k, "p": p, "m": m, "u": u, "tokens": torch.zeros(rows, dtype=torch.int32, device="cuda"), "logprob": torch.zeros(rows, dtype=torch.float32, device="cuda")}


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return {"attend": own_attend, "evict": own_evict, "sample": own_sample}[op](s)
    return {"attend": plain_attend, "evict": plain_evict, "sample": plain_sample}[op](s)


def own_attend(s):
    from speculative_decoding_block_gb300 import binding as B

    c = s["case"]
    B.vsd_decode_attention(s["model"], s["kv"], 0, c["batch"], s["lens"], s["q"], s["k_new"], s["v_new"], s["out"], window=c["window"], score=s["score"], lse=s["lse"])
    return s["out"], s["lse"], s["score"], s["k_pool"], s["v_pool"]


def own_evict(s):
    from speculative_decoding_block_gb300 import binding as B

    c = s["case"]
    B.vsd_kv_evict(s["kv"], c["batch"], s["lens"], s["new_lens"], s["score"], c["budget"], sinks=c["sinks"], recent=c["recent"], kept=s["kept"])
    return s["new_lens"], s["kept"], s["score"], s["k_pool"], s["v_pool"]


def own_sample(s):
    from speculative_decoding_block_gb300 import binding as B

    B.vsd_sample_logits(s["logits"], s["u"], s["tokens"], temperature=s["t"], top_k=s["k"], top_p=s["p"], min_p=s["m"], logprob=s["logprob"])
    return s["tokens"], s["logprob"]


def plain_attend(s):
    c, lens, table = s["case"], s["lens"].long(), s["table"].long()
    batch, n_q, n_kv, hd, room = c["batch"], c["n_q"], c["n_kv"], c["hd"], tokens_room(c)
    # the new token's row joins the cache
    page = table.gather(1, (lens // PAGE)[:, None])[:, 0]
    s["k_pool"][0][page, :, lens % PAGE] = s["k_new"]
    s["v_pool"][0][page, :, lens % PAGE] = s["v_new"]
    k, v = (x[0][table].permute(0, 2, 1, 3, 4).reshape(batch, n_kv, -1, hd)[:, :, :room].float() for x in (s["k_pool"], s["v_pool"]))
    i = torch.arange(room, device="cuda")[None, :]
    n = lens[:, None] + 1
    seen = i < n
    if c["window"]:
        seen = seen & (i >= n - c["window"])
    seen4 = seen[:, None, None, :]
    q = s["q"].view(batch, n_kv, n_q // n_kv, hd).float()
    x = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(hd)
    x = torch.where(seen4, x, torch.full_like(x, -INF))
    top = x.amax(3, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(3, keepdim=True)
    p = e / total
    out = torch.matmul(p, torch.where(seen[:, None, :, None], v, torch.zeros_like(v)))
    s["out"].copy_(out.reshape(batch, n_q * hd))
    s["lse"].copy_((top + torch.log(total)).reshape(batch, n_q))
    if s["score"] is not None:
        mass = p.sum(2)
        old = torch.where((i == lens[:, None])[:, None], torch.zeros_like(mass), s["score"])
        s["score"].copy_(torch.where(seen[:, None], old + mass, s["score"]))
    return s["out"], s["lse"], s["score"], s["k_pool"], s["v_pool"]


def plain_evict(s):
    c, lens, table = s["case"], s["lens"].long(), s["table"].long()
    layers, batch, n_kv, room, budget = c["layers"], c["batch"], c["n_kv"], tokens_room(c), c["budget"]
    i = torch.arange(room, device="cuda")
    n = lens[:, None]
    safe = ((i < c["sinks"]) | (i >= n - c["recent"])) & (i < n)
    key = torch.where(safe[None, :, None], torch.full_like(s["score"], INF), s["score"])
    key = torch.where((i < n)[None, :, None], key, torch.full_like(s["score"], -INF))
    order = torch.sort(key, dim=3, descending=True, stable=True)[1][..., :budget]
    rows = torch.sort(order, dim=3)[0]
    if rows.shape[3] < budget:
        rows = torch.cat([rows, rows.new_zeros(rows.shape[:3] + (budget - rows.shape[3],))], 3)
    j = torch.arange(budget, device="cuda")
    new = torch.minimum(lens, torch.full_like(lens, budget))
    live = (j < new[:, None])[None, :, None].expand(layers, batch, n_kv, budget)
    whole = (lens <= budget)[None, :, None, None]
    rows = torch.where(whole, j.expand_as(rows), rows)
    s["kept"].copy_(torch.where(live, rows, torch.full_like(rows, -1)))
    s["new_lens"].copy_(new)
    # the kept rows, read before any is written
    at = torch.nonzero(live & ~whole)
    layer, b, h, to = at.unbind(1)
    src = rows[layer, b, h, to]
    from_page, to_page = table[b, src // PAGE], table[b, to // PAGE]
    for pool in (s["k_pool"], s["v_pool"]):
        pool[layer, to_page, h, to % PAGE] = pool[layer, from_page, h, src % PAGE]
    s["score"][layer, b, h, to] = s["score"][layer, b, h, src]
    return s["new_lens"], s["kept"], s["score"], s["k_pool"], s["v_pool"]


def plain_sample(s):
    x = s["logits"].double()
    rows, vocab = x.shape
    t = s["t"].double()[:, None]
    w = torch.exp((x - x.amax(1, keepdim=True)) / torch.where(t > 0, t, torch.ones_like(t)))
    order = torch.sort(x, dim=1, descending=True, stable=True)[1]
    ws = w.gather(1, order)
    rank = torch.arange(vocab, device="cuda")[None, :]
    keep = torch.ones_like(ws, dtype=torch.bool)
    if s["k"] is not None:
        k = s["k"].long()[:, None]
        keep = keep & ((rank < k) | (k <= 0))
    if s["p"] is not None:
        p = s["p"].double()[:, None]
        ks = ws * keep
        before = torch.cumsum(ks, 1) - ks
        keep = keep & ((before < p * ks.sum(1, keepdim=True)) | (p >= 1))
    if s["m"] is not None:
        keep = keep & (ws >= s["m"].double()[:, None])
    keep = torch.where(t > 0, keep & (ws > 0), rank == 0)
    kept = torch.zeros_like(w).scatter_(1, order, ws * keep)
    total = torch.cumsum(kept, 1)
    last = total[:, -1:]
    token = torch.searchsorted(total, s["u"].double()[:, None] * last)
    s["tokens"].copy_(token[:, 0])
    s["logprob"].copy_(torch.log(kept.gather(1, token) / last)[:, 0])
    return s["tokens"], s["logprob"]


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"attend": exact_attend, "evict": exact_evict, "sample": exact_sample}[case["op"]](s)


def cache_rows(s, pool, layer, b, n):
    """The first n rows of request b in order: [n_kv, n, hd]."""
    pages = s["table"][b, : -(-n // PAGE)].long()
    x = pool[layer].index_select(0, pages).transpose(0, 1)
    return x.reshape(x.shape[0], -1, x.shape[3])[:, :n]


def exact_attend(s):
    """Request by request, KV head by KV head, with the new row beside the cache until the end."""
    c = s["case"]
    g = c["n_q"] // c["n_kv"]
    out = torch.zeros((c["batch"], c["n_q"], c["hd"]), dtype=torch.float64, device="cuda")
    lse = torch.zeros((c["batch"], c["n_q"]), dtype=torch.float64, device="cuda")
    score = None if s["score"] is None else s["score"].double()
    k_pool, v_pool = s["k_pool"].clone(), s["v_pool"].clone()
    for b, n in enumerate(s["lens"].tolist()):
        first = max(0, n + 1 - c["window"]) if c["window"] else 0
        k = torch.cat([cache_rows(s, s["k_pool"], 0, b, n), s["k_new"][b][:, None]], 1)
        v = torch.cat([cache_rows(s, s["v_pool"], 0, b, n), s["v_new"][b][:, None]], 1)
        for h in range(c["n_kv"]):
            a = s["q"][b, h * g : (h + 1) * g].double() @ k[h, first:].double().T * c["hd"] ** -0.5
            z = torch.logsumexp(a, 1, keepdim=True)
            w = torch.exp(a - z)
            lse[b, h * g : (h + 1) * g] = z[:, 0]
            out[b, h * g : (h + 1) * g] = w @ v[h, first:].double()
            if score is not None:
                score[b, h, n] = 0
                score[b, h, first : n + 1] += w.sum(0)
        page = int(s["table"][b, n // PAGE])
        k_pool[0, page, :, n % PAGE] = s["k_new"][b]
        v_pool[0, page, :, n % PAGE] = s["v_new"][b]
    return out.view(c["batch"], -1), lse, score, k_pool, v_pool


def exact_evict(s):
    """By the smallest kept weight of each head: everything above it, and of its equals the first ones."""
    c = s["case"]
    score, k_pool, v_pool = s["score"].double(), s["k_pool"].clone(), s["v_pool"].clone()
    for b, n in enumerate(s["lens"].tolist()):
        if n <= c["budget"]:
            continue
        lo, hi = c["sinks"], n - c["recent"]
        need = c["budget"] - c["sinks"] - c["recent"]
        x = score[:, b, :, :n].clone()
        mid = x[:, :, lo:hi]
        keep = torch.ones(x.shape, dtype=torch.bool, device="cuda")
        if need:
            edge = mid.kthvalue(mid.shape[2] - need + 1, dim=2, keepdim=True)[0]
            room = need - (mid > edge).sum(2, keepdim=True)
            tie = mid == edge
            keep[:, :, lo:hi] = (mid > edge) | (tie & (tie.long().cumsum(2) <= room))
        else:
            keep[:, :, lo:hi] = False
        rows = keep.nonzero()[:, 2].view(c["layers"], c["n_kv"], c["budget"])
        score[:, b, :, : c["budget"]] = x.gather(2, rows)
        pages = s["table"][b].long()
        to = torch.arange(c["budget"], device="cuda")
        for old, new in ((s["k_pool"], k_pool), (s["v_pool"], v_pool)):
            for layer in range(c["layers"]):
                seq = cache_rows(s, old, layer, b, n)
                got = seq.gather(1, rows[layer][..., None].expand(-1, -1, c["hd"]))
                new[layer][pages[to // PAGE], :, to % PAGE] = got.transpose(0, 1)
    return None, None, score, k_pool, v_pool


def exact_sample(s):
    """Row by row on the host, in the order of falling logits."""
    c = s["case"]
    x_all = s["logits"].cpu().numpy()
    host = {n: None if s[n] is None else s[n].cpu().numpy().astype(np.float64) for n in ("t", "k", "p", "m", "u")}
    got = np.zeros(c["rows"], np.float64)
    for r in range(c["rows"]):
        x = x_all[r].astype(np.float64)
        t, k, p, m = (1.0 if host[n] is None and n == "p" else 0.0 if host[n] is None else float(host[n][r]) for n in ("t", "k", "p", "m"))
        if t <= 0:
            continue
        w = np.exp((x - x.max()) / t)
        if k > 0 or p < 1 or m > 0:
            # only tokens that can be kept are put in order
            ids = np.arange(len(x))
            if 0 < k < len(x):
                ids = np.nonzero(x >= np.partition(x, len(x) - int(k))[len(x) - int(k)])[0]
            ids = ids[np.argsort(-x[ids], kind="stable")]
            if k > 0:
                ids = ids[: int(k)]
            if p < 1:
                mass = np.cumsum(w[ids])
                ids = ids[: int(np.searchsorted(mass, p * mass[-1])) + 1]
            ids = np.sort(ids[w[ids] >= m])
        else:
            ids = np.arange(len(x))
        mass = np.cumsum(w[ids])
        v = ids[int(np.searchsorted(mass, host["u"][r] * mass[-1]))]
        got[r] = math.log(w[v] / mass[-1])
    return None, got
