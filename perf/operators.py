"""Cases of the paged-cache operators: writing tokens into pages, attention of one new token,
attention of a prompt's tokens (both causal, with an optional sliding window and first tokens
that stay visible), attention weights summed by key, and eviction by those weights.

With `own` false every operator is computed in its plain form with elementary torch operations in
fp32; with `own` true by the calls of compressed_kv_cache_dkv_gb300.dkv.

The cache: pools of pages, `page` tokens each, for `hkv` heads of `d` channels.  A sequence's token t
lies in page table[b][t // page], slot t % page.  A query at position p sees token t when t <= p and
(no window, or t > p - window, or t < sinks).  Scores are q . k / sqrt(d).
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _case(name, op, **kw):
    base = dict(name=name, op=op, dtype="fp16", b=1, hq=12, hkv=2, d=128, page=64, order="head", len_min=1,
                len_max=1, tq=0, window=0, sinks=0, weights=False, budget=0, first=0, recent=0)
    assert set(kw) <= set(base), kw
    return base | kw


def listed():
    return [
        # one decode step of 16 sequences writes its tokens (12 query / 2 KV heads, d 128): latency
        _case("append_step", "append", b=16, page=64, len_min=900, len_max=2000, tq=1),
        # prompts of up to 4096 tokens enter the cache, padded to one length, token-major pages
        _case("append_prompts", "append", dtype="bf16", b=8, hq=32, hkv=8, page=16, order="token", len_min=700,
              len_max=4096, tq=4096),
        # one short sequence decodes: latency
        _case("decode_one", "decode", b=1, page=64, len_min=1000, len_max=1000),
        # a serving batch of uneven sequences with a sliding window and 4 sinks, pages of 16
        _case("decode_window", "decode", dtype="bf16", b=64, hq=32, hkv=8, page=16, order="token", len_min=300,
              len_max=8000, window=4096, sinks=4),
        # 16 sequences of 64k tokens, every token visible, the weights kept for a later eviction
        _case("decode_long_weights", "decode", b=16, page=256, len_min=65536, len_max=65536, weights=True),
        # a chunk of 32 new tokens for each of 4 sequences, d 64, equal heads, odd lengths
        _case("prefill_chunk", "prefill", b=4, hq=8, hkv=8, d=64, page=32, len_min=333, len_max=2001, tq=32),
        # a 16k prompt through a sliding window of 1024 and 4 sinks
        _case("prefill_window", "prefill", b=1, page=64, len_min=16384, len_max=16384, tq=16384, window=1024, sinks=4),
        # an 8k prompt, causal, no window
        _case("prefill_full", "prefill", dtype="bf16", b=1, hq=32, hkv=8, page=16, order="token", len_min=8191,
              len_max=8191, tq=8191),
        # the last 32 tokens of 8 prompts weigh the cache before it is cut down
        _case("weights_last", "weights", dtype="bf16", b=8, hq=32, hkv=8, page=16, order="token", len_min=2000,
              len_max=8192, tq=32),
        # a whole prompt weighs its own keys
        _case("weights_prompt", "weights", b=1, page=64, len_min=8192, len_max=8192, tq=8192),
        # two sequences go over their budget by a few pages: latency
        _case("evict_few", "evict", b=2, page=64, len_min=2304, len_max=2304, weights=True, budget=2048, first=4,
              recent=256),
        # a batch is cut to half, pages of 16, uneven lengths, some below the budget
        _case("evict_half", "evict", dtype="bf16", b=32, hq=32, hkv=8, page=16, order="token", len_min=2500,
              len_max=8192, weights=True, budget=4096, first=4, recent=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["append", "decode", "decode", "prefill", "prefill", "weights", "evict"])
        hkv = rng.choice([1, 2, 4, 8])
        c = _case("", op, dtype=rng.choice(["fp16", "bf16"]), hkv=hkv, hq=hkv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8]),
                  d=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128, 256]), order=rng.choice(["head", "token"]))
        del c["name"]
        hi = {"append": 8192, "decode": 65536, "prefill": 16384, "weights": 16384, "evict": 32768}[op]
        c["b"] = _log(rng, 1, 64)
        c["len_max"] = _log(rng, 64, hi)
        c["len_min"] = max(1, int(c["len_max"] * rng.uniform(0.2, 1.0)))
        if op == "append":
            c["tq"] = rng.choice([1, 1, _log(rng, 2, c["len_max"])])
        if op in ("prefill", "weights"):
            c["tq"] = rng.choice([_log(rng, 1, 64), c["len_max"], _log(rng, 1, c["len_max"])])
            c["tq"] = min(c["tq"], c["len_max"])
        if op in ("decode", "prefill", "weights") and rng.random() < 0.6:
            c["window"] = _log(rng, 16, 8192)
            c["sinks"] = rng.choice([0, 1, 4, 70])
        if op == "decode":
            c["weights"] = rng.random() < 0.4
        if op == "evict":
            c["weights"] = True
            c["budget"] = max(16, int(c["len_max"] * rng.uniform(0.2, 0.95)))
            c["first"] = rng.choice([0, 1, 4])
            c["recent"] = rng.randrange(0, c["budget"] // 2 + 1)
        kv = c["b"] * hkv * c["len_max"] * c["d"]
        scores = c["b"] * c["hq"] * c["tq"] * c["len_max"] if op in ("prefill", "weights") else 0
        if kv <= 2 ** 28 and scores <= 2 ** 31:
            return c


def _counts(c):
    """Tokens in the cache and new tokens of every sequence: fixed by the case, spread over its range."""
    lens = []
    for i in range(c["b"]):
        f = (i * 0.6180339887498949 + 1.0) % 1.0 if c["b"] > 1 else 1.0
        f = 1.0 if i == 0 else f
        lens.append(c["len_min"] + int((c["len_max"] - c["len_min"]) * f))
    # new tokens: the last tq of each sequence (padded where it has fewer)
    return lens, [min(c["tq"], n) for n in lens]


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 9176 + 11)
    dt, dev = DTYPES[c["dtype"]], torch.device("cuda")
    b, hq, hkv, d, page = c["b"], c["hq"], c["hkv"], c["d"], c["page"]
    lens, news = _counts(c)
    width = -(-max(lens) // page)
    used = [-(-n // page) for n in lens]
    keep = -(-c["budget"] // page) if c["op"] == "evict" else 0
    n_pages = sum(used) + b * keep + 3
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    at = torch.arange(width, device=dev)
    starts = torch.tensor([sum(used[:i]) for i in range(b)], device=dev)
    have = torch.tensor(used, device=dev)
    table = torch.where(at[None] < have[:, None], perm[(starts[:, None] + at[None]).clamp(max=n_pages - 1)], -1)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).mul_(scale).to(dt)

    def pool(scale, shift):
        shape = (n_pages, hkv, page, d) if c["order"] == "head" else (n_pages, page, hkv, d)
        x = normal(*shape, scale=scale)
        x += normal(*((hkv, 1, d) if c["order"] == "head" else (hkv, d)), scale=shift)  # a mean of each head's channels
        return x if c["order"] == "head" else x.transpose(1, 2)

    s = {"case": c, "k": pool(1.0, 0.5), "v": pool(1.0, 0.3), "table": table.to(torch.int32).contiguous(),
         "lens": torch.tensor(lens, dtype=torch.int32, device=dev), "news": torch.tensor(news, dtype=torch.int32, device=dev)}
    tq, op = c["tq"], c["op"]
    if op == "append":
        # K and V as a projection leaves them: [b][token][head][d]
        s["k_new"] = normal(b, tq, hkv, d).transpose(1, 2)
        s["v_new"] = normal(b, tq, hkv, d).transpose(1, 2)
        s["pos"] = s["lens"] - s["news"]
    if op == "decode":
        s["q"] = normal(b, hq, d, scale=2.0)
        s["out"] = torch.zeros(b, hq, d, dtype=dt, device=dev)
        s["lse"] = torch.zeros(b, hq, device=dev)
    if op in ("prefill", "weights"):
        s["q"] = normal(b, tq, hq, d, scale=2.0).transpose(1, 2)
    if op == "prefill":
        s["out"] = torch.zeros(b, tq, hq, d, dtype=dt, device=dev).transpose(1, 2)
        s["lse"] = torch.zeros(b, hq, tq, device=dev)
    if c["weights"] or op == "weights":
        # weights summed so far: many small, a few large
        s["weights"] = torch.rand(b, hkv, width * page, generator=g, device=dev).pow_(8)
    if op == "weights":
        s["lse"] = _plain_lse(s)
    if op == "evict":
        s["new_table"] = perm[sum(used):sum(used) + b * keep].view(b, keep).contiguous()
        s["kept"] = torch.zeros(b, hkv, c["budget"], dtype=torch.int32, device=dev)
        s["new_lens"] = torch.zeros(b, dtype=torch.int32, device=dev)
        s["new_weights"] = torch.zeros(b, hkv, width * page, device=dev)
    if own:
        from compressed_kv_cache_dkv_gb300 import dkv
        s["p"] = dkv.dkv_paged_layout(s["k"], b, hq, width, window=c["window"], sinks=c["sinks"])
        s["ws"] = torch.zeros(dkv.dkv_paged_workspace_bytes(s["p"], c["weights"]), dtype=torch.uint8, device=dev)
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return {"append": _append, "decode": _decode, "prefill": _prefill, "weights": _weights, "evict": _evict}[op](s)


def _own(s, op):
    from compressed_kv_cache_dkv_gb300 import dkv
    if op == "append":
        dkv.dkv_paged_append(s["p"], s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["pos"], counts=s["news"],
                             workspace=s["ws"])
        return s["k"], s["v"]
    if op == "decode":
        out, lse = dkv.dkv_paged_decode(s["p"], s["q"], s["k"], s["v"], s["table"], s["lens"], out=s["out"],
                                        lse=s["lse"], weights=s.get("weights"), workspace=s["ws"])
        return (out, lse, s["weights"]) if "weights" in s else (out, lse)
    if op == "prefill":
        return dkv.dkv_paged_prefill(s["p"], s["q"], s["k"], s["v"], s["table"], s["lens"], q_lens=s["news"],
                                     out=s["out"], lse=s["lse"], workspace=s["ws"])
    if op == "weights":
        return dkv.dkv_paged_weights(s["p"], s["q"], s["lse"], s["k"], s["table"], s["lens"], s["weights"],
                                     q_lens=s["news"], workspace=s["ws"])
    c = s["case"]
    kept, new_lens, new_weights = dkv.dkv_paged_evict(
        s["p"], s["k"], s["v"], s["table"], s["lens"], s["weights"], c["budget"], c["first"], c["recent"],
        s["new_table"], kept=s["kept"], new_lens=s["new_lens"], new_weights=s["new_weights"], workspace=s["ws"])
    return kept, new_lens, new_weights, s["k"], s["v"]


# ---------------------------------------------------------------- plain forms

def _gathered(pool, table):
    """The sequences' rows in fp32: [b][hkv][tokens][d] (unused pages read page 0)."""
    x = pool[table.clamp(min=0).long()].float()          # [b][pages][hkv][page][d]
    x = x.transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[4])


def _scores(s, q):
    """Masked scores of q [b][hq][tq][d] in fp32: [b][hkv][g * tq][tokens], -inf where a token is not seen."""
    c = s["case"]
    b, hq, tq, d = q.shape
    hkv = c["hkv"]
    k = _gathered(s["k"], s["table"])
    x = (q.float() / math.sqrt(d)).reshape(b, hkv, (hq // hkv) * tq, d) @ k.transpose(2, 3)
    t = torch.arange(k.shape[2], device=q.device)
    new = s["news"] if c["tq"] else torch.ones_like(s["lens"])
    pos = (s["lens"] - new)[:, None] + torch.arange(tq, device=q.device)[None]           # [b][tq]
    seen = (t <= pos[..., None]) & (torch.arange(tq, device=q.device)[None] < new[:, None])[..., None]
    if c["window"]:
        seen &= (t > pos[..., None] - c["window"]) | (t < c["sinks"])
    x = x.view(b, hkv, hq // hkv, tq, -1)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    return x.view(b, hkv, -1, x.shape[-1])


def _softmax(x):
    """In place: the weights of each row and their natural log-sum-exp; a row without tokens has weights 0, -inf."""
    m = x.amax(-1, keepdim=True)
    safe = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x.sub_(safe).exp_()
    n = x.sum(-1, keepdim=True)
    lse = (safe + n.log()).squeeze(-1)
    x.div_(torch.where(n == 0, torch.ones_like(n), n))
    return x, lse


def _plain_lse(s):
    c = s["case"]
    _, lse = _softmax(_scores(s, s["q"]))
    return lse.view(c["b"], c["hq"], c["tq"])


def _append(s):
    page = s["case"]["page"]
    i = torch.arange(s["k_new"].shape[2], device=s["k"].device)
    b_at, i_at = (i[None] < s["news"][:, None]).nonzero(as_tuple=True)
    t = s["pos"].long()[b_at] + i_at
    pages, slots = s["table"][b_at, t // page].long(), t % page
    s["k"][pages, :, slots] = s["k_new"][b_at, :, i_at]
    s["v"][pages, :, slots] = s["v_new"][b_at, :, i_at]
    return s["k"], s["v"]


def _decode(s):
    c = s["case"]
    p, lse = _softmax(_scores(s, s["q"][:, :, None]))
    out = p @ _gathered(s["v"], s["table"])
    out, lse = out.view(c["b"], c["hq"], c["d"]).to(s["q"].dtype), lse.view(c["b"], c["hq"])
    if not c["weights"]:
        return out, lse
    s["weights"] += p.sum(2)
    return out, lse, s["weights"]


def _prefill(s):
    c = s["case"]
    p, lse = _softmax(_scores(s, s["q"]))
    out = (p @ _gathered(s["v"], s["table"])).view(c["b"], c["hq"], c["tq"], c["d"])
    real = (torch.arange(c["tq"], device=out.device) < s["news"][:, None])[:, None]      # rows past a sequence's stay
    s["out"].copy_(torch.where(real[..., None], out, s["out"]))
    s["lse"].copy_(torch.where(real, lse.view(c["b"], c["hq"], c["tq"]), s["lse"]))
    return s["out"], s["lse"]


def _weights(s):
    c = s["case"]
    x = _scores(s, s["q"])
    lse = s["lse"].view(c["b"], c["hkv"], -1, 1)
    x.sub_(torch.where(lse == -math.inf, torch.zeros_like(lse), lse)).exp_()
    s["weights"] += x.sum(2)
    return s["weights"]


def _evict(s):
    c = s["case"]
    page, budget = c["page"], c["budget"]
    b, hkv, cap = s["weights"].shape
    t = torch.arange(cap, device=s["k"].device)
    lens = s["lens"].long()[:, None, None]
    w = s["weights"].clone()
    w[(((t < c["first"]) | (t >= lens - c["recent"])) & (t < lens)).expand_as(w)] = math.inf
    w[(t >= lens).expand_as(w)] = -math.inf
    new = lens.clamp(max=budget)                                                          # [b][1][1]
    j = torch.arange(budget, device=t.device)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices                   # ties: the lowest token
    order = torch.nn.functional.pad(order, (0, max(0, budget - cap)))[..., :budget]
    kept = torch.where(j < new, order, cap).sort(-1).values
    live = (j < new).expand(b, hkv, budget)
    src = kept.clamp(max=cap - 1)
    old_pages = s["table"].clamp(min=0).long()[:, None].expand(b, hkv, -1).gather(2, src // page)
    new_pages = s["new_table"].long()[:, None, j // page].expand(b, hkv, budget)
    heads = torch.arange(hkv, device=t.device)[None, :, None].expand(b, hkv, budget)
    slots = (j % page).expand(b, hkv, budget)
    for x in (s["k"], s["v"]):
        x[new_pages[live], heads[live], slots[live]] = x[old_pages[live], heads[live], (src % page)[live]]
    weights = torch.zeros_like(s["weights"])
    n = min(budget, cap)
    weights[..., :n] = (s["weights"].gather(2, src) * live)[..., :n]
    return torch.where(live, kept, -1).to(torch.int32), new.view(b).to(torch.int32), weights, s["k"], s["v"]


# ---------------------------------------------------------------- work and the 64-bit definition

def _seen(c, p):
    """Tokens that a query at position p sees."""
    if not c["window"] or p + 1 <= c["window"]:
        return p + 1
    return c["window"] + min(c["sinks"], p + 1 - c["window"])


def work(c):
    lens, news = _counts(c)
    row, g = 2 * c["d"], c["hq"] // c["hkv"]
    if c["op"] == "append":
        return {"bytes": 4 * row * c["hkv"] * sum(news), "flops": 0}
    if c["op"] == "decode":
        n = sum(_seen(c, x - 1) for x in lens)
        extra = 8 * n * c["hkv"] if c["weights"] else 0
        return {"bytes": 2 * row * c["hkv"] * n + 2 * row * c["hq"] * c["b"] + extra, "flops": 4 * c["hq"] * c["d"] * n}
    if c["op"] == "evict":
        kept = sum(min(x, c["budget"]) for x in lens)
        return {"bytes": c["hkv"] * (4 * row * kept + 4 * sum(lens) + 8 * kept), "flops": 0}
    pairs = sum(sum(_seen(c, x - n + i) for i in range(n)) for x, n in zip(lens, news))
    # keys that some query sees: the first query's window start on, and the sinks
    keys = 0
    for x, n in zip(lens, news):
        lo = max(0, x - n - c["window"] + 1) if c["window"] else 0
        keys += x - lo + min(c["sinks"], lo)
    if c["op"] == "prefill":
        return {"bytes": 2 * row * c["hkv"] * keys + 2 * row * c["hq"] * sum(news), "flops": 4 * c["hq"] * c["d"] * pairs}
    return {"bytes": row * c["hkv"] * keys + row * c["hq"] * sum(news) + 8 * c["hkv"] * keys,
            "flops": 2 * c["hq"] * c["d"] * pairs}


def exact(c, seed):
    """The operators' definitions in 64 bits, one sequence and head at a time."""
    s = prepare(c, seed)
    lens, news = _counts(c)
    op, page, d, g = c["op"], c["page"], c["d"], c["hq"] // c["hkv"]
    if op == "append":
        for i, (n, new) in enumerate(zip(lens, news)):
            for h in range(c["hkv"]):
                t = torch.arange(n - new, n, device="cuda")
                at = s["table"][i].long()[t // page]
                s["k"][at, h, t % page] = s["k_new"][i, h, :new]
                s["v"][at, h, t % page] = s["v_new"][i, h, :new]
        return s["k"], s["v"]

    def rows(pool, i, h, t):
        return pool[s["table"][i].long()[t // page], h, t % page]

    if op == "evict":
        kept, weights = s["kept"].fill_(-1), s["new_weights"].zero_()
        k, v = s["k"].clone(), s["v"].clone()
        for i, n in enumerate(lens):
            m = min(n, c["budget"])
            for h in range(c["hkv"]):
                w = s["weights"][i, h, :n].double().cpu().numpy()
                must = set(range(min(c["first"], n))) | set(range(max(0, n - c["recent"]), n))
                rest = sorted((t for t in range(n) if t not in must), key=lambda t: (-w[t], t))
                pick = sorted(list(must) + rest[:m - len(must)]) if n > m else list(range(n))
                t = torch.tensor(pick, device="cuda")
                j = torch.arange(m, device="cuda")
                kept[i, h, :m] = t.int()
                weights[i, h, :m] = s["weights"][i, h][t]
                to = s["new_table"][i].long()[j // page]
                k[to, h, j % page] = rows(s["k"], i, h, t)
                v[to, h, j % page] = rows(s["v"], i, h, t)
            s["new_lens"][i] = m
        return kept, s["new_lens"], weights, k, v

    tq = c["tq"] or 1
    q = s["q"][:, :, None] if op == "decode" else s["q"]
    out = torch.zeros(c["b"], c["hq"], tq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(c["b"], c["hq"], tq, dtype=torch.float64, device="cuda")
    weights = s["weights"].double() if "weights" in s else None
    step = max(1, 2 ** 28 // max(lens))
    for i, n in enumerate(lens):
        new = news[i] if c["tq"] else 1
        t = torch.arange(n, device="cuda")
        for h in range(c["hkv"]):
            k, v = rows(s["k"], i, h, t).double(), rows(s["v"], i, h, t).double()
            for j in range(h * g, h * g + g):
                for a in range(0, new, step):
                    e = min(new, a + step)
                    p = torch.arange(n - new + a, n - new + e, device="cuda")[:, None]
                    x = (q[i, j, a:e].double() @ k.T) * d ** -0.5
                    hide = t > p
                    if c["window"]:
                        hide |= (t <= p - c["window"]) & (t >= c["sinks"])
                    x[hide] = -math.inf
                    if op == "weights":
                        weights[i, h, :n] += (x - s["lse"][i, j, a:e].double()[:, None]).exp().sum(0)
                        continue
                    top = x.max(1, keepdim=True).values
                    x = (x - top).exp()
                    total = x.sum(1, keepdim=True)
                    out[i, j, a:e] = (x @ v) / total
                    lse[i, j, a:e] = (top + total.log())[:, 0]
                    if weights is not None:
                        weights[i, h, :n] += (x / total).sum(0)
    if op == "weights":
        return weights
    if op == "prefill":
        return out, lse
    return (out[:, :, 0], lse[:, :, 0], weights) if c["weights"] else (out[:, :, 0], lse[:, :, 0])
