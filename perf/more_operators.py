"""Cases of one serving step over a paged cache that is held in 4 bits: page tables and slot maps
from request lengths, norms of queries and keys with the position rotation, writing new keys and
values in 4 bits (and reading them back), attention of one new token and of several.

With `own` false every operator is computed in its plain form with elementary torch operations; with
`own` true by the calls of compressed_kv_cache_dkv_gb300.dkv.

The cache: bytes [n_pages][hkv][page * 9 d / 8].  A page of a head is a row of blocks of 16 tokens, 18 d
bytes each, g = d / 64 groups of 64 channels:
    K codes [g][16 tokens][32 bytes], V codes the same (channel 2 i in the low half of byte i),
    K (scale, bias) [16 tokens][g][2] fp16, V (scale, bias) the same; value = scale * code + bias.
A group is quantised on the grid u of fp16 numbers next to its largest magnitude L:
    u = 2^(floor(log2(65/64 L)) - 10), at least 2^-24;  b = round(min / u);  n = round(max / u) - b;
    s = ceil(n / 15);  code = round((x / u - b) / s) in 0 .. 15;  scale = s u, bias = b u
(ties to even), so that every value is an fp16 number exactly.

A query at position p sees token t when t <= p and (no window, or t > p - window, or t < sinks).
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _case(name, op, **kw):
    base = dict(name=name, op=op, dtype="fp16", b=1, hq=12, hkv=2, d=128, page=64, len_min=1, len_max=1, tq=0, window=0,
                sinks=0, rope=0, base=1e6, pages=False, gain=True, mixed=False)
    assert set(kw) <= set(base), kw
    return base | kw


def listed():
    return [
        # one decode step of 64 sequences takes its pages: latency
        _case("plan_step", "plan", b=64, page=16, len_min=300, len_max=8000, tq=1),
        # 256 requests at once: prompts, single tokens, finished and cut ones, a list that may run out
        _case("plan_mixed", "plan", b=256, page=16, len_min=100, len_max=4096, tq=4096, mixed=True),
        # queries and keys of one decode step of 16 sequences: latency
        _case("rotate_step", "rotate", b=16, len_min=900, len_max=60000, tq=1, rope=128),
        # those of a 16k prompt, keys and values put into 16-bit pages as they come
        _case("rotate_prompt", "rotate", dtype="bf16", b=1, hq=32, hkv=8, page=16, len_min=16384, len_max=16384, tq=16384,
              rope=128, base=1e4, pages=True),
        # one decode step of 64 sequences enters the cache
        _case("append_step", "append", b=64, hq=32, hkv=8, page=16, len_min=300, len_max=8000, tq=1),
        # prompts of up to 4096 tokens enter the cache
        _case("append_prompts", "append", dtype="bf16", b=8, hq=32, hkv=8, page=16, len_min=700, len_max=4096, tq=4096),
        # one short sequence decodes: latency
        _case("decode_one", "decode", b=1, page=64, len_min=1000, len_max=1000),
        # a serving batch of uneven sequences with a sliding window and 4 sinks, pages of 16
        _case("decode_window", "decode", dtype="bf16", b=64, hq=32, hkv=8, page=16, len_min=300, len_max=8000, window=4096,
              sinks=4),
        # 16 sequences of 64k tokens, every token visible
        _case("decode_long", "decode", b=16, page=256, len_min=65536, len_max=65536),
        # a chunk of 32 new tokens for each of 4 sequences, d 64, equal heads, odd lengths
        _case("prefill_chunk", "prefill", b=4, hq=8, hkv=8, d=64, page=32, len_min=333, len_max=2001, tq=32),
        # a 16k prompt through a sliding window of 1024 and 4 sinks
        _case("prefill_window", "prefill", b=1, page=64, len_min=16384, len_max=16384, tq=16384, window=1024, sinks=4),
        # an 8k prompt, causal, no window
        _case("prefill_full", "prefill", dtype="bf16", b=1, hq=32, hkv=8, page=16, len_min=8191, len_max=8191, tq=8191),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["plan", "rotate", "append", "decode", "decode", "prefill", "prefill"])
        hkv = rng.choice([1, 2, 4, 8])
        c = _case("", op, dtype=rng.choice(["fp16", "bf16"]), hkv=hkv, hq=hkv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8]),
                  d=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128, 256]))
        del c["name"]
        c["b"] = _log(rng, 1, 512 if op == "plan" else 64)
        c["len_max"] = _log(rng, 64, {"plan": 8192, "decode": 65536, "append": 8192}.get(op, 16384))
        c["len_min"] = max(1, int(c["len_max"] * rng.uniform(0.2, 1.0)))
        if op in ("plan", "rotate", "append"):
            c["tq"] = rng.choice([1, _log(rng, 1, 64), _log(rng, 1, c["len_max"])])
            c["mixed"] = op == "plan" and rng.random() < 0.5
        if op == "rotate":
            c["rope"] = rng.choice([16, 32, 48, 64, c["d"], c["d"]])
            c["base"] = rng.choice([1e4, 5e5, 1e6])
            c["pages"], c["gain"] = rng.random() < 0.5, rng.random() < 0.8
        if op == "prefill":
            c["tq"] = min(c["len_max"], rng.choice([_log(rng, 1, 64), c["len_max"], _log(rng, 1, c["len_max"])]))
        if op in ("decode", "prefill") and rng.random() < 0.6:
            c["window"] = _log(rng, 16, 8192)
            c["sinks"] = rng.choice([0, 1, 4, 70])
        kv = c["b"] * hkv * c["len_max"] * c["d"] if op in ("decode", "prefill") else 0
        rows = c["b"] * c["tq"] * (c["hq"] + c["hkv"]) * c["d"] if op in ("rotate", "append") else 0
        scores = c["b"] * c["hq"] * c["tq"] * c["len_max"] if op == "prefill" else 0
        if kv <= 2 ** 28 and scores <= 2 ** 31 and rows <= 2 ** 26 and c["b"] * c["tq"] <= 2 ** 20:
            return c


def _counts(c):
    """Tokens in the cache and new tokens of every sequence: fixed by the case, spread over its range."""
    lens = []
    for i in range(c["b"]):
        f = 1.0 if i == 0 else (i * 0.6180339887498949 + 1.0) % 1.0
        lens.append(c["len_min"] + int((c["len_max"] - c["len_min"]) * f))
    return lens, [min(c["tq"] or 1, n) for n in lens]


# ---------------------------------------------------------------- the cache's bytes

def _quantise(x):
    """x [..., d] -> codes uint8 [..., g, 64], (scale, bias) fp16 [..., g, 2].  In 64 bits: values next to a border."""
    x = x.double().unflatten(-1, (-1, 64))
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    e = torch.frexp(torch.maximum(hi.abs(), lo.abs()) * (65 / 64)).exponent.clamp(min=-13) - 11
    u = ((e.long() + 1023) << 52).view(torch.float64)                                     # 2^e (pow may be a step off)
    b = (lo / u).round()
    s = torch.ceil(((hi / u).round() - b) / 15)
    code = ((x / u - b) / s.clamp(min=1)).round().clamp(0, 15) * (s > 0)
    return code.to(torch.uint8), torch.cat([s * u, b * u], -1).half()


def _put(cache, c, slots, k, v):
    """Writes k, v [rows][hkv][d] to their slots (none below 0)."""
    d, g = c["d"], c["d"] // 64
    live = slots >= 0
    slot, h = slots[live][:, None], torch.arange(c["hkv"], device=slots.device)[None]
    blocks = cache.view(cache.shape[0], c["hkv"], c["page"] // 16, 18 * d)
    at, blk, t = slot // c["page"], slot % c["page"] // 16, slot % 16
    for i, x in enumerate((k, v)):
        code, param = _quantise(x[live])
        packed = code[..., ::2] | (code[..., 1::2] << 4)                                  # [rows][hkv][g][32]
        blocks[..., 8 * d * i:8 * d * (i + 1)].unflatten(-1, (g, 16, 32))[at, h, blk, :, t] = packed
        blocks[..., 16 * d + d * i:17 * d + d * i].unflatten(-1, (16, 4 * g))[at, h, blk, t] = param.flatten(2).view(torch.uint8)


def _values(cache, c, pages):
    """The rows of these pages [b][n] in fp32: K, V [b][hkv][n * page][d]."""
    d, g = c["d"], c["d"] // 64
    x = cache[pages].transpose(1, 2).reshape(pages.shape[0], c["hkv"], -1, 18 * d)        # [b][hkv][blocks][18 d]
    out = []
    for i in range(2):
        code = x[..., 8 * d * i:8 * d * (i + 1)].unflatten(-1, (g, 16, 32)).transpose(-2, -3)
        code = torch.stack([code & 15, code >> 4], -1).flatten(-2).float()                # [b][hkv][blocks][16][g][64]
        param = x[..., 16 * d + d * i:17 * d + d * i].contiguous().view(torch.float16).unflatten(-1, (16, g, 2)).float()
        out.append((code * param[..., :1] + param[..., 1:]).flatten(-2).flatten(2, 3))
    return out


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 23)
    dt, dev = DTYPES[c["dtype"]], torch.device("cuda")
    b, hq, hkv, d, page, op = c["b"], c["hq"], c["hkv"], c["d"], c["page"], c["op"]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).mul_(scale).to(dt)

    def ints(x, dtype=torch.int32):
        return torch.tensor(x, dtype=dtype, device=dev)

    if op == "plan":
        return _prepare_plan(c, seed, g, ints)
    lens, news = _counts(c)
    width = -(-max(lens) // page)
    used = [-(-n // page) for n in lens]
    n_pages = sum(used) + 3
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    at = torch.arange(width, device=dev)
    first = ints([sum(used[:i]) for i in range(b)])
    table = torch.where(at[None] < ints(used)[:, None], perm[(first[:, None] + at[None]).clamp(max=n_pages - 1)], -1)
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    rows = starts[-1]
    s = {"case": c, "table": table.contiguous(), "lens": ints(lens), "news": ints(news), "starts": ints(starts), "rows": rows}
    # the rows' sequences, positions and slots
    seq = torch.repeat_interleave(torch.arange(b, device=dev), ints(news).long())
    pos = torch.arange(rows, device=dev) - s["starts"][seq] + (s["lens"] - s["news"])[seq]
    s["slots"] = (s["table"][seq, pos // page].long() * page + pos % page).contiguous()
    s["positions"] = pos.int()
    if op == "rotate":
        # a projection's output: queries, keys and values side by side
        qkv = normal(rows, hq + 2 * hkv, d, scale=1.5)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_gain"], s["k_gain"] = (normal(d, scale=0.2) + 1, normal(d, scale=0.2) + 1) if c["gain"] else (None, None)
        s["q_out"], s["k_out"] = (torch.zeros(rows, n, d, dtype=dt, device=dev) for n in (hq, hkv))
        if c["pages"]:
            s["k_pages"], s["v_pages"] = (torch.zeros(n_pages, hkv, page, d, dtype=dt, device=dev) for _ in range(2))
        if own:
            from compressed_kv_cache_dkv_gb300 import dkv
            s["p"] = dkv.dkv_paged_layout(s["k_pages"], b, hq, width) if c["pages"] else None
            s["ws"] = torch.zeros(256, dtype=torch.uint8, device=dev)
        return s
    cache = s["cache"] = torch.zeros(n_pages, hkv, page * 9 * d // 8, dtype=torch.uint8, device=dev)
    shift_k, shift_v = normal(hkv, d, scale=0.5), normal(hkv, d, scale=0.3)               # a mean of each head's channels
    if op == "append":
        s["k_new"], s["v_new"] = (normal(rows, hkv, d) + x for x in (shift_k, shift_v))
        n = max(news)
        s["k_out"], s["v_out"] = (torch.zeros(b, hkv, n, d, dtype=dt, device=dev) for _ in range(2))
        s["first"] = s["lens"] - s["news"]
    else:
        step = max(1, 2 ** 25 // (hkv * page * d))
        for i in range(0, n_pages, step):                                                 # fills all pages
            slots = torch.arange(i * page, min(n_pages, i + step) * page, device=dev)
            _put(cache, c, slots, *(normal(len(slots), hkv, d) + x for x in (shift_k, shift_v)))
        s["q"] = normal(rows, hq, d, scale=2.0)
        s["out"] = torch.zeros(rows, hq, d, dtype=dt, device=dev)
        s["lse"] = torch.zeros((rows, hq) if op == "decode" else (hq, rows), device=dev)
    if own:
        from compressed_kv_cache_dkv_gb300 import dkv
        s["p"] = dkv.dkv_qpaged_layout(cache, b, hq, d, width, dtype=dt, window=c["window"], sinks=c["sinks"])
        s["ws"] = torch.zeros(dkv.dkv_qpaged_workspace_bytes(s["p"]), dtype=torch.uint8, device=dev)
    return s


def _prepare_plan(c, seed, g, ints):
    b, page = c["b"], c["page"]
    rng = random.Random(seed * 31 + 5)
    lens = [rng.randint(c["len_min"], c["len_max"]) for _ in range(b)]
    news = [c["tq"]] * b
    if c["mixed"]:  # a new request, a decoding one, a finished one, one cut by some tokens, an idle one
        for i in range(b):
            kind = rng.random()
            if kind < 0.3:
                lens[i], news[i] = 0, rng.randint(1, max(1, c["tq"]))
            elif kind < 0.8:
                news[i] = 1
            else:
                news[i] = -lens[i] if kind < 0.9 else -rng.randint(0, lens[i])
    width = -(-(c["len_max"] + c["tq"]) // page)
    used = [-(-n // page) for n in lens]
    need = sum(max(0, -(-(n + m) // page) - u) for n, m, u in zip(lens, news, used))
    n_free = max(1, int(need * (rng.uniform(0.5, 1.5) if c["mixed"] else 1.0)))
    n_pages = 2 * b * width + 1
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    at = torch.arange(width, device="cuda")
    first = ints([sum(used[:i]) for i in range(b)])
    table = torch.where(at[None] < ints(used)[:, None], perm[(first[:, None] + at[None]).clamp(max=n_pages - 1)], -1)
    free = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
    free[:n_free] = perm[sum(used):sum(used) + n_free]
    rows = -(-b * max(1, c["tq"]) // 64) * 64
    s = {"case": c, "rows": rows, "lens": ints(lens), "news": ints(news), "free": free, "n_free": ints([n_free]),
         "table": table.contiguous(), "n_pages": n_pages,
         "slots": torch.zeros(rows, dtype=torch.int64, device="cuda"), "positions": torch.zeros(rows, dtype=torch.int32, device="cuda"),
         "starts": ints([0] * (b + 1)), "granted": ints([0] * b), "new_lens": ints([0] * b), "new_n_free": ints([0])}
    if own:
        from compressed_kv_cache_dkv_gb300 import dkv
        s["p"] = dkv.dkv_paged(b, 1, 1, 64, page, n_pages, width, 0, 0, 0, page * 64, page * 64, 64)
        s["ws"] = torch.zeros(dkv.dkv_paged_plan_workspace_bytes(s["p"]), dtype=torch.uint8, device="cuda")
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return {"plan": _plan, "rotate": _rotate, "append": _append, "decode": _decode, "prefill": _prefill}[op](s)


def _own(s, op):
    from compressed_kv_cache_dkv_gb300 import dkv
    c = s["case"]
    if op == "plan":
        dkv.dkv_paged_plan(s["p"], s["lens"], s["news"], s["free"], s["n_free"], s["table"], s["rows"], slots=s["slots"],
                           positions=s["positions"], starts=s["starts"], granted=s["granted"], new_lens=s["new_lens"],
                           new_n_free=s["new_n_free"], workspace=s["ws"])
        return (s["slots"], s["positions"], s["starts"], s["granted"], s["new_lens"], s["new_n_free"], s["table"], s["free"])
    if op == "rotate":
        if not c["pages"]:
            return dkv.dkv_qk_norm_rope(s["q"], s["k"], s["positions"], c["rope"], c["base"], q_gain=s["q_gain"],
                                        k_gain=s["k_gain"], eps=1e-6, q_out=s["q_out"], k_out=s["k_out"], workspace=s["ws"])
        q, k = dkv.dkv_qk_norm_rope(s["q"], s["k"], s["positions"], c["rope"], c["base"], q_gain=s["q_gain"],
                                    k_gain=s["k_gain"], eps=1e-6, q_out=s["q_out"], k_out=s["k_out"], p=s["p"], v=s["v"],
                                    k_pages=s["k_pages"], v_pages=s["v_pages"], slots=s["slots"], workspace=s["ws"])
        return q, k, s["k_pages"], s["v_pages"]
    if op == "append":
        dkv.dkv_qpaged_append(s["p"], s["k_new"], s["v_new"], s["cache"], s["slots"], workspace=s["ws"])
        return dkv.dkv_qpaged_gather(s["p"], s["cache"], s["table"], s["first"], s["k_out"], s["v_out"], counts=s["news"],
                                     workspace=s["ws"])
    if op == "decode":
        return dkv.dkv_qpaged_decode(s["p"], s["q"], s["cache"], s["table"], s["lens"], out=s["out"], lse=s["lse"],
                                     workspace=s["ws"])
    return dkv.dkv_qpaged_prefill(s["p"], s["q"], s["starts"], c["tq"], s["cache"], s["table"], s["lens"], out=s["out"],
                                  lse=s["lse"], workspace=s["ws"])


# ---------------------------------------------------------------- plain forms

def _plan(s):
    """Requests are served in order: news > 0 takes pages from the top of the free list until it or the rows run
    out (one that needs no page goes on), news < 0 gives its last pages back first."""
    page, rows = s["case"]["page"], s["rows"]
    lens, news, dev = s["lens"].long(), s["news"].long(), s["lens"].device
    width = s["table"].shape[1]
    grow = news.clamp(min=0)
    have, want = (lens + page - 1) // page, (lens + news + page - 1) // page
    back, need = (have - want).clamp(min=0), (want - have).clamp(min=0)
    # released pages go behind the list
    n_free = s["n_free"].long()
    j = torch.arange(width, device=dev)
    gone = (j[None] >= want[:, None]) & (j[None] < have[:, None])
    n_back = back.sum()
    order = (n_free + back.cumsum(0) - back)[:, None] + j[None] - want[:, None]
    s["free"][order[gone]] = s["table"][gone]
    top = n_free + n_back
    ok = ((need == 0) | (need.cumsum(0) <= top)) & (grow.cumsum(0) <= rows)
    granted, need = grow * ok, need * ok
    got = (j[None] >= have[:, None]) & (j[None] < (have + need)[:, None])
    pick = (top - 1 - (need.cumsum(0) - need))[:, None] - (j[None] - have[:, None])
    s["table"][got] = s["free"][pick[got]]
    s["new_n_free"].copy_(top - need.sum())
    s["granted"].copy_(granted)
    s["new_lens"].copy_(lens + torch.where(news < 0, news, granted))
    s["starts"][1:] = granted.cumsum(0)
    s["starts"][0] = 0
    i = torch.arange(rows, device=dev)
    b = torch.searchsorted(s["starts"][1:].contiguous(), i.int(), right=True).clamp(max=len(lens) - 1)
    live = i < s["starts"][-1]
    t = torch.where(live, lens[b] + i - s["starts"][b], 0)
    s["slots"].copy_(torch.where(live, s["table"][b, (t // page).clamp(max=width - 1)].long() * page + t % page, -1))
    s["positions"].copy_(torch.where(live, t, -1))
    return (s["slots"], s["positions"], s["starts"], s["granted"], s["new_lens"], s["new_n_free"], s["table"], s["free"])


def _rotate(s):
    c = s["case"]
    h, dev = c["rope"] // 2, s["q"].device
    # angles of far positions: in 64 bits
    theta = c["base"] ** (-2.0 * torch.arange(h, device=dev, dtype=torch.float64) / c["rope"])
    angle = s["positions"].double()[:, None, None] * theta
    cos, sin = angle.cos().float(), angle.sin().float()
    for x, gain, out in ((s["q"], s["q_gain"], s["q_out"]), (s["k"], s["k_gain"], s["k_out"])):
        y = x.float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6)
        if gain is not None:
            y = y * gain.float()
        lo, hi = y[..., :h], y[..., h:2 * h]
        out.copy_(torch.cat([lo * cos - hi * sin, hi * cos + lo * sin, y[..., 2 * h:]], -1))
    if not c["pages"]:
        return s["q_out"], s["k_out"]
    pages, slots = s["slots"] // c["page"], s["slots"] % c["page"]
    s["k_pages"][pages, :, slots] = s["k_out"]
    s["v_pages"][pages, :, slots] = s["v"]
    return s["q_out"], s["k_out"], s["k_pages"], s["v_pages"]


def _append(s):
    c = s["case"]
    _put(s["cache"], c, s["slots"], s["k_new"], s["v_new"])
    n = s["k_out"].shape[2]
    i = torch.arange(n, device=s["cache"].device)
    b_at, i_at = (i[None] < s["news"][:, None]).nonzero(as_tuple=True)
    t = (s["first"].long()[b_at] + i_at)
    used, where = torch.unique(s["table"][b_at, t // c["page"]].long(), return_inverse=True)
    for x, out in zip(_values(s["cache"], c, used[:, None]), (s["k_out"], s["v_out"])):
        out[b_at, :, i_at] = x[where, :, t % c["page"]].to(out.dtype)
    return s["k_out"], s["v_out"]


def _attend(s, q, new):
    """q [b][hq][tq][d], the last new[b] tokens of each sequence -> out in fp32 [b][hq][tq][d], lse [b][hq][tq]."""
    c = s["case"]
    b, hq, tq, d = q.shape
    k, v = _values(s["cache"], c, s["table"].clamp(min=0).long())
    x = (q.float() / math.sqrt(d)).reshape(b, c["hkv"], -1, d) @ k.transpose(2, 3)
    t = torch.arange(k.shape[2], device=q.device)
    pos = (s["lens"] - new)[:, None] + torch.arange(tq, device=q.device)[None]            # [b][tq]
    seen = (t <= pos[..., None]) & (t < s["lens"][:, None, None])
    if c["window"]:
        seen &= (t > pos[..., None] - c["window"]) | (t < c["sinks"])
    x.view(b, c["hkv"], -1, tq, len(t)).masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    safe = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x.sub_(safe).exp_()
    n = x.sum(-1, keepdim=True)
    lse = (safe + n.log()).view(b, hq, tq)
    x.div_(torch.where(n == 0, torch.ones_like(n), n))
    return (x @ v).view(b, hq, tq, d), lse


def _decode(s):
    out, lse = _attend(s, s["q"][:, :, None], torch.ones_like(s["lens"]))
    s["out"].copy_(out[:, :, 0])
    s["lse"].copy_(lse[:, :, 0])
    return s["out"], s["lse"]


def _prefill(s):
    c = s["case"]
    i = torch.arange(c["tq"], device=s["q"].device)
    row = (s["starts"][:-1, None] + i[None]).long()                                       # [b][tq]
    live = i[None] < s["news"][:, None]
    out, lse = _attend(s, s["q"][row.clamp(max=s["rows"] - 1)].transpose(1, 2), s["news"])
    s["out"][row[live]] = out.transpose(1, 2)[live].to(s["out"].dtype)
    s["lse"][:, row[live]] = lse.permute(1, 0, 2)[:, live]
    return s["out"], s["lse"]


# ---------------------------------------------------------------- work and the 64-bit definition

def _seen(c, p):
    """Tokens that a query at position p sees."""
    if not c["window"] or p + 1 <= c["window"]:
        return p + 1
    return c["window"] + min(c["sinks"], p + 1 - c["window"])


def work(c):
    lens, news = _counts(c)
    row, g, rows = 2 * c["d"], c["hq"] // c["hkv"], sum(news)
    if c["op"] == "plan":
        # lengths in and out, slots and positions out, the pages that change hands
        rows = -(-c["b"] * max(1, c["tq"]) // 64) * 64
        return {"bytes": 12 * rows + 24 * c["b"] + 8 * c["b"] * (1 + c["tq"] // c["page"]) // 2, "flops": 0}
    if c["op"] == "rotate":
        n = 2 * row * (c["hq"] + c["hkv"]) + 4
        if c["pages"]:
            n += 3 * row * c["hkv"] + 8
        return {"bytes": rows * n, "flops": 8 * rows * (c["hq"] + c["hkv"]) * c["d"]}
    packed = 9 * c["d"] // 8  # bytes of a token's key and value
    if c["op"] == "append":
        return {"bytes": c["hkv"] * rows * (4 * row + packed), "flops": 0}
    if c["op"] == "decode":
        n = sum(_seen(c, x - 1) for x in lens)
        return {"bytes": packed * c["hkv"] * n + 2 * row * c["hq"] * c["b"], "flops": 4 * c["hq"] * c["d"] * n}
    pairs = sum(sum(_seen(c, x - n + i) for i in range(n)) for x, n in zip(lens, news))
    keys = 0  # that some query sees: from the first query's window on, and the sinks
    for x, n in zip(lens, news):
        lo = max(0, x - n - c["window"] + 1) if c["window"] else 0
        keys += x - lo + min(c["sinks"], lo)
    return {"bytes": packed * c["hkv"] * keys + 2 * row * c["hq"] * rows, "flops": 4 * c["hq"] * c["d"] * pairs}


def exact(c, seed):
    """The operators' definitions in 64 bits, one request, row or head at a time."""
    s = prepare(c, seed)
    if c["op"] == "plan":
        return _exact_plan(s, c)
    dev, d, page = s["lens"].device, c["d"], c["page"]
    if c["op"] == "rotate":
        h = c["rope"] // 2
        out = []
        for x, gain in ((s["q"], s["q_gain"]), (s["k"], s["k_gain"])):
            y = torch.empty(x.shape, dtype=torch.float64, device=dev)
            for j in range(x.shape[1]):
                z = x[:, j].double()
                z = z / (z.square().sum(-1, keepdim=True) / d + 1e-6).sqrt()
                z = z * gain.double() if gain is not None else z
                turn = torch.polar(torch.ones(1, dtype=torch.float64, device=dev), torch.outer(
                    s["positions"].double(), torch.tensor([c["base"] ** (-i / h) for i in range(h)], dtype=torch.float64, device=dev)))
                pair = torch.complex(z[:, :h].contiguous(), z[:, h:2 * h].contiguous()) * turn
                y[:, j] = torch.cat([pair.real, pair.imag, z[:, 2 * h:]], -1)
            out.append(y)
        if not c["pages"]:
            return tuple(out)
        pools = []
        for rows in (out[1], s["v"].double()):
            pool = torch.zeros(s["k_pages"].shape, dtype=torch.float64, device=dev)
            for j in range(c["hkv"]):
                pool[s["slots"] // page, j, s["slots"] % page] = rows[:, j]
            pools.append(pool)
        return (*out, *pools)
    if c["op"] == "append":
        lens, news = _counts(c)
        out = []
        grids = torch.tensor([2.0 ** (i - 24) for i in range(32)], dtype=torch.float64, device=dev)
        for x, like in ((s["k_new"], s["k_out"]), (s["v_new"], s["v_out"])):
            y = torch.zeros(like.shape, dtype=torch.float64, device=dev)
            at = 0
            for i, n in enumerate(news):
                for j in range(c["hkv"]):
                    for q in range(0, d, 64):
                        z = x[at:at + n, j, q:q + 64].double()
                        top = z.abs().max(1, keepdim=True).values * 1.015625
                        grid = grids[torch.floor(torch.log2(top.clamp(min=2.0 ** -14))).long() + 14]
                        low = torch.round(z.min(1, keepdim=True).values / grid) * grid
                        span = torch.round(z.max(1, keepdim=True).values / grid) * grid - low
                        step = -torch.floor(-span / grid / 15) * grid
                        code = torch.where(step > 0, torch.round((z - low) / torch.where(step > 0, step, 1.0)), 0.0)
                        y[i, j, :n, q:q + 64] = low + step * code.clamp(0, 15)
                at += n
            out.append(y)
        return tuple(out)
    lens, news = _counts(c)
    rows, g = s["rows"], c["hq"] // c["hkv"]
    out = torch.zeros(rows, c["hq"], d, dtype=torch.float64, device=dev)
    lse = torch.zeros(c["hq"], rows, dtype=torch.float64, device=dev)
    step = max(1, 2 ** 28 // max(lens))
    at = 0
    for i, n in enumerate(lens):
        new = news[i] if c["op"] == "prefill" else 1
        for j in range(c["hkv"]):
            k, v = _exact_rows(s, c, i, j, n)
            for a in range(j * g, j * g + g):
                for f in range(0, new, step):
                    e = min(new, f + step)
                    p = torch.arange(n - new + f, n - new + e, device=dev)[:, None]
                    t = torch.arange(n, device=dev)
                    x = (s["q"][at + f:at + e, a].double() @ k.T) * d ** -0.5
                    hide = t > p
                    if c["window"]:
                        hide |= (t <= p - c["window"]) & (t >= c["sinks"])
                    x[hide] = -math.inf
                    top = x.max(1, keepdim=True).values
                    x = (x - top).exp()
                    total = x.sum(1, keepdim=True)
                    out[at + f:at + e, a] = (x @ v) / total
                    lse[a, at + f:at + e] = (top + total.log())[:, 0]
        at += new
    return (out, lse) if c["op"] == "prefill" else (out, lse.T.contiguous())


def _exact_rows(s, c, i, j, n):
    """K and V of sequence i's head j, byte by byte from its pages: [n][d] in 64 bits."""
    d, page, g = c["d"], c["page"], c["d"] // 64
    t = torch.arange(n, device=s["lens"].device)
    flat = s["cache"][s["table"][i].long()[t // page], j]                                 # [n][bytes of a page]
    base = (t % page // 16 * 18 * d)[:, None]
    ch = torch.arange(d, device=t.device)
    out = []
    for kv in range(2):
        at = base + kv * 8 * d + (ch // 64) * 512 + (t % 16 * 32)[:, None] + ch % 64 // 2
        code = flat.gather(1, at)
        code = torch.where(ch % 2 == 1, code // 16, code % 16).double()
        at = base + (16 + kv) * d + (t % 16 * 4 * g)[:, None] + torch.arange(4 * g, device=t.device)
        param = flat.gather(1, at).view(torch.float16).double().view(n, g, 2)
        out.append(code * param[:, ch // 64, 0] + param[:, ch // 64, 1])
    return out


def _exact_plan(s, c):
    page, rows = c["page"], s["rows"]
    lens, news, table = s["lens"].tolist(), s["news"].tolist(), s["table"].tolist()
    free, n_free = s["free"].tolist(), int(s["n_free"])
    pages_of = lambda n: -(-n // page)  # noqa: E731
    for b, n in enumerate(news):
        if n < 0:
            for j in range(pages_of(lens[b] + n), pages_of(lens[b])):
                free[n_free] = table[b][j]
                n_free += 1
    full = n_free
    slots, positions, starts, granted, new_lens, asked, wanted = [], [], [0], [], [], 0, 0
    for b, n in enumerate(news):
        need = pages_of(lens[b] + n) - pages_of(lens[b]) if n > 0 else 0
        asked, wanted = asked + max(n, 0), wanted + need
        take = n if n > 0 and asked <= rows and (need == 0 or wanted <= full) else 0
        if take:
            for j in range(pages_of(lens[b]), pages_of(lens[b] + n)):
                n_free -= 1
                table[b][j] = free[n_free]
        for t in range(lens[b], lens[b] + take):
            slots.append(table[b][t // page] * page + t % page)
            positions.append(t)
        starts.append(starts[-1] + take)
        granted.append(take)
        new_lens.append(lens[b] + (n if n < 0 else take))
    pad = [-1] * (rows - len(slots))
    dev = lambda x, t=torch.int32: torch.tensor(x, dtype=t, device="cuda")  # noqa: E731
    return (dev(slots + pad, torch.int64), dev(positions + pad), dev(starts), dev(granted), dev(new_lens), dev([n_free]),
            dev(table), dev(free))
