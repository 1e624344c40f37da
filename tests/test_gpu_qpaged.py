"""The operators of a serving step over a paged cache in 4 bits against their definitions in 64 bits: pages and slots,
norm and rotation, append and gather, decode and prefill; types, head layouts, page sizes, lengths from none on,
windows, sinks, ragged batches; slots that nothing may look at hold NaN, unneeded page-table entries numbers out of
range."""
import math
from fractions import Fraction

import pytest
import torch

from compressed_kv_cache_dkv_gb300 import dkv
from tests import paged_ref as R
from tests import qpaged_ref as Q

pytestmark = pytest.mark.gpu


def no_fault(ws):
    assert dkv.dkv_get_error(ws) == (dkv.DKV_OK, 0)


def workspace(p):
    ws = torch.full((dkv.dkv_qpaged_workspace_bytes(p),), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:256] = 0  # only the header has to be zero
    return ws


def randn(shape, dt, seed, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dt)


# ---------------------------------------------------------------- append and gather

@pytest.mark.parametrize("dtype,d,hkv,page,rows,scale", [
    ("fp16", 128, 2, 16, 1, 1.0), ("bf16", 64, 1, 32, 37, 1.0), ("fp16", 64, 3, 256, 700, 30.0),
    ("bf16", 128, 8, 64, 300, 1e-3), ("fp16", 128, 1, 128, 200, 3e-6), ("bf16", 128, 2, 16, 130, 4000.0)])
def test_append_quantises_by_the_definition(dtype, d, hkv, page, rows, scale):
    dt = Q.DT[dtype]
    n_pages = -(-rows // page) + 2
    cache = torch.full((n_pages, hkv, page * 9 * d // 8), 0xA5, dtype=torch.uint8, device="cuda")
    p = dkv.dkv_qpaged_layout(cache, 1, hkv, d, n_pages, dtype=dt)
    ws = workspace(p)
    K, V = (randn((rows, hkv, d), dt, s, scale) for s in (1, 2))
    K[::7, :, :64] += scale * 20          # groups far from zero
    K[::5, :, 64:] = K[::5, :, 64:65]     # groups of one value
    V[::3] = (V[::3] * 4 / scale).round() * scale / 4  # many ties
    slots = torch.randperm(n_pages * page, generator=torch.Generator().manual_seed(3))[:rows]
    if rows > 3:
        slots[1] = -1
    before = cache.clone()
    dkv.dkv_qpaged_append(p, K.cuda(), V.cuda(), cache, slots.cuda(), workspace=ws)
    large = any(bool((x[slots >= 0].double().abs() > 61440).any()) for x in (K, V))
    assert dkv.dkv_get_error(ws)[1] == (dkv.DKV_DEVERR_RANGE if large else 0)
    want = before.cpu()
    blocks = want.view(n_pages, hkv, page // 16, 18 * d)
    G = d // 64
    for i, s in enumerate(slots.tolist()):
        if s < 0:
            continue
        blk = blocks[s // page, :, s % page // 16]
        for kv, x in enumerate((K, V)):
            c, sc, b = Q.quantise(x[i].double())
            c = c.to(torch.uint8)
            for g in range(G):
                at = kv * 8 * d + (g * 16 + s % 16) * 32
                blk[:, at:at + 32] = c[:, g, ::2] | (c[:, g, 1::2] << 4)
            at = (16 + kv) * d + s % 16 * G * 4
            blk[:, at:at + 4 * G] = torch.stack([sc, b], -1).to(torch.float16).reshape(hkv, -1).view(torch.uint8)
    assert torch.equal(cache.cpu(), want)


def test_quantised_values_are_fp16_numbers_near_their_rows():
    """The grid's claims: every value is an fp16 number, off by at most half a step and the grid's rounding."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn(4000, 64, generator=g) * torch.exp(4 * torch.randn(4000, 1, generator=g)) + torch.randn(4000, 1, generator=g) * 3
    x = x.half().double()
    c, s, b = Q.quantise(x)
    v = Q.values(c, s, b)
    assert torch.equal(v.half().double(), v)
    lo, hi = x.min(1).values, x.max(1).values
    top = torch.maximum(lo.abs(), hi.abs())
    u = 2.0 ** torch.clamp(torch.floor(torch.log2(top * 65 / 64)) - 10, min=-24)
    assert bool(((v - x).abs().max(1).values <= (hi - lo) / 30 + u).all())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_append_saturates_and_says_so(dtype):
    dt = Q.DT[dtype]
    cache = torch.zeros(1, 1, 16 * 144, dtype=torch.uint8, device="cuda")
    p = dkv.dkv_qpaged_layout(cache, 1, 1, 128, 1, dtype=dt)
    ws = workspace(p)
    K, V = (randn((4, 1, 128), dt, s) for s in (1, 2))
    K[0, 0, 3], K[1, 0, 70], V[2, 0, 0], V[3, 0, 64] = math.inf, -math.inf, math.nan, 65000.0
    slots = torch.arange(4, device="cuda")
    dkv.dkv_qpaged_append(p, K.cuda(), V.cuda(), cache, slots, workspace=ws)
    assert dkv.dkv_get_error(ws) == (dkv.DKV_ERR_DEVICE, dkv.DKV_DEVERR_RANGE)
    out = [torch.zeros(1, 1, 4, 128, dtype=dt, device="cuda") for _ in range(2)]
    table, first = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    dkv.dkv_qpaged_gather(p, cache, table, first, *out, workspace=ws)
    no_fault(ws)
    for x, y in zip((K, V), out):
        assert torch.equal(y[0, 0].cpu(), Q.values(*Q.quantise(x[:, 0].double())).to(dt))
    dkv.dkv_qpaged_append(p, K.cuda() * 0, V.cuda() * 0, cache, torch.tensor([-1, 16, -2, 3], device="cuda"), workspace=ws)
    assert dkv.dkv_get_error(ws)[1] & dkv.DKV_DEVERR_INDEX


@pytest.mark.parametrize("dtype,d,hkv,page,lens,first,counts", [
    ("fp16", 128, 2, 16, [40], [0], [40]), ("bf16", 64, 3, 32, [100, 1, 65], [7, 0, 3], [90, 1, 0]),
    ("fp16", 64, 1, 256, [600, 300], [255, 17], [300, 1]), ("bf16", 128, 8, 64, [130], [63], [67])])
def test_gather_reads_its_tokens_only(dtype, d, hkv, page, lens, first, counts):
    c = Q.Cache(lens, hkv, d, page, dtype, seed=5, pad_head=16)
    p = c.layout(hkv)
    ws = workspace(p)
    n = max(counts) + 1
    out = [torch.full((c.B, n, hkv, d), 7.0, dtype=c.dt, device="cuda").transpose(1, 2) for _ in range(2)]
    dkv.dkv_qpaged_gather(p, c.cache, c.table.cuda(), c.dev(first), *out, counts=c.dev(counts), workspace=ws)
    no_fault(ws)
    for x, rows in zip(out, (c.K, c.V)):
        for b in range(c.B):
            want = torch.full((hkv, n, d), 7.0, dtype=c.dt)
            want[:, :counts[b]] = rows[b][:, first[b]:first[b] + counts[b]].to(c.dt)
            assert torch.equal(x[b].cpu(), want)


# ---------------------------------------------------------------- decode

CASES = [
    # dtype, d, hq, hkv, page, lens, window, sinks
    ("fp16", 128, 12, 2, 64, [1000], 0, 0),
    ("fp16", 64, 1, 1, 16, [1], 0, 0),
    ("bf16", 128, 8, 1, 16, [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 0], 0, 0),
    ("bf16", 64, 9, 3, 32, [0, 300, 0, 17, 555], 0, 0),
    ("fp16", 128, 7, 7, 256, [5, 2049], 0, 0),
    ("bf16", 128, 5, 1, 128, [777, 1300], 100, 0),
    ("fp16", 128, 12, 4, 16, [50, 64, 65, 500, 1999], 64, 4),
    ("bf16", 64, 16, 2, 64, [1500, 1, 70, 71], 70, 1),
    ("fp16", 64, 4, 2, 32, [900, 130], 1, 0),
    ("fp16", 128, 6, 2, 64, [1500, 333], 200, 130),
    ("bf16", 128, 2, 1, 32, [400, 90], 1000, 5),
]


@pytest.mark.parametrize("dtype,d,hq,hkv,page,lens,window,sinks", CASES)
def test_decode(dtype, d, hq, hkv, page, lens, window, sinks):
    c = Q.Cache(lens, hkv, d, page, dtype, seed=len(lens), pad_head=32)
    p = c.layout(hq, window, sinks)
    ws = workspace(p)
    q = randn((c.B, hq, d), c.dt, 7, 2.0)
    table = c.hidden_table([n - 1 for n in lens], window, sinks)
    out, lse = dkv.dkv_qpaged_decode(p, q.cuda(), c.cache, table, c.dev(lens), workspace=ws)
    no_fault(ws)
    check_decode(c, q, out, lse, lens, hq, window, sinks)
    again, lse2 = dkv.dkv_qpaged_decode(p, q.cuda(), c.cache, table, c.dev(lens), workspace=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("d,hkv,hq,lens", [
    (128, 4, 8, [3] * 700 + [900, 31, 33]),     # many units of a tile: whole in a warp's run, cut by warps and by CTAs
    (64, 1, 2, [1 + i % 150 for i in range(4096)]),
    (128, 2, 16, [20000, 10, 15000, 1]), (64, 8, 8, [2000 + 37 * i for i in range(6)]),
    # a CTA that holds the end of one long unit and the start of the next may be last at both; equal lengths cut evenly
    (128, 2, 8, [4000, 3900]), (64, 2, 2, [4100, 3970, 2000]), (128, 3, 18, [2100, 2000, 1900]), (64, 1, 8, [5000, 4900]),
    (128, 2, 12, [9000]), (64, 8, 16, [200] * 16), (128, 4, 4, [700] * 5)])
def test_decode_deals_units_to_warps(d, hkv, hq, lens):
    page = 32
    used = [-(-n // page) for n in lens]
    n_pages = sum(used)
    pool = torch.zeros(n_pages, hkv, page * 9 * d // 8, dtype=torch.uint8, device="cuda")
    p = dkv.dkv_qpaged_layout(pool, len(lens), hq, d, max(used), dtype=torch.bfloat16)
    ws = workspace(p)
    g = torch.Generator(device="cuda").manual_seed(1)
    K, V = (torch.randn(n_pages * page, hkv, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    dkv.dkv_qpaged_append(p, K, V, pool, torch.arange(n_pages * page, device="cuda"), workspace=ws)
    starts = torch.tensor([sum(used[:i]) for i in range(len(lens))], device="cuda")
    table = (starts[:, None] + torch.arange(max(used), device="cuda")[None]).clamp(max=n_pages - 1).int()
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn(len(lens), hq, d, generator=g, device="cuda").bfloat16() * 2
    out, lse = dkv.dkv_qpaged_decode(p, q, pool, table, L, workspace=ws)
    no_fault(ws)
    back = [torch.zeros(1, hkv, n_pages * page, d, dtype=torch.float16, device="cuda") for _ in range(2)]
    p16 = dkv.dkv_qpaged_layout(pool, 1, hq, d, n_pages)
    dkv.dkv_qpaged_gather(p16, pool, torch.arange(n_pages, dtype=torch.int32, device="cuda")[None], L[:1] * 0, *back)
    for b in range(len(lens)):
        if len(lens) > 1000 and b % 37:
            continue
        at = int(starts[b]) * page
        k, v = (x[0, :, at:at + lens[b]].double().repeat_interleave(hq // hkv, 0) for x in back)
        s = (k @ q[b].double()[:, :, None])[..., 0] / math.sqrt(d)
        w = s.softmax(-1)
        want = (w[:, None] @ v)[:, 0]
        # as in check_decode: what is added up are codes times scale and biases, and 15 scale <= 2 max + a spacing of 2^-10 max,
        # |bias| <= max of the group's largest magnitude: at most 3.1 max each for K and V
        size = 3.1 * (w * v.abs().amax(-1)).sum(-1, keepdim=True)
        ds = R.score_error(d, 3.1 * float((q[b].double().abs().sum(-1) * k.abs().amax((1, 2))).max()) / math.sqrt(d))
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2 * ds) * (1 + 2.0 ** -8) * size + 1e-30
        assert bool(((out[b].double() - want).abs() <= tol).all()), b
        assert bool(((lse[b].double() - s.logsumexp(-1)).abs() <= ds + 2.0 ** -22 * s.logsumexp(-1).abs().clamp(min=1.0)).all()), b
    for _ in range(20):  # the counters in the header are back at zero, and it is the same whoever comes last
        again, lse2 = dkv.dkv_qpaged_decode(p, q, pool, table, L, workspace=ws)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


def check_decode(c, q, out, lse, lens, hq, window, sinks):
    for b in range(c.B):
        for j in range(hq):
            ref, parts, pv = Q.attend(q[b, j:j + 1].double(), c, b, j * c.hkv // hq, torch.tensor([lens[b] - 1]), window, sinks)
            # The products of the codes and of the biases are added up apart, in the scores and with the weights.  A weight
            # times scale over the power of two is one fp16 number (2^-11 relative; the row's largest weight is 2^7 or more,
            # so in the subnormals half of 2^-24 is 2^-32 of it), on codes less 8; the weights' sum and the biases are fp32.
            s, h = c.q[b][1][1], j * c.hkv // hq
            seen = R.seen(torch.tensor([lens[b] - 1]), lens[b], window, sinks).double()
            pv = pv + 2.0 ** (11 - 32) * 16 * (seen @ torch.ones_like(s[h]) * (s[h] * seen[0][:, None]).amax(0) if lens[b] else s[h].sum(0)[None]).repeat_interleave(64, -1)
            R.check_rows(out[b, j:j + 1], lse[b, j:j + 1], (ref[0], ref[1], ref[2], pv, max(ref[4], parts)), c.d, c.dt, 2.0 ** -11,
                         f"sequence {b} head {j}")


@pytest.mark.parametrize("dtype,d,hkv,B,n,page,rising", [
    ("bf16", 128, 1, 1, 40, 16, False), ("fp16", 64, 2, 3, 700, 32, False), ("bf16", 64, 2, 64, 4096, 64, True),
    ("fp16", 128, 2, 60, 4090, 32, True), ("fp16", 128, 1, 2, 9000, 256, False)])
def test_decode_values_far_from_the_heaviest_tokens(dtype, d, hkv, B, n, page, rising):
    """Tokens of hardly any weight with values 2^27 times the others': the others keep their bits.  Rising: they have
    weight when they come, until a later token outweighs them by e^30."""
    dt, G, n_pages = Q.DT[dtype], 4, -(-n // page)
    pool = torch.zeros(n_pages, hkv, page * 9 * d // 8, dtype=torch.uint8, device="cuda")
    p = dkv.dkv_qpaged_layout(pool, B, hkv * G, d, n_pages, dtype=dt)
    ws = workspace(p)
    t = torch.arange(n)
    heavy = n // 2 // 256 * 256 + 32 * 7 + 11 if rising else 7
    odd = (t // 32 % 8 == 6) & (t % 32 == 5) if rising else (t == 3) | (t == n // 2) | (t == n - 1)
    score = torch.zeros(n)
    score[odd] = 0.0 if rising else -30.0
    score[heavy] = 30.0 if rising else 12.0
    K, V = randn((n, hkv, d), dt, 1).double(), randn((n, hkv, d), dt, 2).double() * 2.0 ** -13
    K[:, :, 0] = (score * math.sqrt(d) / 16)[:, None]
    V[odd] = randn((int(odd.sum()), hkv, d), dt, 3).double() * 2.0 ** 13
    dkv.dkv_qpaged_append(p, K.to(dt).cuda(), V.to(dt).cuda(), pool, t.cuda(), workspace=ws)
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda").repeat(B, 1)
    L = torch.full((B,), n, dtype=torch.int32, device="cuda")
    q = randn((B, hkv * G, d), dt, 4, 0.1)
    q[..., 0] = 16.0
    q = q.cuda()
    out, lse = dkv.dkv_qpaged_decode(p, q, pool, table, L, workspace=ws)
    no_fault(ws)
    back = [torch.zeros(1, hkv, n, d, dtype=torch.float16, device="cuda") for _ in range(2)]
    dkv.dkv_qpaged_gather(dkv.dkv_qpaged_layout(pool, 1, hkv * G, d, n_pages), pool, table[:1].contiguous(), L[:1] * 0, *back)
    for h in range(hkv):
        k, v = (x[0, h].double() for x in back)
        x = q[:, h * G:(h + 1) * G].double().flatten(0, 1)
        s = (x @ k.T) / math.sqrt(d)
        w = s.softmax(-1)
        # a weight times scale, on codes less 8, is off by 2^-11 of itself and 2^-32 of the row's largest one; 8 scale is
        # below 3.1 times the largest magnitude (as in exact_rows)
        part = w * v.abs().amax(-1)
        ds = R.score_error(d, 3.1 * float((x.abs() @ k.abs().T).max()) / math.sqrt(d))
        size = 3.1 * (part.sum(-1) + 2.0 ** (11 - 32) * n * part.amax(-1))[:, None]
        want = w @ v
        # (half of fp16's smallest step)
        tol = torch.finfo(dt).eps / 2 * want.abs() + (2.0 ** -11 + 2 * ds) * (1 + 2.0 ** -8) * size + 2.0 ** -25 * (dt == torch.float16)
        err = (out[:, h * G:(h + 1) * G].double().flatten(0, 1) - want).abs()
        assert bool((err <= tol).all()), float((err / tol).max())
        z = s.logsumexp(-1)
        assert bool(((lse[:, h * G:(h + 1) * G].double().flatten() - z).abs() <= ds + 2.0 ** -22 * z.abs().clamp(min=1.0)).all())


# ---------------------------------------------------------------- prefill

PREFILL = [
    # dtype, d, hq, hkv, page, lens, news, window, sinks
    ("fp16", 128, 12, 2, 64, [300], [300], 0, 0),
    ("bf16", 128, 4, 1, 16, [130, 1, 64], [130, 1, 64], 0, 0),
    ("fp16", 64, 3, 3, 32, [65, 200], [1, 70], 0, 0),
    ("bf16", 64, 8, 8, 32, [333, 1001], [32, 32], 0, 0),
    ("fp16", 128, 8, 1, 256, [700], [3], 0, 0),
    ("bf16", 128, 12, 4, 16, [600, 0, 257], [600, 0, 200], 100, 4),
    ("fp16", 128, 2, 2, 128, [513, 100], [513, 1], 64, 0),
    ("bf16", 64, 10, 2, 64, [400], [129], 70, 130),
    ("fp16", 64, 5, 1, 16, [100, 90, 80], [9, 0, 17], 1, 0),
    ("bf16", 128, 16, 2, 64, [2500], [4], 0, 0),
    ("fp16", 128, 6, 6, 32, [520], [260], 300, 70),
    ("fp16", 128, 4, 2, 32, [5, 40], [9, 12], 0, 0),  # more queries than tokens: the first see nothing
]


@pytest.mark.parametrize("dtype,d,hq,hkv,page,lens,news,window,sinks", PREFILL)
def test_prefill(dtype, d, hq, hkv, page, lens, news, window, sinks):
    c = Q.Cache(lens, hkv, d, page, dtype, seed=sum(lens), pad_head=16)
    p = c.layout(hq, window, sinks)
    ws = workspace(p)
    gap = 3  # rows in front of the first span and behind the last belong to nobody
    starts = [gap]
    for n in news:
        starts.append(starts[-1] + n)
    rows = starts[-1] + 5
    q = randn((rows, hq, d), c.dt, 9, 2.0)
    table = c.hidden_table([n - m for n, m in zip(lens, news)], window, sinks)
    fused = torch.full((rows, hq + 1, d), 7.0, dtype=c.dt, device="cuda")
    out, lse = fused[:, :hq], torch.full((hq, rows), 7.0, device="cuda")
    dkv.dkv_qpaged_prefill(p, q.cuda(), c.dev(starts), max(news), c.cache, table, c.dev(lens), out=out, lse=lse, workspace=ws)
    no_fault(ws)
    check_prefill(c, q, out, lse, lens, news, starts, hq, window, sinks)
    mine = torch.zeros(rows, dtype=torch.bool)
    mine[starts[0]:starts[-1]] = True
    assert bool((fused[:, hq] == 7).all()) and bool((out[~mine.cuda()] == 7).all()) and bool((lse[:, ~mine.cuda()] == 7).all())


def check_prefill(c, q, out, lse, lens, news, starts, hq, window, sinks):
    for b in range(c.B):
        if not news[b]:
            continue
        rows = slice(starts[b], starts[b] + news[b])
        pos = torch.arange(lens[b] - news[b], lens[b])
        for j in range(hq):
            ref, parts, _ = Q.attend(q[rows, j].double(), c, b, j * c.hkv // hq, pos, window, sinks)
            # A weight is an fp16 number, the row's largest at 2^7 or more (the reference lies 7 below a maximum, which only
            # grows): in the subnormals it is off by half of 2^-24, 2^-32 of the largest, whatever its own size.
            scale = ref[3] + 2.0 ** (11 - 32) * R.seen(pos, lens[b], window, sinks).double() @ c.V[b][j * c.hkv // hq].abs()
            R.check_rows(out[rows, j], lse[j, rows], (*ref[:3], scale, max(ref[4], parts)), c.d, c.dt, 2.0 ** -11, f"sequence {b} head {j}")


# ---------------------------------------------------------------- norm and rotation

@pytest.mark.parametrize("dtype,d,hq,hkv,rope,rows,gain,eps", [
    ("fp16", 128, 12, 2, 128, 16, True, 1e-6), ("bf16", 64, 1, 1, 64, 1, True, 1e-5), ("bf16", 128, 5, 5, 64, 33, False, 1e-6),
    ("fp16", 64, 9, 3, 48, 7, True, None), ("fp16", 128, 32, 8, 16, 5, True, 1e-6), ("bf16", 128, 3, 1, 0, 4, True, 1e-6),
    ("fp16", 128, 2, 1, 112, 6000, False, None)])
def test_norm_and_rotation(dtype, d, hq, hkv, rope, rows, gain, eps):
    dt = Q.DT[dtype]
    qkv = randn((rows, hq + hkv, d), dt, 1, 3.0)
    gains = [1 + randn((d,), dt, s, 0.3) for s in (2, 3)] if gain else [None, None]
    pos = torch.randint(0, 1 << 20, (rows,), generator=torch.Generator().manual_seed(4)).int()
    pos[0] = (1 << 31) - 1 if rows > 4 else 0
    if rows > 2:
        pos[2] = -1
    fused = qkv.cuda()
    q, k = fused[:, :hq], fused[:, hq:]
    dkv.dkv_qk_norm_rope(q, k, pos.cuda(), rope, 1e4, q_gain=gains[0] if gains[0] is None else gains[0].cuda(),
                         k_gain=gains[1] if gains[1] is None else gains[1].cuda(), eps=eps, q_out=q, k_out=k)
    x = qkv.double()
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() if eps is not None else x
    if gain:
        y = y * torch.cat([gains[0][None].expand(hq, d), gains[1][None].expand(hkv, d)]).double()
    h = rope // 2
    angle = pos.double()[:, None, None] * 1e4 ** (-2.0 * torch.arange(h).double() / max(rope, 1))
    a, b = y[..., :h], y[..., h:2 * h]
    want = torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin(), y[..., 2 * h:]], -1)
    size = torch.cat([a.abs() + b.abs(), a.abs() + b.abs(), y[..., 2 * h:].abs()], -1)
    want[pos < 0] = x[pos < 0]
    # fp32: d additions of squares, the root, three products, the angle (2^-25 of the circle, as steps of pi) and sincospi
    # (2^-23), the last sum; angles of the definition in 64 bits are off by position 2^-52
    f32 = (d / 4 + 24) * 2.0 ** -24 + float(pos.max()) * 2.0 ** -51
    tol = torch.finfo(dt).eps / 2 * want.abs() + 2 * f32 * size + torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    err = (fused.double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def test_rotation_by_given_frequencies_and_into_pages():
    dt, hq, hkv, d, page, rows = torch.bfloat16, 6, 2, 128, 32, 50
    freq = [0.7 / (1 + j) for j in range(32)]
    q, k, v = randn((rows, hq, d), dt, 1), randn((rows, hkv, d), dt, 2), randn((rows, hkv, d), dt, 3)
    pos = torch.arange(rows).int() * 977
    pools = [torch.full((4, page, hkv, d), 5.0, dtype=dt, device="cuda").transpose(1, 2) for _ in range(2)]
    p = dkv.dkv_paged_layout(pools[0], 1, hq, 4)
    slots = torch.randperm(4 * page, generator=torch.Generator().manual_seed(5))[:rows]
    slots[3], slots[4] = -1, 4 * page
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    qo, ko = dkv.dkv_qk_norm_rope(q.cuda(), k.cuda(), pos.cuda(), 64, inv_freq=freq, p=p, v=v.cuda(), k_pages=pools[0],
                                  v_pages=pools[1], slots=slots.cuda(), workspace=ws)
    assert dkv.dkv_get_error(ws) == (dkv.DKV_ERR_DEVICE, dkv.DKV_DEVERR_INDEX)
    y = k.double()
    y = y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    angle = pos.double()[:, None, None] * torch.tensor(freq, dtype=torch.float64)
    want = torch.cat([y[..., :32] * angle.cos() - y[..., 32:64] * angle.sin(), y[..., 32:64] * angle.cos() + y[..., :32] * angle.sin(), y[..., 64:]], -1)
    assert bool(((ko.double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5).all())
    for pool, rows_of in zip(pools, (ko.cpu(), v)):
        expect = torch.full((4, hkv, page, d), 5.0, dtype=dt)
        for i, s in enumerate(slots.tolist()):
            if 0 <= s < 4 * page:
                expect[s // page, :, s % page] = rows_of[i]
        assert torch.equal(pool.cpu(), expect)


PI = Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)


@pytest.mark.parametrize("base", [None, 65536.0])
def test_angles_are_as_exact_as_the_header_says(base):
    """Pairs that turn to almost nothing, so that the angle's error is what is left; the angle itself in whole numbers."""
    h, d = 32, 64
    freq = [65536.0 ** (-j / h) if base else [1.0, 0.7310585786300049, 1e-3, 1.7e-6, 3.7, 1 / 3, 0.9999999, 20.0][j % 8] / (1 + j // 8) for j in range(h)]
    keep = [j for j in range(h) if not base or j % 2 == 0]    # (frequencies that are powers of two: their definition is exact)
    pos = [0, 1, 1000, 65535, (1 << 20) - 1, (1 << 24) + 1, (1 << 30) + 12345, (1 << 31) - 1]
    x, want, tol = torch.zeros(len(pos), 1, d), torch.zeros(len(pos), h, dtype=torch.float64), torch.zeros(len(pos), h, dtype=torch.float64)
    n = torch.arange(1, 2049).double()
    for i, p in enumerate(pos):
        for j in keep:
            turns = Fraction(p) * Fraction(freq[j]) / (2 * PI)
            a = 2 * math.pi * float(turns - math.floor(turns))
            c, s = math.cos(a), math.sin(a)
            m = (n * (s / c if abs(s) < abs(c) else c / s)).round()
            r = (m * c - n * s if abs(s) < abs(c) else n * c - m * s).abs()
            at = int(r.argmin())
            lo, hi = (float(m[at]), float(n[at])) if abs(s) < abs(c) else (float(n[at]), float(m[at]))
            x[i, 0, j], x[i, 0, j + h] = lo, hi
            want[i, j] = lo * c - hi * s
            # fp32: cosine and sine off by 2^-23 (two units), a product and a sum by 2^-24 of what they give
            tol[i, j] = 2.0 ** -11 * abs(want[i, j]) + 2.0 ** -25 + (abs(lo) + abs(hi)) * (2.0 ** -23 + 2.0 ** -24 + 2.0 ** -24) + \
                2 * math.pi * math.hypot(lo, hi) * (2.0 ** -25 + p * 2.0 ** -54 * max(1.0, freq[j]))
    x = x.half().cuda()
    q, k = dkv.dkv_qk_norm_rope(x, x, torch.tensor(pos, dtype=torch.int32, device="cuda"), d, rope_base=base or 1e4,
                                inv_freq=None if base else freq, eps=None)
    for y in (q, k):
        err = (y[:, 0, :h].double().cpu() - want)[:, keep].abs()
        assert bool((err <= tol[:, keep]).all()), float((err / tol[:, keep]).max())


def test_keys_into_pages_alone():
    """The C call without k_out: queries out, keys and values into pages only, the same bits as with it."""
    dt, hq, hkv, d, page, rows = torch.float16, 8, 4, 64, 16, 70
    q, k, v = (randn((rows, n, d), dt, s).cuda() for s, n in ((1, hq), (2, hkv), (3, hkv)))
    pos, slots = torch.arange(rows, dtype=torch.int32, device="cuda"), torch.randperm(80, generator=torch.Generator().manual_seed(4))[:rows].cuda()
    pools = [[torch.full((5, hkv, page, d), 5.0, dtype=dt, device="cuda") for _ in range(2)] for _ in range(2)]
    p = dkv.dkv_paged_layout(pools[0][0], 1, hq, 5)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    want, _ = dkv.dkv_qk_norm_rope(q, k, pos, d, p=p, v=v, k_pages=pools[0][0], v_pages=pools[0][1], slots=slots, workspace=ws)
    out = torch.zeros_like(want)
    r = dkv.dkv_rotate(rows, hq, hkv, d, dkv.DKV_FP16, 1, d, 1e-6, 1e4, None)
    qs, ks = dkv.dkv_strides(0, d, hq * d), dkv.dkv_strides(0, d, hkv * d)
    st = dkv.lib().dkv_qk_norm_rope(r, q.data_ptr(), qs, k.data_ptr(), ks, None, None, pos.data_ptr(), out.data_ptr(), qs, None, None, p,
                                    v.data_ptr(), ks, slots.data_ptr(), pools[1][0].data_ptr(), pools[1][1].data_ptr(), ws.data_ptr(),
                                    ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == dkv.DKV_OK
    no_fault(ws)
    assert torch.equal(out, want) and torch.equal(pools[1][0], pools[0][0]) and torch.equal(pools[1][1], pools[0][1])


# ---------------------------------------------------------------- pages and slots

def plan_ref(page, n_pages, width, lens, news, free, n_free, table, rows):
    """The definition, one request at a time, on lists."""
    of = lambda n: -(-n // page)  # noqa: E731
    cap = width * page
    free, table = list(free), [list(r) for r in table]
    lens = [min(max(n, 0), cap) for n in lens]
    grow = [n if 0 < n <= cap - m else 0 for n, m in zip(news, lens)]
    cut = [min(-n, m) if n < 0 else 0 for n, m in zip(news, lens)]
    stack = free[:n_free]
    for b in range(len(lens)):
        for j in range(of(lens[b] - cut[b]), of(lens[b])):
            stack.append(table[b][j])
    back = stack[n_free:]
    total, need_all, rows_all = len(stack), 0, 0
    slots, positions, starts, granted, new_lens = [], [], [0], [], []
    for b in range(len(lens)):
        need = of(lens[b] + grow[b]) - of(lens[b])
        need_all += need
        rows_all += grow[b]
        take = grow[b] if (need == 0 or need_all <= total) and rows_all <= rows else 0
        if take:
            for j in range(of(lens[b]), of(lens[b] + take)):
                table[b][j] = stack.pop()
        for t in range(lens[b], lens[b] + take):
            pg = table[b][t // page]
            slots.append(pg * page + t % page if 0 <= pg < n_pages else -1)
            positions.append(t)
        starts.append(starts[-1] + take)
        granted.append(take)
        new_lens.append(lens[b] - cut[b] + take)
    for i, x in enumerate(back):
        if n_free + i < len(free):
            free[n_free + i] = x
    pad = [-1] * (rows - len(slots))
    return slots + pad, positions + pad, starts, granted, new_lens, [min(len(stack), len(free))], table, free


def plan_case(B, page, width, seed, most, fill=1.0, share=(0.3, 0.5, 0.1)):
    g = torch.Generator().manual_seed(seed)
    r = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))  # noqa: E731
    cap = width * page
    lens, news = [], []
    for _ in range(B):
        kind = float(torch.rand(1, generator=g))
        n = r(0, max(0, cap - most))
        if kind < share[0]:
            n, m = 0, r(0, most)
        elif kind < share[0] + share[1]:
            m = 1
        elif kind < sum(share):
            m = -n
        else:
            m = -r(0, n)
        lens.append(n)
        news.append(m)
    used = [-(-n // page) for n in lens]
    need = sum(max(0, -(-(n + m) // page) - u) for n, m, u in zip(lens, news, used))
    n_free = max(0, int(need * fill))
    n_pages = sum(used) + max(n_free, 1) + 3
    perm = torch.randperm(n_pages, generator=g).tolist()
    table = [[-9] * width for _ in range(B)]
    for b, u in enumerate(used):
        for j in range(u):
            table[b][j] = perm.pop()
    free = perm[:n_free] + [-5] * (n_pages - n_free)
    return lens, news, free, n_free, n_pages, table


@pytest.mark.parametrize("B,page,width,most,rows,fill,in_place", [
    (1, 16, 4, 5, 8, 1.0, False), (3, 256, 2, 300, 1000, 1.0, True), (64, 16, 30, 1, 64, 1.0, True), (200, 32, 12, 100, 4000, 0.5, False),
    (1024, 16, 4, 20, 9000, 0.9, True), (1025, 64, 8, 300, 60000, 0.7, False), (4096, 16, 6, 70, 100000, 1.2, True),
    (300, 16, 40, 500, 2000, 1.0, False), (5, 128, 3, 200, 0, 1.0, False)])
def test_plan(B, page, width, most, rows, fill, in_place):
    lens, news, free, n_free, n_pages, table = plan_case(B, page, width, B, most, fill)
    want = plan_ref(page, n_pages, width, lens, news, free, n_free, table, rows)
    p = dkv.dkv_qpaged(B, 1, 1, 64, page, n_pages, width, 0, 0, 0, 1 << 20, 1 << 20)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    L, F, N, T = dev(lens), dev(free), dev([n_free]), dev(table)
    ws = torch.full((dkv.dkv_paged_plan_workspace_bytes(p),), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:256] = 0
    got = dkv.dkv_paged_plan(p, L, dev(news), F, N, T, rows, new_lens=L if in_place else None, new_n_free=N if in_place else None,
                             workspace=ws)
    no_fault(ws)
    for name, x, y in zip(("slots", "positions", "starts", "granted", "lens", "n_free", "table", "free"), (*got, T, F), want):
        assert x.tolist() == y, name


def test_plan_refuses_what_does_not_fit():
    page, width = 16, 4
    p = dkv.dkv_qpaged(5, 1, 1, 64, page, 40, width, 0, 0, 0, 1 << 20, 1 << 20)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.zeros(dkv.dkv_paged_plan_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    lens, news = [60, 64, -3, 100, 16], [5, 1, 3, 0, -20]   # over the capacity twice, bad lengths twice, too many dropped
    table = [[0, 1, 2, 3], [4, 5, 6, 7], [9] * 4, [10, 11, 12, 13], [14, 9, 9, 9]]
    free = [20, 21, 77, -1]                                  # the top page does not exist; one place left in the list
    want = plan_ref(page, 40, width, lens, news, free, 3, table, 20)
    F, T = dev(free), dev(table)
    got = dkv.dkv_paged_plan(p, dev(lens), dev(news), F, dev([3]), T, 20, workspace=ws)
    assert dkv.dkv_get_error(ws) == (dkv.DKV_ERR_DEVICE, dkv.DKV_DEVERR_INDEX)
    assert [x.tolist() for x in (*got, T, F)] == list(want)
    # a list without room for a page that comes back
    F, T = dev([20]), dev(table)
    got = dkv.dkv_paged_plan(p, dev([16, 16, 0, 0, 0]), dev([-16, -1, 0, 0, 0]), F, dev([1]), T, 4, workspace=ws)
    assert int(got[5]) == 1 and F.tolist() == [20] and got[4].tolist() == [0, 15, 0, 0, 0]
    assert dkv.dkv_get_error(ws)[1] == dkv.DKV_DEVERR_INDEX


@pytest.mark.parametrize("B,page,width,most,rows,fill,shift", [
    (256, 16, 30, 200, 9001, 0.7, 0), (7, 64, 200, 9000, 30003, 1.0, 0), (100, 32, 40, 500, 20000, 0.5, 1),  # few requests, two grids
    (40, 16, 12, 60, 1000, 1.0, 1), (64, 128, 9, 300, 8192, 0.8, 1), (1000, 16, 8, 60, 12345, 0.9, 1)])      # rows off 16 bytes
def test_plan_of_few_requests_and_of_rows_anywhere(B, page, width, most, rows, fill, shift):
    lens, news, free, n_free, n_pages, table = plan_case(B, page, width, B + 1, most, fill)
    want = plan_ref(page, n_pages, width, lens, news, free, n_free, table, rows)
    p = dkv.dkv_qpaged(B, 1, 1, 64, page, n_pages, width, 0, 0, 0, 1 << 20, 1 << 20)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    L, F, N, T = dev(lens), dev(free), dev([n_free]), dev(table)
    ws = torch.zeros(dkv.dkv_paged_plan_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    around = [torch.full((rows + 8,), 77, dtype=t, device="cuda") for t in (torch.int64, torch.int32)]
    slots, positions = (x[shift:shift + rows] for x in around)
    got = dkv.dkv_paged_plan(p, L, dev(news), F, N, T, rows, slots=slots, positions=positions, workspace=ws)
    no_fault(ws)
    for name, x, y in zip(("slots", "positions", "starts", "granted", "lens", "n_free", "table", "free"), (*got, T, F), want):
        assert x.tolist() == y, name
    for x in around:
        assert bool((x[:shift] == 77).all()) and bool((x[shift + rows:] == 77).all())


@pytest.mark.parametrize("rows", [8, 9000])
@pytest.mark.parametrize("bad", [-1, 40, 1 << 30])
def test_plan_tells_of_pages_given_back_that_do_not_exist(rows, bad):
    """When they come back, not when another request takes them."""
    page, width = 16, 4
    p = dkv.dkv_qpaged(3, 1, 1, 64, page, 40, width, 0, 0, 0, 1 << 20, 1 << 20)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.zeros(dkv.dkv_paged_plan_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    lens, news = [64, 40, 10], [-30, 5, 2]     # two pages back, none taken
    for there in (7, bad):
        table, free = [[0, 1, 2, there], [4, 5, 6, -9], [8, -9, -9, -9]], [20, 21, -5, -5]
        want = plan_ref(page, 40, width, lens, news, free, 2, table, rows)
        F, T = dev(free), dev(table)
        got = dkv.dkv_paged_plan(p, dev(lens), dev(news), F, dev([2]), T, rows, workspace=ws)
        assert dkv.dkv_get_error(ws)[1] == (0 if there == 7 else dkv.DKV_DEVERR_INDEX)
        assert [x.tolist() for x in (*got, T, F)] == list(want)


# ---------------------------------------------------------------- places and numbers at their limits

def filled(d, hkv, page, n_pages, dt, seed=1, scale=1.0, head_pad=0):
    """A pool of random rows, page i holding tokens i * page and up of one long row, and those rows as they are held (fp64)."""
    store = torch.full((n_pages, hkv, page * 9 * d // 8 + head_pad), 0xFF, dtype=torch.uint8, device="cuda")
    pool = store[..., :page * 9 * d // 8]
    p = dkv.dkv_qpaged_layout(pool, 1, hkv, d, n_pages, dtype=dt)
    g = torch.Generator(device="cuda").manual_seed(seed)
    K, V = ((torch.randn(n_pages * page, hkv, d, generator=g, device="cuda") * scale).to(dt) for _ in range(2))
    dkv.dkv_qpaged_append(p, K, V, pool, torch.arange(n_pages * page, device="cuda"))
    back = [torch.zeros(1, hkv, n_pages * page, d, dtype=torch.float16, device="cuda") for _ in range(2)]
    p16 = dkv.dkv_qpaged_layout(pool, 1, hkv, d, n_pages)
    dkv.dkv_qpaged_gather(p16, pool, torch.arange(n_pages, dtype=torch.int32, device="cuda")[None],
                          torch.zeros(1, dtype=torch.int32, device="cuda"), *back)
    return pool, back[0][0].double(), back[1][0].double()


def exact_rows(q, k, v):
    """q [m, d], k, v [n, d] fp64 -> (out, lse, bounds of the parts) of rows that see everything."""
    s = (q @ k.T) / math.sqrt(q.shape[1])
    w = s.softmax(-1)
    size = 3.1 * (w * v.abs().amax(-1)).sum(-1, keepdim=True)
    ds = R.score_error(q.shape[1], 3.1 * float(q.abs().sum(-1).max() * k.abs().max()) / math.sqrt(q.shape[1]))
    return w @ v, s.logsumexp(-1), size, ds


def near(out, lse, ref, dt, p_eps=2.0 ** -11):
    want, want_lse, size, ds = ref
    tol = torch.finfo(dt).eps / 2 * want.abs() + (p_eps + 2 * ds) * (1 + 2.0 ** -8) * size + 1e-30
    assert bool(((out.double() - want).abs() <= tol).all())
    assert bool(((lse.double() - want_lse).abs() <= ds + 2.0 ** -22 * want_lse.abs().clamp(min=1.0)).all())


def test_most_sequences_that_a_call_takes():
    B, d, page = 4096, 128, 16
    pool, k, v = filled(d, 1, page, 64, torch.float16)
    p = dkv.dkv_qpaged_layout(pool, B, 8, d, 2)
    ws = workspace(p)
    lens = torch.arange(B, dtype=torch.int32, device="cuda") % 33
    table = torch.stack([torch.arange(B) % 63, torch.arange(B) % 63 + 1], 1).int().cuda()
    q = randn((B, 8, d), torch.float16, 3, 2.0).cuda()
    out, lse = dkv.dkv_qpaged_decode(p, q, pool, table, lens, workspace=ws)
    no_fault(ws)
    for b in (0, 1, 32, 33, 100, 2047, 4095):
        n, at = int(lens[b]), b % 63 * page
        if n == 0:
            assert not out[b].any() and bool((lse[b] == -math.inf).all())
        else:
            near(out[b], lse[b], exact_rows(q[b].double(), k[0, at:at + n], v[0, at:at + n]), torch.float16)
    starts = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    out2, lse2 = dkv.dkv_qpaged_prefill(p, q, starts, 1, pool, table, lens, workspace=ws)
    no_fault(ws)
    some = lens > 0
    assert bool(((out2[some].double() - out[some].double()).abs() <= 2.0 ** -8 * v.abs().max()).all())


def test_offsets_past_32_bits():
    d, hkv, page, n_pages = 128, 2, 256, 64
    wide = 140 << 20  # bytes from page to page: 8.75 GB in all
    store = torch.empty(n_pages * wide, dtype=torch.uint8, device="cuda")
    bytes_of = page * 9 * d // 8
    pool = store.as_strided((n_pages, hkv, bytes_of), (wide, wide // 2, 1))
    dt = torch.bfloat16
    p = dkv.dkv_qpaged_layout(pool, 1, 4, d, n_pages, dtype=dt)
    ws = workspace(p)
    n = n_pages * page
    K, V = (randn((n, hkv, d), dt, s).cuda() for s in (1, 2))
    table = torch.arange(n_pages - 1, -1, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    t = torch.arange(n, device="cuda")
    dkv.dkv_qpaged_append(p, K, V, pool, table[0].long()[t // page] * page + t % page, workspace=ws)
    back = [torch.zeros(1, hkv, n, d, dtype=dt, device="cuda") for _ in range(2)]
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    dkv.dkv_qpaged_gather(p, pool, table, zero, *back, workspace=ws)
    for x, y in zip((K, V), back):
        want = Q.values(*Q.quantise(x[-300:].double().cpu())).to(dt)
        assert torch.equal(y[0, :, -300:].cpu(), want.transpose(0, 1))
    q = randn((1, 4, d), dt, 3, 2.0).cuda()
    L = torch.tensor([n], dtype=torch.int32, device="cuda")
    out, lse = dkv.dkv_qpaged_decode(p, q, pool, table, L, workspace=ws)
    out2, lse2 = dkv.dkv_qpaged_prefill(p, q, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), 1, pool, table, L, workspace=ws)
    no_fault(ws)
    exact = dkv.dkv_qpaged_layout(pool, 1, 4, d, n_pages)
    back = [torch.zeros(1, hkv, n, d, dtype=torch.float16, device="cuda") for _ in range(2)]
    dkv.dkv_qpaged_gather(exact, pool, table, zero, *back, workspace=ws)
    for h in range(hkv):
        ref = exact_rows(q[0, 2 * h:2 * h + 2].double(), back[0][0, h].double(), back[1][0, h].double())
        near(out[0, 2 * h:2 * h + 2], lse[0, 2 * h:2 * h + 2], ref, dt)
        near(out2[0, 2 * h:2 * h + 2], lse2[2 * h:2 * h + 2, 0], ref, dt)


@pytest.mark.parametrize("page", [16, 64, 128])
def test_pages_and_lengths_out_of_range(page):
    d, hkv, n_pages, dt = 128, 2, 12, torch.float16
    pool, k, v = filled(d, hkv, page, n_pages, dt, seed=page)
    width = 300 // page + 1
    p = dkv.dkv_qpaged_layout(pool, 3, 4, d, width)
    ws = workspace(p)
    table = torch.zeros(3, width, dtype=torch.int32)
    for b in range(3):
        table[b] = (torch.arange(width) * 5 + b) % n_pages
    bad = min(1, width - 1)
    table[0, bad] = n_pages
    table[2, 0] = -1
    lens = torch.tensor([280, 1 << 20, -4], dtype=torch.int32)  # as they are, the capacity, none
    real = [280, width * page, 0]
    q = randn((3, 4, d), dt, 5, 2.0).cuda()
    out, lse = dkv.dkv_qpaged_decode(p, q, pool, table.cuda(), lens.cuda(), workspace=ws)
    assert dkv.dkv_get_error(ws) == (dkv.DKV_ERR_DEVICE, dkv.DKV_DEVERR_INDEX)
    out2, lse2 = dkv.dkv_qpaged_prefill(p, q, torch.arange(4, dtype=torch.int32, device="cuda"), 1, pool, table.cuda(), lens.cuda(), workspace=ws)
    assert dkv.dkv_get_error(ws) == (dkv.DKV_ERR_DEVICE, dkv.DKV_DEVERR_INDEX)
    for b in range(2):
        t = torch.arange(real[b])
        pg = table[b].long()[t // page]
        ok = ((pg >= 0) & (pg < n_pages)).cuda()
        at = (pg.clamp(0, n_pages - 1) * page + t % page).cuda()
        for h in range(hkv):
            K, V = (torch.where(ok[:, None], x[h][at], 0.0) for x in (k, v))
            ref = exact_rows(q[b, 2 * h:2 * h + 2].double(), K, V)
            near(out[b, 2 * h:2 * h + 2], lse[b, 2 * h:2 * h + 2], ref, dt)
            near(out2[b, 2 * h:2 * h + 2], lse2[2 * h:2 * h + 2, b], ref, dt)
    assert not out[2].any() and bool((lse[2] == -math.inf).all()) and not out2[2].any() and bool((lse2[:, 2] == -math.inf).all())
    back = [torch.full((3, hkv, 20, d), 7.0, dtype=dt, device="cuda") for _ in range(2)]
    first = torch.tensor([page - 4, real[1] - 10, -3], dtype=torch.int32, device="cuda")
    dkv.dkv_qpaged_gather(p, pool, table.cuda(), first, *back, counts=torch.tensor([8, 20, 5], dtype=torch.int32, device="cuda"), workspace=ws)
    assert dkv.dkv_get_error(ws)[1] == dkv.DKV_DEVERR_INDEX
    for x, rows in zip(back, (k, v)):
        at = int(table[0, 0]) * page + page - 4
        assert torch.equal(x[0, :, :4].double(), rows[:, at:at + 4]) and not x[0, :, 4:8].any()
        assert not x[1, :, 10:].any() and not x[2, :, :3].any() and bool((x[0, :, 8:] == 7).all())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("power", [10, 20, 24, 30])
def test_scores_of_any_size(dtype, power):
    """Scores around 2^power: the heaviest key takes all, and nothing overflows."""
    dt, d, n, page = Q.DT[dtype], 128, 700, 64
    pool = torch.zeros(11, 1, page * 144, dtype=torch.uint8, device="cuda")
    p = dkv.dkv_qpaged_layout(pool, 1, 8, d, 11, dtype=dt)
    ws = workspace(p)
    size = 2.0 ** (power / 2)
    K = torch.zeros(n, 1, d)
    K[:, 0, 0] = torch.randperm(n, generator=torch.Generator().manual_seed(power)).double().div(n).mul(2).sub(1) * min(size, 4e4)
    K, V = K.to(dt).cuda(), randn((n, 1, d), dt, 2).cuda()
    dkv.dkv_qpaged_append(p, K, V, pool, torch.arange(n, device="cuda"), workspace=ws)
    q = torch.zeros(1, 8, d)
    q[0, :, 0] = torch.linspace(0.5, 1, 8) * min(size * math.sqrt(d), 6e4)  # (an fp16 query of 2^15 sqrt(d) would be infinite)
    q = q.to(dt).cuda()
    table, L = torch.arange(11, dtype=torch.int32, device="cuda")[None].contiguous(), torch.tensor([n], dtype=torch.int32, device="cuda")
    out, lse = dkv.dkv_qpaged_decode(p, q, pool, table, L, workspace=ws)
    out2, lse2 = dkv.dkv_qpaged_prefill(p, q.expand(40, 8, d).contiguous(), torch.tensor([0, 40], dtype=torch.int32, device="cuda"), 40, pool, table, L, workspace=ws)
    no_fault(ws)
    back = [torch.zeros(1, 1, n, d, dtype=torch.float16, device="cuda") for _ in range(2)]
    dkv.dkv_qpaged_gather(dkv.dkv_qpaged_layout(pool, 1, 8, d, 11), pool, table, L * 0, *back, workspace=ws)
    k, v = (x[0, 0].double() for x in back)
    for j in range(8):
        s = (k @ q[0, j].double()) / math.sqrt(d)
        ds = R.score_error(d, 3.1 * float(s.abs().max()))
        for o, l, pos in [(out[0, j], lse[0, j], n - 1), (out2[0, j], lse2[j, 0], n - 40), (out2[39, j], lse2[j, 39], n - 1), (out2[17, j], lse2[j, 17], n - 23)]:
            t = s[:pos + 1]
            assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(l))
            assert abs(float(l) - float(t.logsumexp(0))) <= ds + 1e-4 + 2.0 ** -22 * float(t.abs().max())
            # what is out of reach of the scores' errors has no weight; the output lies within the others' values
            close = v[:pos + 1][t >= t.max() - 2 * ds - 20]
            assert bool((o.double() <= close.amax(0) + 2.0 ** -7 * 5).all()) and bool((o.double() >= close.amin(0) - 2.0 ** -7 * 5).all())


def test_a_query_that_is_not_finite_stays_alone():
    d, dt, page = 128, torch.bfloat16, 32
    pool, k, v = filled(d, 1, page, 20, dt)
    p = dkv.dkv_qpaged_layout(pool, 2, 8, d, 10, dtype=dt)
    ws = workspace(p)
    table = torch.arange(20, dtype=torch.int32, device="cuda").view(2, 10)
    L = torch.tensor([320, 300], dtype=torch.int32, device="cuda")
    q = randn((2, 8, d), dt, 3).cuda()
    clean, lse = dkv.dkv_qpaged_decode(p, q, pool, table, L, workspace=ws)
    q2 = q.clone()
    q2[0, 3, 5], q2[1, 0, 0] = math.nan, math.inf
    out, lse2 = dkv.dkv_qpaged_decode(p, q2, pool, table, L, workspace=ws)
    hit = torch.zeros(2, 8, dtype=torch.bool, device="cuda")
    hit[0, 3] = hit[1, 0] = True
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse2[~hit], lse[~hit]) and not bool(torch.isfinite(out[hit]).all())
    rows = randn((200, 8, d), dt, 4).cuda()
    starts = torch.tensor([0, 150, 200], dtype=torch.int32, device="cuda")
    clean, _ = dkv.dkv_qpaged_prefill(p, rows, starts, 150, pool, table, L, workspace=ws)
    bad = rows.clone()
    bad[70, 2, 1], bad[180, 7, 127] = math.inf, math.nan
    out, _ = dkv.dkv_qpaged_prefill(p, bad, starts, 150, pool, table, L, workspace=ws)
    hit = torch.zeros(200, 8, dtype=torch.bool, device="cuda")
    hit[70, 2] = hit[180, 7] = True
    # (rows of one warp move their references together: the same values but for a rounding of the weights)
    assert bool(((out[~hit].double() - clean[~hit].double()).abs() <= 2.0 ** -8 * v.abs().max() * 2).all())
    assert not bool(torch.isfinite(out[hit]).all())
    zeros, lz = dkv.dkv_qpaged_decode(p, q * 0, pool, table, L, workspace=ws)
    assert bool(((zeros[0, 0].double() - v[0, :320].mean(0)).abs() <= 2.0 ** -7).all())
    assert abs(float(lz[0, 0]) - math.log(320)) < 1e-5
    no_fault(ws)


def test_prefill_spans_out_of_order():
    d, dt, page = 64, torch.float16, 16
    pool, k, v = filled(d, 2, page, 30, dt)
    p = dkv.dkv_qpaged_layout(pool, 4, 4, d, 7)
    ws = workspace(p)
    table = torch.arange(28, dtype=torch.int32, device="cuda").view(4, 7)
    L = torch.tensor([100, 90, 80, 70], dtype=torch.int32, device="cuda")
    q = randn((60, 4, d), dt, 3).cuda()
    good, _ = dkv.dkv_qpaged_prefill(p, q, torch.tensor([0, 20, 40, 50, 60], dtype=torch.int32, device="cuda"), 20, pool, table, L, workspace=ws)
    no_fault(ws)
    for starts, left_out in (([0, 20, 40, 50, 61], [3]), ([0, 20, 40, 39, 60], [2, 3]), ([-1, 20, 40, 50, 60], [0])):
        out, _ = dkv.dkv_qpaged_prefill(p, q, torch.tensor(starts, dtype=torch.int32, device="cuda"), 20, pool, table, L, workspace=ws)
        assert dkv.dkv_get_error(ws) == (dkv.DKV_ERR_DEVICE, dkv.DKV_DEVERR_INDEX)
        for b, (lo, hi) in enumerate(((0, 20), (20, 40), (40, 50), (50, 60))):
            if b not in left_out:
                assert torch.equal(out[lo:hi], good[lo:hi])
    out, _ = dkv.dkv_qpaged_prefill(p, q, torch.tensor([0, 20, 40, 50, 60], dtype=torch.int32, device="cuda"), 19, pool, table, L, workspace=ws)
    assert dkv.dkv_get_error(ws)[1] == dkv.DKV_DEVERR_INDEX and not out[:40].any() and torch.equal(out[40:], good[40:])


def test_few_queries_under_a_wide_table():
    """The keys of few queries are cut into parts; a table many times as wide as the sequences takes the same path."""
    d, dt, page = 128, torch.bfloat16, 64
    pool, k, v = filled(d, 2, page, 80, dt)
    for width in (40, 2000):
        p = dkv.dkv_qpaged_layout(pool, 2, 12, d, width, dtype=dt)
        ws = workspace(p)
        table = torch.full((2, width), -1, dtype=torch.int32)
        table[0, :40], table[1, :40] = torch.arange(40), torch.arange(40, 80)
        L = torch.tensor([2560, 1500], dtype=torch.int32, device="cuda")
        starts = torch.tensor([0, 9, 14], dtype=torch.int32, device="cuda")
        q = randn((14, 12, d), dt, 5, 2.0).cuda()
        out, lse = dkv.dkv_qpaged_prefill(p, q, starts, 9, pool, table.cuda(), L, workspace=ws)
        no_fault(ws)
        for row, n in ((0, 2552), (8, 2560), (9, 1496), (13, 1500)):
            at = 0 if row < 9 else 2560
            for h in range(2):
                ref = exact_rows(q[row, 6 * h:6 * h + 6].double(), k[h, at:at + n], v[h, at:at + n])
                near(out[row, 6 * h:6 * h + 6], lse[6 * h:6 * h + 6, row], ref, dt)


@pytest.mark.parametrize("dtype,d,hq,hkv,page,B,cached,most,window,sinks", [
    ("fp16", 128, 6, 2, 16, 40, 200, 300, 0, 0),      # groups of 128 tokens of one head, the second often short or empty
    ("bf16", 64, 16, 8, 64, 50, 300, 200, 40, 3),     # groups of two heads
    ("bf16", 128, 4, 1, 32, 400, 20, 40, 0, 0),       # hardly a tile for each CTA; requests without a token
    ("fp16", 64, 5, 1, 128, 100, 0, 300, 100, 0),     # five heads: whole prompts
    ("bf16", 128, 10, 5, 16, 200, 1000, 6, 0, 0),     # a few queries of many sequences, three of five groups' heads idle
    ("fp16", 128, 12, 2, 64, 1, 100, 8000, 0, 0)])
def test_prefill_of_more_tiles_than_multiprocessors(dtype, d, hq, hkv, page, B, cached, most, window, sinks):
    """A CTA then goes on with the places of others: every row as alone, and equal calls equal."""
    dt, rnd = Q.DT[dtype], torch.Generator().manual_seed(d + B)
    news = torch.randint(0, most + 1, (B,), generator=rnd).tolist() if B > 1 else [most]
    lens = [n + int(torch.randint(0, cached + 1, (1,), generator=rnd)) for n in news]
    used = [-(-n // page) for n in lens]
    n_pages = sum(used) + 1
    pool, k, v = filled(d, hkv, page, n_pages, dt, seed=B)
    p = dkv.dkv_qpaged_layout(pool, B, hq, d, max(used), dtype=dt, window=window, sinks=sinks)
    ws = workspace(p)
    at = [sum(used[:b]) for b in range(B)]
    table = (torch.tensor(at)[:, None] + torch.arange(max(used))[None]).clamp(max=n_pages - 1).int().cuda()
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    rows = starts[-1] + 2
    q = randn((rows, hq, d), dt, 5, 2.0).cuda()
    out, lse = torch.full((rows, hq, d), 7.0, dtype=dt, device="cuda"), torch.full((hq, rows), 7.0, device="cuda")
    call = lambda o, x: dkv.dkv_qpaged_prefill(p, q, torch.tensor(starts, dtype=torch.int32, device="cuda"), most, pool, table,  # noqa: E731
                                               torch.tensor(lens, dtype=torch.int32, device="cuda"), out=o, lse=x, workspace=ws)
    call(out, lse)
    no_fault(ws)
    assert bool((out[-2:] == 7).all()) and bool((lse[:, -2:] == 7).all())
    for b in range(B):
        n, m = lens[b], news[b]
        if m == 0:
            continue
        pos, t = torch.arange(n - m, n, device="cuda")[:, None], torch.arange(n, device="cuda")[None]
        sees = t <= pos
        if window:
            sees &= (t > pos - window) | (t < sinks)
        for h in range(hq) if B > 1 else (0, hq - 1):
            kk, vv = (x[h * hkv // hq, at[b] * page:at[b] * page + n] for x in (k, v))
            x = q[starts[b]:starts[b] + m, h].double()
            s = ((x @ kk.T) / math.sqrt(d)).masked_fill(~sees, -math.inf)
            w, big = s.softmax(-1), vv.abs().amax(-1)
            # weights below 2^-24 of fp16's unit are off by 2^-32 of the largest, beside 2^-11 of themselves (as in check_prefill)
            size = 3.1 * ((w * big).sum(-1) + 2.0 ** (11 - 32) * sees.double() @ big)[:, None]
            ds = R.score_error(d, 3.1 * float(x.abs().sum(-1).max() * kk.abs().max()) / math.sqrt(d))
            near(out[starts[b]:starts[b] + m, h], lse[h, starts[b]:starts[b] + m], (w @ vv, s.logsumexp(-1), size, ds), dt)
    for _ in range(3):
        out2, lse2 = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
        call(out2, lse2)
        assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype,d,hq,hkv,page,news,cached,window,sinks", [
    ("fp16", 128, 3, 3, 32, [256, 100], [600, 700], 0, 0),         # 256 tokens of a head a unit: both groups, the first alone
    ("bf16", 64, 1, 1, 16, [384, 1, 300, 128], [900, 64], 0, 0),
    ("fp16", 64, 5, 1, 64, [256, 128, 90], [1000], 500, 70),
    ("bf16", 128, 6, 1, 64, [64, 40, 1], [800, 320], 0, 0),        # four heads of six, then two: the second group without a head
    ("fp16", 128, 10, 2, 128, [30, 17], [1500, 640], 900, 3)])
def test_prefill_where_a_group_has_rows_in_some_units_only(dtype, d, hq, hkv, page, news, cached, window, sinks):
    """A CTA goes from units of two groups of rows to units whose second group is empty, and back."""
    dt, B = Q.DT[dtype], 240
    news = [news[b % len(news)] for b in range(B)]
    lens = [n + cached[b % len(cached)] for b, n in enumerate(news)]
    n_pages = -(-max(lens) // page)
    pool, k, v = filled(d, hkv, page, n_pages, dt, seed=hq)
    p = dkv.dkv_qpaged_layout(pool, B, hq, d, n_pages, dtype=dt, window=window, sinks=sinks)
    ws = workspace(p)
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda").repeat(B, 1)    # one row of tokens for all
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    rows = starts[-1]
    q = randn((rows, hq, d), dt, 6, 2.0).cuda()
    pos = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, news)]).cuda()[:, None]
    t = torch.arange(max(lens), device="cuda")[None]
    sees = t <= pos
    if window:
        sees &= (t > pos - window) | (t < sinks)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    refs = []
    for h in range(hq):
        kk, vv = (x[h * hkv // hq, :max(lens)] for x in (k, v))
        x = q[:, h].double()
        s = ((x @ kk.T) / math.sqrt(d)).masked_fill(~sees, -math.inf)
        w, big = s.softmax(-1), vv.abs().amax(-1)
        # weights below 2^-24 of fp16's unit are off by 2^-32 of the largest, beside 2^-11 of themselves (as in check_prefill)
        size = 3.1 * ((w * big).sum(-1) + 2.0 ** (11 - 32) * sees.double() @ big)[:, None]
        refs.append((w @ vv, s.logsumexp(-1), size, R.score_error(d, 3.1 * float(x.abs().sum(-1).max() * kk.abs().max()) / math.sqrt(d))))
    first = None
    for _ in range(10):
        out, lse = torch.full((rows, hq, d), 7.0, dtype=dt, device="cuda"), torch.full((hq, rows), 7.0, device="cuda")
        dkv.dkv_qpaged_prefill(p, q, dev(starts), max(news), pool, table, dev(lens), out=out, lse=lse, workspace=ws)
        no_fault(ws)
        if first is None:
            first = out, lse
            for h in range(hq):
                near(out[:, h], lse[h], refs[h], dt)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


# ---------------------------------------------------------------- streams, graphs, a run of them together

class Server:
    """A decoding loop as a program would write it: plan, rotate, append, attend."""

    def __init__(self, B=3, hq=6, hkv=2, d=64, page=16, width=12, dt=torch.bfloat16, rows=64, window=0, sinks=0):
        self.B, self.hq, self.hkv, self.d, self.page, self.rows, self.dt = B, hq, hkv, d, page, rows, dt
        n_pages = B * width
        dev = lambda *x: torch.zeros(*x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.pool = torch.full((n_pages, hkv, page * 9 * d // 8), 0xFF, dtype=torch.uint8, device="cuda")
        self.p = dkv.dkv_qpaged_layout(self.pool, B, hq, d, width, dtype=dt, window=window, sinks=sinks)
        self.table, self.lens, self.news = dev(B, width) - 1, dev(B), dev(B)
        self.free = torch.randperm(n_pages, generator=torch.Generator().manual_seed(1)).int().cuda()
        self.n_free = dev(1) + n_pages
        self.ws = workspace(self.p)
        self.pws = torch.zeros(dkv.dkv_paged_plan_workspace_bytes(self.p), dtype=torch.uint8, device="cuda")
        self.slots, self.positions = torch.zeros(rows, dtype=torch.int64, device="cuda"), dev(rows)
        self.starts, self.granted = dev(B + 1), dev(B)
        self.gain = (1 + randn((d,), dt, 5, 0.1)).cuda()
        self.q, self.k = (torch.zeros(rows, n, d, dtype=dt, device="cuda") for n in (hq, hkv))
        self.qkv = torch.zeros(rows, hq + 2 * hkv, d, dtype=dt, device="cuda")
        self.out, self.lse = torch.zeros(rows, hq, d, dtype=dt, device="cuda"), torch.zeros(hq, rows, device="cuda")
        self.out1, self.lse1 = torch.zeros(B, hq, d, dtype=dt, device="cuda"), torch.zeros(B, hq, device="cuda")

    def step(self, max_q, stream=None):
        dkv.dkv_paged_plan(self.p, self.lens, self.news, self.free, self.n_free, self.table, self.rows, slots=self.slots,
                           positions=self.positions, starts=self.starts, granted=self.granted, new_lens=self.lens,
                           new_n_free=self.n_free, workspace=self.pws, stream=stream)
        q, k, v = self.qkv.split([self.hq, self.hkv, self.hkv], 1)
        dkv.dkv_qk_norm_rope(q, k, self.positions, 64, 1e4, q_gain=self.gain, k_gain=self.gain, q_out=self.q, k_out=self.k, stream=stream)
        dkv.dkv_qpaged_append(self.p, self.k, v, self.pool, self.slots, workspace=self.ws, stream=stream)
        if max_q == 1:  # every sequence has one new token: row b is sequence b's
            dkv.dkv_qpaged_decode(self.p, self.q[:self.B], self.pool, self.table, self.lens, out=self.out1, lse=self.lse1, workspace=self.ws,
                                  stream=stream)
        dkv.dkv_qpaged_prefill(self.p, self.q, self.starts, max_q, self.pool, self.table, self.lens, out=self.out, lse=self.lse,
                               workspace=self.ws, stream=stream)


def run_server(s, steps, launch, window=0, sinks=0):
    """steps: new tokens of each sequence (below 0: dropped); every step's outputs against attention over the rows that went in."""
    kept = [[[], []] for _ in range(s.B)]
    g = torch.Generator().manual_seed(9)
    for news in steps:
        s.news.copy_(torch.tensor(news, dtype=torch.int32))
        s.qkv.copy_((torch.randn(*s.qkv.shape, generator=g) * 1.5).to(s.dt))
        launch(max(max(news), 1))
        torch.cuda.synchronize()
        assert s.granted.tolist() == [max(n, 0) for n in news]
        starts = s.starts.tolist()
        q, k, v = s.q.cpu(), s.k.cpu(), s.qkv[:, s.hq + s.hkv:].cpu()
        for b, n in enumerate(news):
            if n < 0:
                for x in kept[b]:
                    del x[len(x) + n:]
            for i in range(starts[b], starts[b + 1]):
                assert int(s.positions[i]) == len(kept[b][0])
                kept[b][0].append(Q.values(*Q.quantise(k[i].double())))
                kept[b][1].append(Q.values(*Q.quantise(v[i].double())))
            assert int(s.lens[b]) == len(kept[b][0])
            if n <= 0:
                continue
            K, V = (torch.stack(x, 1) for x in kept[b])          # [hkv][tokens][d]
            pos = torch.arange(K.shape[1] - n, K.shape[1])
            for j in range(s.hq):
                h = j * s.hkv // s.hq
                rows = slice(starts[b], starts[b + 1])
                ref = R.attend(q[rows, j].double(), K[h], V[h], pos, window, sinks)
                size = 3.1 * (ref[2] * V[h].abs().amax(-1)).sum(-1, keepdim=True).expand(-1, s.d)
                parts = 3.1 * float(q[rows, j].double().abs().sum(-1).max() * K[h].abs().max()) / math.sqrt(s.d)
                size = size + 2.0 ** (11 - 32) * 3.1 * V[h].abs().amax(-1).sum()  # weights in fp16's subnormals
                R.check_rows(s.out[rows, j], s.lse[j, rows], (*ref[:3], size, parts), s.d, s.dt, 2.0 ** -11, f"step {news} sequence {b} head {j}")
                if max(news) == 1:
                    assert news == [1] * s.B
                    R.check_rows(s.out1[b:b + 1, j], s.lse1[b:b + 1, j], (*ref[:3], size, parts), s.d, s.dt, 2.0 ** -11, f"decode {b} head {j}")
    no_fault(s.ws)
    no_fault(s.pws)


def test_run_of_them_together():
    s = Server()
    run_server(s, [[20, 5, 33], [1, 1, 1], [1, 1, 1], [0, 30, -33], [7, -20, 16], [1, 1, 1], [-28, 40, 12], [1, 1, 1]], s.step)
    assert int(s.n_free) + sum(-(-n // s.page) for n in s.lens.tolist()) == s.B * 12
    s = Server(window=17, sinks=2)
    run_server(s, [[20, 5, 33], [1, 1, 1], [0, 30, 0], [1, 1, 1]], s.step, window=17, sinks=2)


def test_run_on_another_stream_and_in_a_graph():
    s = Server()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def on_side(max_q):
        side.wait_stream(torch.cuda.current_stream())
        s.step(max_q, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    run_server(s, [[20, 5, 33], [1, 1, 1], [3, 0, 2]], on_side)

    s = Server()
    s.step(1)  # (kernels are loaded before the capture; no sequence grows)
    torch.cuda.synchronize()
    graphs = {}
    for max_q in (1, 64):
        graphs[max_q] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[max_q]):
            s.step(max_q)
    run_server(s, [[20, 5, 33], [1, 1, 1], [0, 30, -33], [7, -20, 16], [1, 1, 1], [1, 1, 1]], lambda n: graphs[1 if n == 1 else 64].replay())


def test_outputs_allocated_in_the_given_stream():
    d, dt, page = 128, torch.float16, 32
    pool, k, v = filled(d, 2, page, 40, dt)
    p = dkv.dkv_qpaged_layout(pool, 1, 8, d, 40)
    table = torch.arange(40, dtype=torch.int32, device="cuda")[None].contiguous()
    L = torch.tensor([1280], dtype=torch.int32, device="cuda")
    q = randn((1, 8, d), dt, 5).cuda()
    want, want_lse = dkv.dkv_qpaged_decode(p, q, pool, table, L)
    starts = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    want2, _ = dkv.dkv_qpaged_prefill(p, q, starts, 1, pool, table, L)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(20):
        busy = torch.randn(2048, 2048, device="cuda")
        busy = busy @ busy                                  # the current stream is behind
        out, lse = dkv.dkv_qpaged_decode(p, q, pool, table, L, stream=side)
        out2, _ = dkv.dkv_qpaged_prefill(p, q, starts, 1, pool, table, L, stream=side)
        side.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse) and torch.equal(out2, want2)


def test_two_calls_at_once():
    """Two streams, a workspace each, over one pool."""
    d, dt, page = 128, torch.bfloat16, 64
    pool, k, v = filled(d, 4, page, 200, dt)
    p = dkv.dkv_qpaged_layout(pool, 2, 8, d, 100, dtype=dt)
    table = torch.arange(200, dtype=torch.int32, device="cuda").view(2, 100)
    L = torch.tensor([6400, 3000], dtype=torch.int32, device="cuda")
    qs = [randn((2, 8, d), dt, s).cuda() for s in (1, 2)]
    ws = [workspace(p) for _ in range(2)]
    want = [dkv.dkv_qpaged_decode(p, q, pool, table, L, workspace=ws[0]) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = [dkv.dkv_qpaged_decode(p, q, pool, table, L, workspace=w, stream=s) for q, w, s in zip(qs, ws, streams)]
        torch.cuda.synchronize()
        for (a, b), (c, e) in zip(got, want):
            assert torch.equal(a, c) and torch.equal(b, e)
    for w in ws:
        no_fault(w)


def test_rows_go_on_to_the_compressed_cache():
    """Tokens of the 4-bit pages, read back, are what the compressed cache is made of."""
    d, hkv, page, n = 64, 2, 64, 3 * 256 + 100
    pool, k, v = filled(d, hkv, page, 14, torch.float16)
    p = dkv.dkv_qpaged_layout(pool, 1, 4, d, 14)
    K, V = (torch.zeros(1, hkv, n, d, dtype=torch.float16, device="cuda") for _ in range(2))
    dkv.dkv_qpaged_gather(p, pool, torch.arange(14, dtype=torch.int32, device="cuda")[None].contiguous(), torch.zeros(1, dtype=torch.int32, device="cuda"), K, V)
    desc = dkv.dkv_layout(1, 4, hkv, d, 3, 100, 16, 32)
    cache = dkv.dkv_compress_layout(desc, K, V)
    q = randn((1, 4, d), torch.float16, 3).cuda()
    out, lse, _ = dkv.dkv_decode_attend(desc, q, cache, 3)
    exact, _ = dkv.dkv_qpaged_decode(dkv.dkv_qpaged_layout(pool, 1, 4, d, 14), q, pool, torch.arange(14, dtype=torch.int32, device="cuda")[None].contiguous(),
                                     torch.tensor([n], dtype=torch.int32, device="cuda"))
    assert bool(torch.isfinite(out).all()) and tuple(out.shape) == (1, 4, d) and tuple(exact.shape) == (1, 4, d)


def test_rows_that_go_on_are_the_rows_that_went_in():
    """Gathered keys and values are the quantised rows of their tokens and heads, the compressed cache made of them is the
    one made of those rows, and the attention over the pages is theirs."""
    d, hkv, page, n, dt = 64, 2, 64, 3 * 256 + 100, torch.float16
    n_pages = -(-n // page)
    pool = torch.zeros(n_pages, hkv, page * 9 * d // 8, dtype=torch.uint8, device="cuda")
    p = dkv.dkv_qpaged_layout(pool, 1, 4, d, n_pages)
    rows = [randn((n, hkv, d), dt, s) for s in (1, 2)]
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(3))
    t = torch.arange(n)
    dkv.dkv_qpaged_append(p, *(x.cuda() for x in rows), pool, (order[t // page] * page + t % page).cuda())
    table, zero = order.int()[None].cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    back = [torch.zeros(1, hkv, n, d, dtype=dt, device="cuda") for _ in range(2)]
    dkv.dkv_qpaged_gather(p, pool, table, zero, *back)
    held = [Q.values(*Q.quantise(x.transpose(0, 1).double())) for x in rows]
    for x, y in zip(back, held):
        assert torch.equal(x[0].double().cpu(), y)
    q = randn((1, 4, d), dt, 3).cuda()
    desc = dkv.dkv_layout(1, 4, hkv, d, 3, 100, 16, 32)
    got, want = (dkv.dkv_decode_attend(desc, q, dkv.dkv_compress_layout(desc, *kv), 3)
                 for kv in (back, [x.to(dt)[None].contiguous().cuda() for x in held]))
    assert all(torch.equal(x, y) for x, y in zip(got, want)) and bool(torch.isfinite(got[0]).all())
    out, lse = dkv.dkv_qpaged_decode(p, q, pool, table, zero + n)
    for h in range(hkv):
        at = slice(2 * h, 2 * h + 2)
        near(out[0, at], lse[0, at], exact_rows(q[0, at].double(), *(x[h].cuda() for x in held)), dt)
