"""The paged-cache operators against their definitions in 64 bits: head layouts, types, page sizes and
orders, lengths from none on, windows, sinks, ragged batches; slots that nothing may look at hold NaN
and infinities, unneeded page-table entries numbers out of range."""
import math

import pytest
import torch

from compressed_kv_cache_dkv_gb300 import dkv, synth
from tests import paged_ref as R

pytestmark = pytest.mark.gpu


def no_fault(ws):
    assert dkv.dkv_get_error(ws) == (dkv.DKV_OK, 0)


def workspace(p, weights=False):
    ws = torch.full((dkv.dkv_paged_workspace_bytes(p, weights),), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:256] = 0  # only the header has to be zero
    return ws


def queries(shape, dt, seed, scale=2.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dt)


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("dtype,d,hkv,page,order,lens,news", [
    ("fp16", 128, 2, 16, "head", [1], [1]),
    ("bf16", 64, 1, 32, "token", [5, 33, 64], [5, 1, 0]),
    ("fp16", 64, 3, 256, "token", [700, 256, 257], [700, 256, 1]),
    ("bf16", 128, 8, 64, "head", [1000, 1, 63], [999, 0, 63]),
])
def test_append_writes_its_tokens_only(dtype, d, hkv, page, order, lens, news):
    c = R.Cache(lens, hkv, d, page, dtype, order, seed=3)
    p, ws = c.layout(hkv), None
    ws = workspace(p)
    n = max(max(news), 1)
    K, V = (queries((c.B, n, hkv, d), c.dt, s).cuda().transpose(1, 2) for s in (1, 2))
    want = [x.clone() for x in (c.k, c.v)]
    for b in range(c.B):
        t = torch.arange(lens[b] - news[b], lens[b])
        for x, new in zip(want, (K, V)):
            x[c.table[b].long()[t // page].cuda(), :, (t % page).cuda()] = new[b, :, :news[b]].transpose(0, 1)
    dkv.dkv_paged_append(p, K, V, c.k, c.v, c.table.cuda(), c.dev([a - x for a, x in zip(lens, news)]), c.dev(news), workspace=ws)
    no_fault(ws)
    for x, y in zip((c.k, c.v), want):
        assert torch.equal(x.contiguous().view(torch.int16), y.contiguous().view(torch.int16))


def test_append_takes_differing_strides_and_skips_bad_places():
    c = R.Cache([40, 20], 2, 64, 16, seed=4)
    p = c.layout(2)
    ws = workspace(p)
    K = queries((2, 2, 8, 64), c.dt, 1).cuda()
    V = queries((2, 8, 2, 64), c.dt, 2).cuda().transpose(1, 2)
    table = c.table.clone()
    table[0, 1] = c.n_pages      # tokens 16..31 of sequence 0 lie on a page that is not there
    before = c.k.clone()
    dkv.dkv_paged_append(p, K, V, c.k, c.v, table.cuda(), c.dev([12, 45]), workspace=ws)  # 48 tokens of room
    assert dkv.dkv_get_error(ws) == (dkv.DKV_ERR_DEVICE, dkv.DKV_DEVERR_INDEX)
    t = torch.arange(12, 16)
    assert torch.equal(c.row(c.k, 0, 1, t), K[0, 1, :4].double().cpu())
    assert torch.equal(c.row(c.v, 0, 1, t), V[0, 1, :4].double().cpu())
    changed = (c.k.view(torch.int16) != before.view(torch.int16)).any(-1).sum()  # rows: 4 tokens x 2 heads ...
    # ... and positions 45..47 of sequence 1, whose third table entry is out of range: skipped
    assert int(changed) == 8


# ---------------------------------------------------------------- decode

DECODE = [
    # dtype, d, hq, hkv, page, order, lens, window, sinks
    ("fp16", 128, 12, 2, 64, "head", [1000], 0, 0),
    ("fp16", 64, 1, 1, 16, "token", [1], 0, 0),
    ("bf16", 128, 8, 1, 16, "token", [1, 2, 63, 64, 65, 127, 128, 129, 0], 0, 0),
    ("bf16", 64, 9, 3, 32, "head", [0, 300, 0, 17, 555], 0, 0),
    ("fp16", 128, 7, 7, 256, "token", [5, 2049], 0, 0),
    ("bf16", 128, 5, 1, 128, "head", [777, 1300], 100, 0),
    ("fp16", 128, 12, 4, 16, "token", [50, 64, 65, 500, 1999], 64, 4),
    ("bf16", 64, 16, 2, 64, "head", [3000, 1, 70, 71], 70, 1),
    ("fp16", 64, 4, 2, 32, "token", [900, 130], 1, 0),
    ("fp16", 128, 6, 2, 64, "head", [1500, 333], 200, 130),
    ("bf16", 128, 2, 1, 32, "token", [400, 90], 1000, 5),
]


@pytest.mark.parametrize("dtype,d,hq,hkv,page,order,lens,window,sinks", DECODE)
@pytest.mark.parametrize("weighed", [False, True])
def test_decode(dtype, d, hq, hkv, page, order, lens, window, sinks, weighed):
    c = R.Cache(lens, hkv, d, page, dtype, order, seed=len(lens))
    p = c.layout(hq, window, sinks)
    ws = workspace(p, weighed)
    q = queries((c.B, hq, d), c.dt, 7)
    weights = torch.rand(c.B, hkv, c.width * page, generator=torch.Generator().manual_seed(1)) if weighed else None
    got = weights.cuda() if weighed else None
    table = c.hidden_table([n - 1 for n in lens], window, sinks)
    out, lse = dkv.dkv_paged_decode(p, q.cuda(), c.k, c.v, table, c.dev(lens), weights=got, workspace=ws)
    no_fault(ws)
    p_eps = 2.0 ** -16 if dtype == "bf16" else 2.0 ** -21  # p as two halves of its type
    for b in range(c.B):
        for h in range(hkv):
            added = torch.zeros(c.width * page, dtype=torch.float64)
            big = 0.0
            for j in range(h * hq // hkv, (h + 1) * hq // hkv):
                ref = R.attend(q[b, j:j + 1].double(), c.K[b][h], c.V[b][h], torch.tensor([lens[b] - 1]), window, sinks)
                R.check_rows(out[b, j:j + 1], lse[b, j:j + 1], ref, d, c.dt, p_eps, f"sequence {b} head {j}")
                added[:lens[b]] += ref[2][0]
                big = max(big, ref[4])
            if weighed:
                want = weights[b, h].double() + added
                # each weight is off by its score's and the lse's errors; fp32 adds the heads and the old value
                tol = (2 * R.score_error(d, big) + 2.0 ** -20 * (1 + math.log(max(2, lens[b])))) * added + 2.0 ** -22 * want
                assert bool(((got[b, h].double().cpu() - want).abs() <= tol).all()), f"weights of sequence {b} head {h}"


def test_decode_takes_strided_queries_and_own_buffers():
    c = R.Cache([130, 70], 2, 128, 64, seed=5)
    p = c.layout(4)
    qkv = queries((2, 8, 128), c.dt, 8).cuda()      # q heads first, K and V heads behind them
    q = qkv[:, :4]
    out = torch.empty(2, 4, 128, dtype=c.dt, device="cuda")
    o, lse = dkv.dkv_paged_decode(p, q, c.k, c.v, c.table.cuda(), c.dev([130, 70]), out=out, lse=False)
    assert o is out and lse is None
    want, _ = dkv.dkv_paged_decode(p, q.contiguous(), c.k, c.v, c.table.cuda(), c.dev([130, 70]))
    assert torch.equal(out, want)


def test_decode_of_many_sequences_covers_every_deal():
    """Units of every length dealt to the multiprocessors: some runs hold many units, some a part of one."""
    lens = [(i * 37) % 400 for i in range(700)]
    c = R.Cache(lens, 1, 64, 32, "bf16", seed=6)
    p = c.layout(2)
    ws = workspace(p)
    q = queries((c.B, 2, 64), c.dt, 9)
    out, lse = dkv.dkv_paged_decode(p, q.cuda(), c.k, c.v, c.table.cuda(), c.dev(lens), workspace=ws)
    no_fault(ws)
    out, lse = out.cpu(), lse.cpu()
    for b in range(c.B):
        ref = R.attend(q[b].double(), c.K[b][0], c.V[b][0], torch.full((2,), lens[b] - 1), 0, 0)
        R.check_rows(out[b], lse[b], ref, 64, c.dt, 2.0 ** -16, f"sequence {b}")


@pytest.mark.parametrize("dtype,hkv,hq,lens,window,sinks", [
    ("fp16", 2, 12, [60000, 20000], 0, 0), ("bf16", 8, 8, [30001], 0, 0), ("fp16", 4, 8, [25000, 9000, 31000], 20000, 100)])
@pytest.mark.parametrize("weighed", [False, True])
def test_decode_of_long_sequences(dtype, hkv, hq, lens, window, sinks, weighed):
    """Many tiles in a row on every multiprocessor: the ring of tiles goes round several times."""
    c = R.Cache(lens, hkv, 128, 256, dtype, seed=8)
    p = c.layout(hq, window, sinks)
    ws = workspace(p, weighed)
    q = queries((c.B, hq, 128), c.dt, 10)
    weights = torch.zeros(c.B, hkv, c.width * 256, device="cuda") if weighed else None
    out, lse = dkv.dkv_paged_decode(p, q.cuda(), c.k, c.v, c.table.cuda(), c.dev(lens), weights=weights, workspace=ws)
    no_fault(ws)
    for b in range(c.B):
        for h in range(hkv):
            added, big = torch.zeros(lens[b], dtype=torch.float64), 0.0
            for j in range(h * hq // hkv, (h + 1) * hq // hkv):
                ref = R.attend(q[b, j:j + 1].double(), c.K[b][h], c.V[b][h], torch.tensor([lens[b] - 1]), window, sinks)
                R.check_rows(out[b, j:j + 1], lse[b, j:j + 1], ref, 128, c.dt, 2.0 ** -16 if dtype == "bf16" else 2.0 ** -21)
                added += ref[2][0]
                big = max(big, ref[4])
            if weighed:
                tol = (2 * R.score_error(128, big) + 2.0 ** -20 * (1 + math.log(lens[b]))) * added + 2.0 ** -40
                assert bool(((weights[b, h, :lens[b]].double().cpu() - added).abs() <= tol).all())


def test_lengths_and_pages_out_of_range_are_reported():
    c = R.Cache([100, 50], 1, 64, 16, seed=7)
    p = c.layout(1)
    ws = workspace(p)
    q = queries((2, 1, 64), c.dt, 3)
    for lens in ([100, -5], [c.width * 16 + 9, 50]):
        table = c.table.clone()
        table[table < 0] = 0
        out, lse = dkv.dkv_paged_decode(p, q.cuda(), c.k, c.v, table.cuda(), c.dev(lens), workspace=ws)
        assert dkv.dkv_get_error(ws) == (dkv.DKV_ERR_DEVICE, dkv.DKV_DEVERR_INDEX)
        good = 0 if lens[1] < 0 else 1
        ref = R.attend(q[good].double(), c.K[good][0], c.V[good][0], torch.tensor([c.lens[good] - 1]), 0, 0)
        R.check_rows(out[good], lse[good], ref, 64, c.dt, 2.0 ** -21)
        if lens[1] < 0:
            assert float(out[1].abs().max()) == 0 and bool(torch.isneginf(lse[1]).all())
    table = c.table.clone()
    table[0, 2] = c.n_pages + 1  # read as a page of zeros: scores 0, values 0
    out, lse = dkv.dkv_paged_decode(p, q.cuda(), c.k, c.v, table.cuda(), c.dev([100, 50]), workspace=ws)
    assert dkv.dkv_get_error(ws) == (dkv.DKV_ERR_DEVICE, dkv.DKV_DEVERR_INDEX)
    K, V = c.K[0][0].clone(), c.V[0][0].clone()
    K[32:48] = V[32:48] = 0
    R.check_rows(out[0], lse[0], R.attend(q[0].double(), K, V, torch.tensor([99]), 0, 0), 64, c.dt, 2.0 ** -21)


# ---------------------------------------------------------------- prefill and weights

PREFILL = [
    # dtype, d, hq, hkv, page, order, lens, q_lens (None: all Tq), Tq, window, sinks
    ("fp16", 128, 2, 1, 64, "head", [128], None, 128, 0, 0),
    ("bf16", 128, 2, 1, 64, "head", [300], None, 300, 0, 0),
    ("fp16", 64, 1, 1, 16, "token", [1], None, 1, 0, 0),
    ("fp16", 128, 3, 1, 32, "token", [513], None, 513, 0, 0),
    ("bf16", 64, 12, 2, 128, "head", [700, 129, 64], [300, 129, 1], 300, 0, 0),
    ("fp16", 64, 5, 1, 256, "token", [1000, 0, 40], [17, 0, 33], 33, 0, 0),
    ("bf16", 128, 8, 8, 16, "token", [600], None, 600, 128, 0),
    ("fp16", 128, 12, 2, 64, "head", [900, 500], [900, 257], 900, 100, 4),
    ("bf16", 64, 7, 1, 32, "head", [777], None, 400, 33, 130),
    ("fp16", 128, 4, 1, 16, "head", [1200], None, 260, 1, 1),
    ("bf16", 128, 2, 2, 64, "token", [640], None, 640, 300, 300),
    ("fp16", 64, 6, 3, 32, "token", [20, 300], [50, 50], 50, 40, 2),   # sequence 0: 30 queries before its first token
    # the first 128 rows of a 256-row block lie before the first token, the others do not
    ("bf16", 128, 1, 1, 64, "head", [100, 40, 300], [256, 200, 256], 256, 0, 0),
    ("fp16", 64, 3, 1, 16, "token", [1], None, 600, 30, 1),
    # few queries over many keys: several heads to a row group, the keys cut into parts
    ("bf16", 128, 8, 1, 16, "token", [5000, 1700, 0, 130], [8, 3, 0, 8], 8, 0, 0),
    ("fp16", 64, 7, 1, 64, "head", [4000], None, 16, 300, 4),
    ("bf16", 128, 6, 2, 32, "head", [2500, 900], [64, 40], 64, 0, 0),
    ("fp16", 128, 3, 1, 128, "token", [1111], None, 50, 0, 0),
    ("bf16", 64, 5, 1, 256, "head", [2049, 64], [9, 1], 9, 1000, 100),
    ("fp16", 128, 4, 4, 64, "head", [1500], None, 1, 0, 0),
    ("bf16", 128, 4, 1, 64, "head", [2300], None, 100, 0, 0),
    ("fp16", 64, 16, 2, 16, "token", [700, 690], None, 33, 128, 64),
    # many tiles: the rings go round
    ("bf16", 64, 2, 1, 64, "head", [4500], None, 4500, 0, 0),
    ("fp16", 128, 3, 1, 16, "token", [2600], None, 2600, 1500, 3),
]


@pytest.mark.parametrize("dtype,d,hq,hkv,page,order,lens,q_lens,Tq,window,sinks", PREFILL)
def test_prefill_and_weights(dtype, d, hq, hkv, page, order, lens, q_lens, Tq, window, sinks):
    c = R.Cache(lens, hkv, d, page, dtype, order, seed=Tq)
    p = c.layout(hq, window, sinks)
    ws = workspace(p)
    n_q = q_lens or [Tq] * c.B
    q = queries((c.B, Tq, hq, d), c.dt, 11).transpose(1, 2)
    for b, n in enumerate(n_q):
        q[b, :, n:] = float("nan")  # rows of padding
    out = torch.full((c.B, Tq, hq, d), 7.0, dtype=c.dt, device="cuda").transpose(1, 2)
    lse = torch.full((c.B, hq, Tq), 7.0, device="cuda")
    table = c.hidden_table([n - m for n, m in zip(lens, n_q)], window, sinks)
    ql = None if q_lens is None else c.dev(q_lens)
    qd = q.cuda()
    dkv.dkv_paged_prefill(p, qd, c.k, c.v, table, c.dev(lens), q_lens=ql, out=out, lse=lse, workspace=ws)
    no_fault(ws)
    old = torch.rand(c.B, hkv, c.width * page, generator=torch.Generator().manual_seed(1))
    weights = old.cuda()
    dkv.dkv_paged_weights(p, qd, lse, c.k, table, c.dev(lens), weights, q_lens=ql, workspace=ws)
    no_fault(ws)
    for b in range(c.B):
        pos = torch.arange(n_q[b]) + lens[b] - n_q[b]
        assert bool((out[b, :, n_q[b]:] == 7).all()) and bool((lse[b, :, n_q[b]:] == 7).all())
        for h in range(hkv):
            added, big, lse_off = torch.zeros(c.width * page, dtype=torch.float64), 0.0, 0.0
            for j in range(h * hq // hkv, (h + 1) * hq // hkv):
                ref = R.attend(q[b, j, :n_q[b]].double(), c.K[b][h], c.V[b][h], pos, window, sinks)
                R.check_rows(out[b, j, :n_q[b]], lse[b, j, :n_q[b]], ref, d, c.dt, torch.finfo(c.dt).eps / 2,
                             f"sequence {b} head {j}")
                added[:lens[b]] += ref[2].sum(0)
                big = max(big, ref[4])
            want = old[b, h].double() + added
            rows = n_q[b] * hq // hkv
            # each weight: its score's and the lse's errors; fp32 adds `rows` weights in 8 partial sums
            tol = (2 * R.score_error(d, big) + 2.0 ** -20 * (1 + math.log(max(2, lens[b]))) + 2.0 ** -23 * (rows / 8 + 8)) * added + 2.0 ** -22 * want
            err = (weights[b, h].double().cpu() - want).abs()
            assert bool((err <= tol).all()), f"weights of sequence {b} head {h}: {float((err - tol).max())}"


@pytest.mark.parametrize("dtype,d,hq,window,sinks", [("fp16", 128, 2, 0, 0), ("bf16", 64, 1, 90, 3), ("bf16", 128, 4, 200, 20)])
def test_prefill_rows_are_not_touched_by_keys_they_do_not_see(dtype, d, hq, window, sinks):
    """NaN and infinities in the values (and keys) of some tokens reach the rows that see them, and no other."""
    n, bad = 500, [3, 130, 260, 261, 444]
    c = R.Cache([n], 1, d, 64, dtype, seed=2)
    p = c.layout(hq, window, sinks)
    q = queries((1, hq, n, d), c.dt, 5).cuda()
    clean, clean_lse = dkv.dkv_paged_prefill(p, q, c.k, c.v, c.table.cuda(), c.dev([n]))
    k, v = c.k.clone(), c.v.clone()
    for i, t in enumerate(bad):
        where = (int(c.table[0, t // 64]), 0, t % 64)
        if i % 2 == 0:
            v[where] = torch.tensor([float("nan"), float("inf")], dtype=c.dt).repeat(d // 2)
        else:
            k[where] = float("nan")
    out, lse = dkv.dkv_paged_prefill(p, q, k, v, c.table.cuda(), c.dev([n]))
    m = R.seen(torch.arange(n), n, window, sinks)
    sees_v = m[:, [t for i, t in enumerate(bad) if i % 2 == 0]].any(1)
    sees_k = m[:, [t for i, t in enumerate(bad) if i % 2 == 1]].any(1)
    good = (~sees_v & ~sees_k).cuda()
    assert torch.equal(out[0][:, good], clean[0][:, good])
    assert torch.equal(lse[0][:, good], clean_lse[0][:, good])
    assert bool(torch.isnan(out[0][:, sees_k.cuda()]).all()) and bool(torch.isnan(lse[0][:, sees_k.cuda()]).all())
    # the values reach the rows that see them: NaN stays NaN (channels 0, 2, ...), +inf stays +inf unless a NaN joins
    only_v = (sees_v & ~sees_k).cuda()
    assert bool(torch.isnan(out[0][:, only_v][..., 0::2]).all())
    assert not bool(torch.isfinite(out[0][:, only_v][..., 1::2]).any())
    assert bool(torch.isfinite(lse[0][:, only_v]).all())


def test_few_queries_are_not_touched_by_keys_they_do_not_see():
    """The same where the keys are cut into parts and joined."""
    n, Tq, d = 3001, 6, 128
    c = R.Cache([n], 1, d, 64, "bf16", seed=21)
    p = c.layout(4, window=2000, sinks=10)
    q = queries((1, 4, Tq, d), c.dt, 5)
    v = c.v.clone()
    for t, x in ((9, "nan"), (10, "nan"), (995, "inf"), (n - 3, "nan"), (n - 1, "inf")):
        v[int(c.table[0, t // 64]), 0, t % 64, :64] = float(x)
    out, lse = dkv.dkv_paged_prefill(p, q.cuda(), c.k, v, c.table.cuda(), c.dev([n]))
    pos = torch.arange(n - Tq, n)
    m = R.seen(pos, n, 2000, 10)
    # token 9 is a sink; the first row, at 2995, sees tokens from 2995 - 2000 + 1 = 996 on, so that none sees 995
    assert bool(m[:, 9].all()) and not bool(m[:, 10].any()) and not bool(m[:, 995].any())
    V = c.V[0][0].clone()
    for j in range(4):
        ref = R.attend(q[0, j].double(), c.K[0][0], V, pos, 2000, 10)
        assert bool(torch.isnan(out[0, j, :, :64]).all())
        sub = (ref[0][:, 64:], ref[1], ref[2], ref[3][:, 64:], ref[4])
        R.check_rows(out[0, j][:, 64:], lse[0, j], sub, d, c.dt, torch.finfo(c.dt).eps / 2)
    v[int(c.table[0, 0]), 0, 9] = 1.0  # now the first rows are free of NaN, the last three are not
    out, _ = dkv.dkv_paged_prefill(p, q.cuda(), c.k, v, c.table.cuda(), c.dev([n]))
    assert bool(torch.isfinite(out[0, :, :Tq - 3]).all()) and bool(torch.isnan(out[0, :, Tq - 3:, :64]).all())
    assert bool(torch.isfinite(out[0, :, :, 64:]).all())


def test_prefill_adds_large_values_of_edge_tiles_exactly():
    """A row that sees one infinite channel keeps its other channels."""
    n, d = 140, 64
    c = R.Cache([n], 1, d, 32, "fp16", seed=12)
    p = c.layout(1)
    q = queries((1, 1, n, d), c.dt, 5)
    v = c.v.clone()
    t = 100
    v[int(c.table[0, t // 32]), 0, t % 32, 5] = float("-inf")
    out, lse = dkv.dkv_paged_prefill(p, q.cuda(), c.k, v, c.table.cuda(), c.dev([n]))
    assert bool((out[0, 0, t:, 5] == float("-inf")).all())
    ref = R.attend(q[0, 0].double(), c.K[0][0], c.V[0][0], torch.arange(n), 0, 0)
    keep = [i for i in range(d) if i != 5]
    sub = (ref[0][:, keep], ref[1], ref[2], ref[3][:, keep], ref[4])
    R.check_rows(out[0, 0][:, keep], lse[0, 0], sub, d, c.dt, torch.finfo(c.dt).eps / 2)


# ---------------------------------------------------------------- evict

def _evict_check(c, p, weights, budget, first, recent, kept, new_lens, new_weights, table, k, v):
    """k, v: the pools before; the kept rows lie at positions 0.. of `table`."""
    for b, n in enumerate(c.lens):
        m = min(n, budget)
        assert int(new_lens[b]) == m
        for h in range(c.hkv):
            want = R.evict(weights[b, h, :n].tolist(), n, budget, first, recent)
            assert kept[b, h, :m].tolist() == want, f"sequence {b} head {h}"
            assert bool((kept[b, h, m:] == -1).all())
            t, j = torch.tensor(want, dtype=torch.long), torch.arange(m)
            for pool, before in ((c.k, k), (c.v, v)):
                now = pool.cpu()[table[b].long()[j // c.page], h, j % c.page]
                assert torch.equal(now.view(torch.int16), before.cpu()[c.table[b].long()[t // c.page], h, t % c.page].view(torch.int16))
            got = new_weights[b, h].cpu()
            w = weights[b, h][t]
            assert torch.equal(got[:m].nan_to_num(-1.0), w.nan_to_num(-1.0)) and bool((got[m:] == 0).all())


@pytest.mark.parametrize("dtype,d,hkv,page,order,lens,budget,first,recent", [
    ("fp16", 128, 2, 64, "head", [300, 200, 0, 128, 129], 128, 4, 16),
    ("bf16", 64, 1, 16, "token", [1000], 17, 0, 0),
    ("fp16", 64, 3, 32, "token", [65, 64, 40], 64, 32, 32),       # no room for a candidate
    ("bf16", 128, 1, 256, "head", [5000, 2100], 2047, 1, 700),
    ("fp16", 128, 2, 16, "head", [33, 2], 1, 0, 1),
    ("bf16", 64, 2, 64, "head", [700], 500, 0, 0),
])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["spread", "ties"])
def test_evict(dtype, d, hkv, page, order, lens, budget, first, recent, in_place, kind):
    keep_pages = -(-budget // page)
    width = max(max(-(-n // page) for n in lens), keep_pages)
    c = R.Cache(lens, hkv, d, page, dtype, order, seed=budget, spare=len(lens) * keep_pages, width=width)
    p = c.layout(hkv)
    ws = workspace(p)
    g = torch.Generator().manual_seed(5)
    weights = torch.rand(c.B, hkv, width * page, generator=g) ** 8
    if kind == "ties":  # few values, zeros of both signs, infinities, NaN, negative ones
        weights = torch.tensor([0.0, -0.0, 1.0, 2.0, math.inf, -math.inf, math.nan, -1.0, 1e-40])[
            torch.randint(0, 9, weights.shape, generator=g)]
    lens_d, w_d, k, v = c.dev(lens), weights.cuda(), c.k.clone(), c.v.clone()
    table = c.table.cuda()
    if in_place:
        kept, new_lens, new_weights = dkv.dkv_paged_evict(p, c.k, c.v, table, lens_d, w_d, budget, first, recent, table,
                                                          new_lens=lens_d, new_weights=w_d, workspace=ws)
        assert new_lens is lens_d and new_weights is w_d
        to = c.table
    else:
        to = c.free[:c.B * keep_pages].view(c.B, keep_pages)
        kept, new_lens, new_weights = dkv.dkv_paged_evict(p, c.k, c.v, table, lens_d, w_d, budget, first, recent, to.cuda(),
                                                          workspace=ws)
    no_fault(ws)
    _evict_check(c, p, weights, budget, first, recent, kept.cpu(), new_lens.cpu(), new_weights, to, k, v)


@pytest.mark.parametrize("lens,budget,kind", [([40000, 30001, 25], 20000, "spread"), ([33333], 30000, "ties"), ([24577], 3, "ties"),
                                              ([210000], 100000, "spread")])
def test_evict_of_long_sequences(lens, budget, kind):
    """Capacities past what one block of threads holds; the last one past what all of them hold."""
    page = 256
    width = max(-(-n // page) for n in lens)
    c = R.Cache(lens, 1, 64, page, "bf16", seed=budget, width=width)
    p = c.layout(2)
    ws = workspace(p)
    g = torch.Generator().manual_seed(6)
    weights = torch.rand(c.B, 1, width * page, generator=g)
    if kind == "ties":
        weights = torch.tensor([0.0, 1.0, 2.0, math.nan])[torch.randint(0, 4, weights.shape, generator=g)]
    lens_d, w_d, k, v, table = c.dev(lens), weights.cuda(), c.k.clone(), c.v.clone(), c.table.cuda()
    kept, new_lens, new_weights = dkv.dkv_paged_evict(p, c.k, c.v, table, lens_d, w_d, budget, 1, 1, table, new_lens=lens_d,
                                                      new_weights=w_d, workspace=ws)
    no_fault(ws)
    _evict_check(c, p, weights, budget, 1, 1, kept.cpu(), new_lens.cpu(), new_weights, c.table, k, v)


def _evict_mixed(c, stays, budget, first, recent, own_weights):
    """Sequences with stays[b] are compacted in place, the others move to free pages."""
    keep = -(-budget // c.page)
    to = c.free[:c.B * keep].view(c.B, keep).clone()
    for b in range(c.B):
        if stays[b]:
            to[b] = c.table[b, :keep]
    p = c.layout(c.hkv)
    ws = workspace(p)
    weights = torch.rand(c.B, c.hkv, c.width * c.page, generator=torch.Generator().manual_seed(5)) ** 8
    w_d, k, v = weights.cuda(), c.k.cpu(), c.v.cpu()
    kept, new_lens, new_weights = dkv.dkv_paged_evict(p, c.k, c.v, c.table.cuda(), c.dev(c.lens), w_d, budget, first, recent,
                                                      to.cuda(), new_weights=w_d if own_weights else None, workspace=ws)
    no_fault(ws)
    c.k, c.v = c.k.cpu(), c.v.cpu()
    _evict_check(c, p, weights, budget, first, recent, kept.cpu(), new_lens.cpu(), new_weights.cpu(), to, k, v)


@pytest.mark.parametrize("dtype,d,hkv,page,order", [("fp16", 128, 4, 16, "head"), ("bf16", 64, 2, 64, "token")])
@pytest.mark.parametrize("who", [0, 2, 4])
@pytest.mark.parametrize("own_weights", [False, True])
def test_evict_in_place_of_pages_that_others_are_moved_from(dtype, d, hkv, page, order, who, own_weights):
    """Five sequences share their first tokens; one is compacted in place, over rows that the others keep."""
    lens = [6000, 5000, 5500, 1200, 4800]
    keep, shared = -(-2000 // page), 1024 // page
    c = R.Cache(lens, hkv, d, page, dtype, order, seed=7, spare=len(lens) * keep)
    c.table[:, :shared] = c.table[who, :shared].clone()
    _evict_mixed(c, [b == who for b in range(len(lens))], 2000, 4, 64, own_weights)


@pytest.mark.parametrize("own_weights", [False, True])
def test_evict_of_many_sequences_in_place_and_not(own_weights):
    """More sequences than one block of threads puts in order at once."""
    lens = [(i * 29) % 60 for i in range(1300)]
    c = R.Cache(lens, 1, 64, 16, "bf16", seed=8, spare=2 * 1300, width=4)
    _evict_mixed(c, [n > 20 and b % 3 == 0 for b, n in enumerate(lens)], 20, 1, 5, own_weights)


# ---------------------------------------------------------------- together

def test_a_serving_run():
    """Prompts enter in two chunks, their last tokens weigh the cache, it is cut down in place, and tokens
    follow one by one with their weights, through a second eviction: every step against 64 bits."""
    B, hq, hkv, d, page, budget, first, recent = 3, 6, 2, 128, 32, 160, 4, 32
    dt = torch.bfloat16
    lens0, width = [300, 170, 90], 12
    g = torch.Generator().manual_seed(77)
    table = torch.randperm(B * width, generator=g).int().view(B, width).cuda()
    k, v = (torch.full((B * width, hkv, page, d), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    p = dkv.dkv_paged_layout(k, B, hq, width, window=150, sinks=first)
    ws = workspace(p, True)
    weights = torch.zeros(B, hkv, width * page, device="cuda")
    K = [[torch.empty(0, d, dtype=torch.float64) for _ in range(hkv)] for _ in range(B)]
    V = [[torch.empty(0, d, dtype=torch.float64) for _ in range(hkv)] for _ in range(B)]
    W = [[torch.empty(0, dtype=torch.float64) for _ in range(hkv)] for _ in range(B)]
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    u = torch.finfo(dt).eps / 2

    def add(counts):
        n = max(counts)
        kn, vn = (torch.randn(B, n, hkv, d, generator=g).to(dt).transpose(1, 2) for _ in range(2))
        cn = torch.tensor(counts, dtype=torch.int32, device="cuda")
        dkv.dkv_paged_append(p, kn.cuda(), vn.cuda(), k, v, table, lens, counts=cn, workspace=ws)
        lens.add_(cn)
        for b in range(B):
            for h in range(hkv):
                K[b][h] = torch.cat([K[b][h], kn[b, h, :counts[b]].double()])
                V[b][h] = torch.cat([V[b][h], vn[b, h, :counts[b]].double()])
                W[b][h] = torch.cat([W[b][h], torch.zeros(counts[b], dtype=torch.float64)])
        return cn

    def cut():
        kept, _, _ = dkv.dkv_paged_evict(p, k, v, table, lens, weights, budget, first, recent, table, new_lens=lens,
                                         new_weights=weights, workspace=ws)
        kept = kept.cpu()
        for b in range(B):
            for h in range(hkv):
                n = W[b][h].numel()
                m = min(n, budget)
                t = kept[b, h, :m].long()
                # the choice is made by the fp32 weights: against the 64-bit ones it may differ among near equals only
                order = W[b][h].clone()
                order[:first], order[n - recent:] = math.inf, math.inf
                assert float(order[t].min()) >= float(order.sort(descending=True).values[m - 1]) - 1e-3
                assert bool((t[1:] > t[:-1]).all())
                K[b][h], V[b][h], W[b][h] = K[b][h][t], V[b][h][t], W[b][h][t]

    for part in range(2):
        counts = [n // 2 if part == 0 else n - n // 2 for n in lens0]
        cn = add(counts)
        q = (torch.randn(B, hq, max(counts), d, generator=g) * 2).to(dt)
        out, lse = dkv.dkv_paged_prefill(p, q.cuda(), k, v, table, lens, q_lens=cn, workspace=ws)
        if part == 1:
            dkv.dkv_paged_weights(p, q.cuda(), lse, k, table, lens, weights, q_lens=cn, workspace=ws)
        for b in range(B):
            n = K[b][0].shape[0]
            for j in range(hq):
                h = j // 3
                ref = R.attend(q[b, j, :counts[b]].double(), K[b][h], V[b][h], torch.arange(n - counts[b], n), 150, first)
                R.check_rows(out[b, j, :counts[b]], lse[b, j, :counts[b]], ref, d, dt, u, f"chunk {part} {b} {j}")
                if part == 1:
                    W[b][h] += ref[2].sum(0)
    cut()
    for step in range(40):
        add([1] * B)
        q = (torch.randn(B, hq, d, generator=g) * 2).to(dt)
        out, lse = dkv.dkv_paged_decode(p, q.cuda(), k, v, table, lens, weights=weights, workspace=ws)
        for b in range(B):
            n = K[b][0].shape[0]
            for j in range(hq):
                h = j // 3
                ref = R.attend(q[b, j:j + 1].double(), K[b][h], V[b][h], torch.tensor([n - 1]), 150, first)
                R.check_rows(out[b, j:j + 1], lse[b, j:j + 1], ref, d, dt, 2.0 ** -16, f"step {step} {b} {j}")
                W[b][h] += ref[2][0]
        if step == 30:
            cut()
    no_fault(ws)
    assert lens.tolist() == [169, 169, 130] or lens.tolist() == [n.numel() for n in (W[0][0], W[1][0], W[2][0])]
    for b in range(B):
        for h in range(hkv):
            n = W[b][h].numel()
            assert float((weights[b, h, :n].double().cpu() - W[b][h]).abs().max()) < 1e-3
            assert bool((weights[b, h, n:] == 0).all())


def test_calls_in_a_graph_and_on_a_stream_of_their_own():
    c = R.Cache([400, 90], 2, 128, 64, "fp16", seed=9)
    p = c.layout(4, window=128, sinks=4)
    table, lens = c.table.cuda(), c.dev(c.lens)
    ws = workspace(p, True)
    q = queries((2, 4, 128), c.dt, 1).cuda()
    qp = queries((2, 4, 40, 128), c.dt, 2).cuda()
    ql = c.dev([40, 33])
    weights = torch.zeros(2, 2, c.width * 64, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(2, 4, device="cuda")
    po, pl = torch.zeros_like(qp), torch.zeros(2, 4, 40, device="cuda")

    def step():
        dkv.dkv_paged_decode(p, q, c.k, c.v, table, lens, out=out, lse=lse, weights=weights, workspace=ws)
        dkv.dkv_paged_prefill(p, qp, c.k, c.v, table, lens, q_lens=ql, out=po, lse=pl, workspace=ws)
        dkv.dkv_paged_weights(p, qp, pl, c.k, table, lens, weights, q_lens=ql, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    want = [x.clone() for x in (out, lse, po, pl, weights)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x in (out, lse, po, pl, weights):
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip((out, lse, po, pl, weights), want):
        assert torch.equal(x, y)
    # new contents of the same buffers are taken up by the next replay
    lens.copy_(c.dev([399, 1]))
    graph.replay()
    torch.cuda.synchronize()
    fresh, _ = dkv.dkv_paged_decode(p, q, c.k, c.v, table, lens)
    assert torch.equal(out, fresh) and not torch.equal(out, want[0])
    no_fault(ws)


def test_pools_that_interleave_keys_and_values():
    c = R.Cache([333, 64], 2, 64, 32, "bf16", seed=30)
    both = torch.empty(c.n_pages, 2, 2, 32, 64, dtype=c.dt, device="cuda")
    both[:, 0], both[:, 1] = c.k, c.v
    k, v = both[:, 0], both[:, 1]
    p = dkv.dkv_paged_layout(k, 2, 6, c.width)
    q, table, lens = queries((2, 6, 64), c.dt, 1).cuda(), c.table.cuda(), c.dev(c.lens)
    out, lse = dkv.dkv_paged_decode(p, q, k, v, table, lens)
    want, want_lse = dkv.dkv_paged_decode(c.layout(6), q, c.k, c.v, table, lens)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    qp = queries((2, 6, 20, 64), c.dt, 2).cuda()
    out, _ = dkv.dkv_paged_prefill(p, qp, k, v, table, lens)
    want, _ = dkv.dkv_paged_prefill(c.layout(6), qp, c.k, c.v, table, lens)
    assert torch.equal(out, want)
    new = queries((2, 2, 3, 64), c.dt, 3).cuda()
    dkv.dkv_paged_append(p, new, new + 1, k, v, table, c.dev([40, 7]))
    assert torch.equal(k[int(c.table[0, 1]), :, 8:11], new[0]) and torch.equal(v[int(c.table[1, 0]), :, 7:10], new[1] + 1)


def test_runs_are_alike_and_two_streams_do_not_meet():
    """The same bits every time; two calls at once, each with its workspace, give what they give alone."""
    c = R.Cache([3000, 2000, 100], 2, 128, 64, "bf16", seed=31)
    p = c.layout(8, window=1500, sinks=4)
    table, lens = c.table.cuda(), c.dev(c.lens)
    qs = [queries((3, 8, 128), c.dt, s).cuda() for s in (1, 2)]
    qp = [queries((3, 8, 50, 128), c.dt, s).cuda() for s in (3, 4)]

    def run(i, ws):
        w = torch.zeros(3, 2, c.width * 64, device="cuda")
        o, l = dkv.dkv_paged_decode(p, qs[i], c.k, c.v, table, lens, weights=w, workspace=ws)
        po, pl = dkv.dkv_paged_prefill(p, qp[i], c.k, c.v, table, lens, workspace=ws)
        dkv.dkv_paged_weights(p, qp[i], pl, c.k, table, lens, w, workspace=ws)
        return o, l, po, pl, w

    alone = [run(i, workspace(p, True)) for i in range(2)]
    torch.cuda.synchronize()
    streams, spaces = [torch.cuda.Stream() for _ in range(2)], [workspace(p, True) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [None, None]
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i] = run(i, spaces[i])
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_nothing_to_do():
    c = R.Cache([0, 0], 1, 64, 16, seed=32, width=2)
    p = c.layout(2)
    q = queries((2, 2, 64), c.dt, 1).cuda()
    table, lens = c.table.cuda(), c.dev([0, 0])
    weights = torch.ones(2, 1, 32, device="cuda")
    out, lse = dkv.dkv_paged_decode(p, q, c.k, c.v, table, lens, weights=weights)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all()) and bool((weights == 1).all())
    qp = queries((2, 2, 5, 64), c.dt, 1).cuda()
    out, lse = dkv.dkv_paged_prefill(p, qp, c.k, c.v, table, lens)  # five queries before the first token
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    dkv.dkv_paged_weights(p, qp, lse, c.k, table, lens, weights)
    assert bool((weights == 1).all())
    none = qp[:, :, :0]
    out, lse = dkv.dkv_paged_prefill(p, none, c.k, c.v, table, lens)
    assert out.shape == (2, 2, 0, 64) and lse.shape == (2, 2, 0)
    dkv.dkv_paged_append(p, none[:, :1], none[:, :1], c.k, c.v, table, lens)
    kept, new_lens, new_weights = dkv.dkv_paged_evict(p, c.k, c.v, table, lens, weights, 8, 1, 2, table)
    assert bool((kept == -1).all()) and bool((new_lens == 0).all()) and bool((new_weights == 0).all())


def test_tensors_that_do_not_fit_are_refused():
    c = R.Cache([100], 2, 64, 16, seed=33)
    p = c.layout(4)
    table, lens = c.table.cuda(), c.dev([100])
    q = queries((1, 4, 64), c.dt, 1).cuda()
    ok = dict(q=q, k_pages=c.k, v_pages=c.v, page_table=table, lens=lens)
    for change in (dict(q=q.bfloat16()), dict(q=q[:, :3]), dict(q=q.cpu()), dict(lens=lens.long()), dict(lens=lens.cpu()),
                   dict(page_table=table[:, :-1]), dict(k_pages=c.k[:-1]), dict(v_pages=c.v.float()),
                   dict(v_pages=c.v.transpose(1, 2).contiguous().transpose(1, 2)), dict(out=q.float()),
                   dict(lse=torch.zeros(1, 3, device="cuda")), dict(weights=torch.zeros(1, 2, 5, device="cuda")),
                   dict(q=queries((1, 64, 4), c.dt, 1).cuda().transpose(1, 2)),
                   dict(workspace=torch.zeros(1 << 25, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            dkv.dkv_paged_decode(p, **(ok | change))
    wide = queries((1, 1, 64), c.dt, 1).cuda().expand(1, 4, 64)  # one row for four heads: stride 0
    with pytest.raises(dkv.DkvError) as e:
        dkv.dkv_paged_decode(p, **(ok | dict(q=wide)))
    assert e.value.status == dkv.DKV_ERR_ALIGN
    with pytest.raises(dkv.DkvError) as e:
        dkv.dkv_paged_decode(p, **ok, workspace=torch.zeros(512, dtype=torch.uint8, device="cuda"))
    assert e.value.status == dkv.DKV_ERR_WORKSPACE
    with pytest.raises(dkv.DkvError) as e:
        dkv.dkv_paged_evict(p, c.k, c.v, table, lens, torch.zeros(1, 2, c.width * 16, device="cuda"), 10, 6, 5, table)
    assert e.value.status == dkv.DKV_ERR_SHAPE


def test_eviction_to_a_page_that_is_not_there():
    c = R.Cache([100], 1, 64, 16, seed=34, spare=3)
    p = c.layout(1)
    ws = workspace(p)
    to = torch.tensor([[int(c.free[0]), c.n_pages, int(c.free[1])]], dtype=torch.int32, device="cuda")
    w = torch.rand(1, 1, c.width * 16, device="cuda")
    k, v = c.k.clone(), c.v.clone()
    kept, new_lens, _ = dkv.dkv_paged_evict(p, c.k, c.v, c.table.cuda(), c.dev([100]), w, 40, 0, 0, to, workspace=ws)
    assert dkv.dkv_get_error(ws) == (dkv.DKV_ERR_DEVICE, dkv.DKV_DEVERR_INDEX)
    want = R.evict(w[0, 0, :100].tolist(), 100, 40, 0, 0)
    assert kept[0, 0].tolist() == want and int(new_lens[0]) == 40
    for j, t in enumerate(want):
        if not 16 <= j < 32:
            got = c.k[int(to[0, j // 16]), 0, j % 16]
            assert torch.equal(got, k[int(c.table[0, t // 16]), 0, t % 16])
    changed = (c.v.view(torch.int16) != v.view(torch.int16)).any(-1).any(-1).any(-1).nonzero().flatten().tolist()
    assert sorted(changed) == sorted([int(c.free[0]), int(c.free[1])])


def test_pools_past_two_to_the_31_elements():
    """Offsets inside a pool that do not fit 32 bits: a sequence on the first and last pages."""
    page, hkv, d = 256, 8, 128
    n_pages = 2 ** 31 // (page * hkv * d) + 40
    k, v = (torch.empty(n_pages, hkv, page, d, dtype=torch.float16, device="cuda") for _ in range(2))
    lens, B = [700, 300], 2
    table = torch.tensor([[n_pages - 1, 0, n_pages - 7], [n_pages - 3, 5, -1]], dtype=torch.int32, device="cuda")
    p = dkv.dkv_paged_layout(k, B, hkv, 3)
    ws = workspace(p)
    kn, vn = (queries((B, hkv, 700, d), torch.float16, s, 1.0) for s in (1, 2))
    counts = torch.tensor(lens, dtype=torch.int32, device="cuda")
    dkv.dkv_paged_append(p, kn.cuda(), vn.cuda(), k, v, table, torch.zeros_like(counts), counts=counts, workspace=ws)
    q = queries((B, hkv, d), torch.float16, 3)
    out, lse = dkv.dkv_paged_decode(p, q.cuda(), k, v, table, counts, workspace=ws)
    qp = queries((B, hkv, 5, d), torch.float16, 4)
    po, pl = dkv.dkv_paged_prefill(p, qp.cuda(), k, v, table, counts, workspace=ws)
    no_fault(ws)
    for b in range(B):
        for h in range(hkv):
            K, V = kn[b, h, :lens[b]].double(), vn[b, h, :lens[b]].double()
            R.check_rows(out[b, h:h + 1], lse[b, h:h + 1], R.attend(q[b, h:h + 1].double(), K, V, torch.tensor([lens[b] - 1]), 0, 0),
                         d, torch.float16, 2.0 ** -21)
            R.check_rows(po[b, h], pl[b, h], R.attend(qp[b, h].double(), K, V, torch.arange(lens[b] - 5, lens[b]), 0, 0),
                         d, torch.float16, 2.0 ** -11)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_many_small_weights_beside_a_large_one_count(dtype):
    """Token 0 scores 18, every other one 0: weights of e^-18, which a half of its own cannot hold, and
    only they have values in the upper channels."""
    n, d, hkv = 2048, 64, 8
    c = R.Cache([n] * 4, hkv, d, 64, dtype, seed=2)
    K, V = torch.zeros(n, d, dtype=torch.float64), torch.zeros(n, d, dtype=torch.float64)
    K[0, 0] = 18.0
    V[0, :32] = 1.0
    V[1:, 32:] = 1000.0
    t = torch.arange(n)
    for b in range(c.B):
        for pool, rows in ((c.k, K), (c.v, V)):
            pool[c.table[b].long()[t // 64].cuda(), :, (t % 64).cuda()] = rows.to(c.dt).cuda()[:, None]
    q = torch.zeros(c.B, hkv, n, d, dtype=c.dt)
    q[..., 0] = 8.0  # 1 / c
    p, lens = c.layout(hkv), c.dev([n] * 4)
    V = V.to(c.dt).double()
    ref = R.attend(q[0, 0].double(), K, V, t, 0, 0)
    out, lse = dkv.dkv_paged_prefill(p, q.cuda(), c.k, c.v, c.table.cuda(), lens)
    # p as one value of the pools' type: e^-18 is above 2^-26, and 2^7 p in fp16 off by half a subnormal
    # step, 2^-25, at most: relative 2^-25 / 2^-19
    p_eps = 2.0 ** -6 if dtype == "fp16" else torch.finfo(c.dt).eps / 2
    for b, h in ((0, 0), (3, 7), (1, 4)):
        R.check_rows(out[b, h], lse[b, h], ref, d, c.dt, p_eps, f"prefill {b} {h}")
    out, lse = dkv.dkv_paged_decode(p, q[:, :, -1].cuda(), c.k, c.v, c.table.cuda(), lens)
    last = tuple(x[-1:] for x in ref[:2]) + (ref[2],) + (ref[3][-1:],) + (ref[4],)
    p_eps = 2.0 ** -16 if dtype == "bf16" else 2.0 ** -21
    p_eps = max(p_eps, 2.0 ** -13)  # (the low half of 2^14 p > 2^-12 is in steps of 2^-24)
    for b in range(c.B):
        for h in range(hkv):
            R.check_rows(out[b, h][None], lse[b, h][None], last, d, c.dt, p_eps, f"decode {b} {h}")


@pytest.mark.parametrize("handle", [False, True])
def test_what_a_call_allocates_is_in_its_streams_order(handle):
    """The current stream is busy while calls on another one allocate outputs and workspaces."""
    lens, q_lens = [150, 70], [40, 5]
    c = R.Cache(lens, 2, 64, 16, "bf16", seed=6)
    p = c.layout(4)
    q, table, n, nq = queries((2, 4, 40, 64), c.dt, 3).cuda(), c.table.cuda(), c.dev(lens), c.dev(q_lens)
    q1 = q[:, :, 0].contiguous()
    want, wlse = dkv.dkv_paged_prefill(p, q, c.k, c.v, table, n, nq)
    want1, wlse1 = dkv.dkv_paged_decode(p, q1, c.k, c.v, table, n)
    side = torch.cuda.Stream()
    x = torch.randn(8192, 8192, device="cuda", dtype=c.dt)
    torch.cuda.synchronize()
    for _ in range(30):
        y = x @ x  # about 20 ms
    stream = side.cuda_stream if handle else side
    out, lse = dkv.dkv_paged_prefill(p, q, c.k, c.v, table, n, nq, stream=stream)
    out1, lse1 = dkv.dkv_paged_decode(p, q1, c.k, c.v, table, n, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    assert torch.equal(out1, want1) and torch.equal(lse1, wlse1)
    del y


def test_a_prefill_has_ended_before_what_follows_reads_its_rows():
    """The stage calls' attention grid may start before the grid in front of it has ended, if that one allows
    it; it reads its queries at once.  Here they are the rows that a long prefill writes last."""
    w = synth.WORKLOADS["8k"]
    desc = dkv.dkv_layout(1, w.n_q_heads, w.n_kv_heads, w.head_dim, w.n_blocks, w.window, w.rank(0), w.n_residual)
    K, V = (torch.from_numpy(x[:1]).cuda() for x in synth.layer_kv(w, 0))
    packed = dkv.dkv_compress_layout(desc, K, V)
    Tq = 4096
    c = R.Cache([Tq], w.n_kv_heads, w.head_dim, 64, "fp16", seed=40)
    p, table, lens = c.layout(w.n_q_heads), c.table.cuda(), c.dev([Tq])
    q = queries((1, w.n_q_heads, Tq, w.head_dim), c.dt, 41).cuda()
    rows = torch.zeros(Tq, 1, w.n_q_heads, w.head_dim, dtype=c.dt, device="cuda")
    ws, pws = torch.zeros(dkv.dkv_decode_workspace_bytes(desc, w.top_k), dtype=torch.uint8, device="cuda"), workspace(p)

    def run(wait):
        rows.zero_()
        out = torch.full((1, w.n_q_heads, w.head_dim), float("nan"), device="cuda")
        dkv.dkv_decode_route(desc, q[:, :, 0].contiguous(), packed, w.top_k, ws)
        dkv.dkv_paged_prefill(p, q, c.k, c.v, table, lens, out=rows.permute(1, 2, 0, 3), lse=False, workspace=pws)
        if wait:
            torch.cuda.synchronize()
        dkv.dkv_decode_blocks(desc, rows[0], packed, w.top_k, ws)
        dkv.dkv_decode_combine(desc, w.top_k, out, ws)
        torch.cuda.synchronize()
        return out

    want = run(True)
    assert bool(want.isfinite().all())
    for _ in range(5):
        assert torch.equal(run(False), want)
    no_fault(ws)
    no_fault(pws)


@pytest.mark.parametrize("dtype,d,hq,hkv,Tq", [("fp16", 128, 2, 1, 20), ("bf16", 64, 8, 2, 32), ("fp16", 64, 3, 1, 300),
                                               ("bf16", 128, 6, 2, 256)])
def test_a_query_whose_lse_is_minus_infinity_adds_no_weight(dtype, d, hq, hkv, Tq):
    """Whatever its row holds: NaN and infinities, as rows that nothing has written may."""
    n = 700
    c = R.Cache([n], hkv, d, 64, dtype, seed=50)
    p = c.layout(hq)
    ws = workspace(p)
    q = queries((1, hq, Tq, d), c.dt, 51)
    table, lens = c.table.cuda(), c.dev([n])
    _, lse = dkv.dkv_paged_prefill(p, q.cuda(), c.k, c.v, table, lens, workspace=ws)
    out = torch.zeros(hq, Tq, dtype=torch.bool)
    out[:, 3] = out[0, 7:12] = out[-1, Tq - 1] = True
    bad = q.clone()
    bad[0, out] = torch.tensor([float("nan"), float("inf")], dtype=c.dt).repeat(d // 2)
    lse[0, out.cuda()] = float("-inf")
    weights = torch.zeros(1, hkv, c.width * 64, device="cuda")
    dkv.dkv_paged_weights(p, bad.cuda(), lse, c.k, table, lens, weights, workspace=ws)
    no_fault(ws)
    pos = torch.arange(n - Tq, n)
    for h in range(hkv):
        added, big = torch.zeros(n, dtype=torch.float64), 0.0
        for j in range(h * hq // hkv, (h + 1) * hq // hkv):
            ref = R.attend(q[0, j].double(), c.K[0][h], c.V[0][h], pos, 0, 0)
            added += ref[2][~out[j]].sum(0)
            big = max(big, ref[4])
        rows = Tq * hq // hkv  # (as for the weights of all queries)
        tol = (2 * R.score_error(d, big) + 2.0 ** -20 * (1 + math.log(n)) + 2.0 ** -23 * (rows / 8 + 8)) * added
        assert bool(((weights[0, h, :n].double().cpu() - added).abs() <= tol).all())


@pytest.mark.parametrize("dtype,size", [("fp16", 4e4), ("fp16", 1.5e4), ("bf16", 1e7), ("bf16", 2e4)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_of_any_size(dtype, size, sign):
    """Scores past 2^24, where neighbouring fp32 values are further apart than the exponentials reach: the
    key with the largest one has all the weight, and keys with equal ones share it.  One channel of q and k is
    not zero, so that the products are exact; its steps are worth more than 1000 in a score, so that every
    other weight is below e^-1000."""
    d, n, hq = 64, 700, 2
    c = R.Cache([n], 1, d, 64, dtype, seed=60)
    g = torch.Generator().manual_seed(61)
    K = torch.zeros(n, d, dtype=torch.float64)
    K[:, 0] = ((0.5 + 0.5 * torch.rand(n, generator=g)) * size).to(c.dt).double()
    t = torch.arange(n)
    c.k[c.table[0].long()[t // 64].cuda(), 0, (t % 64).cuda()] = K.to(c.dt).cuda()
    q = torch.zeros(1, hq, n, d, dtype=c.dt)
    q[..., 0] = sign * 0.9 * size
    scores = q[0, 0, 0, 0].double() * K[:, 0] / math.sqrt(d)
    table, lens, u = c.table.cuda(), c.dev([n]), torch.finfo(c.dt).eps / 2
    apart = scores.unique().diff()
    assert float(apart.min()) > 1000 and float(scores.abs().min()) * 1.4427 > 2 ** 23
    p = c.layout(hq)
    V = c.V[0][0]

    def check(out, lse, pos, p_eps, what):
        for i, at in enumerate(pos):
            s = scores[:at + 1]
            top = float(s.max())
            best = s == top
            want = V[:at + 1][best].mean(0)
            tol = u * want.abs() + p_eps * (1 + u) * V[:at + 1][best].abs().mean(0)
            assert bool(((out[i].double().cpu() - want).abs() <= tol).all()), f"{what}: row at {at}"
            # the product with log2(e) / sqrt(d), the maximum's part, the logarithm of the count and the way back to base e
            exact = top + math.log(int(best.sum()))
            assert abs(float(lse[i]) - exact) <= 2.0 ** -21 * abs(exact), f"{what}: lse at {at}"

    some = [0, 1, 2, 63, 64, 200, 511, 512, 698, 699]
    out, lse = dkv.dkv_paged_prefill(p, q.cuda(), c.k, c.v, table, lens)
    for j in range(hq):
        check(out[0, j][some], lse[0, j][some], some, u, f"prefill {j}")
    out, lse = dkv.dkv_paged_prefill(p, q[:, :, -5:].cuda(), c.k, c.v, table, lens)  # few queries, keys in parts
    for j in range(hq):
        check(out[0, j], lse[0, j], range(n - 5, n), u, f"few queries {j}")
    for at in some:
        out, lse = dkv.dkv_paged_decode(p, q[:, :, at].contiguous().cuda(), c.k, c.v, table, c.dev([at + 1]))
        for j in range(hq):
            check(out[:, j], lse[:, j], [at], 2.0 ** -16 if dtype == "bf16" else 2.0 ** -21, f"decode {j}")


WIDE = [
    # dtype, d, hq, hkv, page, lens, q_lens, Tq, window, sinks: tables for many times the lengths
    ("bf16", 128, 4, 2, 64, [1024], None, 16, 0, 0),
    ("fp16", 64, 8, 8, 16, [333, 2001, 1, 700], [32, 32, 1, 9], 32, 0, 0),
    ("bf16", 64, 3, 1, 256, [300, 4000], [1, 100], 100, 500, 4),
    ("fp16", 128, 6, 1, 32, [1300, 600, 700], [1300, 600, 500], 1300, 0, 0),
    ("bf16", 64, 2, 1, 64, [700] * 40, None, 300, 256, 3),
    # more units than there is room for: each walks its blocks of keys alone
    ("fp16", 64, 1, 1, 32, [(i * 389) % 1900 for i in range(170)], [(i * 101) % 301 for i in range(170)], 300, 0, 0),
    ("bf16", 128, 3, 1, 16, [2000 - 11 * i for i in range(160)], None, 200, 900, 300),
]


@pytest.mark.parametrize("dtype,d,hq,hkv,page,lens,q_lens,Tq,window,sinks", WIDE)
def test_a_wide_page_table_changes_no_result(dtype, d, hq, hkv, page, lens, q_lens, Tq, window, sinks):
    """A table for 131072 tokens: grids that are reckoned from it find most of their work missing."""
    c = R.Cache(lens, hkv, d, page, dtype, seed=70, width=131072 // page)
    p = c.layout(hq, window, sinks)
    ws = workspace(p)
    n_q = q_lens or [Tq] * c.B
    q = queries((c.B, hq, Tq, d), c.dt, 71)
    ql = None if q_lens is None else c.dev(q_lens)
    table = c.hidden_table([n - m for n, m in zip(lens, n_q)], window, sinks)
    out, lse = dkv.dkv_paged_prefill(p, q.cuda(), c.k, c.v, table, c.dev(lens), q_lens=ql, workspace=ws)
    no_fault(ws)
    weights = torch.zeros(c.B, hkv, c.width * page, device="cuda")
    dkv.dkv_paged_weights(p, q.cuda(), lse, c.k, table, c.dev(lens), weights, q_lens=ql, workspace=ws)
    no_fault(ws)
    for b in range(0, c.B, 7 if c.B > 10 else 1):
        pos = torch.arange(n_q[b]) + lens[b] - n_q[b]
        assert bool((weights[b, :, lens[b]:] == 0).all())
        for h in range(hkv):
            added, big = torch.zeros(lens[b], dtype=torch.float64), 0.0
            for j in range(h * hq // hkv, (h + 1) * hq // hkv):
                ref = R.attend(q[b, j, :n_q[b]].double(), c.K[b][h], c.V[b][h], pos, window, sinks)
                R.check_rows(out[b, j, :n_q[b]], lse[b, j, :n_q[b]], ref, d, c.dt, torch.finfo(c.dt).eps / 2, f"sequence {b} head {j}")
                added += ref[2].sum(0)
                big = max(big, ref[4])
            rows = n_q[b] * hq // hkv
            tol = (2 * R.score_error(d, big) + 2.0 ** -20 * (1 + math.log(max(2, lens[b]))) + 2.0 ** -23 * (rows / 8 + 8)) * added
            assert bool(((weights[b, h, :lens[b]].double().cpu() - added).abs() <= tol + 2.0 ** -40).all()), f"weights of {b} {h}"


def _microseconds(f):
    """The quickest of a dozen calls, each replayed from a graph."""
    f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(4):
            f()
    best = math.inf
    for _ in range(12):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 250)
    return best


def _tight_and_wide(call):
    """Times of call(width of the table in tokens) on a table of the sequences' length and on one for 131072."""
    return _microseconds(call(1024)), _microseconds(call(131072))


def _uniform(B, hkv, d, tokens, G):
    n, page = 1024, 64
    c = R.Cache([n] * B, hkv, d, page, "bf16", seed=72, width=tokens // page)
    return c, c.layout(G * hkv), c.table.cuda(), c.dev(c.lens)


@pytest.mark.parametrize("B,hkv,G,Tq,d", [(16, 2, 4, 1024, 64), (8, 2, 8, 32, 128)])
def test_the_time_of_weights_goes_by_the_lengths(B, hkv, G, Tq, d):
    """Twice the time on a table of 128 times the length would be the table's (it was 10 to 15 times)."""
    def call(tokens):
        c, p, table, lens = _uniform(B, hkv, d, tokens, G)
        ws, q = workspace(p), queries((B, G * hkv, Tq, d), c.dt, 73).cuda()
        lse, weights = torch.full((B, G * hkv, Tq), 8.0, device="cuda"), torch.zeros(B, hkv, tokens, device="cuda")
        return lambda: dkv.dkv_paged_weights(p, q, lse, c.k, table, lens, weights, workspace=ws)

    tight, wide = _tight_and_wide(call)
    assert wide < 2 * tight, f"{wide:.1f} us, {tight:.1f} on the narrow table"


@pytest.mark.parametrize("B,hkv,G,Tq,d", [(1, 1, 8, 16, 128), (8, 1, 8, 8, 64)])
def test_the_time_of_few_queries_goes_by_the_lengths(B, hkv, G, Tq, d):
    """On a table of 128 times the length the grid is one of more parts, which return at once (it took 1.5 to
    2 times the time, while every part left and joined its rows)."""
    def call(tokens):
        c, p, table, lens = _uniform(B, hkv, d, tokens, G)
        ws, q = workspace(p), queries((B, G * hkv, Tq, d), c.dt, 74).cuda()
        out, lse = torch.empty_like(q), torch.empty(B, G * hkv, Tq, device="cuda")
        return lambda: dkv.dkv_paged_prefill(p, q, c.k, c.v, table, lens, out=out, lse=lse, workspace=ws)

    tight, wide = _tight_and_wide(call)
    assert wide < 1.3 * tight, f"{wide:.1f} us, {tight:.1f} on the narrow table"


def test_the_time_of_eviction_goes_by_the_lengths():
    """The selection took a cluster's time for every sequence under a table for more tokens than one block of
    threads holds, however short they were (110 us here, 11 on the narrow table)."""
    B, hkv, n, m, page = 16, 4, 1024, 512, 64

    def call(tokens):
        c = R.Cache([n] * B, hkv, 64, page, "bf16", seed=75, width=tokens // page, spare=B * m // page)
        p, ws, to = c.layout(hkv), None, c.free.view(B, m // page).cuda()
        ws, weights = workspace(p), torch.rand(B, hkv, tokens, device="cuda")
        kept, lens = torch.empty(B, hkv, m, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
        table, n_d, after = c.table.cuda(), c.dev(c.lens), torch.empty_like(weights)
        return lambda: dkv.dkv_paged_evict(p, c.k, c.v, table, n_d, weights, m, 4, 16, to, kept=kept, new_lens=lens,
                                           new_weights=after, workspace=ws)

    tight, wide = _microseconds(call(n)), _microseconds(call(131072))
    zeros = B * hkv * 131072 * 4 / 3e6  # us to write the weights' tails at 3 TB/s
    assert wide < 2 * tight + zeros, f"{wide:.1f} us, {tight:.1f} on the narrow table"


def test_eviction_refuses_numbers_past_32_bits():
    c = R.Cache([100], 1, 64, 16, seed=76)
    p, table = c.layout(1), c.table.cuda()
    w = torch.rand(1, 1, c.width * 16, device="cuda")
    before = c.k.clone()
    for budget, first, recent in (((1 << 32) + 40, 4, 8), (40, 1 << 32, 8), (40, 4, (1 << 32) + 8), (40, 4, -(1 << 32))):
        with pytest.raises(dkv.DkvError) as e:
            dkv.dkv_paged_evict(p, c.k, c.v, table, c.dev([100]), w, budget, first, recent, table)
        assert e.value.status == dkv.DKV_ERR_ARG
    assert torch.equal(c.k.view(torch.int16), before.view(torch.int16))
