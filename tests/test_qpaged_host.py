"""Host side of the serving-step operators (no GPU): descriptor and argument checks, every one of which returns before a
launch.  The arguments are integers that stand for device addresses."""
import ctypes
import math

import pytest
import torch

from compressed_kv_cache_dkv_gb300 import dkv
from tests import qpaged_ref as Q

A = 1 << 20  # a 16-byte aligned stand-in address
BIG = 1 << 40


def desc(**kw):
    base = dict(batch=2, n_q_heads=12, n_kv_heads=2, head_dim=128, page_size=64, n_pages=40, max_pages=16, dtype=0,
                window=0, sinks=0)
    base.update({k: v for k, v in kw.items() if not k.startswith("stride")})
    page = base["page_size"] * base["head_dim"] * 9 // 8
    return dkv.dkv_qpaged(**base, stride_head=kw.get("stride_head", page), stride_page=kw.get("stride_page", page * base["n_kv_heads"]))


def st(h=128, t=12 * 128, b=12 * 128):
    return dkv.dkv_strides(b, h, t)


BAD = [
    (dict(batch=0), dkv.DKV_ERR_ARG), (dict(n_pages=0), dkv.DKV_ERR_ARG), (dict(max_pages=0), dkv.DKV_ERR_ARG),
    (dict(window=-1), dkv.DKV_ERR_ARG), (dict(sinks=-1), dkv.DKV_ERR_ARG), (dict(dtype=2), dkv.DKV_ERR_ARG),
    (dict(n_q_heads=13), dkv.DKV_ERR_SHAPE), (dict(head_dim=96), dkv.DKV_ERR_UNSUPPORTED),
    (dict(n_q_heads=18), dkv.DKV_ERR_UNSUPPORTED), (dict(page_size=8), dkv.DKV_ERR_UNSUPPORTED),
    (dict(page_size=48), dkv.DKV_ERR_UNSUPPORTED), (dict(page_size=512), dkv.DKV_ERR_UNSUPPORTED),
    (dict(batch=4097), dkv.DKV_ERR_UNSUPPORTED), (dict(max_pages=16385), dkv.DKV_ERR_UNSUPPORTED),
    (dict(batch=4096, n_kv_heads=16, n_q_heads=16), dkv.DKV_ERR_UNSUPPORTED),
    (dict(stride_head=64 * 144 - 16), dkv.DKV_ERR_ALIGN), (dict(stride_head=64 * 144 + 8), dkv.DKV_ERR_ALIGN),
    (dict(stride_page=-(1 << 20)), dkv.DKV_ERR_ALIGN), (dict(stride_page=1 << 38), dkv.DKV_ERR_ALIGN),
]


@pytest.mark.parametrize("change,status", BAD)
def test_descriptor_checks(change, status):
    p, L = desc(**change), dkv.lib()
    assert L.dkv_qpaged_check(p) == status
    assert L.dkv_qpaged_workspace_bytes(p) == 0
    # every call refuses it before anything else
    assert L.dkv_qpaged_append(p, A, A, st(), 1, A, A, A, BIG, None) == status
    assert L.dkv_qpaged_gather(p, A, A, A, None, 1, A, A, st(), A, BIG, None) == status
    assert L.dkv_qpaged_decode(p, A, st(), A, A, A, A, A, A, BIG, None) == status
    assert L.dkv_qpaged_prefill(p, A, st(), 4, 4, A, A, A, A, A, st(), None, A, BIG, None) == status


@pytest.mark.parametrize("change", [dict(), dict(head_dim=64), dict(dtype=1), dict(page_size=16), dict(page_size=256),
                                    dict(n_q_heads=2), dict(n_q_heads=16), dict(window=1 << 30, sinks=1 << 30),
                                    dict(n_pages=1, stride_page=0), dict(n_kv_heads=1, n_q_heads=8, stride_head=0)])
def test_descriptors_that_are_taken(change):
    p = desc(**change)
    assert dkv.lib().dkv_qpaged_check(p) == dkv.DKV_OK
    assert dkv.dkv_qpaged_workspace_bytes(p) > 256
    assert dkv.lib().dkv_qpaged_check(None) == dkv.DKV_ERR_ARG


def refuser(f, args):
    def call(i, x):
        return f(*(args[:i] + [x] + args[i + 1:]))
    return call


def test_append_and_gather_checks():
    p, L = desc(), dkv.lib()
    need = dkv.dkv_qpaged_workspace_bytes(p)
    call = refuser(L.dkv_qpaged_append, [p, A, A, st(), 3, A, A, A, BIG, None])
    for i in (1, 2, 3, 5, 6, 7):
        assert call(i, None) == dkv.DKV_ERR_ARG, i
    for i in (1, 2, 6, 7):
        assert call(i, A + 8) == dkv.DKV_ERR_ALIGN, i
    assert call(5, A + 4) == dkv.DKV_ERR_ALIGN
    assert call(4, -1) == dkv.DKV_ERR_ARG
    assert call(4, 0) == dkv.DKV_OK  # nothing to write, nothing launched
    assert call(8, need - 1) == dkv.DKV_ERR_WORKSPACE
    for bad in (st(t=132), st(h=64)):
        assert call(3, bad) == dkv.DKV_ERR_ALIGN
    call = refuser(L.dkv_qpaged_gather, [p, A, A, A, None, 5, A, A, st(), A, BIG, None])
    for i in (1, 2, 3, 6, 7, 8, 9):
        assert call(i, None) == dkv.DKV_ERR_ARG, i
    for i in (1, 6, 7, 9):
        assert call(i, A + 8) == dkv.DKV_ERR_ALIGN, i
    for i in (2, 3, 4):
        assert call(i, A + 2) == dkv.DKV_ERR_ALIGN, i
    assert call(5, -1) == dkv.DKV_ERR_ARG
    assert call(5, 0) == dkv.DKV_OK
    assert call(5, 16 * 64 + 1) == dkv.DKV_ERR_SHAPE
    assert call(10, need - 1) == dkv.DKV_ERR_WORKSPACE
    assert call(8, st(b=100)) == dkv.DKV_ERR_ALIGN


def test_decode_and_prefill_checks():
    p, L = desc(), dkv.lib()
    need = dkv.dkv_qpaged_workspace_bytes(p)
    call = refuser(L.dkv_qpaged_decode, [p, A, st(), A, A, A, A, None, A, BIG, None])
    for i in (1, 2, 3, 4, 5, 6, 8):
        assert call(i, None) == dkv.DKV_ERR_ARG, i
    for i in (1, 3, 6, 8):
        assert call(i, A + 8) == dkv.DKV_ERR_ALIGN, i
    for i in (4, 5, 7):
        assert call(i, A + 2) == dkv.DKV_ERR_ALIGN, i
    assert call(9, need - 1) == dkv.DKV_ERR_WORKSPACE
    assert call(2, st(h=100)) == dkv.DKV_ERR_ALIGN
    call = refuser(L.dkv_qpaged_prefill, [p, A, st(), 9, 4, A, A, A, A, A, st(), None, A, BIG, None])
    for i in (1, 2, 5, 6, 7, 8, 9, 10, 12):
        assert call(i, None) == dkv.DKV_ERR_ARG, i
    for i in (1, 6, 9, 12):
        assert call(i, A + 8) == dkv.DKV_ERR_ALIGN, i
    for i in (5, 7, 8, 11):
        assert call(i, A + 2) == dkv.DKV_ERR_ALIGN, i
    assert call(3, -1) == call(4, -1) == dkv.DKV_ERR_ARG
    assert call(3, 0) == call(4, 0) == dkv.DKV_OK
    assert call(3, (1 << 30) + 1) == dkv.DKV_ERR_UNSUPPORTED
    assert call(13, need - 1) == dkv.DKV_ERR_WORKSPACE
    assert call(2, st(t=100)) == call(10, st(h=64)) == dkv.DKV_ERR_ALIGN


def test_plan_checks():
    call = refuser(dkv.lib().dkv_paged_plan, [4, 16, 100, 8, A, A, A, 50, A, A, 64, A, A, A, A, A, A, A, BIG, None])
    for i in (0, 1, 2, 3):
        assert call(i, 0) == dkv.DKV_ERR_ARG, i
    assert call(7, -1) == call(10, -1) == dkv.DKV_ERR_ARG
    for i in (4, 5, 6, 8, 9, 11, 12, 13, 14, 15, 16, 17):
        assert call(i, None) == dkv.DKV_ERR_ARG, i
        assert call(i, A + 2) == dkv.DKV_ERR_ALIGN, i
    assert call(11, A + 4) == call(17, A + 8) == dkv.DKV_ERR_ALIGN
    assert call(0, 4097) == call(1, 8) == call(1, 24) == call(1, 512) == call(3, 65537) == call(10, (1 << 30) + 1) == dkv.DKV_ERR_UNSUPPORTED
    assert call(18, dkv.lib().dkv_paged_plan_workspace_bytes(4) - 1) == dkv.DKV_ERR_WORKSPACE
    assert dkv.lib().dkv_paged_plan_workspace_bytes(0) == dkv.lib().dkv_paged_plan_workspace_bytes(4097) == 0


def test_rotation_checks():
    L = dkv.lib()

    def rot(**kw):
        base = dict(rows=5, n_q_heads=4, n_kv_heads=2, head_dim=128, dtype=1, norm=1, rope_dims=64, eps=1e-6, rope_base=1e4)
        return dkv.dkv_rotate(**(base | kw))

    pool = dkv.dkv_paged(1, 4, 2, 128, 16, 4, 4, 1, 0, 0, 4096, 2048, 128)
    args = [rot(), A, st(), A, st(), A, A, A, A, st(), A, st(), pool, A, st(), A, A, A, A, 256, None]
    call = refuser(L.dkv_qk_norm_rope, args)
    for i in (1, 2, 3, 4, 7, 8, 9, 11, 12, 13, 14, 15, 16, 17):
        assert call(i, None) == dkv.DKV_ERR_ARG, i
    for i in (1, 3, 5, 6, 8, 10, 13, 16, 17, 18):
        assert call(i, A + 8) == dkv.DKV_ERR_ALIGN, i
    assert call(7, A + 2) == call(15, A + 4) == dkv.DKV_ERR_ALIGN
    for i in (2, 4, 9, 11, 14):
        assert call(i, st(t=100)) == dkv.DKV_ERR_ALIGN, i
    assert call(19, 255) == dkv.DKV_ERR_WORKSPACE
    plain = refuser(L.dkv_qk_norm_rope, args[:12] + [None] * 7 + [0, None])
    assert plain(10, None) == dkv.DKV_ERR_ARG  # keys that go nowhere
    assert call(0, None) == dkv.DKV_ERR_ARG
    for kw in (dict(rows=-1), dict(n_q_heads=0), dict(n_kv_heads=0), dict(dtype=2), dict(rope_dims=-16), dict(rope_dims=144),
               dict(eps=-1.0), dict(eps=math.nan), dict(rope_base=1.0), dict(rope_base=math.inf)):
        assert plain(0, rot(**kw)) == dkv.DKV_ERR_ARG, kw
    for kw in (dict(head_dim=96), dict(rope_dims=24)):
        assert plain(0, rot(**kw)) == dkv.DKV_ERR_UNSUPPORTED, kw
    bad = rot()
    bad.inv_freq = (ctypes.c_double * 32)(*([1.0] * 31 + [math.inf]))
    assert plain(0, bad) == dkv.DKV_ERR_ARG
    assert plain(0, rot(rows=0)) == dkv.DKV_OK
    for kw in (dict(n_kv_heads=4), dict(head_dim=64), dict(dtype=0)):
        assert call(0, rot(**kw)) == dkv.DKV_ERR_SHAPE, kw


def test_layout_from_a_pool():
    pool = torch.zeros(10, 2, 32 * 144, dtype=torch.uint8)
    p = dkv.dkv_qpaged_layout(pool, 3, 8, 128, 7, dtype=torch.bfloat16, window=5, sinks=1)
    assert (p.page_size, p.n_pages, p.n_kv_heads, p.dtype, p.stride_page, p.stride_head) == (32, 10, 2, 1, 2 * 32 * 144, 32 * 144)
    for args in ((pool[0], 3, 8, 128, 7), (pool.float(), 3, 8, 128, 7), (pool[..., ::2], 3, 8, 128, 7)):
        with pytest.raises(dkv.DkvError):
            dkv.dkv_qpaged_layout(*args)
    for d, dt, width, status in ((96, torch.float16, 7, dkv.DKV_ERR_UNSUPPORTED), (128, torch.float32, 7, dkv.DKV_ERR_ARG),
                                 (128, torch.float16, 1 << 33, dkv.DKV_ERR_ARG), (128, torch.float16, 0, dkv.DKV_ERR_ARG)):
        with pytest.raises(dkv.DkvError) as e:
            dkv.dkv_qpaged_layout(pool, 3, 8, d, width, dtype=dt)
        assert e.value.status == status
    with pytest.raises(dkv.DkvError):
        dkv.dkv_qpaged_layout(torch.zeros(10, 2, 1000, dtype=torch.uint8), 3, 8, 128, 7)


def test_host_tensors_are_refused():
    pool = torch.zeros(4, 1, 16 * 72, dtype=torch.uint8)
    p = dkv.dkv_qpaged_layout(pool, 1, 1, 64, 4)
    row, slot, one = torch.zeros(1, 1, 64, dtype=torch.float16), torch.zeros(1, dtype=torch.int64), torch.zeros(1, dtype=torch.int32)
    table = torch.zeros(1, 4, dtype=torch.int32)
    for call in (lambda: dkv.dkv_qpaged_append(p, row, row, pool, slot), lambda: dkv.dkv_qpaged_decode(p, row, pool, table, one),
                 lambda: dkv.dkv_qpaged_prefill(p, row, torch.zeros(2, dtype=torch.int32), 1, pool, table, one),
                 lambda: dkv.dkv_qpaged_gather(p, pool, table, one, row[None], row[None]), lambda: dkv.dkv_qk_norm_rope(row, row, one, 64),
                 lambda: dkv.dkv_paged_plan(p, one, one, one, one, table, 4)):
        with pytest.raises(ValueError):
            call()


def test_reference_grid_is_exact():
    """The quantiser's claims on the definition itself: fp16 numbers, within half a step and a spacing."""
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(2000, 128, generator=g) * torch.exp(5 * torch.randn(2000, 1, generator=g)) + torch.randn(2000, 1, generator=g)).bfloat16().double()
    x[:10] = 0.0
    x[10:20] = 61440.0
    c, s, b = Q.quantise(x)
    v = Q.values(c, s, b)
    assert torch.equal(v.half().double(), v)
    y = x.clamp(-61440, 61440).view(2000, 2, 64)
    span = y.amax(-1) - y.amin(-1)
    u = 2.0 ** torch.clamp(torch.floor(torch.log2(y.abs().amax(-1).clamp(min=1e-30) * 65 / 64)) - 10, min=-24)
    assert bool(((v.view(2000, 2, 64) - y).abs().amax(-1) <= span / 30 + u).all())
