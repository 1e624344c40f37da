"""Host side of the paged-cache operators (no GPU): descriptor and argument checks, every one of which
returns before a launch.  The arguments are integers that stand for device addresses."""
import ctypes

import pytest

from compressed_kv_cache_dkv_gb300 import dkv

A = 1 << 20  # a 16-byte aligned stand-in address
BIG = 1 << 40


def desc(**kw):
    base = dict(batch=2, n_q_heads=12, n_kv_heads=2, head_dim=128, page_size=64, n_pages=40, max_pages=16, dtype=0,
                window=0, sinks=0)
    base.update({k: v for k, v in kw.items() if not k.startswith("stride")})
    p = dkv.dkv_paged(**base)
    p.stride_token = kw.get("stride_token", base["head_dim"])
    p.stride_head = kw.get("stride_head", base["head_dim"] * base["page_size"])
    p.stride_page = kw.get("stride_page", base["head_dim"] * base["page_size"] * base["n_kv_heads"])
    return p


def st(b=12 * 128, h=128, t=128):
    return dkv.dkv_strides(b, h, t)


BAD = [
    (dict(batch=0), dkv.DKV_ERR_ARG), (dict(n_pages=0), dkv.DKV_ERR_ARG), (dict(max_pages=0), dkv.DKV_ERR_ARG),
    (dict(window=-1), dkv.DKV_ERR_ARG), (dict(sinks=-1), dkv.DKV_ERR_ARG), (dict(dtype=2), dkv.DKV_ERR_ARG),
    (dict(n_q_heads=13), dkv.DKV_ERR_SHAPE), (dict(head_dim=96), dkv.DKV_ERR_UNSUPPORTED),
    (dict(n_q_heads=18), dkv.DKV_ERR_UNSUPPORTED), (dict(page_size=8), dkv.DKV_ERR_UNSUPPORTED),
    (dict(page_size=48), dkv.DKV_ERR_UNSUPPORTED), (dict(page_size=512), dkv.DKV_ERR_UNSUPPORTED),
    (dict(batch=4097), dkv.DKV_ERR_UNSUPPORTED), (dict(max_pages=16385), dkv.DKV_ERR_UNSUPPORTED),
    (dict(batch=4096, n_kv_heads=16, n_q_heads=16), dkv.DKV_ERR_UNSUPPORTED),
    (dict(stride_token=130), dkv.DKV_ERR_ALIGN), (dict(stride_token=64), dkv.DKV_ERR_ALIGN),
    (dict(stride_head=0), dkv.DKV_ERR_ALIGN), (dict(stride_page=-128), dkv.DKV_ERR_ALIGN),
    (dict(stride_page=1 << 38), dkv.DKV_ERR_ALIGN),
]


@pytest.mark.parametrize("change,status", BAD)
def test_descriptor_checks(change, status):
    p = desc(**change)
    L = dkv.lib()
    assert L.dkv_paged_check(p) == status
    assert L.dkv_paged_workspace_bytes(p, 0) == 0
    # every call refuses it before anything else
    assert L.dkv_paged_append(p, A, A, st(), 1, A, None, A, A, A, A, BIG, None) == status
    assert L.dkv_paged_decode(p, A, st(), A, A, A, A, A, A, None, A, BIG, None) == status
    assert L.dkv_paged_prefill(p, A, st(), 4, A, A, A, A, None, A, st(), None, A, BIG, None) == status
    assert L.dkv_paged_weights(p, A, st(), 4, A, A, A, A, None, A, A, BIG, None) == status
    assert L.dkv_paged_evict(p, A, A, A, A, A, 100, 4, 10, A, 2, A, A, A, A, BIG, None) == status


@pytest.mark.parametrize("change", [dict(), dict(head_dim=64), dict(dtype=1), dict(page_size=16), dict(page_size=256),
                                    dict(n_q_heads=2), dict(n_q_heads=16), dict(window=1 << 30, sinks=1 << 30),
                                    dict(n_pages=1, stride_page=0), dict(n_kv_heads=1, n_q_heads=8, stride_head=0)])
def test_descriptors_that_are_taken(change):
    p = desc(**change)
    assert dkv.lib().dkv_paged_check(p) == dkv.DKV_OK
    small, large = dkv.dkv_paged_workspace_bytes(p), dkv.dkv_paged_workspace_bytes(p, True)
    assert 256 < small < large
    assert dkv.lib().dkv_paged_check(None) == dkv.DKV_ERR_ARG


def test_append_checks():
    p, f = desc(), dkv.lib().dkv_paged_append
    args = [p, A, A, st(), 3, A, None, A, A, A, A, BIG, None]

    def call(i, x):
        return f(*(args[:i] + [x] + args[i + 1:]))

    for i in (1, 2, 3, 5, 7, 8, 9, 10):
        assert call(i, None) == dkv.DKV_ERR_ARG, i
    for i in (1, 2, 7, 8, 10):
        assert call(i, A + 8) == dkv.DKV_ERR_ALIGN, i
    assert call(5, A + 2) == call(6, A + 2) == call(9, A + 1) == dkv.DKV_ERR_ALIGN
    assert call(4, -1) == dkv.DKV_ERR_ARG
    assert call(4, 0) == dkv.DKV_OK  # nothing to write, nothing launched
    assert call(4, 16 * 64 + 1) == dkv.DKV_ERR_SHAPE
    assert call(11, 255) == dkv.DKV_ERR_WORKSPACE
    for bad in (st(t=132), st(h=64), st(b=0)):
        assert call(3, bad) == dkv.DKV_ERR_ALIGN


def test_decode_checks():
    p, f = desc(), dkv.lib().dkv_paged_decode
    args = [p, A, st(), A, A, A, A, A, A, None, A, BIG, None]

    def call(i, x, **more):
        a = args[:i] + [x] + args[i + 1:]
        for k, v in more.items():
            a[int(k[1:])] = v
        return f(*a)

    for i in (1, 2, 3, 4, 5, 6, 7, 10):
        assert call(i, None) == dkv.DKV_ERR_ARG, i
    assert call(8, None, _9=A) == dkv.DKV_ERR_ARG  # weights need the lse
    for i in (1, 3, 4, 7, 10):
        assert call(i, A + 8) == dkv.DKV_ERR_ALIGN, i
    for i in (5, 6, 8, 9):
        assert call(i, A + 2) == dkv.DKV_ERR_ALIGN, i
    assert call(11, dkv.dkv_paged_workspace_bytes(p) - 1) == dkv.DKV_ERR_WORKSPACE
    assert call(11, dkv.dkv_paged_workspace_bytes(p, True) - 1, _9=A) == dkv.DKV_ERR_WORKSPACE
    assert call(2, st(h=100)) == dkv.DKV_ERR_ALIGN


def test_prefill_and_weights_checks():
    p, L = desc(), dkv.lib()
    pre = [p, A, st(), 7, A, A, A, A, None, A, st(), None, A, BIG, None]
    wts = [p, A, st(), 7, A, A, A, A, None, A, A, BIG, None]

    def call(f, args, i, x):
        return f(*(args[:i] + [x] + args[i + 1:]))

    for i in (1, 2, 4, 5, 6, 7, 9, 10, 12):
        assert call(L.dkv_paged_prefill, pre, i, None) == dkv.DKV_ERR_ARG, i
    for i in (1, 4, 5, 9, 12):
        assert call(L.dkv_paged_prefill, pre, i, A + 8) == dkv.DKV_ERR_ALIGN, i
    for i in (6, 7, 8, 11):
        assert call(L.dkv_paged_prefill, pre, i, A + 2) == dkv.DKV_ERR_ALIGN, i
    for i in (1, 2, 4, 5, 6, 7, 9, 10):
        assert call(L.dkv_paged_weights, wts, i, None) == dkv.DKV_ERR_ARG, i
    for i in (1, 5, 10):
        assert call(L.dkv_paged_weights, wts, i, A + 8) == dkv.DKV_ERR_ALIGN, i
    for i in (4, 6, 7, 8, 9):
        assert call(L.dkv_paged_weights, wts, i, A + 2) == dkv.DKV_ERR_ALIGN, i
    for f, args in ((L.dkv_paged_prefill, pre), (L.dkv_paged_weights, wts)):
        assert call(f, args, 3, -1) == dkv.DKV_ERR_ARG
        assert call(f, args, 3, 0) == dkv.DKV_OK
        assert call(f, args, 3, (1 << 20) + 1) == dkv.DKV_ERR_UNSUPPORTED
        assert call(f, args, 2, st(t=100)) == dkv.DKV_ERR_ALIGN
        assert call(f, args, len(args) - 2, 255) == dkv.DKV_ERR_WORKSPACE
    assert call(L.dkv_paged_prefill, pre, 10, st(t=100)) == dkv.DKV_ERR_ALIGN


def test_evict_checks():
    p, f = desc(), dkv.lib().dkv_paged_evict
    #       0  1  2  3  4  5  6    7  8   9  10 11 12 13 14 15   16
    args = [p, A, A, A, A, A, 100, 4, 10, A, 2, A, A, A, A, BIG, None]

    def call(**kw):
        a = list(args)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)

    for i in (1, 2, 3, 4, 5, 9, 11, 12, 13, 14):
        assert call(**{f"_{i}": None}) == dkv.DKV_ERR_ARG, i
    for i in (1, 2, 14):
        assert call(**{f"_{i}": A + 8}) == dkv.DKV_ERR_ALIGN, i
    for i in (3, 4, 5, 9, 11, 12, 13):
        assert call(**{f"_{i}": A + 2}) == dkv.DKV_ERR_ALIGN, i
    assert call(_6=0) == call(_7=-1) == call(_8=-1) == call(_10=0) == dkv.DKV_ERR_ARG
    assert call(_7=60, _8=41) == dkv.DKV_ERR_SHAPE                  # first + recent > budget
    assert call(_6=129) == dkv.DKV_ERR_SHAPE                        # two pages hold 128
    assert call(_6=16 * 64 + 1, _10=100) == dkv.DKV_ERR_SHAPE       # over the capacity
    assert call(_7=(1 << 31) - 1, _8=(1 << 31) - 1) == dkv.DKV_ERR_SHAPE
    assert call(_15=300 - 256) == dkv.DKV_ERR_WORKSPACE


def test_status_reaches_python():
    with pytest.raises(dkv.DkvError) as e:
        import torch
        dkv.dkv_paged_layout(torch.zeros(3, 2, 24, 64, dtype=torch.float16), 1, 4, 2)
    assert e.value.status == dkv.DKV_ERR_UNSUPPORTED
    for bad in (torch.zeros(3, 2, 16, 64), torch.zeros(3, 2, 64, dtype=torch.float16),
                torch.zeros(3, 2, 64, 16, dtype=torch.float16).transpose(2, 3)):
        with pytest.raises(dkv.DkvError) as e:
            dkv.dkv_paged_layout(bad, 1, 4, 2)
        assert e.value.status == dkv.DKV_ERR_ARG
    assert ctypes.sizeof(dkv.dkv_paged) == 64 and ctypes.sizeof(dkv.dkv_strides) == 24


def test_numbers_past_32_bits_are_refused_in_python():
    """They would arrive as others: 2^32 + 16 as 16."""
    import torch
    pool = torch.zeros(3, 2, 16, 64, dtype=torch.float16)
    dkv.dkv_paged_layout(pool, 1, 4, 2, window=(1 << 31) - 1, sinks=(1 << 31) - 1)
    for more in (dict(window=1 << 32), dict(window=(1 << 32) + 16), dict(sinks=1 << 32), dict(window=1 << 31), dict(sinks=-(1 << 32)),
                 dict(batch=(1 << 32) + 1), dict(n_q_heads=(1 << 32) + 4), dict(max_pages=(1 << 32) + 2)):
        with pytest.raises(dkv.DkvError) as e:
            dkv.dkv_paged_layout(pool, **(dict(batch=1, n_q_heads=4, max_pages=2) | more))
        assert e.value.status == dkv.DKV_ERR_ARG, more
