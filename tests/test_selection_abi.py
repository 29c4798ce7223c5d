"""The ordered selections reject bad arguments on the host, before any launch (no GPU needed)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def om():
    import ordered_merge_gb300

    return ordered_merge_gb300


def _route(L, vt=0, x=0x10000, t=4, e=64, stride=64, bias=None, score=0, groups=1, picks=1, best=1, k=2, ids=0x90000,
           w=0xA0000):
    return L.om_route_topk(vt, x, t, e, stride, bias, score, groups, picks, best, k, 0, 1.0, ids, w, None)


def test_route_refusals(om):
    L = om.lib()
    for bad in (dict(vt=3), dict(vt=-1), dict(score=2), dict(t=-1), dict(e=0), dict(k=0), dict(k=65), dict(groups=0),
                dict(groups=5), dict(groups=4, picks=5), dict(groups=4, picks=0), dict(best=3), dict(best=0),
                dict(groups=32, picks=1, k=3), dict(x=None), dict(ids=None), dict(w=None), dict(x=0x10002),
                dict(vt=1, x=0x10001), dict(ids=0x90001), dict(bias=0x20002), dict(stride=-1), dict(w=0x90008),
                dict(ids=0x10040), dict(bias=0x90010), dict(w=0x10000 - 16)):
        assert _route(L, **bad) == om.OM_EINVAL, bad
    for bad in (dict(e=1025, stride=1025), dict(k=33), dict(groups=64, picks=64), dict(t=1 << 33), dict(t=1 << 32, stride=1 << 40), dict(stride=1 << 57)):
        assert _route(L, **bad) == om.OM_ERANGE, bad
    assert _route(L, t=0, x=None, ids=None, w=None) == om.OM_OK


def test_route_backward_refusals(om):
    L = om.lib()

    def call(vt=0, x=0x10000, t=4, e=64, stride=64, ids=0x90000, g=0xA0000, score=0, k=2, out=0xB0000):
        return L.om_route_topk_backward(vt, x, t, e, stride, ids, g, score, k, 0, 1.0, out, None)

    for bad in (dict(vt=9), dict(score=-1), dict(t=-2), dict(k=0), dict(k=65), dict(ids=None), dict(g=None),
                dict(out=None), dict(out=0xB0002), dict(out=0x10010), dict(out=0x90000 - 8), dict(out=0xA0004)):
        assert call(**bad) == om.OM_EINVAL, bad
    assert call(e=2000, stride=2000) == om.OM_ERANGE
    assert call(t=0, x=None, ids=None, g=None, out=None) == om.OM_OK


def test_group_refusals(om):
    L = om.lib()

    def call(ids=0x10000, n=100, groups=8, off=0x20000, order=0x30000, place=0x40000):
        return L.om_group_by_id(ids, n, groups, off, order, place, None)

    for bad in (dict(n=-1), dict(groups=0), dict(ids=None), dict(off=None), dict(order=None), dict(place=None),
                dict(ids=0x10001), dict(order=0x30002), dict(order=0x10000), dict(place=0x30010), dict(off=0x10000),
                dict(off=0x30000), dict(off=0x40000 - 4)):
        assert call(**bad) == om.OM_EINVAL, bad
    assert call(n=1 << 31) == om.OM_ERANGE
    assert call(groups=1025) == om.OM_ERANGE


def test_accumulate_refusals(om):
    L = om.lib()

    def call(vt=0, w=0x100000, b=2, hq=4, h=2, q=1, s=64, wb=256, wh=64, wq=64, score=0x10000, sb=128, sh=64,
             lengths=None, out=0x20000, ob=128, oh=64):
        return L.om_accumulate_weights(vt, w, b, hq, h, q, s, wb, wh, wq, score, sb, sh, lengths, 1.0, out, ob, oh, None)

    for bad in (dict(vt=4), dict(b=-1), dict(h=3), dict(h=0), dict(hq=0), dict(q=-1), dict(s=-1), dict(wb=-1), dict(oh=-4),
                dict(w=None), dict(out=None), dict(w=0x100002), dict(score=0x10002), dict(out=0x20001), dict(lengths=0x30002),
                dict(oh=32), dict(ob=64), dict(ob=0), dict(out=0x100000), dict(out=0x10004), dict(out=0x10000, ob=256),
                dict(lengths=0x20010)):
        assert call(**bad) == om.OM_EINVAL, bad
    for bad in (dict(b=40000), dict(q=70000), dict(wb=1 << 41), dict(s=1 << 32)):
        assert call(**bad) == om.OM_ERANGE, bad
    assert call(b=0, w=None, out=None) == om.OM_OK


def test_select_refusals(om):
    L = om.lib()

    def call(score=0x10000, b=2, h=2, s=64, sb=128, sh=64, lengths=None, budget=16, first=2, last=4, keep=0x20000,
             kept=0x30000):
        return L.om_evict_select(score, b, h, s, sb, sh, lengths, budget, first, last, keep, kept, None)

    for bad in (dict(b=-1), dict(h=0), dict(s=-1), dict(sb=-1), dict(budget=0), dict(first=-1), dict(last=-1),
                dict(first=10, last=7), dict(first=17, last=0), dict(score=None), dict(keep=None), dict(kept=None),
                dict(score=0x10002), dict(keep=0x20002), dict(kept=0x20004), dict(keep=0x10000), dict(kept=0x10010),
                dict(lengths=0x20000), dict(lengths=0x30004)):
        assert call(**bad) == om.OM_EINVAL, bad
    for bad in (dict(s=1 << 31), dict(b=1 << 16), dict(sb=1 << 41)):
        assert call(**bad) == om.OM_ERANGE, bad
    assert call(b=0, keep=None, kept=None) == om.OM_OK


def test_gather_refusals(om):
    L = om.lib()

    def call(keep=0x1000, b=1, h=2, budget=8, length=32, count=1, arrays=True, **field):
        one = dict(src=0x10000, dst=0x20000, entry_bytes=64, src_batch=4096, src_head=2048, src_entry=64,
                   dst_batch=1024, dst_head=512, dst_entry=64)
        one.update(field)
        table = (om.CacheArray * 9)(*[om.CacheArray(**one) for _ in range(9)])
        for i in range(1, 9):
            table[i].dst = (one["dst"] or 0) + 0x10000 * i
        return L.om_evict_gather(keep, b, h, budget, length, table if arrays else None, count, None)

    for bad in (dict(b=-1), dict(h=0), dict(budget=0), dict(length=-1), dict(count=0), dict(arrays=False), dict(keep=None),
                dict(keep=0x1002), dict(src=None), dict(dst=None), dict(entry_bytes=0), dict(src_entry=-1),
                dict(dst_entry=32), dict(dst_head=256), dict(dst=0x10000), dict(dst=0x10800), dict(dst=0x1000),
                dict(dst_entry=0)):
        assert call(**bad) == om.OM_EINVAL, bad
    # in place: rows that reach into each other's entries; one array of two; two arrays in one place
    same = dict(dst=0x10000, dst_batch=4096, dst_entry=64)
    assert call(**same, src_head=1024, dst_head=1024) == om.OM_EINVAL
    assert call(**same, dst_head=2048, count=2) == om.OM_EINVAL
    for bad in (dict(count=9), dict(b=1 << 16), dict(src_entry=1 << 31), dict(dst_batch=1 << 41), dict(entry_bytes=1 << 25)):
        assert call(**bad) == om.OM_ERANGE, bad
    assert call(b=0, keep=None) == om.OM_OK


def test_binding_refusals(om):
    """The binding rejects CPU tensors, wrong types, shapes and layouts with ValueError."""
    import torch

    x = torch.zeros(4, 8)
    for call in (lambda: om.route_topk(x, 2), lambda: om.route_topk(x.double(), 2), lambda: om.route_topk(x[0], 2),
                 lambda: om.route_topk(x.t(), 2), lambda: om.route_topk(x, 2, score="relu"),
                 lambda: om.route_topk(x, 2, bias=torch.zeros(7)),
                 lambda: om.route_topk_backward(x, torch.zeros(4, 2), torch.zeros(4, 2)),
                 lambda: om.group_by_id(torch.zeros(4), 8), lambda: om.group_by_id(torch.zeros(4, dtype=torch.int32), 8),
                 lambda: om.accumulate_weights(torch.zeros(1, 2, 3, 4)),
                 lambda: om.accumulate_weights(torch.zeros(1, 2, 3, 4), torch.zeros(1, 1, 5)),
                 lambda: om.evict_select(torch.zeros(1, 2, 3).half(), 2),
                 lambda: om.evict_gather(torch.zeros(1, 2, 3, dtype=torch.int32), ()),
                 lambda: om.evict_gather(torch.zeros(1, 2, 3, dtype=torch.int64), (torch.zeros(1, 2, 9, 4),))):
        with pytest.raises(ValueError) if not torch.cuda.is_available() else pytest.raises((ValueError, RuntimeError)):
            call()
    assert ctypes.sizeof(om.CacheArray) == 72
    with pytest.raises(AttributeError):
        om.no_such_name
