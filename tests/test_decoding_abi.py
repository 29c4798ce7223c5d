"""Beam search, embedding rows and routed experts reject bad arguments on the host, before any launch (no GPU needed)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def om():
    import ordered_merge_gb300

    return ordered_merge_gb300


def test_beam_select_refusals(om):
    L = om.lib()

    def call(vt=0, x=0x100000, b=2, n=3, v=100, bs=300, ns=100, scores=0x10000, fin=0x20000, end=5, top=4, out=0x30000,
             par=0x40000, tok=0x50000):
        return L.om_beam_select(vt, x, b, n, v, bs, ns, scores, fin, end, top, out, par, tok, None)

    for bad in (dict(vt=3), dict(vt=-1), dict(b=-1), dict(n=0), dict(v=0), dict(top=0), dict(bs=-1), dict(ns=-1),
                dict(end=-1), dict(end=100), dict(x=None), dict(out=None), dict(par=None), dict(tok=None), dict(x=0x100002),
                dict(vt=1, x=0x100001), dict(scores=0x10002), dict(out=0x30002), dict(par=0x40001), dict(tok=0x50003),
                dict(out=0x100000), dict(tok=0x100000 + 2396), dict(par=0x30000), dict(tok=0x40000 + 28), dict(out=0x10000),
                dict(par=0x20004), dict(out=0x100000 - 28)):
        assert call(**bad) == om.OM_EINVAL, bad
    for bad in (dict(n=65), dict(top=65), dict(v=(1 << 30) + 1), dict(b=(1 << 24) + 1), dict(bs=1 << 41), dict(ns=1 << 41),
                dict(b=1 << 24, bs=1 << 40)):
        assert call(**bad) == om.OM_ERANGE, bad
    assert call(b=0, x=None, out=None) == om.OM_OK


def test_beam_gather_refusals(om):
    L = om.lib()

    def call(parents=0x1000, b=2, n=4, h=2, s=8, starts=0x2000, lengths=0x3000, count=1, arrays=True, step=0x100000, **field):
        one = dict(src=0x100000, dst=0x10000000, entry_bytes=64, src_batch=4096, src_beam=1024, src_head=512, src_entry=64,
                   dst_batch=4096, dst_beam=1024, dst_head=512, dst_entry=64)
        one.update(field)
        table = (om.BeamArray * 65)(*[om.BeamArray(**one) for _ in range(65)])
        for i in range(1, 65):
            table[i].dst = (one["dst"] or 0) + step * i
            if one["src"] == one["dst"]:
                table[i].src = table[i].dst
        return L.om_beam_gather(parents, b, n, h, s, starts, lengths, table if arrays else None, count, None)

    for bad in (dict(b=-1), dict(n=0), dict(h=0), dict(s=-1), dict(count=0), dict(arrays=False), dict(parents=None),
                dict(parents=0x1002), dict(starts=0x2001), dict(lengths=0x3002), dict(src=None), dict(dst=None),
                dict(entry_bytes=0), dict(src_head=-1), dict(dst_entry=-64), dict(dst_entry=32), dict(dst_beam=256),
                dict(dst_entry=0), dict(dst=0x100040), dict(dst=0x100000, dst_entry=128), dict(dst=0x1000), dict(dst=0x2000 - 64),
                dict(dst=0x3004), dict(count=2, step=64)):
        assert call(**bad) == om.OM_EINVAL, bad
    same = dict(dst=0x100000)
    assert call(**same, dst_beam=2048, count=1) == om.OM_EINVAL  # same place, other strides
    assert call(**same, count=2, step=512) == om.OM_EINVAL       # two arrays of which one reaches into the other
    for bad in (dict(n=65), dict(count=65), dict(h=65536), dict(b=32768), dict(s=1 << 31), dict(entry_bytes=(1 << 30) + 16),
                dict(src_entry=1 << 31), dict(dst_batch=1 << 41)):
        assert call(**bad) == om.OM_ERANGE, bad
    assert call(b=0, parents=None) == om.OM_OK
    assert call(s=0, parents=None) == om.OM_OK


def test_embed_lookup_refusals(om):
    L = om.lib()

    def call(vt=1, table=0x100000, rows=100, w=64, ts=64, ids=0x10000, ib=8, n=10, out=0x20000, os=64):
        return L.om_embed_lookup(vt, table, rows, w, ts, ids, ib, n, 1.0, out, os, None)

    for bad in (dict(vt=5), dict(rows=-1), dict(w=0), dict(ts=-1), dict(os=-1), dict(n=-1), dict(ib=2), dict(ib=0),
                dict(table=None), dict(ids=None), dict(out=None), dict(table=0x100001), dict(ids=0x10004), dict(ib=4, ids=0x10002),
                dict(out=0x20001), dict(os=63), dict(out=0x100000), dict(out=0x10000), dict(out=0x100000 - 1278)):
        assert call(**bad) == om.OM_EINVAL, bad
    for bad in (dict(rows=(1 << 31) - 1), dict(n=1 << 31), dict(w=(1 << 24) + 1, ts=1 << 25, os=1 << 25), dict(ts=1 << 41),
                dict(os=1 << 41), dict(rows=1 << 30, ts=1 << 40), dict(n=1 << 30, os=1 << 40)):
        assert call(**bad) == om.OM_ERANGE, bad
    assert call(n=0, table=None, ids=None, out=None) == om.OM_OK


def test_embed_backward_refusals(om):
    L = om.lib()

    def call(vt=1, grad=0x100000, n=10, w=64, gs=64, ids=0x10000, ib=8, rows=100, acc=0, tt=1, table=0x200000, ts=64):
        return L.om_embed_lookup_backward(vt, grad, n, w, gs, ids, ib, rows, 1.0, acc, tt, table, ts, None)

    for bad in (dict(vt=3), dict(tt=2), dict(tt=4), dict(vt=0, tt=1), dict(n=-1), dict(w=0), dict(gs=-1), dict(ts=-1), dict(rows=-1),
                dict(ib=3), dict(grad=None), dict(ids=None), dict(table=None), dict(grad=0x100001), dict(table=0x200001),
                dict(tt=0, table=0x200002), dict(ids=0x10004), dict(ts=32), dict(table=0x100000), dict(table=0x10000 - 12800 + 2),
                dict(table=0x10040)):
        assert call(**bad) == om.OM_EINVAL, bad
    for bad in (dict(rows=(1 << 31) - 1), dict(n=(1 << 30) + 1), dict(w=(1 << 20) + 1, gs=1 << 21, ts=1 << 21), dict(gs=1 << 41),
                dict(ts=1 << 41), dict(n=1 << 30, gs=1 << 40), dict(rows=1 << 30, ts=1 << 40), dict(n=1 << 22, w=1 << 20, gs=1 << 20, ts=1 << 20, grad=0x10000000000000, ids=0x20000000000000)):
        assert call(**bad) == om.OM_ERANGE, bad
    assert call(rows=0, table=None) == om.OM_OK


def test_expert_mlp_refusals(om):
    L = om.lib()

    def call(vt=1, x=0x100000, t=4, h=64, xs=64, ids=0x10000, w=0x20000, k=2, e=8, i=32, up=0x200000, ue=2048, ur=64,
             gate=0x300000, ge=2048, gr=64, down=0x400000, de=2048, dr=32, act=0, out=0x30000, os=64):
        return L.om_expert_mlp(vt, x, t, h, xs, ids, w, k, e, i, up, ue, ur, gate, ge, gr, down, de, dr, act, out, os, None)

    for bad in (dict(vt=0), dict(vt=3), dict(t=-1), dict(h=0), dict(k=0), dict(e=0), dict(i=0), dict(act=3), dict(act=-1),
                dict(xs=-1), dict(ue=-1), dict(gr=-1), dict(dr=-2), dict(os=-1), dict(x=None), dict(ids=None), dict(w=None),
                dict(up=None), dict(down=None), dict(out=None), dict(x=0x100001), dict(ids=0x10002), dict(w=0x20001),
                dict(up=0x200001), dict(gate=0x300001), dict(down=0x400001), dict(out=0x30001), dict(os=63), dict(out=0x100000),
                dict(out=0x10000), dict(out=0x20010), dict(out=0x200000 + 32000), dict(out=0x300000), dict(out=0x400000)):
        assert call(**bad) == om.OM_EINVAL, bad
    for bad in (dict(t=65), dict(k=33), dict(e=1025), dict(h=(1 << 20) + 1), dict(i=(1 << 20) + 1), dict(xs=1 << 41), dict(de=1 << 41)):
        assert call(**bad) == om.OM_ERANGE, bad
    assert call(t=0, x=None, out=None) == om.OM_OK


def test_binding_refusals(om):
    """The binding rejects CPU tensors, wrong types, shapes and layouts with ValueError."""
    import torch

    x, i32 = torch.zeros(2, 3, 8), torch.zeros(2, 3, dtype=torch.int32)
    state, table, ids = torch.zeros(2, 3, 1, 4, 8), torch.zeros(9, 8), torch.zeros(4, dtype=torch.int64)
    h, up, down = torch.zeros(4, 16).bfloat16(), torch.zeros(5, 8, 16).bfloat16(), torch.zeros(5, 16, 8).bfloat16()
    eid, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for call in (lambda: om.beam_select(x, 2), lambda: om.beam_select(x[0], 2), lambda: om.beam_select(x.transpose(1, 2), 2),
                 lambda: om.beam_select(x, 2, torch.zeros(2, 4)), lambda: om.beam_select(x, 2, torch.zeros(2, 3).double()),
                 lambda: om.beam_select(x, 2, finished=i32), lambda: om.beam_select(x.double(), 2),
                 lambda: om.beam_gather(i32, (state,)), lambda: om.beam_gather(i32, ()), lambda: om.beam_gather(i32.long(), (state,)),
                 lambda: om.beam_gather(i32, (state,), out=()), lambda: om.beam_gather(i32, (state,), lengths=torch.zeros(3, dtype=torch.int32)),
                 lambda: om.beam_gather(i32, (state,), starts=torch.zeros(2)), lambda: om.beam_gather(i32[0], (state,)),
                 lambda: om.embed_lookup(ids, table), lambda: om.embed_lookup(ids.float(), table),
                 lambda: om.embed_lookup(ids, table, out=torch.zeros(4, 9)), lambda: om.embed_lookup(ids, table.t()),
                 lambda: om.embed_lookup(ids, table.requires_grad_(), out=torch.zeros(4, 8)),
                 lambda: om.embed_lookup_backward(torch.zeros(4, 8), ids, 9), lambda: om.embed_lookup_backward(torch.zeros(3, 8), ids, 9),
                 lambda: om.embed_lookup_backward(torch.zeros(4, 8), ids, 9, accumulate=True),
                 lambda: om.embed_lookup_backward(torch.zeros(4, 8), ids, 9, grad_table=torch.zeros(9, 8).half()),
                 lambda: om.embed_lookup_backward(torch.zeros(8, 4).t(), ids, 9),
                 lambda: om.expert_mlp(h, eid, w, up, down), lambda: om.expert_mlp(h.float(), eid, w, up.float(), down.float()),
                 lambda: om.expert_mlp(h, eid, w, up, down, act="tanh"), lambda: om.expert_mlp(h, eid, w.double(), up, down),
                 lambda: om.expert_mlp(h, eid, w, up, up), lambda: om.expert_mlp(h, eid, w, up, down, gate=down),
                 lambda: om.expert_mlp(h, eid, w, up.half(), down), lambda: om.expert_mlp(h, eid, w, up.transpose(1, 2), down)):
        with pytest.raises(ValueError) if not torch.cuda.is_available() else pytest.raises((ValueError, RuntimeError)):
            call()
    assert ctypes.sizeof(om.BeamArray) == 88
