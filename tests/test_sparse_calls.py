"""Host-side validation of the append with norms, the bounds of keys, the
selection of records and the attention over listed ones: every refusal is a
status before anything is launched, struct layouts match the header, workspace
sizes are host-only.  No GPU needed."""
import ctypes
import math
import os
import subprocess

import pytest

from test_cache_calls import INV, UNS, WSP, _append, _codec, _query

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "tq.h")


@pytest.fixture(scope="module")
def tq():
    from rotated_lloyd_max_gb300 import build
    build.build()
    import rotated_lloyd_max_gb300 as m
    m.load()
    return m


def test_struct_layouts_match_header(tq, tmp_path):
    names = ("tq_head_norm", "tq_bounds_args", "tq_select_args", "tq_record_lists")
    lines = ["#include <stdio.h>", "#include <stddef.h>", f'#include "{HEADER}"', "int main(void) {"]
    for name in names:
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        for f, _ in getattr(tq, name)._fields_:
            lines.append(f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));')
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.check_call(["gcc", "-std=c11", "-Wall", "-Werror", str(src), "-o", str(exe)])
    got = dict(x.split() for x in subprocess.check_output([str(exe)], text=True).splitlines())
    for name in names:
        cls = getattr(tq, name)
        assert int(got[name]) == ctypes.sizeof(cls), name
        for f, _ in cls._fields_:
            assert int(got[f"{name}.{f}"]) == getattr(cls, f).offset, f"{name}.{f}"


def _set(a, v, kw):
    for k, x in {**v, **kw}.items():
        setattr(a, k, x)
    return a


NORM_BAD = [dict(q_weight=None, k_weight=None), dict(q_weight=0x10004), dict(k_weight=0x10008), dict(q_head_stride=2),
            dict(k_head_stride=-4), dict(eps=-1e-6), dict(eps=math.nan), dict(eps=math.inf)]


@pytest.mark.parametrize("kw", NORM_BAD)
def test_norm_refusals(tq, kw):
    n = _set(tq.tq_head_norm(), dict(q_weight=0x10000, k_weight=0x20000, eps=1e-6), kw)
    assert tq.load().tq_norm_append(ctypes.byref(_append(tq)), ctypes.byref(n), None) == INV


def test_norm_needs_queries_for_their_weights_and_the_appends_arguments(tq):
    L = tq.load()
    n = _set(tq.tq_head_norm(), dict(q_weight=0x10000, eps=1e-6), {})
    no_q = _append(tq, q=None, q_out=None, n_q_heads=0)
    assert L.tq_norm_append(ctypes.byref(no_q), ctypes.byref(n), None) == INV
    assert L.tq_norm_append(ctypes.byref(_append(tq)), None, None) == INV
    assert L.tq_norm_append(None, ctypes.byref(n), None) == INV
    for kw, status in ((dict(head_dim=96), UNS), (dict(tail_cap=0), INV), (dict(rot_dim=40), UNS)):
        assert L.tq_norm_append(ctypes.byref(_append(tq, **kw)), ctypes.byref(n), None) == status


def _bounds(tq, **kw):
    return _set(tq.tq_bounds_args(), dict(n_layers=1, batch=2, n_kv_heads=2, k_rec=0x100000, rec_cap=8, n_chunks=0x200000,
                                          max_chunks=8, max_new=8, bounds=0x300000), kw)


BOUNDS_BAD = [
    (dict(n_layers=0), INV), (dict(batch=0), INV), (dict(n_kv_heads=0), INV), (dict(k_rec=None), INV),
    (dict(bounds=None), INV), (dict(n_chunks=None), INV), (dict(k_rec=0x100008), INV), (dict(bounds=0x300008), INV),
    (dict(n_chunks=0x200002), INV), (dict(first=0x200001), INV), (dict(k_rec_layer_stride=8), INV),
    (dict(bounds_layer_stride=4), INV), (dict(rec_cap=0), INV), (dict(max_chunks=9), INV), (dict(max_chunks=-1), INV),
    (dict(max_new=0), INV), (dict(block_table=0x400000), INV), (dict(block_table=0x400000, table_stride=7), INV),
    (dict(n_layers=2, bounds_layer_stride=2 * 2 * 8 * 256 - 8), INV),
    (dict(n_layers=2, block_table=0x400000, table_stride=8, bounds_layer_stride=2 * 8 * 256 - 8), INV),
    (dict(max_chunks=1 << 25, rec_cap=1 << 25), UNS), (dict(batch=1 << 30), UNS),
]


@pytest.mark.parametrize("kw,status", BOUNDS_BAD)
def test_bounds_refusals(tq, kw, status):
    a, c = _bounds(tq, **kw), _codec(tq)
    assert tq.load().tq_key_bounds(ctypes.byref(c), ctypes.byref(a), None) == status


def test_bounds_codecs(tq):
    L, a = tq.load(), _bounds(tq)
    assert L.tq_key_bounds(None, ctypes.byref(a), None) == INV
    assert L.tq_key_bounds(ctypes.byref(_codec(tq)), None, None) == INV
    assert L.tq_key_bounds(ctypes.byref(_codec(tq, T=-1.0)), ctypes.byref(a), None) == INV


def _select(tq, **kw):
    return _set(tq.tq_select_args(),
                dict(n_layers=1, batch=2, t_q=5, n_q_heads=4, n_kv_heads=2, head_dim=128, causal=1, q=0x10000,
                     q_batch_stride=5 * 512, q_token_stride=512, bounds=0x300000, rec_cap=8, n_chunks=0x200000,
                     tail_len=0x200100, max_chunks=8, max_tail=20, q_block=2, keep=4, sink=1, recent=2, list=0x500000,
                     count=0x600000), kw)


SELECT_BAD = [
    (dict(head_dim=96), UNS), (dict(n_layers=0), INV), (dict(t_q=0), INV), (dict(n_q_heads=3), INV), (dict(q=None), INV),
    (dict(q=0x10008), INV), (dict(q_token_stride=510), INV), (dict(q_batch_stride=-8), INV), (dict(bounds=None), INV),
    (dict(bounds=0x300008), INV), (dict(bounds_layer_stride=4), INV), (dict(n_chunks=None), INV), (dict(list=None), INV),
    (dict(count=None), INV), (dict(list=0x500002), INV), (dict(count=0x600001), INV), (dict(q_lens=0x700002), INV),
    (dict(tail_len=None), INV), (dict(max_chunks=9), INV), (dict(max_chunks=-1), INV), (dict(max_tail=-1), INV),
    (dict(rec_cap=0), INV), (dict(block_table=0x800000), INV), (dict(block_table=0x800000, table_stride=7), INV),
    (dict(q_block=0), INV), (dict(keep=0), INV), (dict(sink=-1), INV), (dict(recent=-1), INV), (dict(sink=3), INV),
    (dict(sink=0x7FFFFFFF, recent=0x7FFFFFFF), INV), (dict(max_chunks=16385, rec_cap=16385), UNS), (dict(t_q=1 << 28), UNS),
    (dict(batch=1 << 26, n_layers=1 << 10), UNS),
]


@pytest.mark.parametrize("kw,status", SELECT_BAD)
def test_select_refusals(tq, kw, status):
    L, a = tq.load(), _select(tq, **kw)
    assert L.tq_select_records_workspace_size(ctypes.byref(a)) == 0
    assert L.tq_select_records(ctypes.byref(a), 0x1000000, 1 << 50, None) == status


def test_select_workspace(tq):
    L, a = tq.load(), _select(tq)
    need = L.tq_select_records_workspace_size(ctypes.byref(a))
    assert need >= 2 * 2 * 3 * 8 * 12
    for w, n, st in ((0x1000000, need - 1, WSP), (None, need, INV), (0x1000010, need, INV)):
        assert L.tq_select_records(ctypes.byref(a), w, n, None) == st
    assert L.tq_select_records_workspace_size(ctypes.byref(_select(tq, max_chunks=16384, rec_cap=16384))) > 0


def _lists(tq, **kw):
    return _set(tq.tq_record_lists(), dict(list=0x500000, count=0x600000, list_stride=4, q_block=2), kw)


@pytest.mark.parametrize("kw,status", [
    (dict(list=None), INV), (dict(count=None), INV), (dict(list=0x500002), INV), (dict(count=0x600001), INV),
    (dict(list_stride=0), INV), (dict(list_stride=-1), INV), (dict(q_block=0), INV), (dict(list_stride=1 << 25), UNS)])
def test_list_refusals(tq, kw, status):
    L, kc, vc = tq.load(), _codec(tq), _codec(tq, bits=2)
    a, r = _query(tq), _lists(tq, **kw)
    refs = [ctypes.byref(x) for x in (a, r, kc, vc)]
    assert L.tq_sparse_attn_workspace_size(*refs) == 0
    assert L.tq_sparse_attn(*refs, 0x1000000, 1 << 50, None) == status


def test_attention_over_lists_takes_the_prefills_arguments(tq):
    L, kc, vc, r = tq.load(), _codec(tq), _codec(tq, bits=2), _lists(tq)

    def call(a, k=kc, v=vc, rr=r, w=0x1000000, n=1 << 50):
        return L.tq_sparse_attn(ctypes.byref(a), rr and ctypes.byref(rr), k and ctypes.byref(k), v and ctypes.byref(v), w, n, None)

    for kw, status in ((dict(head_dim=320), UNS), (dict(q=None), INV), (dict(out=None), INV), (dict(scale=math.inf), INV),
                       (dict(softcap=-1.0), INV), (dict(max_chunks=9), INV), (dict(v_rec=None), INV), (dict(splits=-1), INV),
                       (dict(out_token_stride=0), INV), (dict(batch=40000), UNS),
                       (dict(k_rec=None, v_rec=None, n_chunks=None, max_chunks=0), INV)):
        assert call(_query(tq, **kw)) == status, kw
    a = _query(tq)
    assert call(a, rr=None) == INV and call(a, k=None) == INV and call(a, v=None) == INV
    assert call(a, v=_codec(tq, d=64)) == INV
    for outl in (0.0, 2.0):
        k = _codec(tq, T=outl, cap=1312 if outl else 0)
        need = L.tq_sparse_attn_workspace_size(ctypes.byref(a), ctypes.byref(r), ctypes.byref(k), ctypes.byref(vc))
        assert need > 0
        assert call(a, k=k, n=need - 1) == WSP and call(a, k=k, w=None) == INV and call(a, k=k, w=0x1000010) == INV
    one = _query(tq, splits=1)
    assert 0 < L.tq_sparse_attn_workspace_size(ctypes.byref(one), ctypes.byref(r), ctypes.byref(kc), ctypes.byref(vc)) <= need


def test_binding_refuses_wrong_tensors(tq):
    """Shapes, dtypes and layouts are checked in Python before any pointer is taken (CPU tensors here)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("CPU tensors are refused by their device there")
    bf, i32 = torch.bfloat16, torch.int32
    w = torch.zeros(4, 64)
    tq.make_head_norm(q_weight=w, k_weight=w[0])
    for bad in (dict(q_weight=w.to(bf)), dict(k_weight=w.t()), dict(q_weight=w[None])):
        with pytest.raises(ValueError):
            tq.make_head_norm(**bad)
    rec, n = torch.zeros(1, 2, 2, 3, 1536, dtype=torch.uint8), torch.zeros(1, 2, dtype=i32)
    bounds = torch.zeros(1, 2, 2, 3, 2, 64, dtype=bf)
    good = dict(k_rec=rec, bounds=bounds, n_chunks=n, max_chunks=3)
    tq.make_bounds_args(**good)
    for bad in (dict(bounds=bounds[:, :, :, :2]), dict(bounds=bounds.float()), dict(n_chunks=n.long()), dict(first=n[:, :1]),
                dict(k_rec=rec[..., ::2]), dict(block_table=torch.zeros(2, 3, dtype=i32))):
        with pytest.raises(ValueError):
            tq.make_bounds_args(**{**good, **bad})
    pool = dict(k_rec=torch.zeros(1, 7, 2, 1536, dtype=torch.uint8), bounds=torch.zeros(1, 7, 2, 2, 64, dtype=bf),
                block_table=torch.zeros(2, 3, dtype=i32))
    tq.make_bounds_args(**{**good, **pool})
    q = torch.zeros(1, 2, 5, 4, 64, dtype=bf)
    lists = dict(list=torch.zeros(1, 2, 3, 2, 2, dtype=i32), count=torch.zeros(1, 2, 3, 2, dtype=i32))
    good = dict(q=q, bounds=bounds, n_chunks=n, max_chunks=3, q_block=2, keep=2, **lists)
    tq.make_select_args(**good)
    for bad in (dict(q=q[..., :3]), dict(bounds=bounds[:1, :1]), dict(q_block=5), dict(keep=3), dict(q_block=0),
                dict(list=lists["list"].long()), dict(list=lists["list"].transpose(2, 3)), dict(tail_len=n.t()),
                dict(block_table=torch.zeros(2, 3, dtype=i32))):
        with pytest.raises(ValueError):
            tq.make_select_args(**{**good, **bad})
    tq.make_record_lists(**lists)
    for bad in (dict(count=lists["count"][:, :1]), dict(list=lists["list"][..., 0]), dict(count=lists["count"].long())):
        with pytest.raises(ValueError):
            tq.make_record_lists(**{**lists, **bad})


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("T_out", [0.0, 2.0])
@pytest.mark.parametrize("T,G,q_block", [(2048, 4, 1), (2048, 1, 1), (2047, 4, 5), (300, 5, 4), (1000, 16, 8), (513, 4, 64),
                                         (300, 5, 100), (5, 64, 5), (1, 4, 1)])
def test_partials_take_the_rows_that_there_are(tq, d, T_out, T, G, q_block):
    """One split of the records and one of the ring: the workspace holds two partials of every row (f32 outputs, two
    numbers), a unit's rows (not a block's) padded to 128."""
    B, Hkv = 2, 8
    outl = dict(T=T_out, cap=4 * math.ceil(0.08 * 128 * d / 4)) if T_out else {}
    kc, vc = _codec(tq, d=d, **outl), _codec(tq, d=d, bits=2, **outl)
    row = Hkv * G * d
    a = _query(tq, batch=B, t_q=T, n_q_heads=Hkv * G, n_kv_heads=Hkv, head_dim=d, q_batch_stride=T * row, q_token_stride=row,
               out_batch_stride=T * row, out_token_stride=row, splits=1, max_tail=60)
    r = _lists(tq, list_stride=1, q_block=q_block)
    need = tq.load().tq_sparse_attn_workspace_size(*[ctypes.byref(x) for x in (a, r, kc, vc)])
    assert 0 < need <= B * Hkv * (-(-T * G // 128) * 128) * 2 * (4 * d + 8) + 1024


@pytest.mark.parametrize("T,layers,max_tail,keep", [(1 << 20, 64, 1 << 30, 32), (1 << 20, 64, 1 << 29, 256),
                                                    (1 << 20, 64, 1 << 30, 1), (1 << 17, 1, 1 << 20, 32), (1, 1, 1 << 30, 1)])
def test_runs_of_very_long_rings_are_planned(tq, T, layers, max_tail, keep):
    """Lists x ring tiles past 2^31 a run (a division by zero ended the process): the workspace holds one partial of the
    records and one of the ring for every row, and few more."""
    Hkv, d = 8, 64
    row = Hkv * d
    a = _query(tq, n_layers=layers, batch=1, t_q=T, n_q_heads=Hkv, n_kv_heads=Hkv, head_dim=d, q_layer_stride=T * row,
               q_batch_stride=T * row, q_token_stride=row, out_layer_stride=T * row, out_batch_stride=T * row,
               out_token_stride=row, max_tail=max_tail, tail_cap=max_tail)
    kc, vc, r = _codec(tq, d=d), _codec(tq, d=d, bits=2), _lists(tq, list_stride=keep, q_block=1)
    need = tq.load().tq_sparse_attn_workspace_size(*[ctypes.byref(x) for x in (a, r, kc, vc)])
    one = layers * T * Hkv * (4 * d + 8)
    assert 2 * one <= need <= (4 if T > 1 else 700) * one + 1024
