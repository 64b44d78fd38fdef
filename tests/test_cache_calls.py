"""Host-side validation of the append, the several-query calls and the eviction
by weight: every refusal is a status before anything is launched, struct
layouts match the header, workspace sizes are host-only.  No GPU needed."""
import ctypes
import math
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "tq.h")
INV, UNS, WSP = 1, 2, 3


@pytest.fixture(scope="module")
def tq():
    from rotated_lloyd_max_gb300 import build
    build.build()
    import rotated_lloyd_max_gb300 as m
    m.load()
    return m


def _codec(tq, d=128, bits=3, T=0.0, cap=0):
    c = tq.tq_codec()
    c.head_dim, c.bits, c.outlier_T, c.outlier_cap = d, bits, T, cap
    K = 1 << bits
    for k in range(K):
        c.centroids[k] = (k - (K - 1) / 2) / 10
    for k in range(K - 1):
        c.boundaries[k] = (c.centroids[k] + c.centroids[k + 1]) / 2
    c.boundaries[K // 2 - 1] = 0.0
    return c


def test_struct_layouts_match_header(tq, tmp_path):
    structs = {"tq_append_args": tq.tq_append_args, "tq_query_args": tq.tq_query_args,
               "tq_evict_mass_args": tq.tq_evict_mass_args}
    lines = ["#include <stdio.h>", "#include <stddef.h>", f'#include "{HEADER}"', "int main(void) {"]
    for name, cls in structs.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        for f, _ in cls._fields_:
            lines.append(f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));')
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.check_call(["gcc", "-std=c11", "-Wall", "-Werror", str(src), "-o", str(exe)])
    got = dict(l.split() for l in subprocess.check_output([str(exe)], text=True).splitlines())
    for name, cls in structs.items():
        assert int(got[name]) == ctypes.sizeof(cls), name
        for f, _ in cls._fields_:
            assert int(got[f"{name}.{f}"]) == getattr(cls, f).offset, f"{name}.{f}"


def _append(tq, **kw):
    a = tq.tq_append_args()
    v = dict(n_layers=1, batch=2, t_q=3, n_q_heads=4, n_kv_heads=2, head_dim=128, q=0x10000, k=0x20000, v=0x30000,
             q_layer_stride=0, q_batch_stride=1536, q_token_stride=512, kv_layer_stride=0, kv_batch_stride=768,
             kv_token_stride=256, q_out=0x40000, q_out_batch_stride=1536, q_out_token_stride=512, positions=0x50000,
             n_axes=2, rot_start=0, rot_dim=128, inv_freq=0x60000, rot_scale=1.0, k_tail=0x70000, v_tail=0x80000,
             tail_layer_stride=0, tail_cap=64, tail_len=0x90000, tail_len_out=0xA0000)
    v.update(kw)
    for k, x in v.items():
        setattr(a, k, x)
    return a


APPEND_BAD = [
    (dict(head_dim=96), UNS), (dict(n_layers=0), INV), (dict(t_q=0), INV), (dict(k=None), INV), (dict(k_tail=None), INV),
    (dict(v=None), INV), (dict(v_tail=None), INV), (dict(v_tail=0x70000), INV), (dict(q=None), INV),
    (dict(q_out=None), INV), (dict(n_q_heads=0), INV), (dict(k=0x20008), INV), (dict(q_token_stride=510), INV),
    (dict(kv_batch_stride=-8), INV), (dict(tail_len=None), INV), (dict(tail_len_out=None), INV),
    (dict(tail_len_out=0xA0002), INV), (dict(tail_cap=0), INV), (dict(rot_dim=40), UNS), (dict(rot_dim=144), INV),
    (dict(rot_dim=64, rot_start=72), INV), (dict(rot_dim=64, rot_start=4), UNS), (dict(n_axes=0), INV),
    (dict(n_axes=5), INV), (dict(positions=None), INV), (dict(inv_freq=None), INV), (dict(rot_scale=math.inf), INV),
    (dict(q_out=0x10000, q_out_token_stride=520), INV), (dict(mass=0xB0000, mass_cap=0), INV),
    (dict(mass=0xB0002, mass_cap=9), INV), (dict(pair_axis=(ctypes.c_uint8 * 256)(*[2] * 256)), INV),
]


@pytest.mark.parametrize("kw,status", APPEND_BAD)
def test_append_refusals(tq, kw, status):
    assert tq.load().tq_append(ctypes.byref(_append(tq, **kw)), None) == status
    assert tq.load().tq_append(None, None) == INV


def _query(tq, **kw):
    a = tq.tq_query_args()
    v = dict(n_layers=1, batch=2, t_q=5, n_q_heads=4, n_kv_heads=2, head_dim=128, scale=1.0, causal=1, q=0x10000,
             q_batch_stride=2560, q_token_stride=512, out=0x20000, out_batch_stride=2560, out_token_stride=512,
             k_rec=0x100000, v_rec=0x200000, rec_cap=8, k_tail=0x300000, v_tail=0x400000, tail_cap=64,
             n_chunks=0x500000, tail_start=0x500100, tail_len=0x500200, max_chunks=8, max_tail=64)
    v.update(kw)
    for k, x in v.items():
        setattr(a, k, x)
    return a


QUERY_BAD = [
    (dict(head_dim=320), UNS), (dict(n_q_heads=5), INV), (dict(t_q=0), INV), (dict(q=None), INV), (dict(q=0x10004), INV),
    (dict(q_token_stride=12), INV), (dict(scale=math.nan), INV), (dict(softcap=-1.0), INV), (dict(softcap=math.inf), INV),
    (dict(max_chunks=9), INV), (dict(max_tail=65), INV), (dict(max_chunks=-1), INV), (dict(splits=-1), INV),
    (dict(n_chunks=None), INV), (dict(tail_len=None), INV), (dict(k_rec=None), INV), (dict(k_tail=None), INV),
    (dict(k_rec=0x100008), INV), (dict(k_rec_layer_stride=8), INV), (dict(rec_cap=0), INV), (dict(tail_cap=0), INV),
    (dict(tail_layer_stride=4), INV), (dict(block_table=0x600000, table_stride=0), INV),
    (dict(block_table=0x600000, table_stride=7), INV), (dict(n_chunks=0x500002), INV), (dict(batch=40000), UNS),
    (dict(t_q=1 << 29), UNS), (dict(max_chunks=1 << 25, rec_cap=1 << 25), UNS),
]


@pytest.mark.parametrize("kw,status", QUERY_BAD)
def test_query_refusals(tq, kw, status):
    L, kc, vc = tq.load(), _codec(tq), _codec(tq, bits=2)
    a, ws = _query(tq, **kw), ctypes.c_void_p(0x1000000)
    assert L.tq_prefill_attn_workspace_size(ctypes.byref(a), ctypes.byref(kc), ctypes.byref(vc)) == 0
    assert L.tq_prefill_attn(ctypes.byref(a), ctypes.byref(kc), ctypes.byref(vc), ws, 1 << 40, None) == status
    assert L.tq_attn_mass_workspace_size(ctypes.byref(a), ctypes.byref(kc)) == 0
    assert L.tq_attn_mass(ctypes.byref(a), ctypes.byref(kc), 0x2000000, 0, 1 << 30, 1.0, ws, 1 << 40, None) == status


def test_query_codecs_values_and_workspaces(tq):
    L, kc, vc = tq.load(), _codec(tq), _codec(tq, bits=2)
    ws = ctypes.c_void_p(0x1000000)

    def prefill(a, k=kc, v=vc, w=ws, n=1 << 40):
        return L.tq_prefill_attn(ctypes.byref(a), k and ctypes.byref(k), v and ctypes.byref(v), w, n, None)

    a = _query(tq)
    need = L.tq_prefill_attn_workspace_size(ctypes.byref(a), ctypes.byref(kc), ctypes.byref(vc))
    assert need > 0
    assert prefill(a, n=need - 1) == WSP
    assert prefill(a, w=None) == INV and prefill(a, w=ctypes.c_void_p(0x1000010)) == INV
    assert prefill(a, k=None) == INV and prefill(a, v=None) == INV
    assert prefill(a, k=_codec(tq, d=64)) == INV and prefill(a, v=_codec(tq, d=64)) == INV
    assert prefill(a, k=_codec(tq, bits=3, T=-1.0)) == INV
    for bad in (dict(out=None), dict(v_rec=None), dict(v_tail=None), dict(out=0x20002), dict(out_token_stride=4)):
        assert prefill(_query(tq, **bad)) == INV
    shared = _query(tq, v_rec=0x100000)  # one record for both needs one codec
    assert prefill(shared) == INV
    # the weights need no values and no output
    b = _query(tq, out=None, v_rec=None, v_tail=None)
    need = L.tq_attn_mass_workspace_size(ctypes.byref(b), ctypes.byref(kc))
    assert need > 0

    def mass(a, m=0x2000000, cap=8 * 128 + 64, decay=1.0, w=ws, n=need, stride=0):
        return L.tq_attn_mass(ctypes.byref(a), ctypes.byref(kc), m, stride, cap, decay, w, n, None)

    assert mass(b, m=None) == INV and mass(b, m=0x2000002) == INV and mass(b, cap=8 * 128 + 63) == INV
    assert mass(b, decay=-0.5) == INV and mass(b, decay=math.nan) == INV and mass(b, stride=-1) == INV
    assert mass(b, n=need - 1) == WSP and mass(b, w=None) == INV


def _evict(tq, in_place=False, **kw):
    a = tq.tq_evict_mass_args()
    v = dict(n_layers=1, batch=2, n_kv_heads=2, k_rec=0x100000, v_rec=0x200000, rec_cap=8, k_dst=0x300000, v_dst=0x400000,
             dst_cap=4, mass=0x500000, mass_dst=0x600000, mass_cap=8 * 128 + 16, mass_dst_cap=4 * 128 + 16,
             n_chunks=0x700000, n_chunks_dst=0x700100, tail_len=0x700200, max_chunks=8, max_tail=16, keep_chunks=4,
             sink=4, recent=100)
    if in_place:
        v.update(k_dst=v["k_rec"], v_dst=v["v_rec"], mass_dst=v["mass"], n_chunks_dst=v["n_chunks"])
    v.update(kw)
    for k, x in v.items():
        setattr(a, k, x)
    return a


EVICT_BAD = [
    (False, dict(n_layers=0), INV), (False, dict(k_rec=None), INV), (False, dict(k_dst=None), INV),
    (False, dict(mass=None), INV), (False, dict(n_chunks_dst=None), INV), (False, dict(k_dst=0x300008), INV),
    (False, dict(mass_dst=0x500000), INV), (False, dict(v_dst=0x200000), INV), (False, dict(v_dst=0x300000), INV),
    (False, dict(n_chunks_dst=0x700000), INV), (True, dict(v_dst=0x400000), INV), (True, dict(mass_dst=0x600000), INV),
    (True, dict(n_chunks_dst=0x700100), INV), (False, dict(keep_chunks=0), INV), (False, dict(sink=-1), INV),
    (False, dict(sink=413), INV), (False, dict(max_chunks=9), INV), (False, dict(mass_cap=8 * 128 + 15), INV),
    (False, dict(mass_dst_cap=4 * 128 + 15), INV), (False, dict(dst_cap=3), INV), (False, dict(rec_cap=0), INV),
    (False, dict(block_table=0x800000, table_stride=0), INV), (False, dict(dst_table=0x800000, dst_table_stride=3), INV),
    (False, dict(k_dst_layer_stride=8), INV), (False, dict(kept=0x900002), INV), (True, dict(batch=65536), UNS),
    (True, dict(max_chunks=1 << 25, rec_cap=1 << 25, mass_cap=0x7FFFFFFF), UNS),
]


@pytest.mark.parametrize("in_place,kw,status", EVICT_BAD)
def test_evict_mass_refusals(tq, in_place, kw, status):
    L, kc, vc = tq.load(), _codec(tq), _codec(tq, bits=2)
    a = _evict(tq, in_place, **kw)
    assert L.tq_evict_mass_workspace_size(ctypes.byref(a), ctypes.byref(kc), ctypes.byref(vc)) == 0
    assert L.tq_evict_mass(ctypes.byref(a), ctypes.byref(kc), ctypes.byref(vc), 0x1000000, 1 << 40, None) == status


def test_evict_mass_workspace(tq):
    L, kc, vc = tq.load(), _codec(tq), _codec(tq, bits=2)
    for in_place in (False, True):
        a = _evict(tq, in_place)
        need = L.tq_evict_mass_workspace_size(ctypes.byref(a), ctypes.byref(kc), ctypes.byref(vc))
        assert need >= 4 * 4 * 128 * 4
        for w, n, st in ((0x1000000, need - 1, WSP), (None, need, INV), (0x1000010, need, INV)):
            assert L.tq_evict_mass(ctypes.byref(a), ctypes.byref(kc), ctypes.byref(vc), w, n, None) == st
        assert L.tq_evict_mass(ctypes.byref(a), ctypes.byref(_codec(tq, d=64)), ctypes.byref(vc), 0x1000000, need,
                               None) == INV


def test_pair_axes_of_sections(tq):
    assert tq.rope_pair_axis([2, 1, 1]) == [0, 0, 1, 2]
    assert tq.rope_pair_axis([3, 1, 2], interleaved=True) == [0, 1, 2, 0, 2, 0]


def test_binding_refuses_wrong_tensors(tq):
    """Shapes, dtypes and layouts are checked in Python before any pointer is taken (CPU tensors here)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("CPU tensors are refused by their device there")
    bf, i32 = torch.bfloat16, torch.int32
    k, ring = torch.zeros(1, 2, 3, 2, 64, dtype=bf), torch.zeros(1, 2, 2, 8, 64, dtype=bf)
    ln = torch.zeros(1, 2, dtype=i32)
    good = dict(k=k, v=k, k_tail=ring, v_tail=ring.clone(), tail_len=ln)
    tq.make_append_args(**good)
    for bad in (dict(k=k.float()), dict(k=k.transpose(2, 3)), dict(k_tail=ring[:, :1]), dict(v_tail=ring[..., :4, :]),
                dict(tail_len=ln.long()), dict(tail_len=ln[:, :1]), dict(q=k), dict(inv_freq=torch.ones(4)),
                dict(inv_freq=torch.ones(4), positions=torch.zeros(1, 2, 4, dtype=i32)),
                dict(inv_freq=torch.ones(4), positions=torch.zeros(1, 2, 3, dtype=i32), pair_axis=[0]),
                dict(mass=torch.zeros(1, 2, 3, 9))):
        with pytest.raises(ValueError):
            tq.make_append_args(**{**good, **bad})
    q = torch.zeros(1, 2, 3, 4, 64, dtype=bf)
    rec = torch.zeros(1, 2, 2, 3, 1536, dtype=torch.uint8)
    good = dict(q=q, scale=1.0, out=q.clone(), k_rec=rec, v_rec=rec, n_chunks=ln, max_chunks=3)
    tq.make_query_args(**good)
    for bad in (dict(out=q[:, :, :2]), dict(k_rec=rec[:, :1]), dict(k_rec=rec[..., ::2]), dict(n_chunks=ln.long()),
                dict(v_rec=rec[:, :, :, :2]), dict(q_lens=torch.zeros(3, dtype=i32)),
                dict(block_table=torch.zeros(2, 3, dtype=i32))):
        with pytest.raises(ValueError):
            tq.make_query_args(**{**good, **bad})
    m = torch.zeros(1, 2, 2, 400)
    good = dict(k_rec=rec, v_rec=rec, mass=m, n_chunks=ln, max_chunks=3, keep_chunks=2)
    tq.make_evict_mass_args(**good)
    for bad in (dict(mass=m[:, :1]), dict(k_dst=rec), dict(kept=torch.zeros(1, 2, 2, 255, dtype=i32)),
                dict(dst_table=torch.zeros(2, 3, dtype=i32)), dict(mass=m.double())):
        with pytest.raises(ValueError):
            tq.make_evict_mass_args(**{**good, **bad})


def test_outputs_that_overlap_themselves_are_refused(tq):
    """Two rows, or two layers, of an output in the same place would be written in any order."""
    L, kc, vc, ws = tq.load(), _codec(tq), _codec(tq, bits=2), ctypes.c_void_p(0x1000000)
    for kw in (dict(q_out_token_stride=504), dict(q_out_batch_stride=0), dict(n_layers=2, q_out_layer_stride=256, tail_layer_stride=1 << 20),
               dict(n_layers=2, q_out_layer_stride=4096, tail_layer_stride=2 * 2 * 64 * 128 - 8),
               dict(n_layers=2, q_out_layer_stride=4096, tail_layer_stride=2 * 2 * 64 * 128, mass=0xB0000, mass_cap=9,
                    mass_layer_stride=35)):
        assert L.tq_append(ctypes.byref(_append(tq, **kw)), None) == INV
    for kw in (dict(out_token_stride=0), dict(out_batch_stride=504), dict(n_layers=2)):
        a = _query(tq, **kw)
        assert L.tq_prefill_attn(ctypes.byref(a), ctypes.byref(kc), ctypes.byref(vc), ws, 1 << 40, None) == INV
    a = _query(tq, n_layers=2, tail_layer_stride=1 << 20)
    assert L.tq_attn_mass(ctypes.byref(a), ctypes.byref(kc), 0x2000000, 4 * 1088 - 1, 1088, 1.0, ws, 1 << 40, None) == INV
    two = dict(n_layers=2, mass_layer_stride=4 * (8 * 128 + 16), mass_dst_layer_stride=4 * (4 * 128 + 16),
               k_dst_layer_stride=1 << 20, v_dst_layer_stride=1 << 20)
    assert L.tq_evict_mass_workspace_size(ctypes.byref(_evict(tq, **two)), ctypes.byref(kc), ctypes.byref(vc)) > 0
    for kw in (dict(mass_layer_stride=4159), dict(mass_dst_layer_stride=2111), dict(k_dst_layer_stride=0),
               dict(v_dst_layer_stride=4 * 4 * (128 * 128 * 2 // 8 + 512) - 16)):
        a = _evict(tq, **dict(two, **kw))
        assert L.tq_evict_mass(ctypes.byref(a), ctypes.byref(kc), ctypes.byref(vc), ws, 1 << 40, None) == INV


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("paged", [False, True])
def test_layers_that_overlap_in_place_are_refused(tq, shared, paged):
    """In place the source is the destination: two layers in the same records would be compacted at once."""
    L, kc, vc, ws = tq.load(), _codec(tq), _codec(tq, bits=3 if shared else 2), ctypes.c_void_p(0x1000000)
    heads = 2 if paged else 2 * 8 * 2
    kb, vb = ((128 * 128 * b // 8 + 512) * heads for b in (3, 3 if shared else 2))
    kw = dict(n_layers=2, mass_layer_stride=4 * (8 * 128 + 16), k_rec_layer_stride=kb, v_rec_layer_stride=vb)
    if paged:
        kw.update(block_table=0x800000, table_stride=8)
    if shared:
        kw.update(v_rec=0x100000, v_dst=0x100000)

    def size(**more):
        a = _evict(tq, True, **dict(kw, **more))
        n = L.tq_evict_mass_workspace_size(ctypes.byref(a), ctypes.byref(kc), ctypes.byref(vc))
        if n == 0:
            assert L.tq_evict_mass(ctypes.byref(a), ctypes.byref(kc), ctypes.byref(vc), ws, 1 << 40, None) == INV
        return n

    assert size() > 0
    assert size(k_rec_layer_stride=kb - 16) == 0 and size(k_rec_layer_stride=0) == 0
    if not shared:
        assert size(v_rec_layer_stride=vb - 16) == 0 and size(v_rec_layer_stride=0) == 0
    assert size(n_layers=1, k_rec_layer_stride=0, v_rec_layer_stride=0) > 0


def test_sizes_whose_indices_would_wrap_are_refused(tq):
    """Token indices are 32-bit, with room for a launch's last threads and a split's length behind them; a
    merge's grid has 2^31 - 1 blocks at most."""
    L, kc, vc = tq.load(), _codec(tq, d=64, bits=1), _codec(tq, d=64, bits=1)
    most = ((1 << 31) - (1 << 20)) // 128

    def sizes(a):
        return (L.tq_prefill_attn_workspace_size(ctypes.byref(a), ctypes.byref(kc), ctypes.byref(vc)),
                L.tq_attn_mass_workspace_size(ctypes.byref(a), ctypes.byref(kc)))

    def query(n, tail, **kw):
        return _query(tq, **dict(dict(head_dim=64, batch=1, n_kv_heads=1, n_q_heads=1, t_q=1, max_chunks=n, rec_cap=max(n, 1),
                                      max_tail=tail, tail_cap=max(tail, 1)), **kw))

    assert all(sizes(query(most - 1, 0))) and all(sizes(query(most - 1, 128)))
    assert sizes(query(most, 1)) == (0, 0) and sizes(query(most + 1, 0)) == (0, 0)
    assert all(sizes(query(0, 128 * most))) and sizes(query(0, 128 * most + 1)) == (0, 0)
    a = query(most + 1, 0)
    ws = ctypes.c_void_p(0x1000000)
    assert L.tq_prefill_attn(ctypes.byref(a), ctypes.byref(kc), ctypes.byref(vc), ws, 1 << 60, None) == UNS
    # nothing cached, rows of 2^32 - 2^17 (layer, sequence, kv head) units: the merge alone would run
    none = dict(k_rec=None, v_rec=None, n_chunks=None, k_tail=None, v_tail=None, tail_start=None, tail_len=None, rec_cap=0,
                tail_cap=0, out_batch_stride=64, out_layer_stride=1 << 22, q_batch_stride=64, q_token_stride=64)
    a = query(0, 0, n_layers=65535, batch=65535, **none)
    assert L.tq_prefill_attn_workspace_size(ctypes.byref(a), ctypes.byref(kc), ctypes.byref(vc)) == 0
    assert L.tq_prefill_attn(ctypes.byref(a), ctypes.byref(kc), ctypes.byref(vc), ws, 1 << 60, None) == UNS
    b = dict(n_kv_heads=1, batch=1, max_tail=0, tail_len=None, keep_chunks=1, recent=0, sink=0, dst_cap=1)
    ev = lambda n, **kw: L.tq_evict_mass_workspace_size(  # noqa: E731
        ctypes.byref(_evict(tq, False, **dict(b, max_chunks=n, rec_cap=n, mass_cap=128 * n, mass_dst_cap=128, **kw))),
        ctypes.byref(kc), ctypes.byref(vc))
    assert ev(most) > 0 and ev(most + 1) == 0
