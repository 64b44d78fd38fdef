"""GPU tests of tq_evict_mass: the selection against a stable sort, records bit
for bit, side lists, in place and into another cache, pages, ties, NaN."""
import math

import numpy as np
import pytest

import tq_testlib as tl
from cache_cases import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rotated_lloyd_max_gb300 import build
    build.build()
    import rotated_lloyd_max_gb300 as m
    m.load()
    return m


def _chosen(m, N, keep, sink, recent):
    """Indices that remain, ascending: protected ones, then the largest, the lower index first."""
    if N <= keep:
        return np.arange(N)
    at = np.arange(N)
    key = np.where(np.isnan(m[:N]), -np.inf, m[:N].astype(np.float64))
    rank = np.where((at < sink) | (at >= N - recent), 2, np.where(np.isnan(m[:N]), 0, 1))
    return np.sort(np.lexsort((at, -key, -rank))[:keep])


def _rows(rec, codec, n):
    """Per token: code row bytes, scale bytes, side-list entries of host records [R, bytes]."""
    T = codec.c.outlier_T
    lay = tl.record_layout(codec.head_dim, codec.bits, bool(T), codec.c.outlier_cap if T else 0)
    rb = codec.head_dim * codec.bits // 8
    out = []
    for r in range(n):
        e = 0
        for s in range(128):
            ent = b""
            if T:
                c = int(rec[r, lay["count"] + s])
                ent = rec[r, lay["entries"] + 4 * e: lay["entries"] + 4 * (e + c)].tobytes()
                e += c
            out.append((rec[r, rb * s: rb * (s + 1)].tobytes(),
                        rec[r, lay["norm"] + 4 * s: lay["norm"] + 4 * s + 4].tobytes(), ent))
    return out


def _mass(c, kind, seed):
    g = np.random.default_rng(seed)
    cap = 128 * c.max_chunks + c.max_tail + 3
    m = np.exp(2 * g.standard_normal((c.L, c.B, c.Hkv, cap))).astype(np.float32)
    if kind == "ties":
        m = np.floor(m).astype(np.float32)
        m[..., ::3] = 0.0
        m[..., 1::7] = -0.0
    if kind == "equal":
        m[:] = 0.25
    if kind == "wild":
        m[..., ::5] = math.nan
        m[..., 1::11] = math.inf
        m[..., 2::13] = -math.inf
        m[..., 3::17] *= -1
        m[..., 4::19] = 1e-42
    return m


def _case(tq, orc, *, keep, sink=0, recent=0, kind="spread", in_place=False, dst_paged=False, T=0.0, **kw):
    import torch
    c = Cache(tq, orc, T=T, seed=31, **kw)
    mass0 = _mass(c, kind, 5)
    mass = torch.from_numpy(mass0.copy()).cuda()
    host = c._host
    kept = torch.full((c.L, c.B, c.Hkv, 128 * keep), -7, dtype=torch.int32, device="cuda")
    call = dict(k_rec=c.rec["k"], v_rec=c.rec["v"], mass=mass, n_chunks=c.d_n, max_chunks=c.max_chunks,
                keep_chunks=keep, tail_len=c.d_len, max_tail=c.max_tail, sink=sink, recent=recent, kept=kept,
                block_table=c.table)
    src = {w: c.rec[w].clone() for w in "kv"}
    if in_place:
        n_dst, mass_dst, dst, table = c.d_n, mass, c.rec, c.table
    else:
        slots = min(keep, c.max_chunks)
        n_dst = torch.full_like(c.d_n, -1)
        mass_dst = torch.full((c.L, c.B, c.Hkv, 128 * slots + c.max_tail + 1), -3.0, device="cuda")
        table = None
        if dst_paged:
            table = torch.randperm(c.B * slots + 1, device="cuda")[: c.B * slots].to(torch.int32).view(c.B, slots)
            shape = lambda w: (c.L, c.B * slots + 1, c.Hkv, c.rec[w].shape[-1])  # noqa: E731
        else:
            shape = lambda w: (c.L, c.B, c.Hkv, slots, c.rec[w].shape[-1])  # noqa: E731
        dst = {"k": torch.full(shape("k"), 0xCD, dtype=torch.uint8, device="cuda")}
        dst["v"] = dst["k"] if c.shared else torch.full(shape("v"), 0xCD, dtype=torch.uint8, device="cuda")
        call.update(k_dst=dst["k"], v_dst=dst["v"], mass_dst=mass_dst, n_chunks_dst=n_dst, dst_table=table)
    tq.evict_mass(k_codec=c.kc, v_codec=c.vc, **call)
    torch.cuda.synchronize()
    if not in_place:
        assert torch.equal(src["k"], c.rec["k"]) and torch.equal(src["v"], c.rec["v"])
        np.testing.assert_array_equal(mass.cpu().numpy(), mass0)
    got_n, got_m, got_kept = n_dst.cpu().numpy(), mass_dst.cpu().numpy(), kept.cpu().numpy()
    for l in range(c.L):
        for b in range(c.B):
            n, ln = int(c.n[l, b]), int(c.len[l, b])
            left = min(n, keep)
            assert got_n[l, b] == left
            for h in range(c.Hkv):
                want = _chosen(mass0[l, b, h], 128 * n, 128 * keep, sink, recent)
                np.testing.assert_array_equal(got_kept[l, b, h, :128 * left], want)
                assert np.all(got_kept[l, b, h, 128 * left:] == -7)
                m, m0 = got_m[l, b, h], mass0[l, b, h]
                np.testing.assert_array_equal(m[:128 * left], m0[want])
                np.testing.assert_array_equal(m[128 * left:128 * left + ln], m0[128 * n:128 * n + ln])
                rest = m[128 * left + ln:]
                if in_place:
                    gone = 128 * (n - left)
                    assert np.all(rest[:gone] == 0)
                    np.testing.assert_array_equal(rest[gone:], m0[128 * n + ln:])
                else:
                    assert np.all(rest == -3.0)
                for w, codec in (("k", c.kc), ("v", c.vc)):
                    if table is not None:
                        t = table.cpu().numpy()
                        rec = dst[w][l].cpu().numpy()[t[b], h]
                    else:
                        rec = dst[w][l, b, h].cpu().numpy()
                    old = _rows(host[w][l, b, h], codec, n)
                    new = _rows(rec, codec, left)
                    if codec.c.outlier_T:  # a list that outgrows its record loses the entries at its end
                        for r in range(left):
                            room = int(codec.c.outlier_cap)
                            for s in range(128):
                                e = old[want[128 * r + s]]
                                have = new[128 * r + s]
                                assert have[:2] == e[:2]
                                assert have[2] == e[2][: 4 * room]
                                room -= len(have[2]) // 4
                    else:
                        assert new == [old[i] for i in want]
    return c


CASES = {
    "half": dict(d=128, n=6, keep=3, B=3, L=2),
    "to_one_record": dict(d=64, kb=3, vb=1, n=9, keep=1, sink=5, recent=17),
    "nothing_to_do": dict(d=64, n=3, keep=3),
    "room_to_spare": dict(d=64, n=3, keep=40),
    "all_protected": dict(d=64, n=4, keep=2, sink=100, recent=156),
    "ties": dict(d=128, n=8, keep=3, kind="ties", sink=3),
    "all_equal": dict(d=64, n=8, keep=5, kind="equal", recent=9),
    "wild": dict(d=128, n=7, keep=4, kind="wild"),
    "shared_d512": dict(d=512, kb=4, shared=True, Hkv=1, n=5, keep=2),
    "d256_two_bits": dict(d=256, kb=2, vb=2, n=4, keep=3),
    "one_bit_rows_of_8_bytes": dict(d=64, kb=1, vb=3, n=4, keep=2),
    "side_lists": dict(d=128, T=2.0, n=6, keep=3),
    "side_lists_shared": dict(d=64, kb=3, T=1.5, shared=True, n=6, keep=2),
    "paged": dict(d=128, n=6, keep=4, B=3, L=2, paged=True),
    "no_ring": dict(d=128, n=5, keep=2, tail=0, cap=8),
    "thirty_two_records": dict(d=64, n=32, keep=16, B=1, sink=4, recent=30),
    "forty_records": dict(d=64, kb=2, vb=2, n=40, keep=7, B=1, Hkv=3),
    "many_records": dict(d=64, kb=1, vb=1, n=300, keep=170, B=1, Hkv=1, sink=4, recent=64),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", CASES)
def test_eviction(tq, orc, name, in_place):
    _case(tq, orc, in_place=in_place, **CASES[name])


def test_into_pages(tq, orc):
    _case(tq, orc, d=128, n=6, keep=4, B=3, paged=True, dst_paged=True)


def test_a_side_list_that_outgrows_its_record(tq, orc):
    """Lists near their capacity gathered from the densest tokens: entries past the capacity go."""
    import torch
    import rotated_lloyd_max_gb300 as m
    orig = m.tq_make_codebook
    try:
        m.tq_make_codebook = lambda b, d, **kw: orig(b, d, **{**kw, "outlier_cap": 160})
        for in_place in (False, True):
            _case(tq, orc, d=64, T=1.5, n=5, keep=2, in_place=in_place)
    finally:
        m.tq_make_codebook = orig


def test_long_stream_uses_every_pass(tq):
    """300 000 tokens of one stream whose weights share their leading digits: every digit decides."""
    import torch
    L = B = Hkv = 1
    n, keep, d = 2344, 1000, 64
    kc = tq.tq_make_codebook(1, d)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    rec = torch.randint(0, 256, (1, 1, 1, n, kc.record_bytes), dtype=torch.uint8, device="cuda", generator=g)
    mass = 1.0 + torch.rand((1, 1, 1, 128 * n), device="cuda", generator=g) * 2.0 ** -12
    for in_place in (False, True):
        cnt = torch.full((1, 1), n, dtype=torch.int32, device="cuda")
        m, r = mass.clone(), rec.clone()
        kept = torch.zeros((1, 1, 1, 128 * keep), dtype=torch.int32, device="cuda")
        kw = {}
        if not in_place:
            kw = dict(k_dst=torch.zeros_like(rec[:, :, :, :keep]), mass_dst=torch.zeros((1, 1, 1, 128 * keep), device="cuda"),
                      n_chunks_dst=torch.zeros_like(cnt))
            kw["v_dst"] = kw["k_dst"]
        tq.evict_mass(k_codec=kc, v_codec=kc, k_rec=r, v_rec=r, mass=m, n_chunks=cnt, max_chunks=n, keep_chunks=keep,
                      kept=kept, **kw)
        best = torch.sort(mass[0, 0, 0], descending=True, stable=True).indices[:128 * keep].sort().values
        assert torch.equal(kept[0, 0, 0].long(), best)
        out = kw.get("k_dst", r)[0, 0, 0, :keep]
        rows = rec[0, 0, 0, :, :1024].reshape(-1, 8)[best].reshape(keep, 1024)
        assert torch.equal(out[:, :1024], rows)
        assert torch.equal(out[:, 1024:], rec[0, 0, 0, :, 1024:].reshape(-1, 4)[best].reshape(keep, 512))
        assert torch.equal(kw.get("mass_dst", m)[0, 0, 0, :128 * keep], mass[0, 0, 0][best])


@pytest.mark.parametrize("T", [0.0, 2.0])
@pytest.mark.parametrize("in_place", [False, True])
def test_captured_and_replayed(tq, orc, in_place, T):
    """A captured call, replayed after the weights and counters have changed, does what a fresh call does."""
    import torch
    c = Cache(tq, orc, B=2, Hkv=2, d=128, kb=4, vb=3, n=9, tail=33, T=T, seed=41)
    rec0 = {w: c.rec[w].clone() for w in "kv"}
    masses = [torch.from_numpy(_mass(c, kind, s)).cuda() for kind, s in (("spread", 1), ("ties", 2))]
    counts = [torch.tensor([x], dtype=torch.int32, device="cuda") for x in ([9, 4], [7, 9])]

    def buffers():
        b = dict(rec={w: rec0[w].clone() for w in "kv"}, mass=masses[0].clone(), n=counts[0].clone())
        if in_place:
            return b, dict()
        d = dict(k_dst=torch.zeros_like(rec0["k"][:, :, :, :5]).contiguous(), mass_dst=torch.zeros_like(masses[0]),
                 v_dst=torch.zeros_like(rec0["v"][:, :, :, :5]).contiguous(), n_chunks_dst=torch.zeros_like(counts[0]))
        return b, d

    def call(b, d, ws=None):
        return tq.evict_mass(k_codec=c.kc, v_codec=c.vc, k_rec=b["rec"]["k"], v_rec=b["rec"]["v"], mass=b["mass"],
                             n_chunks=b["n"], max_chunks=9, keep_chunks=5, tail_len=c.d_len, max_tail=33, sink=3, recent=50,
                             workspace=ws, **d)

    def results(b, d):
        return [d["k_dst"], d["v_dst"], d["mass_dst"], d["n_chunks_dst"]] if d else [*b["rec"].values(), b["mass"], b["n"]]

    def refill(b, d, i):
        for w in "kv":
            b["rec"][w].copy_(rec0[w])
        b["mass"].copy_(masses[i])
        b["n"].copy_(counts[i])
        for x in d.values():
            x.zero_()

    b, d = buffers()
    ws = call(b, d)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        call(b, d, ws)
    for i in (0, 1):
        refill(b, d, i)
        g.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in results(b, d)]
        fb, fd = buffers()
        refill(fb, fd, i)
        call(fb, fd)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, results(fb, fd)))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n", [3104, 3207])
def test_streams_longer_than_a_cluster_keeps(tq, in_place, n):
    """More records than a cluster of eight CTAs keeps in shared memory (192 KB each): the weights are read again in
    every pass; the last CTA has fewer records, or all have the same number."""
    import torch
    keep, d = 1500, 64
    kc = tq.tq_make_codebook(1, d)
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    rec = torch.randint(0, 256, (1, 1, 1, n, kc.record_bytes), dtype=torch.uint8, device="cuda", generator=g)
    mass = 1.0 + torch.rand((1, 1, 1, 128 * n + 77), device="cuda", generator=g) * 2.0 ** -12
    mass[..., 5:128 * n:3] = mass[..., 5:6]  # a third of the weights are equal
    cnt = torch.full((1, 1), n, dtype=torch.int32, device="cuda")
    ln = torch.full((1, 1), 77, dtype=torch.int32, device="cuda")
    m, r = mass.clone(), rec.clone()
    kept = torch.zeros((1, 1, 1, 128 * keep), dtype=torch.int32, device="cuda")
    kw = {}
    if not in_place:
        kw = dict(k_dst=torch.zeros_like(rec[:, :, :, :keep]), mass_dst=torch.zeros((1, 1, 1, 128 * keep + 77), device="cuda"),
                  n_chunks_dst=torch.zeros_like(cnt))
        kw["v_dst"] = kw["k_dst"]
    tq.evict_mass(k_codec=kc, v_codec=kc, k_rec=r, v_rec=r, mass=m, n_chunks=cnt, max_chunks=n, keep_chunks=keep,
                  kept=kept, tail_len=ln, max_tail=77, sink=9, recent=200, **kw)
    rank = mass[0, 0, 0, :128 * n].clone()
    rank[:9] = rank[-200:] = math.inf
    best = torch.sort(rank, descending=True, stable=True).indices[:128 * keep].sort().values
    assert torch.equal(kept[0, 0, 0].long(), best)
    out = kw.get("k_dst", r)[0, 0, 0, :keep]
    assert torch.equal(out[:, :1024], rec[0, 0, 0, :, :1024].reshape(-1, 8)[best].reshape(keep, 1024))
    assert torch.equal(out[:, 1024:], rec[0, 0, 0, :, 1024:].reshape(-1, 4)[best].reshape(keep, 512))
    md = kw.get("mass_dst", m)[0, 0, 0]
    assert torch.equal(md[:128 * keep], mass[0, 0, 0, best])
    assert torch.equal(md[128 * keep:128 * keep + 77], mass[0, 0, 0, 128 * n:])
    assert torch.all(md[128 * keep + 77:128 * n + 77] == 0)


def test_more_than_a_million_records_remain(tq):
    """2^20 + 2 records of one stream with side lists, into another cache: 134 million tokens remain."""
    import torch
    n, keep, d = (1 << 20) + 5, (1 << 20) + 2, 64
    kc = tq.tq_make_codebook(1, d, outlier_T=3.0, outlier_cap=8)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rec = torch.zeros((1, 1, 1, n, kc.record_bytes), dtype=torch.uint8, device="cuda")
    rec[..., :1536].random_(0, 256, generator=g)  # codes and scales; no entries
    mass = torch.ones((1, 1, 1, 128 * n + 9), device="cuda")
    gone = torch.randperm(128 * n, device="cuda", generator=g)[:128 * (n - keep)]
    mass[0, 0, 0, gone] = 0.0
    cnt = torch.full((1, 1), n, dtype=torch.int32, device="cuda")
    ln = torch.full((1, 1), 9, dtype=torch.int32, device="cuda")
    dst = torch.zeros((1, 1, 1, keep, kc.record_bytes), dtype=torch.uint8, device="cuda")
    mass_dst = torch.zeros((1, 1, 1, 128 * keep + 9), device="cuda")
    n_dst = torch.zeros_like(cnt)
    kept = torch.zeros((1, 1, 1, 128 * keep), dtype=torch.int32, device="cuda")
    tq.evict_mass(k_codec=kc, k_rec=rec, v_rec=rec, mass=mass, n_chunks=cnt, max_chunks=n, keep_chunks=keep, kept=kept,
                  tail_len=ln, max_tail=9, k_dst=dst, v_dst=dst, mass_dst=mass_dst, n_chunks_dst=n_dst)
    assert int(n_dst) == keep and torch.all(mass_dst == 1)
    best = mass[0, 0, 0, :128 * n].nonzero().view(-1)
    assert torch.equal(kept[0, 0, 0].long(), best)
    for lo, hi, row in ((0, 1024, 8), (1024, 1536, 4)):
        rows = rec[0, 0, 0, :, lo:hi].reshape(-1, row)[best].view(keep, hi - lo)
        assert torch.equal(dst[0, 0, 0, :, lo:hi], rows)
    assert not dst[0, 0, 0, :, 1536:1664].any()
