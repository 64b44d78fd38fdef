"""GPU tests of tq_sparse_attn against softmax attention in 64 bits over the
oracle's decode of the listed records and the ring: head dims, rows on either
side of the kernels' border, bit widths, side lists, pages, ragged batches,
empty lists, entries that name nothing or come twice, splits."""
import math

import numpy as np
import pytest

import synth
import tq_testlib as tl
from cache_cases import CHUNK, Cache, queries

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


def lists(c, T, qb, keep, seed, order="ascending"):
    """Random lists [L][B][blocks][Hkv][keep] of records the sequences hold, -1 behind them; counts."""
    g = np.random.default_rng(seed)
    blocks = -(-T // qb)
    out = np.full((c.L, c.B, blocks, c.Hkv, keep), -1, np.int32)
    cnt = np.zeros((c.L, c.B, blocks, c.Hkv), np.int32)
    for i in np.ndindex(*cnt.shape):
        n = int(c.n[i[0], i[1]])
        m = min(n, keep)
        pick = g.permutation(n)[:m]
        out[i][:m] = np.sort(pick) if order == "ascending" else pick
        cnt[i] = m
    return out, cnt


def run(tq, c, q, ls, qb, lens=None, *, causal=True, softcap=0.0, scale=1.0, splits=0, fill=9.0):
    import torch
    L, B, T, Hq, d = q.shape
    wide = torch.full((L, B, T, Hq + 1, d), fill, dtype=torch.bfloat16, device="cuda")  # a strided output
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
    tq.sparse_attn(k_codec=c.kc, v_codec=c.vc, q=tl.to_bf16_tensor(q, "cuda"), out=wide[..., :Hq, :], scale=scale,
                   softcap=softcap, causal=causal, q_lens=None if lens is None else i32(lens), splits=splits,
                   list=i32(ls[0]), count=i32(ls[1]), q_block=qb, **c.kw())
    torch.cuda.synchronize()
    assert torch.all(wide[..., Hq:, :] == fill)
    return wide[..., :Hq, :]


def reference(c, q, ls, qb, l, b, h, t, hq, m, causal, softcap, scale):
    """Weights, keys and values of one row, float64: (w, k, v) of the tokens it sees."""
    n, ln = int(c.n[l, b]), int(c.len[l, b])
    total = n * CHUNK + ln
    limit = total - m + t + 1 if causal else total
    j = t // qb
    ids = [int(e) for e in ls[0][l, b, j, h][: max(0, int(ls[1][l, b, j, h]))] if 0 <= e < n]
    at = np.concatenate([e * CHUNK + np.arange(CHUNK) for e in ids] + [n * CHUNK + np.arange(ln)]).astype(int)
    at = at[at < limit]
    key = (l, b, h)
    if key not in c.__dict__.setdefault("_vec", {}):
        c._vec[key] = (c.vectors("k", l, b, h), c.vectors("v", l, b, h))
    k, v = (x[at] for x in c._vec[key])
    x = scale * (k @ q)
    if softcap:
        x = softcap * np.tanh(x / softcap)
    if len(at) == 0:
        return np.zeros(0), k, v
    w = np.exp(x - x.max())
    return w / w.sum(), k, v


def check(c, q, ls, qb, got, lens=None, *, causal=True, softcap=0.0, scale=1.0, fill=9.0):
    """The bounds of the several-query attention (its operands' roundings are these, or finer): a score off by
    2^-10 |q| |k| at most, a weight by twice that of itself, the weighted value by 2^-7.5, a record's values in
    the rotated basis by 2^-10 |v|; over everything 2^-8 of the output's norm."""
    L, B, T, Hq, d = q.shape
    G = Hq // c.Hkv
    qf = synth.bf16_bits_to_f32(q).astype(np.float64)
    g = synth.bf16_bits_to_f32(tl.bf16_tensor_bits(got.contiguous())).astype(np.float64)
    err2 = ref2 = 0.0
    for l in range(L):
        for b in range(B):
            m = T if lens is None else int(lens[b])
            assert np.all(g[l, b, m:] == fill)
            for t in range(m):
                for hq in range(Hq):
                    w, k, v = reference(c, qf[l, b, t, hq], ls, qb, l, b, hq // G, t, hq, m, causal, softcap, scale)
                    want = w @ v
                    ds = 2.0 ** -10 * abs(scale) * np.linalg.norm(qf[l, b, t, hq]) * (
                        np.linalg.norm(k, axis=-1).max() if len(k) else 0.0)
                    turned = 2.0 ** -10 * (w @ np.linalg.norm(v, axis=-1))
                    tol = 2.0 ** -8 * np.abs(want) + (np.expm1(2 * ds) + 2.0 ** -7.5) * (w @ np.abs(v)) * 1.01 + turned + 1e-6
                    e = np.abs(g[l, b, t, hq] - want)
                    assert np.all(e <= tol), (l, b, t, hq, float((e / tol).max()))
                    err2 += float((e ** 2).sum())
                    ref2 += float((want ** 2).sum())
    assert math.sqrt(err2) <= 2.0 ** -8 * math.sqrt(ref2) + 1e-6, math.sqrt(err2 / max(ref2, 1e-30))


CASES = {
    "one_token": dict(d=128, G=6, T=1, n=9, keep=4),
    "one_row": dict(d=128, G=1, T=1, n=5, keep=2, Hkv=3),
    "drafted_d64": dict(d=64, G=7, T=5, n=7, keep=3, kb=3, vb=2, B=3, lens=[5, 2, 4]),
    "sixteen_rows": dict(d=128, G=8, T=4, qb=2, n=6, keep=3, kb=4, vb=4),
    "eleven_rows_d64": dict(d=64, G=11, T=2, n=6, keep=3, kb=2, vb=3),
    "seventeen_rows": dict(d=128, G=17, T=2, n=6, keep=3),
    "blocks": dict(d=128, G=4, T=150, qb=64, n=7, keep=3, tail=170, B=3, lens=[150, 0, 70]),
    "blocks_past_a_tile_d64": dict(d=64, G=5, T=130, qb=100, n=6, keep=4, tail=140),
    "one_bit": dict(d=128, G=2, T=2, n=5, keep=2, kb=1, vb=1),
    "one_bit_d64": dict(d=64, G=2, T=2, n=5, keep=2, kb=1, vb=1),
    "two_bits": dict(d=128, G=3, T=2, n=5, keep=3, kb=2, vb=2),
    "three_bits": dict(d=128, G=5, T=3, n=5, keep=3, kb=3, vb=3),
    "three_bits_d64": dict(d=64, G=5, T=3, n=5, keep=3, kb=3, vb=3),
    "four_and_one": dict(d=64, G=3, T=2, n=5, keep=3, kb=4, vb=1),
    "side_lists": dict(d=128, G=4, T=3, T_out=2.0, kb=4, vb=3, n=5, keep=3),
    "side_lists_d64_shared": dict(d=64, G=2, T=4, T_out=1.5, kb=2, shared=True, n=4, keep=2),
    "side_lists_d256": dict(d=256, G=4, T=2, T_out=2.0, kb=4, vb=3, n=4, keep=2),
    "shared": dict(d=128, G=4, T=2, kb=4, shared=True, n=5, keep=2),
    "d256": dict(d=256, G=3, T=5, kb=2, vb=3, n=5, keep=2),
    "d512_mqa": dict(d=512, G=64, T=3, kb=4, shared=True, Hkv=1, n=6, keep=3, B=1),
    "d512_blocks": dict(d=512, G=16, T=9, qb=5, kb=4, vb=2, Hkv=1, n=4, keep=2, lens=[9, 3]),
    "paged": dict(d=128, G=3, T=2, kb=2, vb=3, paged=True, n=6, keep=3, B=3, L=2),
    "paged_blocks": dict(d=128, G=5, T=40, qb=20, paged=True, n=6, keep=3, tail=50),
    "softcap": dict(d=128, G=2, T=3, softcap=4.0, n=5, keep=3),
    "softcap_blocks": dict(d=64, G=8, T=20, qb=10, softcap=4.0, n=5, keep=3),
    "softcap_d256": dict(d=256, G=2, T=3, softcap=4.0, n=5, keep=3),
    "not_causal": dict(d=64, G=4, T=3, causal=False, n=4, keep=2),
    "records_only": dict(d=128, G=2, T=3, tail=0, n=5, keep=2),
    "records_only_blocks": dict(d=128, G=6, T=9, qb=4, tail=0, n=5, keep=2),
    "records_only_d512": dict(d=512, G=4, T=3, tail=0, n=3, keep=2, Hkv=1),
    "queries_in_the_records": dict(d=128, G=3, T=200, n=4, keep=3, tail=60),
    "queries_in_the_records_blocks": dict(d=128, G=3, T=200, qb=50, n=4, keep=3, tail=60),
    "queries_in_the_records_d256": dict(d=256, G=3, T=200, qb=50, n=4, keep=3, tail=60),
    "long_ring": dict(d=128, G=4, T=2, n=2, keep=1, tail=700),
    "long_lists_d64": dict(d=64, G=2, T=2, n=300, keep=290, Hkv=1, lens=[2, 1]),
    "long_lists_blocks_d64": dict(d=64, G=10, T=4, qb=2, n=300, keep=290, Hkv=1, B=1),
    "long_lists_d256": dict(d=256, G=3, T=1, n=270, keep=265, Hkv=1, B=1, kb=2, shared=True),
}


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("name", CASES)
def test_sparse_against_the_formula(tq, orc, name, splits):
    kw = dict(CASES[name])
    G, T, lens, keep, qb = kw.pop("G"), kw.pop("T"), kw.pop("lens", None), kw.pop("keep"), kw.pop("qb", 1)
    causal, softcap, T_out = kw.pop("causal", True), kw.pop("softcap", 0.0), kw.pop("T_out", 0.0)
    c = Cache(tq, orc, T=T_out, seed=3, **kw)
    q = queries(c.L, c.B, T, c.Hkv * G, c.d, 77)
    ls = lists(c, T, qb, keep, 5)
    out = run(tq, c, q, ls, qb, lens, causal=causal, softcap=softcap, splits=splits)
    check(c, q, ls, qb, out, lens, causal=causal, softcap=softcap)


ROUTES = {"few": dict(d=128, G=3, T=3, qb=1), "few_d64": dict(d=64, G=9, T=2, qb=1), "tiles": dict(d=128, G=5, T=9, qb=5),
          "wide": dict(d=256, G=2, T=3, qb=1)}


@pytest.mark.parametrize("name", ROUTES)
def test_lists_in_any_order_with_entries_that_name_nothing_or_come_twice(tq, orc, name):
    r = ROUTES[name]
    c = Cache(tq, orc, B=2, Hkv=2, d=r["d"], kb=4, vb=3, n=5, tail=40, seed=6, lens=([5, 3], [40, 11]))
    q = queries(1, 2, r["T"], 2 * r["G"], r["d"], 7)
    ls = lists(c, r["T"], r["qb"], 6, 8, order="any")
    ls[0][0, 0, 0, 0] = [4, -1, 2, 5, 2, 1 << 30]   # holes, a record past the last, one twice
    ls[1][0, 0, 0, 0] = 6
    ls[0][0, 1, 0, 1] = [-7, 3, 99, -1, 5, 4]       # nothing but the ring
    ls[1][0, 1, 0, 1] = 6
    ls[1][0, 0, 0, 1] = 100                         # past the list's end
    ls[0][0, 0, 0, 1] = [0, 1, 2, 3, 4, -1]
    for splits in (0, 1, 2):
        out = run(tq, c, q, ls, r["qb"], splits=splits)
        check(c, q, ls, r["qb"], out)


@pytest.mark.parametrize("name", ROUTES)
def test_rows_that_see_nothing_are_zero(tq, orc, name):
    """Empty lists and no ring (count 0, or negative, or entries that name nothing, or a cache without records)."""
    import torch
    r = ROUTES[name]
    c = Cache(tq, orc, B=4, Hkv=1, d=r["d"], kb=4, vb=3, n=3, tail=0, seed=9, lens=([3, 3, 3, 0], [0, 0, 0, 0]))
    q = queries(1, 4, r["T"], r["G"], r["d"], 10)
    ls = lists(c, r["T"], r["qb"], 3, 11)
    ls[1][0, 0] = 0
    ls[1][0, 1] = -5
    ls[0][0, 2] = 3
    ls[1][0, 3] = 3
    ls[0][0, 3] = 0
    out = run(tq, c, q, ls, r["qb"])
    assert torch.all(out == 0)


@pytest.mark.parametrize("name", ROUTES)
def test_all_records_are_the_prefill_attention(tq, orc, name):
    import torch
    r = ROUTES[name]
    c = Cache(tq, orc, B=2, Hkv=2, d=r["d"], kb=4, vb=3, n=5, tail=40, seed=12)
    q = queries(1, 2, r["T"], 2 * r["G"], r["d"], 13)
    out = run(tq, c, q, lists(c, r["T"], r["qb"], 5, 14), r["qb"])
    ref = torch.empty_like(out)
    tq.prefill_attn(k_codec=c.kc, v_codec=c.vc, q=tl.to_bf16_tensor(q, "cuda"), out=ref, scale=1.0, **c.kw())
    e = (out.float() - ref.float()).norm() / ref.float().norm()
    assert float(e) <= 2.0 ** -7  # each within 2^-8 of the formula


@pytest.mark.parametrize("name", ROUTES)
def test_a_dominating_token_leaves_the_others_theirs(tq, orc, name):
    """One token of a record with most of the weight (60 to 99.9%, by how far chance takes the other keys along
    the query) and a value of zero: the output is the others'."""
    import torch
    r = ROUTES[name]
    d = r["d"]
    c = Cache(tq, orc, B=1, Hkv=1, d=d, kb=4, vb=4, n=12, tail=0, seed=15)
    off = 128 * d * 4 // 8
    T, G = r["T"], r["G"]
    ls = (np.broadcast_to(np.arange(12, dtype=np.int32), (1, 1, -(-T // r["qb"]), 1, 12)).copy(),
          np.full((1, 1, -(-T // r["qb"]), 1), 12, np.int32))
    # a query along a key: its logit far above the others', whose own are small
    k = c.vectors("k", 0, 0, 0)
    for at, nats in ((5, 14.5), (700, 14.5), (5 + 11 * 128, 16.0)):
        c.rec["v"][0, 0, 0, :, off:off + 512] = tl_scale(c, off)
        c.rec["v"][0, 0, 0, at // 128, off + 4 * (at % 128):off + 4 * (at % 128) + 4] = 0
        c._host["v"] = c.rec["v"].cpu().numpy()
        c.__dict__.pop("_vec", None)
        q = np.zeros((1, 1, T, G, d))
        q[...] = k[at] / np.linalg.norm(k[at]) ** 2 * nats
        qb = synth.f32_to_bf16_bits(q.astype(np.float32))
        out = run(tq, c, qb, ls, r["qb"], causal=False)
        qf = synth.bf16_bits_to_f32(qb).astype(np.float64)
        got = synth.bf16_bits_to_f32(tl.bf16_tensor_bits(out.contiguous())).astype(np.float64)
        w, _, v = reference(c, qf[0, 0, 0, 0], ls, r["qb"], 0, 0, 0, 0, 0, T, False, 0.0, 1.0)
        assert w.max() > 0.5
        want = w @ v
        # the dominating logit's own error, 2^-12 of it (a weight's denominator off by 2^-7.9 at 16 nats at most).
        # Kernels on tcgen05 keep the weights of the tile that holds the token in f16 below 2^-2 for the largest
        # (a scale in (1/2, 1] on top where it is folded in): half a step of f16's subnormals, 2^-25, is 2^-22 of
        # the largest weight then; 128 such roundings, independent and uniform, add up to sqrt(128 / 3) of one,
        # four standard deviations of which are allowed.  The kernel for few rows keeps 11 bits there.
        tile = 0.0 if name.startswith("few") else 4 * math.sqrt(128 / 3) * 2.0 ** -22 * w.max() * np.linalg.norm(v, axis=-1).max()
        e = np.linalg.norm(got[0, 0, 0, 0] - want)
        assert e <= 2.0 ** -7 * np.linalg.norm(want) + tile, (at, e, tile)


def tl_scale(c, off):
    if "_vscale" not in c.__dict__:
        c._vscale = c.rec["v"][0, 0, 0, :, off:off + 512].clone()
    return c._vscale


def test_scales_from_tiny_to_huge(tq, orc):
    """Values of norms 1e-20 .. 1e20 in one list, and zero vectors, in either order: the weights' exponent follows."""
    import torch
    c = Cache(tq, orc, B=1, Hkv=1, d=128, kb=4, vb=4, n=4, tail=5, seed=16)
    off = 128 * 128 * 4 // 8
    sc = c.rec["v"][0, 0, 0, :, off:off + 512].contiguous().view(torch.float32)
    c.rec["v"][0, 0, 0, :, off:off + 512] = (sc * torch.tensor([1e-20, 1.0, 0.0, 1e20], device="cuda")[:, None]).view(torch.uint8)
    c._host["v"] = c.rec["v"].cpu().numpy()
    q = queries(1, 1, 2, 2, 128, 17)
    for order in ([0, 1, 2, 3], [3, 2, 1, 0], [0, 2, 1], [2, 0], [2]):
        ls = (np.full((1, 1, 2, 1, 4), -1, np.int32), np.full((1, 1, 2, 1), len(order), np.int32))
        ls[0][..., :len(order)] = order
        check(c, q, ls, 1, run(tq, c, q, ls, 1, splits=1))


@pytest.mark.parametrize("name", ROUTES)
def test_growing_logits_move_the_reference(tq, orc, name):
    """Keys whose scales grow from record to record, in the list's order and against it."""
    import torch
    r = ROUTES[name]
    d, T, G = r["d"], r["T"], r["G"]
    c = Cache(tq, orc, B=1, Hkv=1, d=d, kb=4, vb=4, n=6, tail=T, seed=18)
    off = 128 * d * 4 // 8
    sc = c.rec["k"][0, 0, 0, :, off:off + 512].contiguous().view(torch.float32)
    c.rec["k"][0, 0, 0, :, off:off + 512] = (sc * torch.tensor([0.1, 1, 3, 6, 9, 12], device="cuda")[:, None]).view(torch.uint8)
    c._host["k"] = c.rec["k"].cpu().numpy()
    q = queries(1, 1, T, G, d, 19)
    qf = synth.bf16_bits_to_f32(q).astype(np.float64)
    for order in (range(6), range(5, -1, -1)):
        blocks = -(-T // r["qb"])
        ls = (np.broadcast_to(np.array(list(order), np.int32), (1, 1, blocks, 1, 6)).copy(), np.full((1, 1, blocks, 1), 6, np.int32))
        got = synth.bf16_bits_to_f32(tl.bf16_tensor_bits(run(tq, c, q, ls, r["qb"], splits=1).contiguous())).astype(np.float64)
        # a logit of up to 60 is off by 2^-12 of itself: 2^-6 of a weight, and so of the output
        for t in range(T):
            for i in range(G):
                w, _, v = reference(c, qf[0, 0, t, i], ls, r["qb"], 0, 0, 0, t, i, T, True, 0.0, 1.0)
                assert np.linalg.norm(got[0, 0, t, i] - w @ v) <= 2.0 ** -5 * np.linalg.norm(w @ v)


@pytest.mark.parametrize("name", ROUTES)
def test_rows_that_are_not_finite(tq, orc, name):
    """A query row of NaN or an infinity, a listed key scale that is not finite: NaN rows, the others as they were;
    a record that no list names, and keys of tokens that a query does not see, may hold anything."""
    import torch
    r = ROUTES[name]
    d, T, G = r["d"], r["T"], r["G"]
    c = Cache(tq, orc, B=1, Hkv=1, d=d, kb=4, vb=4, n=4, tail=30, seed=20)
    q = queries(1, 1, T, G, d, 21)
    blocks = -(-T // r["qb"])
    ls = (np.broadcast_to(np.array([0, 3], np.int32), (1, 1, blocks, 1, 2)).copy(), np.full((1, 1, blocks, 1), 2, np.int32))
    clean = run(tq, c, q, ls, r["qb"])
    for bad in (0x7FC0, 0x7F80, 0xFF80):
        x = q.copy()
        x[0, 0, 1, 0, 9] = bad
        out = run(tq, c, x, ls, r["qb"])
        assert torch.all(out[0, 0, 1, 0].isnan())
        out[0, 0, 1, 0] = clean[0, 0, 1, 0]  # the others: a warp's rows may take another order of roundings beside it
        assert float((out.float() - clean.float()).norm() / clean.float().norm()) <= 2.0 ** -8
    off = 128 * d * 4 // 8
    for value in (math.nan, math.inf):
        word = torch.tensor([value], device="cuda").view(torch.uint8)
        keep = c.rec["k"].clone()
        c.rec["k"][0, 0, 0, 1:3, off:off + 4] = word  # records that no list names
        slot = (int(c.start[0, 0]) + 29) % c.cap
        row = c.ring["k"][0, 0, :, slot].clone()
        c.ring["k"][0, 0, :, slot] = value            # the last token's own key
        out = run(tq, c, q, ls, r["qb"])
        assert torch.equal(out[0, 0, : T - 1], clean[0, 0, : T - 1]) and torch.all(out[0, 0, T - 1].isnan())
        c.ring["k"][0, 0, :, slot] = row
        c.rec["k"][0, 0, 0, 3, off + 40:off + 44] = word
        assert torch.all(run(tq, c, q, ls, r["qb"]).isnan())
        c.rec["k"].copy_(keep)


@pytest.mark.parametrize("name", ROUTES)
def test_entries_that_name_nothing_read_no_other_record(tq, orc, name):
    """Holes in a list beside records that it does not name and that hold NaN and infinities, keys and values; the
    first of a run's entries, the last, and all of them."""
    import torch
    r = ROUTES[name]
    d, T, G = r["d"], r["T"], r["G"]
    c = Cache(tq, orc, B=1, Hkv=1, d=d, kb=4, vb=4, n=5, tail=30, seed=41)
    q = queries(1, 1, T, G, d, 42)
    blocks = -(-T // r["qb"])
    same = lambda e: (np.broadcast_to(np.array(e, np.int32), (1, 1, blocks, 1, len(e))).copy(),  # noqa: E731
                      np.full((1, 1, blocks, 1), len(e), np.int32))
    clean, alone = run(tq, c, q, same([1, 3]), r["qb"], splits=1), run(tq, c, q, same([-1]), r["qb"], splits=1)
    off = 128 * d * 4 // 8
    bad = torch.tensor([math.nan, math.inf, -math.inf, math.nan], device="cuda").view(torch.uint8)
    for w in "kv":
        for x in (0, 2, 4):
            c.rec[w][0, 0, 0, x, off:off + 16] = bad
    for e in ([-1, 1, 3], [1, 9, 3], [-1, 5, 1, 1 << 30, 3, -1, -2, 7]):
        for splits in (0, 1, 2):
            out = run(tq, c, q, same(e), r["qb"], splits=splits)
            assert float((out.float() - clean.float()).norm() / clean.float().norm()) <= 2.0 ** -8
    for splits in (0, 1, 3):
        assert torch.equal(run(tq, c, q, same([-1, 5, -3]), r["qb"], splits=splits), alone)


@pytest.mark.parametrize("scale", [-1.0, 0.0])
@pytest.mark.parametrize("name", ROUTES)
def test_negative_and_zero_scales(tq, orc, name, scale):
    r = ROUTES[name]
    c = Cache(tq, orc, B=1, Hkv=1, d=r["d"], kb=4, vb=2, n=4, tail=30, seed=22)
    q = queries(1, 1, r["T"], r["G"], r["d"], 23)
    ls = lists(c, r["T"], r["qb"], 2, 24)
    check(c, q, ls, r["qb"], run(tq, c, q, ls, r["qb"], scale=scale), scale=scale)


@pytest.mark.parametrize("name", ROUTES)
def test_captured_and_replayed(tq, orc, name):
    import torch
    r = ROUTES[name]
    c = Cache(tq, orc, B=2, Hkv=2, d=r["d"], kb=4, vb=4, n=5, tail=64, seed=25)
    qt = tl.to_bf16_tensor(queries(1, 2, r["T"], 2 * r["G"], r["d"], 26), "cuda")
    ls = [torch.from_numpy(x).cuda() for x in lists(c, r["T"], r["qb"], 3, 27)]
    eager, out = torch.zeros_like(qt), torch.zeros_like(qt)
    tq.sparse_attn(k_codec=c.kc, v_codec=c.vc, q=qt, out=eager, scale=1.0, list=ls[0], count=ls[1], q_block=r["qb"], **c.kw())
    a = tq.make_query_args(q=qt, out=out, scale=1.0, **c.kw())
    rl = tq.make_record_lists(list=ls[0], count=ls[1], q_block=r["qb"])
    ws = torch.empty(tq.tq_sparse_attn_workspace_size(a, rl, c.kc, c.vc), dtype=torch.uint8, device="cuda")
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        tq.tq_sparse_attn(a, rl, c.kc, c.vc, ws)
    for _ in range(2):
        out.zero_()
        ws.fill_(0xFF)  # nothing is left from the call before
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ROUTES)
def test_a_dropped_workspace_is_not_handed_out_under_the_call(tq, orc, name, raw):
    """A call queued on a busy side stream; its workspace is dropped and memory of its size is filled meanwhile."""
    import torch
    r = ROUTES[name]
    c = Cache(tq, orc, B=1, Hkv=2, d=r["d"], kb=4, vb=4, n=16, tail=40, seed=30)
    q = tl.to_bf16_tensor(queries(1, 1, r["T"], 2 * r["G"], r["d"], 31), "cuda")
    ls = [torch.from_numpy(x).cuda() for x in lists(c, r["T"], r["qb"], 12, 32)]
    ref, out = torch.zeros_like(q), torch.zeros_like(q)
    kw = dict(k_codec=c.kc, v_codec=c.vc, q=q, scale=1.0, list=ls[0], count=ls[1], q_block=r["qb"], **c.kw())
    need = tq.sparse_attn(out=ref, **kw).numel()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    tq.sparse_attn(out=out, stream=side.cuda_stream if raw else side, **kw)
    junk = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and len(junk) == 4


@pytest.mark.parametrize("name", ROUTES)
def test_two_calls_at_once(tq, orc, name):
    """Calls of two streams over one cache, each with its own workspace: both as if alone."""
    import torch
    r = ROUTES[name]
    c = Cache(tq, orc, B=2, Hkv=2, d=r["d"], kb=4, vb=3, n=30, tail=64, seed=33)
    qs = [tl.to_bf16_tensor(queries(1, 2, r["T"], 2 * r["G"], r["d"], s), "cuda") for s in (34, 35)]
    ls = [[torch.from_numpy(x).cuda() for x in lists(c, r["T"], r["qb"], 20, s)] for s in (36, 37)]
    call = lambda i, out: tq.sparse_attn(k_codec=c.kc, v_codec=c.vc, q=qs[i], out=out, scale=1.0, list=ls[i][0],  # noqa: E731
                                         count=ls[i][1], q_block=r["qb"], **c.kw())
    alone = [torch.zeros_like(q) for q in qs]
    for i in range(2):
        call(i, alone[i])
    outs = [[torch.zeros_like(qs[i]) for _ in range(8)] for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for k in range(8):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                call(i, outs[i][k])
    torch.cuda.synchronize()
    assert all(torch.equal(o, alone[i]) for i in range(2) for o in outs[i])


@pytest.mark.parametrize("name", ROUTES)
def test_records_past_32_bits_of_a_pool(tq, orc, name):
    """Pages more than 2^32 bytes into their pool."""
    import torch
    r = ROUTES[name]
    c = Cache(tq, orc, B=2, Hkv=1, d=r["d"], kb=4, vb=4, n=4, tail=30, shared=True, paged=True, seed=38)
    q = queries(1, 2, r["T"], r["G"], r["d"], 39)
    ls = lists(c, r["T"], r["qb"], 3, 40)
    near = run(tq, c, q, ls, r["qb"])
    pool = c.rec["k"]
    blocks = (1 << 32) // pool.shape[-1] + 100
    far = torch.empty((1, blocks, 1, pool.shape[-1]), dtype=torch.uint8, device="cuda")
    far[:, -pool.shape[1]:] = pool
    c.rec = dict(k=far, v=far)
    c.table = c.table + (blocks - pool.shape[1])
    assert torch.equal(run(tq, c, q, ls, r["qb"]), near)


def test_lists_of_another_shape_are_refused(tq, orc):
    import torch
    c = Cache(tq, orc, B=2, Hkv=2, d=128, kb=4, vb=4, n=3, tail=9, seed=28)
    q = tl.to_bf16_tensor(queries(1, 2, 4, 4, 128, 29), "cuda")
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    for shape, qb in (((1, 2, 2, 2), 1), ((1, 2, 4, 1), 1), ((1, 1, 4, 2), 1), ((1, 2, 4, 2), 2), ((1, 2, 4, 2), 0)):
        with pytest.raises((ValueError, tq.TqError)):
            tq.sparse_attn(k_codec=c.kc, v_codec=c.vc, q=q, out=torch.empty_like(q), scale=1.0, list=z(*shape, 3),
                           count=z(*shape), q_block=qb, **c.kw())


@pytest.mark.parametrize("splits", [1, 7])
@pytest.mark.parametrize("G,qb,d", [(17, 1, 64), (5, 7, 128), (16, 4, 128), (64, 2, 64), (43, 3, 128), (65, 3, 64), (128, 2, 128),
                                    (43, 7, 64), (65, 8, 64)])
def test_blocks_of_17_to_520_rows(tq, orc, G, qb, d, splits):
    """Blocks whose rows end inside the partials' tiles of 128, or take several; the last one is short."""
    c = Cache(tq, orc, B=2, Hkv=1, d=d, kb=4, vb=3, n=9, tail=40, seed=43, lens=([9, 4], [40, 17]))
    T = 2 * qb + 1
    q = queries(1, 2, T, G, d, 44)
    ls = lists(c, T, qb, 8, 45)
    lens = [T, max(1, qb - 1)]
    check(c, q, ls, qb, run(tq, c, q, ls, qb, lens, splits=splits), lens)
