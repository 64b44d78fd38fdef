"""The calls for a part of a long cache together, as a server runs them: tokens
appended with norms and rotation, aged into records, the records bounded,
chosen and attended; against the same steps in 64 bits on the host."""
import math

import numpy as np
import pytest

import synth
import tq_testlib as tl
from cache_cases import Cache, ocodec, queries
from test_gpu_append import _turned
from test_gpu_key_bounds import at, check, place
from test_gpu_select import want as wanted

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


@pytest.mark.parametrize("d,G,paged", [(128, 3, False), (64, 8, True), (256, 2, False)])
def test_append_age_bound_choose_attend(tq, orc, d, G, paged):
    import torch
    B, Hkv, kb, vb, cap, recs, keep = 2, 2, 4, 3, 800, 10, 3
    Hq = Hkv * G
    kc, vc = tq.tq_make_codebook(kb, d), tq.tq_make_codebook(vb, d)
    zeros = lambda *s, **k: torch.zeros(s, device="cuda", **k)  # noqa: E731
    lead = (1, B * recs + 1, Hkv) if paged else (1, B, Hkv, recs)
    table, perm = None, None
    if paged:
        perm = np.random.default_rng(1).permutation(B * recs + 1)[: B * recs].reshape(B, recs).astype(np.int32)
        table = torch.from_numpy(perm).cuda()
    krec, vrec = zeros(*lead, kc.record_bytes, dtype=torch.uint8), zeros(*lead, vc.record_bytes, dtype=torch.uint8)
    bounds = torch.full((*lead, 2, d), math.nan, dtype=torch.bfloat16, device="cuda")
    ring = {w: zeros(1, B, Hkv, cap, d, dtype=torch.bfloat16) for w in "kv"}
    cnt = {w: zeros(1, B, dtype=torch.int32) for w in ("n", "start", "len", "bounded")}
    freq = (10000.0 ** (-np.arange(d // 4) / (d // 4))).astype(np.float32)
    wt = {s: torch.from_numpy(np.random.default_rng(i).normal(1, 0.2, d).astype(np.float32)).cuda() for i, s in enumerate("qk")}
    norm = tq.make_head_norm(q_weight=wt["q"] * (1.5 / math.sqrt(d)), k_weight=wt["k"])
    done = np.zeros(B, int)

    def cached(b, which):
        """float64 keys or values [Hkv][tokens][d] as the device holds them, in order."""
        n, s, ln = (int(cnt[w][0, b]) for w in ("n", "start", "len"))
        rec, c = (krec, kc) if which == "k" else (vrec, vc)
        rec = rec[0, b] if table is None else rec[0, perm[b].astype(np.int64)].transpose(0, 1)
        at = (s + np.arange(ln)) % cap
        out = []
        for h in range(Hkv):
            old = orc.decode_records(rec[h].cpu().numpy(), 128 * n, ocodec(orc, c)) if n else np.zeros((0, d))
            out.append(np.concatenate([old, synth.bf16_bits_to_f32(tl.bf16_tensor_bits(ring[which][0, b, h]))[at]]))
        return np.stack(out)

    for step, (T, qb) in enumerate(((600, 64), (1, 1), (5, 1), (230, 100), (2, 2))):
        lens = np.array([T, max(1, T - 30 * step)])
        x = tl.to_bf16_tensor(synth.gaussian_bf16((1, B, T, Hq + 2 * Hkv, d), 100 + step), "cuda")
        pos = np.stack([np.arange(T) + done[b] for b in range(B)])[None]
        q = torch.zeros((1, B, T, Hq, d), dtype=torch.bfloat16, device="cuda")
        q_lens = torch.from_numpy(lens.astype(np.int32)).cuda()
        before = {b: cached(b, "k").shape[1] for b in range(B)}
        tq.tq_norm_append(tq.make_append_args(
            q=x[..., :Hq, :], k=x[..., Hq:Hq + Hkv, :], v=x[..., Hq + Hkv:, :], q_out=q, k_tail=ring["k"],
            v_tail=ring["v"], tail_start=cnt["start"], tail_len=cnt["len"], q_lens=q_lens,
            positions=torch.from_numpy(pos.astype(np.int32)).cuda(), inv_freq=torch.from_numpy(freq).cuda()), norm)
        xf = synth.bf16_bits_to_f32(tl.bf16_tensor_bits(x)).astype(np.float64)[0]
        for b in range(B):  # the new keys
            k = xf[b, : lens[b], Hq:Hq + Hkv]
            k = k * wt["k"].cpu().numpy() / np.sqrt((k ** 2).mean(-1, keepdims=True) + 1e-6)
            z, size = _turned(k, pos[:, b, : lens[b]], freq, [0] * len(freq), 0, False, 1.0)
            e = np.abs(cached(b, "k")[:, before[b]:].transpose(1, 0, 2) - z)
            assert np.all(e <= 2.0 ** -8 * np.abs(z) + 2.0 ** -19 * (size + np.abs(z)))
        done += lens
        # the queries read what was there before this step's tokens age
        n_max = recs
        nb = -(-T // qb)
        lst, count = zeros(1, B, nb, Hkv, keep, dtype=torch.int32), zeros(1, B, nb, Hkv, dtype=torch.int32)
        common = dict(n_chunks=cnt["n"], tail_len=cnt["len"], max_chunks=n_max, max_tail=cap, q_lens=q_lens, block_table=table)
        tq.select_records(q=q, bounds=bounds, q_block=qb, keep=keep, sink=1, recent=1, list=lst, count=count, **common)
        out = torch.zeros_like(q)
        tq.sparse_attn(k_codec=kc, v_codec=vc, q=q, out=out, scale=1.0, k_rec=krec, v_rec=vrec, k_tail=ring["k"],
                       v_tail=ring["v"], tail_start=cnt["start"], list=lst, count=count, q_block=qb, **common)
        qf = synth.bf16_bits_to_f32(tl.bf16_tensor_bits(q)).astype(np.float64)[0]
        of = synth.bf16_bits_to_f32(tl.bf16_tensor_bits(out)).astype(np.float64)[0]
        bf = synth.bf16_bits_to_f32(tl.bf16_tensor_bits(bounds)).astype(np.float64)[0]
        for b in range(B):
            m, n, ln = int(lens[b]), int(cnt["n"][0, b]), int(cnt["len"][0, b])
            bb = bf[b][:, :n] if table is None else bf[perm[b][:n]].transpose(1, 0, 2, 3)
            w = wanted(qf[b], bb[:, :, 0], bb[:, :, 1], n, ln, m, G, qb, keep, 1, 1)
            np.testing.assert_array_equal(lst[0, b].cpu().numpy(), w)
            k, v = cached(b, "k"), cached(b, "v")
            err2 = ref2 = 0.0
            for h in range(Hkv):
                for r in range(n):  # a bound is one: no key passes it by more than its f32 error
                    kk = k[h, 128 * r:128 * r + 128]
                    off = 2.0 ** -20 * np.linalg.norm(kk, axis=-1).max()
                    assert np.all(bb[h, r, 0] <= kk.min(0) + off) and np.all(bb[h, r, 1] >= kk.max(0) - off)
                for t in range(m):
                    ids = w[t // qb, h]
                    at = np.concatenate([128 * e + np.arange(128) for e in ids[ids >= 0]] +
                                        [np.arange(128 * n, 128 * n + ln - m + t + 1)]).astype(int)
                    for i in range(G):
                        s = k[h][at] @ qf[b, t, h * G + i]
                        p = np.exp(s - s.max())
                        ref = p @ v[h][at] / p.sum()
                        err2 += ((of[b, t, h * G + i] - ref) ** 2).sum()
                        ref2 += (ref ** 2).sum()
            assert np.all(of[b, m:] == 0)
            assert math.sqrt(err2 / ref2) <= 2.0 ** -8, (step, b)
        tq.tq_evict(kc, vc, k_rec=krec, v_rec=vrec, k_tail=ring["k"], v_tail=ring["v"], n_chunks=cnt["n"],
                    tail_start=cnt["start"], tail_len=cnt["len"], window=64, margin=16, max_evict=4, block_table=table)
        tq.key_bounds(k_codec=kc, k_rec=krec, bounds=bounds, n_chunks=cnt["n"], first=cnt["bounded"], max_chunks=recs,
                      max_new=4, block_table=table)
        cnt["bounded"].copy_(cnt["n"])
    assert int(cnt["n"].min()) >= 4


@pytest.mark.parametrize("paged", [False, True])
def test_bounds_and_lists_after_an_eviction_by_weight_and_a_rollback(tq, orc, paged):
    """When bounds expire: all of them after an eviction by weight; from the records that a rollback leaves on, where
    others have been written in the dropped ones' places."""
    import torch
    c = Cache(tq, orc, B=2, Hkv=2, d=128, kb=4, vb=3, n=9, tail=40, cap=700, paged=paged, seed=51, lens=([9, 7], [40, 21]))
    bounds = place(c)
    ring = dict(k_tail=c.ring["k"], v_tail=c.ring["v"])
    counts = dict(n_chunks=c.d_n, tail_start=c.d_start, tail_len=c.d_len)
    recs = dict(k_rec=c.rec["k"], v_rec=c.rec["v"], block_table=c.table)
    q = queries(1, 2, 3, 8, 128, 52)

    def bound(first=None):
        tq.key_bounds(k_codec=c.kc, k_rec=c.rec["k"], bounds=bounds, n_chunks=c.d_n, first=first, max_chunks=9,
                      block_table=c.table)

    def agree():
        """Every record's bounds are those of its keys, and the lists those of its bounds."""
        c.n[:], c.len[:] = c.d_n.cpu().numpy(), c.d_len.cpu().numpy()
        k = c.rec["k"]
        if c.table is not None:
            k = torch.stack([torch.stack([k[0, c.table[b].long()] for b in range(2)])]).transpose(2, 3)
        c._host["k"] = k.contiguous().cpu().numpy()
        lst = torch.zeros((1, 2, 3, 2, 4), dtype=torch.int32, device="cuda")
        tq.select_records(q=tl.to_bf16_tensor(q, "cuda"), bounds=bounds, n_chunks=c.d_n, max_chunks=9, tail_len=c.d_len,
                          max_tail=c.cap, keep=4, sink=1, recent=1, list=lst, count=lst[..., 0].clone(), block_table=c.table)
        qf = synth.bf16_bits_to_f32(q).astype(np.float64)[0]
        for b in range(2):
            n = int(c.n[0, b])
            for h in range(2):
                for r in range(n):
                    check(c, bounds, 0, b, h, r)
            bb = np.array([[at(c, bounds, 0, b, h, r) for r in range(n)] for h in range(2)])
            w = wanted(qf[b], bb[:, :, 0], bb[:, :, 1], n, int(c.len[0, b]), 3, 4, 1, 4, 1, 1)
            np.testing.assert_array_equal(lst[0, b].cpu().numpy(), w)

    bound()
    agree()
    old = bounds.clone()
    mass = torch.rand((1, 2, 2, 9 * 128 + c.cap), device="cuda")
    tq.evict_mass(k_codec=c.kc, v_codec=c.vc, mass=mass, n_chunks=c.d_n, max_chunks=9, tail_len=c.d_len, max_tail=c.cap,
                  keep_chunks=5, sink=4, recent=128, **recs)
    bound()
    assert int(c.d_n.max()) == 5 and not torch.equal(old, bounds)
    agree()
    bounded = c.d_n.clone()
    tq.tq_rollback(c.kc, c.vc, torch.tensor([[2 * 128 + 50, 3 * 128 + 7]], dtype=torch.int32, device="cuda"),
                   max_evict=1, **recs, **ring, **counts)
    assert c.d_n.tolist() == [[2, 3]] and c.d_len.tolist() == [[50, 7]]
    bounded = torch.minimum(bounded, c.d_n)  # (5 would skip the next ones)
    x = tl.to_bf16_tensor(queries(1, 2, 400, 4, 128, 53, gain=5.0), "cuda")
    tq.tq_append(tq.make_append_args(q=None, q_out=None, k=x[..., :2, :], v=x[..., 2:, :],
                                     positions=torch.zeros((1, 2, 400), dtype=torch.int32, device="cuda"),
                                     inv_freq=torch.ones(64, device="cuda"), **ring,
                                     **{w: counts[w] for w in ("tail_start", "tail_len")}))
    tq.tq_evict(c.kc, c.vc, window=0, margin=0, max_evict=4, **recs, **ring, **counts)
    assert c.d_n.tolist() == [[5, 6]]
    bound(bounded)
    agree()
