"""The calls for a part of a long cache together, as a server runs them: tokens
appended with norms and rotation, aged into records, the records bounded,
chosen and attended; against the same steps in 64 bits on the host."""
import math

import numpy as np
import pytest

import synth
import tq_testlib as tl
from cache_cases import ocodec
from test_gpu_append import _turned
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
