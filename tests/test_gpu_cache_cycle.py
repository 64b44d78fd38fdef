"""The several-token calls together, as a server runs them: prompts appended and
attended in slices, aged into records, weighed, cut to the heaviest tokens, and
decoded from; against the same steps in 64 bits on the host."""
import math

import numpy as np
import pytest

import synth
import tq_testlib as tl
from cache_cases import ocodec, weights

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


def test_prompt_slices_then_eviction_then_decode(tq, orc):
    import torch
    B, Hkv, G, d, kb, vb = 2, 2, 3, 128, 4, 3
    Hq, cap, recs = Hkv * G, 544, 8
    kc, vc = tq.tq_make_codebook(kb, d), tq.tq_make_codebook(vb, d)
    zeros = lambda *s, **k: torch.zeros(s, device="cuda", **k)  # noqa: E731
    krec = zeros(1, B, Hkv, recs, kc.record_bytes, dtype=torch.uint8)
    vrec = zeros(1, B, Hkv, recs, vc.record_bytes, dtype=torch.uint8)
    ring = {w: zeros(1, B, Hkv, cap, d, dtype=torch.bfloat16) for w in "kv"}
    cnt = {w: zeros(1, B, dtype=torch.int32) for w in ("n", "start", "len")}
    mass = zeros(1, B, Hkv, 128 * recs + cap)
    freq = torch.from_numpy((10000.0 ** (-np.arange(d // 2) / (d // 2))).astype(np.float32)).cuda()
    axis = tq.rope_pair_axis([24, 20, 20], interleaved=True)
    keys = [[np.zeros((Hkv, 0, d))] for _ in range(B)]
    vals = [[np.zeros((Hkv, 0, d))] for _ in range(B)]
    ref_mass = [np.zeros((Hkv, 0)) for _ in range(B)]
    done = np.zeros(B, int)

    def cached(b, which):
        """float64 keys or values as the device holds them, in order."""
        n, s, ln = (int(cnt[w][0, b]) for w in ("n", "start", "len"))
        rec, c = (krec, kc) if which == "k" else (vrec, vc)
        at = (s + np.arange(ln)) % cap
        out = []
        for h in range(Hkv):
            old = orc.decode_records(rec[0, b, h].cpu().numpy(), 128 * n, ocodec(orc, c)) if n else np.zeros((0, d))
            out.append(np.concatenate([old, synth.bf16_bits_to_f32(tl.bf16_tensor_bits(ring[which][0, b, h]))[at]]))
        return np.stack(out)

    for step, T in enumerate((200, 131, 1, 250)):
        lens = np.array([T, max(1, T - 37 * step)])
        bits = synth.gaussian_bf16((1, B, T, Hq + 2 * Hkv, d), 100 + step)
        x = tl.to_bf16_tensor(bits, "cuda")
        x[..., :Hq, :] *= 2.0 / math.sqrt(d)
        pos = np.stack([np.stack([np.arange(T) // (a + 1) + done[b] for b in range(B)]) for a in range(3)])
        q = torch.zeros((1, B, T, Hq, d), dtype=torch.bfloat16, device="cuda")
        q_lens = torch.from_numpy(lens.astype(np.int32)).cuda()
        tq.tq_append(tq.make_append_args(
            q=x[..., :Hq, :], k=x[..., Hq:Hq + Hkv, :], v=x[..., Hq + Hkv:, :], q_out=q, k_tail=ring["k"],
            v_tail=ring["v"], tail_start=cnt["start"], tail_len=cnt["len"], q_lens=q_lens,
            positions=torch.from_numpy(pos.astype(np.int32)).cuda(), inv_freq=freq, pair_axis=axis, mass=mass,
            n_chunks=cnt["n"]))
        done += lens
        out = torch.zeros_like(q)
        cache = dict(k_rec=krec, k_tail=ring["k"], n_chunks=cnt["n"], tail_start=cnt["start"], tail_len=cnt["len"],
                     max_chunks=recs, max_tail=cap, q_lens=q_lens, q=q, scale=1.0)
        tq.prefill_attn(k_codec=kc, v_codec=vc, out=out, v_rec=vrec, v_tail=ring["v"], **cache)
        tq.attn_mass(k_codec=kc, mass=mass, decay=0.75, **cache)
        qf = synth.bf16_bits_to_f32(tl.bf16_tensor_bits(q)).astype(np.float64)
        of = synth.bf16_bits_to_f32(tl.bf16_tensor_bits(out)).astype(np.float64)
        for b in range(B):
            m, k, v = int(lens[b]), cached(b, "k"), cached(b, "v")
            total = k.shape[1]
            ref_mass[b] = np.concatenate([ref_mass[b], np.zeros((Hkv, total - ref_mass[b].shape[1]))], 1) * 0.75
            for h in range(Hkv):
                for i in range(G):
                    w = weights(qf[0, b, :, h * G + i], k[h], m, total, True, 0.0, 1.0)[:m]
                    want = w @ v[h]
                    e = np.linalg.norm(of[0, b, :m, h * G + i] - want) / np.linalg.norm(want)
                    assert e <= 2.0 ** -7.5, (step, b, h, i, e)  # |q||k| / sqrt(d) is about 2 here
                    ref_mass[b][h] += w.sum(0)
            got = mass[0, b, :, :total].cpu().numpy()
            assert np.linalg.norm(got - ref_mass[b]) <= 1e-4 * np.linalg.norm(ref_mass[b])
        tq.tq_evict(kc, vc, k_rec=krec, v_rec=vrec, k_tail=ring["k"], v_tail=ring["v"], n_chunks=cnt["n"],
                    tail_start=cnt["start"], tail_len=cnt["len"], window=64, margin=16, max_evict=4)
    n = cnt["n"].cpu().numpy()[0]
    assert n.max() >= 3
    before = {w: [cached(b, w) for b in range(B)] for w in "kv"}
    got = mass.cpu().numpy()
    tq.evict_mass(k_codec=kc, v_codec=vc, k_rec=krec, v_rec=vrec, mass=mass, n_chunks=cnt["n"], tail_len=cnt["len"],
                  max_chunks=recs, max_tail=cap, keep_chunks=2, sink=4, recent=32)
    assert cnt["n"].cpu().numpy()[0].tolist() == [min(2, int(v)) for v in n]
    q = tl.to_bf16_tensor(synth.gaussian_bf16((1, B, Hq, d), 9, scale=1.5 / math.sqrt(d)), "cuda")
    out = torch.empty((1, B, Hq, d), device="cuda")
    tq.decode_attn(k_codec=kc, v_codec=vc, q=q, out=out, scale=1.0, k_rec=krec, v_rec=vrec, k_tail=ring["k"],
                   v_tail=ring["v"], n_chunks=cnt["n"], tail_start=cnt["start"], tail_len=cnt["len"], max_chunks=recs,
                   max_tail=cap)
    qf = q.float().cpu().numpy().astype(np.float64)[0]
    for b in range(B):
        N = 128 * int(n[b])
        for h in range(Hkv):
            at, m = np.arange(N), got[0, b, h, :N].astype(np.float64)
            safe = (at < 4) | (at >= N - 32)
            stay = np.sort(np.lexsort((at, -m, ~safe))[:256]) if N > 256 else at
            rows = np.concatenate([stay, np.arange(N, before["k"][b].shape[1])])
            k, v = before["k"][b][h][rows], before["v"][b][h][rows]
            for i in range(G):
                w = weights(qf[b, h * G + i][None], k, 1, len(rows), True, 0.0, 1.0)
                assert np.abs(out[0, b, h * G + i].cpu().numpy() - w @ v).max() <= 2e-3
            np.testing.assert_array_equal(mass[0, b, h, :len(rows)].cpu().numpy(), got[0, b, h][rows])
