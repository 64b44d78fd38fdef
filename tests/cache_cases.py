"""Caches and 64-bit references shared by the tests of the several-token calls
(append, prefill attention, accumulated weights, eviction by them).  The
references are plain numpy over the oracle's fp64 decode of the same records."""
from __future__ import annotations

import math

import numpy as np

import synth
import tq_testlib as tl

CHUNK = 128


def ocodec(orc, c):
    return orc.Codec(d=c.head_dim, bits=c.bits, seed=int(c.c.sign_seed), T=float(c.c.outlier_T),
                     cap=int(c.c.outlier_cap) if c.c.outlier_T else 0)


class Cache:
    """A cache of L layers and B sequences of different lengths, and its float64 image."""

    def __init__(self, tq, orc, *, L=1, B=2, Hkv=2, d=128, kb=4, vb=3, n=3, tail=70, cap=None, T=0.0, shared=False,
                 paged=False, seed=0, lens=None):
        import torch
        self.L, self.B, self.Hkv, self.d, self.max_chunks, self.max_tail = L, B, Hkv, d, n, tail
        self.kc = tq.tq_make_codebook(kb, d, sign_seed=1, outlier_T=T)
        self.vc = self.kc if shared else tq.tq_make_codebook(vb, d, sign_seed=1, outlier_T=T)
        self.shared = shared
        g = np.random.default_rng(seed)
        # the first sequence is full, the others hold less (one nothing at all where there are three)
        self.n = g.integers(0, n + 1, (L, B))
        self.len = g.integers(0, tail + 1, (L, B))
        self.n[:, 0], self.len[:, 0] = n, tail
        if B > 2:
            self.n[:, 2], self.len[:, 2] = 0, 0
        if lens is not None:
            self.n[:], self.len[:] = lens
        cap = cap or tail + 13
        self.cap = cap
        self.start = g.integers(0, cap, (L, B))
        units = L * B * Hkv
        kw = dict(lognormal_sigma=0.3, outlier_frac=0.02 if T else 0.0)
        rings = []
        self.rec, self.ring = {}, {}
        for which, codec in (("k", self.kc), ("v", self.vc)):
            if which == "v" and shared:
                self.rec["v"], self.ring["v"] = self.rec["k"], self.ring["k"]
                continue
            rec = torch.zeros((L, B, Hkv, max(n, 1), codec.record_bytes), dtype=torch.uint8, device="cuda")
            if n:
                x = synth.gaussian_bf16((units, n * CHUNK, d), seed + (1 if which == "k" else 2), **kw)
                tq.tq_encode(codec, tl.to_bf16_tensor(x, "cuda"), rec.view(units, max(n, 1), -1))
            self.rec[which] = rec
            ring = synth.gaussian_bf16((L, B, Hkv, cap, d), seed + (3 if which == "k" else 4))
            self.ring[which] = tl.to_bf16_tensor(ring, "cuda")
            rings.append(self.ring[which])
        for ring in rings:  # slots of no token hold NaN: nothing may read them
            for l in range(L):
                for b in range(B):
                    used = (self.start[l, b] + np.arange(self.len[l, b])) % cap
                    free = np.setdiff1d(np.arange(cap), used)
                    ring[l, b][:, torch.from_numpy(free).cuda()] = math.nan
        self.table = None
        self.orc = orc
        self._host = {w: self.rec[w].cpu().numpy() for w in ("k", "v")}
        if paged:
            blocks = B * max(n, 1) + 2
            perm = g.permutation(blocks)[: B * max(n, 1)].reshape(B, max(n, 1)).astype(np.int32)
            pools = {}
            for which in ("k", "v"):
                if which == "v" and shared:
                    pools["v"] = pools["k"]
                    continue
                pool = torch.randint(0, 256, (L, blocks, Hkv, self.rec[which].shape[-1]), dtype=torch.uint8,
                                     device="cuda")
                for b in range(B):
                    for r in range(max(n, 1)):
                        pool[:, int(perm[b, r])] = self.rec[which][:, b, :, r]
                pools[which] = pool
            self.rec = pools
            self.table = torch.from_numpy(perm).cuda()
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
        self.d_n, self.d_len, self.d_start = i32(self.n), i32(self.len), i32(self.start)

    def vectors(self, which, l, b, h):
        """float64 keys or values of a sequence in the order of its tokens."""
        oc = ocodec(self.orc, self.kc if which == "k" else self.vc)
        n = int(self.n[l, b])
        old = (self.orc.decode_records(self._host[which][l, b, h], n * CHUNK, oc) if n
               else np.zeros((0, self.d)))
        at = (self.start[l, b] + np.arange(self.len[l, b])) % self.cap
        new = synth.bf16_bits_to_f32(tl.bf16_tensor_bits(self.ring[which][l, b, h]))[at]
        return np.concatenate([np.asarray(old, np.float64), new.astype(np.float64)])

    def kw(self, values=True):
        """Keyword arguments of make_query_args."""
        k = dict(k_rec=self.rec["k"], n_chunks=self.d_n, max_chunks=self.max_chunks, k_tail=self.ring["k"],
                 tail_start=self.d_start, tail_len=self.d_len, max_tail=self.max_tail, block_table=self.table)
        if values:
            k.update(v_rec=self.rec["v"], v_tail=self.ring["v"])
        if self.max_chunks == 0:
            for name in ("k_rec", "v_rec", "n_chunks", "block_table"):
                k.pop(name, None)
        if self.max_tail == 0:
            for name in ("k_tail", "v_tail", "tail_start", "tail_len"):
                k.pop(name, None)
            k["max_tail"] = 0
        return k


def queries(L, B, T, Hq, d, seed, gain=1.5):
    return synth.gaussian_bf16((L, B, T, Hq, d), seed, scale=gain / math.sqrt(d))


def weights(q, k, lens, total, causal, softcap, scale):
    """Softmax weights [T, N] of one query head in float64; rows that see nothing are zero.
    q [T, d], k [N, d] float64."""
    T, N = q.shape[0], k.shape[0]
    x = scale * (q @ k.T)
    if softcap:
        x = softcap * np.tanh(x / softcap)
    t, j = np.arange(T)[:, None], np.arange(N)[None, :]
    seen = (t < lens) & (j < total)
    if causal:
        seen = seen & (j <= total - lens + t)
    w = np.zeros((T, N))
    for i in range(T):
        if seen[i].any():
            e = np.exp(x[i, seen[i]] - x[i, seen[i]].max())
            w[i, seen[i]] = e / e.sum()
    return w
