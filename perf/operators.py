"""Cases of the cache operators that serve prompts and long contexts.

Four operators around the rotated Lloyd-Max cache (records of 128 tokens, a
dense bf16 ring behind them):

  append   rotary positions with several axes on queries and keys, keys and
           values appended to the ring
  prefill  attention of several new tokens per sequence over records and ring
  mass     the attention weight every cached token receives, accumulated
  evict    the records compacted to the tokens of the largest accumulated weight

`run` computes them in plain torch operations, or, where `own` is true, through
the library's entry points.  A case is a dict of sizes; `prepare` draws its
inputs from the seed alone.
"""
import functools
import math

import numpy as np
import torch

own = False

CHUNK = 128
DEV = "cuda"


# ---------------------------------------------------------------- cases
def _append(**kw):
    case = dict(op="append", L=1, B=1, T=1, Hkv=2, G=6, d=128, rot=128, axes=3, adjacent=False, ragged=False,
                shared=False, window=300, far=4096)
    return {**case, **kw}


def _attend(op, **kw):
    case = dict(op=op, L=1, B=1, T=1, Hkv=2, G=6, d=128, kb=4, vb=4, ctx=2048, tail=256, shared=False, causal=True,
                softcap=0.0, ragged=False, paged=False, gain=2.0)
    return {**case, **kw}


def _evict(**kw):
    case = dict(op="evict", L=1, B=1, Hkv=2, d=128, kb=4, vb=4, ctx=4096, keep=2048, sink=4, recent=128, tail=200,
                shared=False, ragged=False, paged=False)
    return {**case, **kw}


def listed():
    return [
        # one new token of one sequence: the latency of a decode step's smallest call
        _append(name="append_token", T=1, Hkv=2, G=6, far=2048),
        # one new token for each of 32 sequences of a served batch, three axes
        _append(name="append_batch32", B=32, T=1, Hkv=8, G=4, far=32768),
        # prompts with images, padded to one length, of which the last rows are not tokens
        _append(name="append_prompts", B=4, T=4099, Hkv=8, G=4, ragged=True, far=262144),
        # verification of five drafted tokens against a short cache
        _attend("prefill", name="prefill_verify", T=5, Hkv=2, G=6, ctx=2048, kb=3, vb=2, tail=133),
        # a slice of a long prompt: 1024 tokens over a 4-bit cache of 32768
        _attend("prefill", name="prefill_slice", T=1024, Hkv=8, G=4, ctx=32768, kb=4, vb=4, tail=1280),
        # ragged prompts of a batch at head dim 64, 3-bit keys and 2-bit values, paged
        _attend("prefill", name="prefill_ragged_d64", B=6, T=257, Hkv=4, G=7, d=64, ctx=6144, kb=3, vb=2, tail=401,
                ragged=True, paged=True),
        # one key/value head for 64 query heads, keys and values in one record
        _attend("prefill", name="prefill_mqa_d512", T=64, Hkv=1, G=64, d=512, ctx=16384, tail=272, shared=True),
        # weights of one decode step, one sequence
        _attend("mass", name="mass_token", T=1, Hkv=2, G=6, ctx=2048, kb=3, vb=2, tail=256),
        # weights of one decode step of a served batch
        _attend("mass", name="mass_batch32", B=32, T=1, Hkv=8, G=4, ctx=32768, kb=4, vb=3, tail=144),
        # the last 32 tokens of a long prompt vote on what to keep
        _attend("mass", name="mass_window", T=32, Hkv=8, G=4, ctx=131072, kb=3, vb=2, tail=1024),
        # a short cache cut to half
        _evict(name="evict_half", ctx=4096, keep=2048, kb=3, vb=2),
        # every sequence of a served batch cut to a quarter
        _evict(name="evict_batch32", B=32, Hkv=8, ctx=32768, keep=8192, kb=4, vb=3, tail=144),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "prefill", "mass", "evict"])
    d = rng.choice([64, 128, 128, 256, 512])
    kb, vb = rng.choice([(4, 4), (4, 3), (3, 2), (2, 2), (1, 4), (3, 3)])
    Hkv = 1 if d == 512 else rng.choice([1, 2, 3, 4, 8])
    ragged, paged = rng.random() < 0.5, rng.random() < 0.3
    if op == "append":
        T = _log(rng, 1, 4099)
        B = _log(rng, 1, max(1, min(48, 8192 // T)))
        G = rng.choice([1, 4, 5, 6, 7, 8]) if d < 512 else 16
        rot = rng.choice([d, d // 2, 32])
        return _append(B=B, T=T, Hkv=Hkv, G=G, d=d, rot=rot, axes=rng.choice([1, 2, 3, 4]),
                       adjacent=rng.random() < 0.4, ragged=ragged and T > 1, shared=d == 512 and rng.random() < 0.5,
                       window=rng.randrange(1, 400), far=_log(rng, 1000, 1000000))
    shared = d == 512 and rng.random() < 0.7
    if shared:
        kb = vb = 4
    if op == "evict":
        ctx = CHUNK * _log(rng, 2, 512)
        B = _log(rng, 1, max(1, min(32, 2097152 // (ctx * Hkv * (d // 64)))))
        keep = CHUNK * rng.randrange(1, ctx // CHUNK)
        return _evict(B=B, Hkv=Hkv, d=d, kb=kb, vb=vb, ctx=ctx, keep=keep, sink=rng.randrange(0, 65),
                      recent=rng.choice([0, 17, 63]), tail=rng.randrange(0, 400), shared=shared, ragged=ragged,
                      paged=paged)
    T = _log(rng, 1, 700) if op == "prefill" else _log(rng, 1, 48)
    G = rng.choice([1, 4, 5, 6, 7, 8]) if d < 512 else rng.choice([16, 64])
    if d == 512:
        T = min(T, 96)
    ctx = CHUNK * _log(rng, 1, 256)
    B = _log(rng, 1, max(1, min(16, (1 << 31) // (ctx * Hkv * G * T * d // 64))))
    return _attend(op, B=B, T=T, Hkv=Hkv, G=G, d=d, kb=kb, vb=vb, ctx=ctx,
                   tail=max(T, rng.randrange(1, 900)), shared=shared, causal=rng.random() < 0.8,
                   softcap=rng.choice([0.0, 0.0, 20.0]), ragged=ragged, paged=paged, gain=rng.choice([1.0, 2.0, 3.0]))


# ---------------------------------------------------------------- the codec's constants
@functools.lru_cache(maxsize=None)
def _unit_table(bits):
    """Centroids of the Lloyd-Max quantiser of N(0, 1) with 2^bits levels (float64)."""
    n = 1 << bits
    c = np.linspace(-2.0, 2.0, n) if n > 2 else np.array([-0.8, 0.8])
    phi = lambda x: math.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)  # noqa: E731
    cdf = lambda x: 0.5 * math.erfc(-x / math.sqrt(2))  # noqa: E731
    for _ in range(20000):
        t = 0.5 * (c[1:] + c[:-1])
        f = np.array([0.0, *map(phi, t), 0.0])
        F = np.array([0.0, *map(cdf, t), 1.0])
        new = (f[:-1] - f[1:]) / (F[1:] - F[:-1])
        new = 0.5 * (new - new[::-1])
        if np.max(np.abs(new - c)) < 1e-14:
            break
        c = new
    return new


def _signs(d, seed=1):
    """+-1 per coordinate: the top bit of SplitMix64's outputs."""
    m, out, z = (1 << 64) - 1, [], seed
    for _ in range(d):
        z = (z + 0x9E3779B97F4A7C15) & m
        x = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & m
        x = ((x ^ (x >> 27)) * 0x94D049BB133111EB) & m
        out.append(-1.0 if (x ^ (x >> 31)) >> 63 else 1.0)
    return torch.tensor(out, device=DEV)


def _hadamard(d):
    h = torch.ones((1, 1), device=DEV)
    while h.shape[0] < d:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def _codec(d, bits):
    return dict(bits=bits, cent=torch.from_numpy((_unit_table(bits) / math.sqrt(d)).astype(np.float32)).to(DEV),
                rot=_hadamard(d) * _signs(d) / math.sqrt(d))  # decoded = scale * (code values @ rot)


def _rec_bytes(d, bits):
    return CHUNK * d * bits // 8 + 4 * CHUNK


def _records(lead, n_rec, d, bits, gen):
    """Records of Gaussian vectors: Gaussian rotated coordinates quantised, log-normal norms."""
    edges = torch.from_numpy(0.5 * (_unit_table(bits)[1:] + _unit_table(bits)[:-1])).float().to(DEV)
    rows = math.prod(lead) * n_rec * CHUNK
    out = torch.empty((math.prod(lead) * n_rec, _rec_bytes(d, bits)), dtype=torch.uint8, device=DEV)
    step = CHUNK * max(1, (1 << 25) // (CHUNK * d))
    for r in range(0, rows, step):
        m = min(step, rows - r)
        codes = torch.bucketize(torch.randn((m, d), generator=gen, device=DEV), edges, out_int32=True)
        if bits == 3:
            w = (codes.view(m, d // 8, 8) << (3 * torch.arange(8, device=DEV, dtype=torch.int32))).sum(-1)
            by = torch.stack([w & 255, (w >> 8) & 255, w >> 16], -1)
        else:
            k = 8 // bits
            by = (codes.view(m, d // k, k) << (bits * torch.arange(k, device=DEV, dtype=torch.int32))).sum(-1)
        norm = math.sqrt(d) * torch.exp(0.25 * torch.randn(m, generator=gen, device=DEV))
        a, b = r // CHUNK, (r + m) // CHUNK
        out[a:b, : CHUNK * d * bits // 8] = by.to(torch.uint8).view(b - a, -1)
        out[a:b, CHUNK * d * bits // 8:] = norm.view(b - a, CHUNK).view(torch.uint8)
    return out.view(*lead, n_rec, -1)


# ---------------------------------------------------------------- inputs
def _bf16(shape, gen, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * scale).to(torch.bfloat16)


def _ints(v, shape=None):
    t = torch.as_tensor(v, dtype=torch.int32, device=DEV)
    return t if shape is None else t.expand(shape).contiguous()


def _positions(c, gen):
    """[axes][B][T]: running text with one picture in the middle, whose patches share a time and have a row and a column."""
    B, T, n = c["B"], c["T"], c["axes"]
    at = torch.arange(T, device=DEV)
    base = torch.randint(0, c["far"], (B, 1), generator=gen, device=DEV)
    first, size = T // 4, T // 2
    inside = (at >= first) & (at < first + size)
    k, w = at - first, max(1, math.isqrt(max(1, size)))
    axes = [at, torch.where(inside, first + k // w, at), torch.where(inside, first + k % w, at), at // 2]
    if n > 1:
        axes[0] = torch.where(inside, first, at)
    return torch.stack([(a + base).to(torch.int32) for a in axes[:n]]).contiguous()


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    host = np.random.RandomState(int(seed) % (1 << 31))
    L, B, Hkv, d = c["L"], c["B"], c["Hkv"], c["d"]
    s = dict(case=c)
    if c["op"] == "append":
        T, G = c["T"], c["G"]
        Hq, half = Hkv * G, c["rot"] // 2
        # one projection's output holds queries, keys and values of a token side by side
        s["qkv"] = _bf16((L, B, T, (Hq + 2 * Hkv) * d), gen)
        heads = s["qkv"].view(L, B, T, Hq + 2 * Hkv, d)
        s["q"], s["k"], s["v"] = heads[..., :Hq, :], heads[..., Hq:Hq + Hkv, :], heads[..., Hq + Hkv:, :]
        s["q_out"] = torch.zeros((L, B, T, Hq, d), dtype=torch.bfloat16, device=DEV)
        cap = c["window"] + T + 37
        s["k_tail"] = _bf16((L, B, Hkv, cap, d), gen)
        s["v_tail"] = None if c["shared"] else _bf16((L, B, Hkv, cap, d), gen)
        s["start"] = _ints(host.randint(0, cap, (L, B)))
        s["len"] = _ints(host.randint(0, c["window"] + 1, (L, B)))
        s["len_out"] = torch.zeros_like(s["len"])
        s["lens"] = _ints(host.randint(T // 2, T + 1, B)) if c["ragged"] else None
        s["pos"] = _positions(c, gen)
        s["freq"] = (10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)).float()
        # each axis turns its own run of frequencies
        s["axis"] = [min(c["axes"] - 1, p * c["axes"] // half) for p in range(half)]
        s["rot_start"] = d - c["rot"]
        return s
    n_max = c["ctx"] // CHUNK
    n = host.randint(n_max // 2, n_max + 1, (L, B)) if c["ragged"] else np.full((L, B), n_max)
    s["n"] = _ints(n)
    for key, bits in (("k", c["kb"]), ("v", c["vb"])):
        s[key + "_codec"] = _codec(d, bits)
    if c["paged"]:  # blocks of a pool, in no order
        pool = B * n_max + 3
        s["table"] = _ints(host.permutation(pool)[: B * n_max].reshape(B, n_max))
        lead = (L, pool)
        shape = lambda bits: _records(lead, Hkv, d, bits, gen)  # noqa: E731
    else:
        s["table"] = None
        shape = lambda bits: _records((L, B, Hkv), n_max, d, bits, gen)  # noqa: E731
    s["k_rec"] = shape(c["kb"])
    s["v_rec"] = s["k_rec"] if c["shared"] else shape(c["vb"])
    if c["op"] == "evict":
        total = c["ctx"] + c["tail"]
        s["mass"] = torch.exp(2.0 * torch.randn((L, B, Hkv, total), generator=gen, device=DEV))
        s["mass"] *= (torch.rand((L, B, Hkv, total), generator=gen, device=DEV) > 0.1)  # some tokens got nothing
        s["tail_len"] = _ints(c["tail"], (L, B))
        kc = c["keep"] // CHUNK
        s["k_dst"] = torch.zeros((L, B, Hkv, kc, _rec_bytes(d, c["kb"])), dtype=torch.uint8, device=DEV)
        s["v_dst"] = s["k_dst"] if c["shared"] else torch.zeros((L, B, Hkv, kc, _rec_bytes(d, c["vb"])),
                                                                dtype=torch.uint8, device=DEV)
        s["mass_dst"] = torch.zeros((L, B, Hkv, c["keep"] + c["tail"]), device=DEV)
        s["kept"] = torch.full((L, B, Hkv, c["keep"]), -1, dtype=torch.int32, device=DEV)
        s["n_dst"] = torch.zeros((L, B), dtype=torch.int32, device=DEV)
        return s
    T, Hq = c["T"], Hkv * c["G"]
    s["q"] = _bf16((L, B, T, Hq, d), gen, c["gain"] / math.sqrt(d))
    cap = c["tail"] + 19
    s["k_tail"] = _bf16((L, B, Hkv, cap, d), gen)
    s["v_tail"] = s["k_tail"] if c["shared"] else _bf16((L, B, Hkv, cap, d), gen)
    s["start"] = _ints(host.randint(0, cap, (L, B)))
    lens = host.randint(T // 2, T + 1, B) if c["ragged"] else np.full(B, T)
    s["lens"] = _ints(lens) if c["ragged"] else None
    low = np.minimum(lens, c["tail"])[None, :]
    s["len"] = _ints(np.maximum(low, host.randint(0, c["tail"] + 1, (L, B))) if c["ragged"] else c["tail"], (L, B))
    if c["op"] == "prefill":
        s["out"] = torch.zeros((L, B, T, Hq, d), dtype=torch.bfloat16, device=DEV)
    else:
        # what steps of this kind have left: the decayed sum's steady state, spread over the tokens
        level = 2 * c["G"] * T / (1 - DECAY) / (c["ctx"] + c["tail"])
        s["mass"] = level * torch.rand((L, B, Hkv, c["ctx"] + c["tail"]), generator=gen, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms
def _rows(x, order):
    """Batched row gather: x [..., n, w], order [..., m] -> [..., m, w]."""
    return torch.gather(x, -2, order.long()[..., None].expand(*order.shape, x.shape[-1]))


def _contiguous(rec, table, heads):
    """[L][B][Hkv][n][bytes] of a pool [L][blocks][Hkv][bytes]."""
    return rec if table is None else rec[:, table.long()].permute(0, 1, 3, 2, 4)


def _unpack(rec, d, bits):
    """Codes [..., n * 128, d] and scales [..., n * 128] of records [..., n, bytes]."""
    lead, cut = rec.shape[:-2], CHUNK * d * bits // 8
    by = rec[..., :cut].reshape(*lead, -1, d * bits // 8).to(torch.int32)
    if bits == 3:
        g = by.view(*by.shape[:-1], d // 8, 3)
        word, k = g[..., 0] | (g[..., 1] << 8) | (g[..., 2] << 16), 8
    else:
        word, k = by, 8 // bits
    codes = (word[..., None] >> (bits * torch.arange(k, device=rec.device, dtype=torch.int32))) & ((1 << bits) - 1)
    return codes.reshape(*by.shape[:-1], d), rec[..., cut:].contiguous().view(torch.float32).reshape(*lead, -1)


def _decoded(rec, codec, d):
    codes, scale = _unpack(rec, d, codec["bits"])
    return codec["cent"][codes.long()] @ codec["rot"] * scale[..., None]


def _ring(x, start):
    """The ring's tokens in order: x [L][B][Hkv][cap][d]."""
    cap = x.shape[3]
    at = (start.long()[..., None] + torch.arange(cap, device=x.device)) % cap
    return _rows(x, at[:, :, None, :].expand(*x.shape[:4]))


def _cached(s, which):
    """Keys or values [L][B][Hkv][n * 128 + tail][d] in f32: decoded records, then the ring."""
    c = s["case"]
    old = _decoded(_contiguous(s[which + "_rec"], s["table"], c["Hkv"]), s[which + "_codec"], c["d"])
    return torch.cat([old, _ring(s[which + "_tail"], s["start"])[..., : c["tail"], :].float()], 3)


def _weights(s, keys):
    """Softmax weights [L][B][Hkv][G][T][n * 128 + tail]; rows of no token or without any key are zero."""
    c = s["case"]
    L, B, T, Hkv, G, d, ctx = (c[k] for k in ("L", "B", "T", "Hkv", "G", "d", "ctx"))
    at = torch.arange(ctx + c["tail"], device=DEV)
    n, ln = 128 * s["n"].long()[..., None], s["len"].long()[..., None]
    index = torch.where(at < ctx, at, at - ctx + n)                 # the token's place in its sequence
    there = torch.where(at < ctx, at < n, at - ctx < ln)            # [L][B][columns]
    lens = torch.full((B,), T, device=DEV) if s["lens"] is None else s["lens"].long()
    t = torch.arange(T, device=DEV)
    seen = there[:, :, None, :] & (t < lens[:, None])[None, :, :, None]
    if c["causal"]:
        last = (n + ln - lens[:, None]) + t                         # [L][B][T]
        seen = seen & (index[:, :, None, :] <= last[..., None])
    q = s["q"].float().view(L, B, T, Hkv, G, d).permute(0, 1, 3, 4, 2, 5)
    x = (q.reshape(L, B, Hkv, G * T, d) @ keys.transpose(-1, -2)).view(L, B, Hkv, G, T, -1)
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    x = x.masked_fill(~seen[:, :, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(x - top)
    return p / p.sum(-1, keepdim=True).clamp_min(1e-30)


def _plain_prefill(s):
    c = s["case"]
    L, B, T, Hkv, G, d = (c[k] for k in ("L", "B", "T", "Hkv", "G", "d"))
    w = _weights(s, _cached(s, "k")).view(L, B, Hkv, G * T, -1)
    o = (w @ _cached(s, "v")).view(L, B, Hkv, G, T, d).permute(0, 1, 4, 2, 3, 5).reshape(L, B, T, Hkv * G, d)
    if s["lens"] is None:
        s["out"].copy_(o)
    else:
        tokens = torch.arange(T, device=DEV) < s["lens"][:, None]
        s["out"].copy_(torch.where(tokens[None, :, :, None, None], o.to(torch.bfloat16), s["out"]))
    return s["out"]


DECAY = 0.96875


def _plain_mass(s):
    c = s["case"]
    ctx, m = c["ctx"], s["mass"]
    got = _weights(s, _cached(s, "k")).sum((3, 4))                  # [L][B][Hkv][columns]
    at = torch.arange(ctx + c["tail"], device=DEV)
    n, ln = 128 * s["n"].long()[..., None], s["len"].long()[..., None]
    column = torch.where(at < n, at, (at - n + ctx).clamp_max(ctx + c["tail"] - 1))  # of the token at place `at`
    got = torch.gather(got, 3, column[:, :, None].expand_as(got))
    m.copy_(torch.where((at < n + ln)[:, :, None], DECAY * m + got, m))
    return m


def _rotated(x, s, cos, sin):
    """x [L][B][T][heads][d] with the pairs of its rotated coordinates turned."""
    c = s["case"]
    a, half = s["rot_start"], c["rot"] // 2
    r = x[..., a: a + c["rot"]].float()
    x0, x1 = (r[..., 0::2], r[..., 1::2]) if c["adjacent"] else (r[..., :half], r[..., half:])
    y0, y1 = x0 * cos - x1 * sin, x1 * cos + x0 * sin
    y = torch.stack([y0, y1], -1).flatten(-2) if c["adjacent"] else torch.cat([y0, y1], -1)
    return torch.cat([x[..., :a].float(), y, x[..., a + c["rot"]:].float()], -1).to(torch.bfloat16)


def _plain_append(s):
    c = s["case"]
    L, B, T = c["L"], c["B"], c["T"]
    pos = s["pos"][torch.tensor(s["axis"], device=DEV)]             # [pairs][B][T]
    angle = pos.permute(1, 2, 0).double() * s["freq"].double()      # far positions need more than 24 bits
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    lens = torch.full((B,), T, device=DEV, dtype=torch.int32) if s["lens"] is None else s["lens"]
    token = (torch.arange(T, device=DEV) < lens[:, None])[None, :, :, None, None]
    s["q_out"].copy_(torch.where(token, _rotated(s["q"], s, cos, sin), s["q_out"]))
    cap = s["k_tail"].shape[3]
    slot = (s["start"] + s["len"]).long()[..., None] + torch.arange(T, device=DEV)
    slot = (slot % cap)[:, :, None, :, None].expand(L, B, c["Hkv"], T, c["d"])
    for ring, new in ((s["k_tail"], _rotated(s["k"], s, cos, sin)), (s["v_tail"], s["v"])):
        if ring is not None:
            new = new.permute(0, 1, 3, 2, 4)
            old = torch.gather(ring, 3, slot)
            ring.scatter_(3, slot, torch.where(token.permute(0, 1, 3, 2, 4), new, old))
    s["len_out"].copy_(s["len"] + lens)
    return [s["q_out"], s["k_tail"], s["v_tail"], s["len_out"]]


def _plain_evict(s):
    c = s["case"]
    L, B, Hkv, d, ctx, keep = (c[k] for k in ("L", "B", "Hkv", "d", "ctx", "keep"))
    at = torch.arange(ctx, device=DEV)
    n = 128 * s["n"].long()[..., None]
    left = torch.clamp(n, max=keep)                                 # tokens that remain
    key = s["mass"][..., :ctx]
    safe = ((at < c["sink"]) | (at >= n - c["recent"])) & (at < n)
    key = torch.where(safe[:, :, None], torch.full_like(key, math.inf), key)
    key = key.masked_fill((at >= n)[:, :, None], -math.inf)
    best = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :keep]
    slot = torch.arange(keep, device=DEV)
    live = (slot < left)[:, :, None]
    best = torch.sort(torch.where(live, best, torch.full_like(best, ctx)), -1).values  # in the tokens' order
    s["kept"].copy_(torch.where(live, best, s["kept"].long()))
    best = best.clamp_max(ctx - 1)
    for key_, bits in (("k", c["kb"]), ("v", c["vb"])):
        if key_ == "k" or not c["shared"]:
            rec, row, cut = _contiguous(s[key_ + "_rec"], s["table"], Hkv), d * bits // 8, CHUNK * d * bits // 8
            codes = _rows(rec[..., :cut].reshape(L, B, Hkv, ctx, row), best)
            scale = _rows(rec[..., cut:].reshape(L, B, Hkv, ctx, 4), best)
            new = torch.cat([codes.view(L, B, Hkv, keep // CHUNK, cut), scale.view(L, B, Hkv, keep // CHUNK, -1)], -1)
            whole = live.expand(L, B, Hkv, keep)[..., ::CHUNK][..., None]
            s[key_ + "_dst"].copy_(torch.where(whole, new, s[key_ + "_dst"]))
    # accumulated weights follow their tokens, the ring's behind them
    place = torch.arange(keep + c["tail"], device=DEV)
    src = torch.where(place < left, 0, (place - left + n).clamp(0, ctx + c["tail"] - 1))[:, :, None].expand(
        L, B, Hkv, keep + c["tail"])
    src = torch.where((place < left)[:, :, None], torch.nn.functional.pad(best, (0, c["tail"])), src)
    got = torch.gather(s["mass"], 3, src)
    s["mass_dst"].copy_(torch.where((place < left + s["tail_len"][..., None])[:, :, None], got, s["mass_dst"]))
    s["n_dst"].copy_(torch.clamp(s["n"], max=keep // CHUNK))
    return [s["k_dst"], None if c["shared"] else s["v_dst"], s["mass_dst"], s["kept"], s["n_dst"]]


# ---------------------------------------------------------------- the library's entry points
@functools.lru_cache(maxsize=None)
def _handle(bits, d):
    import rotated_lloyd_max_gb300 as tq
    return tq.tq_make_codebook(bits, d, sign_seed=1)


def _own_args(s):
    """Argument blocks, codecs and workspaces that a program keeps with its cache."""
    import rotated_lloyd_max_gb300 as tq
    c = s["case"]
    if c["op"] == "append":
        return tq, (tq.make_append_args(
            q=s["q"], k=s["k"], v=None if c["shared"] else s["v"], q_out=s["q_out"], positions=s["pos"],
            inv_freq=s["freq"], pair_axis=s["axis"], rot_start=s["rot_start"], pair_adjacent=c["adjacent"],
            k_tail=s["k_tail"], v_tail=s["v_tail"], tail_start=s["start"], tail_len=s["len"],
            tail_len_out=s["len_out"], q_lens=s["lens"]),)
    kc, vc = _handle(c["kb"], c["d"]), _handle(c["vb"], c["d"])
    if c["op"] == "evict":
        a = tq.make_evict_mass_args(
            k_rec=s["k_rec"], v_rec=s["v_rec"], k_dst=s["k_dst"], v_dst=s["v_dst"], mass=s["mass"],
            mass_dst=s["mass_dst"], n_chunks=s["n"], n_chunks_dst=s["n_dst"], tail_len=s["tail_len"],
            max_chunks=c["ctx"] // CHUNK, max_tail=c["tail"], keep_chunks=c["keep"] // CHUNK, sink=c["sink"],
            recent=c["recent"], kept=s["kept"], block_table=s["table"])
        need = tq.tq_evict_mass_workspace_size(a, kc, vc)
        return tq, (a, kc, vc, torch.empty(need, dtype=torch.uint8, device=DEV))
    a = tq.make_query_args(
        q=s["q"], out=s.get("out"), scale=1.0, softcap=c["softcap"], causal=c["causal"], q_lens=s["lens"],
        k_rec=s["k_rec"], v_rec=s["v_rec"], k_tail=s["k_tail"], v_tail=s["v_tail"], n_chunks=s["n"],
        tail_start=s["start"], tail_len=s["len"], max_chunks=c["ctx"] // CHUNK, max_tail=c["tail"],
        block_table=s["table"])
    if c["op"] == "prefill":
        need = tq.tq_prefill_attn_workspace_size(a, kc, vc)
        return tq, (a, kc, vc, torch.empty(need, dtype=torch.uint8, device=DEV))
    need = tq.tq_attn_mass_workspace_size(a, kc)
    return tq, (a, kc, s["mass"], torch.empty(need, dtype=torch.uint8, device=DEV))


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"append": _plain_append, "prefill": _plain_prefill, "mass": _plain_mass, "evict": _plain_evict}[op](s)
    if "call" not in s:
        s["call"] = _own_args(s)
    tq, args = s["call"]
    if op == "append":
        tq.tq_append(*args)
        return [s["q_out"], s["k_tail"], s["v_tail"], s["len_out"]]
    if op == "prefill":
        tq.tq_prefill_attn(*args)
        return s["out"]
    if op == "mass":
        tq.tq_attn_mass(*args, decay=DECAY)
        return s["mass"]
    tq.tq_evict_mass(*args)
    return [s["k_dst"], None if s["case"]["shared"] else s["v_dst"], s["mass_dst"], s["kept"], s["n_dst"]]


def work(case):
    """Bytes and operations that a pass cannot do without (uniform lengths; ragged ones hold three quarters)."""
    c = case
    part = 0.75 if c["ragged"] else 1.0
    units, d = c["L"] * c["B"] * c["Hkv"], c["d"]
    if c["op"] == "append":
        rows = units * c["T"] * part * (c["G"] + (1 if c["shared"] else 2))
        return {"bytes": rows * d * 4 + 4 * c["axes"] * c["B"] * c["T"], "flops": rows * c["rot"] * 3}
    kb, vb = (d * c[k] / 8 + 4 for k in ("kb", "vb"))
    if c["op"] == "evict":
        ctx = c["ctx"] * part
        kept = min(c["keep"], ctx)
        moved = kept * 2 * (kb + (0 if c["shared"] else vb))
        return {"bytes": units * (4 * ctx + 4 * kept + moved + 4 * (kept + 2 * c["tail"])), "flops": units * ctx}
    ctx, tail, rows = c["ctx"] * part, c["tail"] * part, units * c["G"] * c["T"] * part
    keys = ctx + tail - (rows / units / c["G"] / 2 if c["causal"] else 0)
    if c["op"] == "mass":
        return {"bytes": units * (ctx * kb + tail * d * 2 + 8 * (ctx + tail)) + rows * d * 2,
                "flops": rows * keys * (2 * d + 4)}
    kv = kb + (0 if c["shared"] else vb)
    return {"bytes": units * (ctx * kv + tail * d * (2 if c["shared"] else 4)) + rows * d * 4,
            "flops": rows * keys * 4 * d}


# ---------------------------------------------------------------- the definition, in 64 bits
def _exact_vectors(s, which, l, b, h):
    """Keys or values of one sequence and head, float64, in the order of the tokens."""
    c = s["case"]
    d, n, ln = c["d"], int(s["n"][l, b]), int(s["len"][l, b])
    rec = s[which + "_rec"][l, b, h, :n] if s["table"] is None else s[which + "_rec"][l, s["table"][b, :n].long(), h]
    bits = s[which + "_codec"]["bits"]
    row = d * bits // 8
    by = rec[:, : CHUNK * row].reshape(n * CHUNK, row)
    bit = ((by[:, :, None] >> torch.arange(8, device=DEV, dtype=torch.uint8)) & 1).reshape(n * CHUNK, d, bits)
    code = (bit.to(torch.int16) << torch.arange(bits, device=DEV, dtype=torch.int16)).sum(-1)
    scale = rec[:, CHUNK * row:].contiguous().view(torch.float32).reshape(-1).double()
    x = s[which + "_codec"]["cent"].double()[code] * scale[:, None]
    block = 1
    while block < d:  # the butterflies of the transform
        x = x.view(-1, d // (2 * block), 2, block)
        x = torch.stack([x[:, :, 0] + x[:, :, 1], x[:, :, 0] - x[:, :, 1]], 2)
        block *= 2
    x = x.reshape(-1, d) * _signs(d).double() / math.sqrt(d)
    cap = s[which + "_tail"].shape[3]
    slots = (int(s["start"][l, b]) + torch.arange(ln, device=DEV)) % cap
    return torch.cat([x, s[which + "_tail"][l, b, h, slots].double()])


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "evict":
        return None  # moves bytes and selects: nothing computed
    L, B, T, Hkv, G, d = (c[k] for k in ("L", "B", "T", "Hkv", "G", "d"))
    lens = [T] * B if s["lens"] is None else s["lens"].tolist()
    if c["op"] == "append":
        q_out, k_tail = s["q_out"].double(), s["k_tail"].double()
        v_tail = None if s["v_tail"] is None else s["v_tail"].double()
        half, a, cap = c["rot"] // 2, s["rot_start"], s["k_tail"].shape[3]
        first = torch.arange(half, device=DEV) * (2 if c["adjacent"] else 1) + a
        second = first + (1 if c["adjacent"] else half)
        for b in range(B):
            m = lens[b]
            pos = s["pos"][torch.tensor(s["axis"], device=DEV), b, :m].double()
            z = torch.polar(torch.ones_like(pos), pos * s["freq"].double()[:, None]).T[:, None]  # [m][1][pairs]
            for l in range(L):
                at = (int(s["start"][l, b]) + int(s["len"][l, b]) + torch.arange(m, device=DEV)) % cap
                for x, put in ((s["q"], None), (s["k"], k_tail)):
                    y = x[l, b, :m].double()
                    w = torch.complex(y[..., first], y[..., second]) * z
                    y[..., first], y[..., second] = w.real, w.imag
                    if put is None:
                        q_out[l, b, :m] = y
                    else:
                        put[l, b][:, at] = y.transpose(0, 1)
                if v_tail is not None:
                    v_tail[l, b][:, at] = s["v"][l, b, :m].double().transpose(0, 1)
        return [q_out, k_tail, v_tail, None]
    out = s["out"].double() if c["op"] == "prefill" else s["mass"].double()
    for l in range(L):
        for b in range(B):
            total, m = CHUNK * int(s["n"][l, b]) + int(s["len"][l, b]), lens[b]
            for h in range(Hkv):
                k = _exact_vectors(s, "k", l, b, h)
                got = torch.zeros(total, dtype=torch.float64, device=DEV)
                v = _exact_vectors(s, "v", l, b, h) if c["op"] == "prefill" else None
                for g in range(G):
                    x = s["q"][l, b, :m, h * G + g].double() @ k.T
                    if c["softcap"]:
                        x = c["softcap"] * torch.tanh(x / c["softcap"])
                    if c["causal"]:
                        row = torch.arange(m, device=DEV)[:, None] + total - m
                        x = x.masked_fill(torch.arange(total, device=DEV) > row, -math.inf)
                    w = torch.softmax(x, -1)
                    if v is None:
                        got += w.sum(0)
                    else:
                        out[l, b, :m, h * G + g] = w @ v
                if v is None:
                    out[l, b, h, :total] = DECAY * out[l, b, h, :total] + got
    return out
