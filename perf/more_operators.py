"""Cases of the operators that attend to a part of a long cache.

Four operators around the rotated Lloyd-Max cache (records of 128 tokens, a
dense bf16 ring behind them), in the order in which a model calls them:

  append   RMS norms of every query and key head, rotary positions, keys and
           values appended to the ring
  bounds   the smallest and largest value that each coordinate of a record's
           keys takes
  select   records chosen for blocks of queries by an upper bound of their
           logits, formed from the bounds
  sparse   attention over the chosen records and the ring

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
EPS = 1e-6


# ---------------------------------------------------------------- cases
def _append(**kw):
    case = dict(op="append", L=1, B=1, T=1, Hkv=2, G=6, d=128, rot=128, adjacent=False, ragged=False, shared=False,
                per_head=False, window=300, far=4096)
    return {**case, **kw}


def _bounds(**kw):
    case = dict(op="bounds", L=1, B=1, Hkv=2, d=128, kb=4, n=64, new=64, ragged=False, paged=False)
    return {**case, **kw}


def _select(**kw):
    case = dict(op="select", L=1, B=1, T=1, Hkv=2, G=6, d=128, n=64, keep=16, qb=1, sink=1, recent=2, tail=200,
                ragged=False, paged=False)
    return {**case, **kw}


def _sparse(**kw):
    case = dict(op="sparse", L=1, B=1, T=1, Hkv=2, G=6, d=128, kb=4, vb=4, n=64, keep=16, qb=1, tail=200,
                shared=False, softcap=0.0, ragged=False, paged=False, gain=2.0)
    return {**case, **kw}


def listed():
    return [
        # one new token of one sequence: the latency of a decode step's smallest call
        _append(name="append_token"),
        # prompts padded to one length, of which the last rows are not tokens
        _append(name="append_prompts", B=4, T=2049, Hkv=8, G=4, ragged=True, far=131072),
        # a decode step of a served batch has moved one chunk of every sequence into a record
        _bounds(name="bounds_step32", B=32, Hkv=8, n=256, new=1),
        # a prompt of 131072 tokens has just been encoded, 3-bit keys
        _bounds(name="bounds_prompt", Hkv=8, kb=3, n=1024, new=1024),
        # the same of a model with one wide key/value head, 65536 tokens
        _bounds(name="bounds_mqa_d512", Hkv=1, d=512, n=512, new=512),
        # a decode step of one sequence of 8192 tokens
        _select(name="select_token"),
        # a decode step of a served batch, 32768 tokens each
        _select(name="select_batch32", B=32, Hkv=8, G=4, n=256, keep=32),
        # a slice of a prompt, one list for 64 tokens
        _select(name="select_slice", T=1024, Hkv=8, G=4, n=256, keep=32, qb=64, tail=1280),
        # a decode step of one sequence: 16 of 64 records
        _sparse(name="sparse_token", kb=3, vb=2),
        # a decode step of a served batch: 32 of 256 records for every sequence and head
        _sparse(name="sparse_batch32", B=32, Hkv=8, G=4, n=256, keep=32, vb=3, tail=144),
        # a slice of a prompt of 32768 tokens, one list for 64 tokens
        _sparse(name="sparse_slice", T=1024, Hkv=8, G=4, n=256, keep=32, qb=64, tail=1280),
        # one key/value head for 64 query heads, keys and values in one record, four drafted tokens of
        # four sequences, each token with a list of its own
        _sparse(name="sparse_mqa_d512", B=4, T=4, Hkv=1, G=64, d=512, n=128, keep=32, tail=272, shared=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "bounds", "select", "sparse"])
    d = rng.choice([64, 128, 128, 256, 512])
    Hkv = 1 if d == 512 else rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 4, 5, 6, 7, 8]) if d < 512 else rng.choice([16, 64])
    kb, vb = rng.choice([(4, 4), (4, 3), (3, 2), (2, 2), (1, 4), (3, 3)])
    ragged, paged = rng.random() < 0.5, rng.random() < 0.3
    if op == "append":
        T = _log(rng, 1, 2049)
        B = _log(rng, 1, max(1, min(48, 4096 // T)))
        return _append(B=B, T=T, Hkv=Hkv, G=min(G, 16), d=d, rot=rng.choice([d, d // 2, 32]),
                       adjacent=rng.random() < 0.4, ragged=ragged and T > 1, shared=d == 512 and rng.random() < 0.5,
                       per_head=rng.random() < 0.3, window=rng.randrange(1, 400), far=_log(rng, 1000, 1000000))
    if op == "bounds":
        n = _log(rng, 1, 512)
        B = _log(rng, 1, max(1, min(32, 65536 // (n * Hkv * d))))
        return _bounds(B=B, Hkv=Hkv, d=d, kb=kb, n=n, new=rng.choice([1, n, _log(rng, 1, n)]), ragged=ragged,
                       paged=paged)
    n = _log(rng, 2, 256)
    keep = _log(rng, 2, min(48, n))
    if rng.random() < 0.5:   # decode steps and drafted tokens: a list for every token
        T, qb = _log(rng, 1, 8), 1
        B = _log(rng, 1, max(1, min(32, 65536 // (keep * Hkv * T * d))))
    else:                    # slices of prompts: a list for a block of tokens
        qb = rng.choice([16, 32, 64, 100])
        T, B = _log(rng, qb, max(qb, 12288 // (Hkv * G))), 1
    if op == "select":
        sink = rng.randrange(0, 2)
        return _select(B=B, T=T, Hkv=Hkv, G=G, d=d, n=n, keep=keep, qb=qb, sink=sink,
                       recent=rng.randrange(0, keep - sink + 1), tail=T + rng.randrange(0, 400), ragged=ragged,
                       paged=paged)
    shared = d == 512 and rng.random() < 0.7
    return _sparse(B=B, T=T, Hkv=Hkv, G=G, d=d, kb=4 if shared else kb, vb=4 if shared else vb, n=n, keep=keep, qb=qb,
                   tail=T + rng.randrange(0, 300), shared=shared, softcap=rng.choice([0.0, 0.0, 20.0]), ragged=ragged,
                   paged=paged, gain=rng.choice([1.0, 2.0, 3.0]))


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


def _blocks(c):
    return -(-c["T"] // c["qb"])


def _prepare_append(c, s, gen, host):
    L, B, T, Hkv, G, d = (c[k] for k in ("L", "B", "T", "Hkv", "G", "d"))
    Hq, half = Hkv * G, c["rot"] // 2
    # one projection's output holds queries, keys and values of a token side by side
    heads = _bf16((L, B, T, Hq + 2 * Hkv, d), gen, 1.7)
    s["q"], s["k"], s["v"] = heads[..., :Hq, :], heads[..., Hq:Hq + Hkv, :], heads[..., Hq + Hkv:, :]
    s["q_out"] = torch.zeros((L, B, T, Hq, d), dtype=torch.bfloat16, device=DEV)
    weight = lambda h: 1.0 + 0.3 * torch.randn((h, d) if c["per_head"] else (d,), generator=gen, device=DEV)  # noqa: E731
    s["wq"], s["wk"] = weight(Hq), weight(Hkv)
    cap = c["window"] + T + 37
    s["k_tail"] = _bf16((L, B, Hkv, cap, d), gen)
    s["v_tail"] = None if c["shared"] else _bf16((L, B, Hkv, cap, d), gen)
    s["start"] = _ints(host.randint(0, cap, (L, B)))
    s["len"] = _ints(host.randint(0, c["window"] + 1, (L, B)))
    s["len_out"] = torch.zeros_like(s["len"])
    s["lens"] = _ints(host.randint(T // 2, T + 1, B)) if c["ragged"] else None
    base = torch.randint(0, c["far"], (B, 1), generator=gen, device=DEV)
    s["pos"] = (base + torch.arange(T, device=DEV)).to(torch.int32)[None].contiguous()
    s["freq"] = (10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)).float()
    s["rot_start"] = d - c["rot"]


def _prepare_bounds(c, s, gen, host):
    L, B, Hkv, d, n = (c[k] for k in ("L", "B", "Hkv", "d", "n"))
    have = host.randint(n // 2, n + 1, (L, B)) if c["ragged"] else np.full((L, B), n)
    s["n"] = _ints(have)
    s["first"] = _ints(np.maximum(have - c["new"], 0))
    s["codec"] = _codec(d, c["kb"])
    lead, per = ((L, B, Hkv), n)
    s["table"] = None
    if c["paged"]:
        pool = B * n + 3
        s["table"] = _ints(host.permutation(pool)[: B * n].reshape(B, n))
        lead, per = (L, pool), Hkv
    s["k_rec"] = _records(lead, per, d, c["kb"], gen)
    s["bounds"] = torch.zeros((*lead, per, 2, d), dtype=torch.bfloat16, device=DEV)


def _prepare_select(c, s, gen, host):
    L, B, T, Hkv, G, d, n = (c[k] for k in ("L", "B", "T", "Hkv", "G", "d", "n"))
    have = host.randint((n + 1) // 2, n + 1, (L, B)) if c["ragged"] else np.full((L, B), n)
    s["n"] = _ints(have)
    s["lens"] = _ints(host.randint(T // 2, T + 1, B)) if c["ragged"] else None
    s["len"] = _ints(c["tail"], (L, B))
    lead = (L, B, Hkv, n)
    s["table"] = None
    if c["paged"]:
        pool = B * n + 3
        s["table"] = _ints(host.permutation(pool)[: B * n].reshape(B, n))
        lead = (L, pool, Hkv)
    # keys with a mean that drifts from record to record, and a few channels that are larger than the others
    wide = torch.ones(d, device=DEV)
    wide[torch.from_numpy(host.permutation(d)[:4]).to(DEV)] = 6.0
    mean = 0.4 * torch.randn((*lead, d), generator=gen, device=DEV) * wide
    half = (2.2 + torch.rand((*lead, d), generator=gen, device=DEV)) * wide
    s["bounds"] = torch.stack([mean - half, mean + half], -2).to(torch.bfloat16)
    s["q"] = _bf16((L, B, T, Hkv * G, d), gen, 2.0 / math.sqrt(d))
    s["list"] = torch.zeros((L, B, _blocks(c), Hkv, c["keep"]), dtype=torch.int32, device=DEV)
    s["count"] = torch.zeros((L, B, _blocks(c), Hkv), dtype=torch.int32, device=DEV)


def _prepare_sparse(c, s, gen, host):
    L, B, T, Hkv, G, d, n, keep = (c[k] for k in ("L", "B", "T", "Hkv", "G", "d", "n", "keep"))
    have = host.randint((n + 1) // 2, n + 1, (L, B)) if c["ragged"] else np.full((L, B), n)
    s["n"] = _ints(have)
    for key, bits in (("k", c["kb"]), ("v", c["vb"])):
        s[key + "_codec"] = _codec(d, bits)
    lead, per = (L, B, Hkv), n
    s["table"] = None
    if c["paged"]:  # blocks of a pool, in no order
        pool = B * n + 3
        s["table"] = _ints(host.permutation(pool)[: B * n].reshape(B, n))
        lead, per = (L, pool), Hkv
    s["k_rec"] = _records(lead, per, d, c["kb"], gen)
    s["v_rec"] = s["k_rec"] if c["shared"] else _records(lead, per, d, c["vb"], gen)
    # what a selection leaves: the first record, the last one, others in between, in their order
    nb = _blocks(c)
    at = torch.arange(n, device=DEV)
    last = s["n"].long()[:, :, None, None, None]
    score = torch.rand((L, B, nb, Hkv, n), generator=gen, device=DEV)
    score = torch.where((at == 0) | (at == last - 1), score + 2.0, score).masked_fill(at >= last, -1.0)
    best = score.topk(keep, -1).indices
    best = torch.where(torch.gather(score, -1, best) < 0, n, best).sort(-1).values
    s["list"] = torch.where(best < n, best, -1).to(torch.int32)
    s["count"] = (best < n).sum(-1).to(torch.int32)
    s["q"] = _bf16((L, B, T, Hkv * G, d), gen, c["gain"] / math.sqrt(d))
    cap = c["tail"] + 19
    s["k_tail"] = _bf16((L, B, Hkv, cap, d), gen)
    s["v_tail"] = s["k_tail"] if c["shared"] else _bf16((L, B, Hkv, cap, d), gen)
    s["start"] = _ints(host.randint(0, cap, (L, B)))
    lens = host.randint(T // 2, T + 1, B) if c["ragged"] else np.full(B, T)
    s["lens"] = _ints(lens) if c["ragged"] else None
    low = np.minimum(lens, c["tail"])[None, :]
    s["len"] = _ints(np.maximum(low, host.randint(0, c["tail"] + 1, (L, B))) if c["ragged"] else c["tail"], (L, B))
    s["out"] = torch.zeros((L, B, T, Hkv * G, d), dtype=torch.bfloat16, device=DEV)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    host = np.random.RandomState(int(seed) % (1 << 31))
    s = dict(case=c)
    {"append": _prepare_append, "bounds": _prepare_bounds, "select": _prepare_select,
     "sparse": _prepare_sparse}[c["op"]](c, s, gen, host)
    return s


# ---------------------------------------------------------------- plain forms
def _normed(x, w):
    """RMS norm of every head [L][B][T][heads][d], in f32."""
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w


def _rotated(x, s, cos, sin):
    """x [L][B][T][heads][d] (f32) with the pairs of its rotated coordinates turned."""
    c = s["case"]
    a, half = s["rot_start"], c["rot"] // 2
    r = x[..., a: a + c["rot"]]
    x0, x1 = (r[..., 0::2], r[..., 1::2]) if c["adjacent"] else (r[..., :half], r[..., half:])
    y0, y1 = x0 * cos - x1 * sin, x1 * cos + x0 * sin
    y = torch.stack([y0, y1], -1).flatten(-2) if c["adjacent"] else torch.cat([y0, y1], -1)
    return torch.cat([x[..., :a], y, x[..., a + c["rot"]:]], -1).to(torch.bfloat16)


def _plain_append(s):
    c = s["case"]
    L, B, T, cap = c["L"], c["B"], c["T"], s["k_tail"].shape[3]
    angle = s["pos"][0].double()[..., None] * s["freq"].double()    # far positions need more than 24 bits
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    lens = torch.full((B,), T, device=DEV, dtype=torch.int32) if s["lens"] is None else s["lens"]
    token = (torch.arange(T, device=DEV) < lens[:, None])[None, :, :, None, None]
    s["q_out"].copy_(torch.where(token, _rotated(_normed(s["q"], s["wq"]), s, cos, sin), s["q_out"]))
    slot = (s["start"] + s["len"]).long()[..., None] + torch.arange(T, device=DEV)
    slot = (slot % cap)[:, :, None, :, None].expand(L, B, c["Hkv"], T, c["d"])
    token = token.permute(0, 1, 3, 2, 4)
    new = _rotated(_normed(s["k"], s["wk"]), s, cos, sin).permute(0, 1, 3, 2, 4)
    s["k_tail"].scatter_(3, slot, torch.where(token, new, torch.gather(s["k_tail"], 3, slot)))
    if s["v_tail"] is not None:
        new = s["v"].permute(0, 1, 3, 2, 4)
        s["v_tail"].scatter_(3, slot, torch.where(token, new, torch.gather(s["v_tail"], 3, slot)))
    s["len_out"].copy_(s["len"] + lens)
    return [s["q_out"], s["k_tail"], s["v_tail"], s["len_out"]]


def _unpack(rec, d, bits):
    """Codes [..., 128, d] and scales [..., 128] of records [..., bytes]."""
    lead, cut = rec.shape[:-1], CHUNK * d * bits // 8
    by = rec[..., :cut].reshape(*lead, CHUNK, d * bits // 8).to(torch.int32)
    if bits == 3:
        g = by.view(*by.shape[:-1], d // 8, 3)
        word, k = g[..., 0] | (g[..., 1] << 8) | (g[..., 2] << 16), 8
    else:
        word, k = by, 8 // bits
    codes = (word[..., None] >> (bits * torch.arange(k, device=rec.device, dtype=torch.int32))) & ((1 << bits) - 1)
    return codes.reshape(*by.shape[:-1], d), rec[..., cut:].contiguous().view(torch.float32)


def _decoded(rec, codec, d):
    """Vectors [..., 128, d] of records [..., bytes], in f32."""
    codes, scale = _unpack(rec, d, codec["bits"])
    return codec["cent"][codes.long()] @ codec["rot"] * scale[..., None]


def _outward(x, down):
    """f32 to the next bf16 below (down) or above."""
    bits = x.contiguous().view(torch.int32)
    cut = bits & -65536                                             # towards zero
    away = (cut != bits) & ((bits < 0) == down)
    return torch.where(away, cut + 65536, cut).view(torch.float32).to(torch.bfloat16)


def _plain_bounds(s):
    c = s["case"]
    d, n = c["d"], c["n"]
    new = min(c["new"], n)
    at = (s["first"].long()[..., None] + torch.arange(new, device=DEV))             # [L][B][new]
    live = at < s["n"].long()[..., None]
    at = at.clamp(max=n - 1)
    if s["table"] is None:
        pick = at[:, :, None, :, None]
        rec = torch.gather(s["k_rec"], 3, pick.expand(c["L"], c["B"], c["Hkv"], new, s["k_rec"].shape[-1]))
    else:  # [L][B][new][Hkv][bytes]
        block = torch.gather(s["table"].long()[None].expand(c["L"], -1, -1), 2, at)
        layer = torch.arange(c["L"], device=DEV)[:, None, None]
        rec = s["k_rec"][layer, block]
    x = _decoded(rec, s["codec"], d)
    b = torch.stack([_outward(x.amin(-2), True), _outward(x.amax(-2), False)], -2)
    if s["table"] is None:
        pick = at[:, :, None, :, None, None].expand_as(b)
        keep = live[:, :, None, :, None, None]
        s["bounds"].scatter_(3, pick, torch.where(keep, b, torch.gather(s["bounds"], 3, pick)))
    else:
        old = s["bounds"][layer, block]
        s["bounds"].index_put_((layer, block), torch.where(live[..., None, None, None], b, old))
    return s["bounds"]


def _plain_select(s):
    c = s["case"]
    L, B, T, Hkv, G, d, n, keep, qb = (c[k] for k in ("L", "B", "T", "Hkv", "G", "d", "n", "keep", "qb"))
    nb = _blocks(c)
    lens = torch.full((B,), T, device=DEV) if s["lens"] is None else s["lens"].long()
    bnd = s["bounds"] if s["table"] is None else s["bounds"][:, s["table"].long()].permute(0, 1, 3, 2, 4, 5)
    lo, hi = bnd[..., 0, :].double(), bnd[..., 1, :].double()       # neighbours in rank may differ by little
    q = torch.nn.functional.pad(s["q"], (0, 0, 0, 0, 0, nb * qb - T)).double()
    q = q.view(L, B, nb * qb, Hkv, G, d).permute(0, 1, 3, 2, 4, 5).reshape(L, B, Hkv, nb * qb * G, d)
    score = q.clamp_min(0) @ hi.transpose(-1, -2) + q.clamp_max(0) @ lo.transpose(-1, -2)
    t = torch.arange(nb * qb, device=DEV)
    live = (t < lens[:, None])[None, :, None, :, None, None]
    score = score.view(L, B, Hkv, nb * qb, G, n).masked_fill(~live, -math.inf)
    score = score.view(L, B, Hkv, nb, qb * G, n).amax(-2).transpose(2, 3)           # [L][B][blocks][Hkv][n]
    first = torch.arange(nb, device=DEV) * qb
    last = torch.minimum(lens[:, None], first + qb) - 1                             # [B][blocks]
    total = 128 * s["n"].long() + s["len"].long()
    limit = total[..., None] - lens[:, None] + last + 1
    m = torch.minimum(s["n"].long()[..., None], (limit + CHUNK - 1) // CHUNK)
    m = torch.where(last >= first, m, 0)[..., None, None]                           # records a block may read
    at = torch.arange(n, device=DEV)
    safe = ((at < c["sink"]) | (at >= m - c["recent"])) & (at < m)
    score = score.masked_fill(safe, math.inf)
    rank = torch.sort(torch.where(at < m, score, torch.full_like(score, -math.inf)), dim=-1, descending=True,
                      stable=True).indices[..., :keep]
    best = torch.where(torch.arange(keep, device=DEV) < m, rank, n).sort(-1).values
    s["list"].copy_(torch.where(best < n, best, -1))
    s["count"].copy_((best < n).sum(-1))
    return [s["list"], s["count"]]


def _ring(x, start, tail):
    """The ring's first `tail` tokens in order: x [L][B][Hkv][cap][d]."""
    at = (start.long()[..., None] + torch.arange(tail, device=x.device)) % x.shape[3]
    return torch.gather(x, 3, at[:, :, None, :, None].expand(*x.shape[:3], tail, x.shape[4])).float()


def _listed(s, which):
    """Vectors [L][B][blocks][Hkv][keep * 128][d] of the listed records, in f32."""
    c = s["case"]
    L, B, Hkv, d = c["L"], c["B"], c["Hkv"], c["d"]
    at = s["list"].clamp_min(0).long()
    layer = torch.arange(L, device=DEV)[:, None, None, None, None]
    seq = torch.arange(B, device=DEV)[:, None, None, None]
    head = torch.arange(Hkv, device=DEV)[:, None]
    if s["table"] is None:
        rec = s[which + "_rec"][layer, seq, head, at]
    else:
        rec = s[which + "_rec"][layer, s["table"].long()[seq, at], head]
    return _decoded(rec, s[which + "_codec"], d).flatten(-3, -2)


def _plain_sparse(s):
    c = s["case"]
    L, B, T, Hkv, G, d, keep, qb, tail = (c[k] for k in ("L", "B", "T", "Hkv", "G", "d", "keep", "qb", "tail"))
    nb = _blocks(c)
    lens = torch.full((B,), T, device=DEV) if s["lens"] is None else s["lens"].long()
    q = torch.nn.functional.pad(s["q"], (0, 0, 0, 0, 0, nb * qb - T)).float()
    q = q.view(L, B, nb, qb, Hkv, G, d).permute(0, 1, 2, 4, 3, 5, 6).reshape(L, B, nb, Hkv, qb * G, d)
    ring = lambda x: _ring(x, s["start"], tail)[:, :, None]         # noqa: E731  [L][B][1][Hkv][tail][d]
    x = torch.cat([q @ _listed(s, "k").transpose(-1, -2), q @ ring(s["k_tail"]).transpose(-1, -2)], -1)
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    there = (s["list"] >= 0).repeat_interleave(CHUNK, -1)[..., None, :]             # [L][B][blocks][Hkv][1][keep * 128]
    t = (torch.arange(nb, device=DEV)[:, None] * qb + torch.arange(qb, device=DEV)).repeat_interleave(G, -1)
    last = s["len"].long()[:, :, None, None] - lens[:, None, None] + t              # in the ring: [L][B][blocks][rows]
    j = torch.arange(tail, device=DEV)
    near = (j <= last[..., None]) & (j < s["len"].long()[:, :, None, None, None])
    seen = torch.cat([there.expand(-1, -1, -1, -1, qb * G, -1),
                      near[:, :, :, None].expand(-1, -1, -1, Hkv, -1, -1)], -1)
    x = x.masked_fill(~seen, -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True).clamp_min(-3e38))
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
    o = p[..., : keep * CHUNK] @ _listed(s, "v") + p[..., keep * CHUNK:] @ ring(s["v_tail"])
    o = o.view(L, B, nb, Hkv, qb, G, d).permute(0, 1, 2, 4, 3, 5, 6).reshape(L, B, nb * qb, Hkv * G, d)[:, :, :T]
    token = (torch.arange(T, device=DEV) < lens[:, None])[None, :, :, None, None]
    s["out"].copy_(torch.where(token, o.to(torch.bfloat16), s["out"]))
    return s["out"]


# ---------------------------------------------------------------- the library's entry points
@functools.lru_cache(maxsize=None)
def _handle(bits, d):
    import rotated_lloyd_max_gb300 as tq
    return tq.tq_make_codebook(bits, d, sign_seed=1)


def _own_call(s):
    """The call with the argument blocks, codecs and workspace that a program keeps with its cache."""
    import rotated_lloyd_max_gb300 as tq
    c = s["case"]
    space = lambda size: torch.empty(size, dtype=torch.uint8, device=DEV)  # noqa: E731
    if c["op"] == "append":
        a = tq.make_append_args(
            q=s["q"], k=s["k"], v=None if c["shared"] else s["v"], q_out=s["q_out"], positions=s["pos"],
            inv_freq=s["freq"], rot_start=s["rot_start"], pair_adjacent=c["adjacent"], k_tail=s["k_tail"],
            v_tail=s["v_tail"], tail_start=s["start"], tail_len=s["len"], tail_len_out=s["len_out"], q_lens=s["lens"])
        norm = tq.make_head_norm(q_weight=s["wq"], k_weight=s["wk"], eps=EPS)
        return lambda: tq.tq_norm_append(a, norm)
    if c["op"] == "bounds":
        a = tq.make_bounds_args(k_rec=s["k_rec"], bounds=s["bounds"], n_chunks=s["n"], first=s["first"],
                                max_chunks=c["n"], max_new=min(c["new"], c["n"]), block_table=s["table"])
        codec = _handle(c["kb"], c["d"])
        return lambda: tq.tq_key_bounds(a, codec)
    if c["op"] == "select":
        a = tq.make_select_args(q=s["q"], bounds=s["bounds"], n_chunks=s["n"], max_chunks=c["n"], tail_len=s["len"],
                                max_tail=c["tail"], q_lens=s["lens"], block_table=s["table"], q_block=c["qb"],
                                keep=c["keep"], sink=c["sink"], recent=c["recent"], list=s["list"], count=s["count"])
        ws = space(tq.tq_select_records_workspace_size(a))
        return lambda: tq.tq_select_records(a, ws)
    kc, vc = _handle(c["kb"], c["d"]), _handle(c["vb"], c["d"])
    a = tq.make_query_args(
        q=s["q"], out=s["out"], scale=1.0, softcap=c["softcap"], q_lens=s["lens"], k_rec=s["k_rec"], v_rec=s["v_rec"],
        k_tail=s["k_tail"], v_tail=s["v_tail"], n_chunks=s["n"], tail_start=s["start"], tail_len=s["len"],
        max_chunks=c["n"], max_tail=c["tail"], block_table=s["table"])
    lists = tq.make_record_lists(list=s["list"], count=s["count"], q_block=c["qb"])
    ws = space(tq.tq_sparse_attn_workspace_size(a, lists, kc, vc))
    return lambda: tq.tq_sparse_attn(a, lists, kc, vc, ws)


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"append": _plain_append, "bounds": _plain_bounds, "select": _plain_select, "sparse": _plain_sparse}[op](s)
    if "call" not in s:
        s["call"] = _own_call(s)
    s["call"]()
    return {"append": lambda: [s["q_out"], s["k_tail"], s["v_tail"], s["len_out"]], "bounds": lambda: s["bounds"],
            "select": lambda: [s["list"], s["count"]], "sparse": lambda: s["out"]}[op]()


def work(case):
    """Bytes and operations that a pass cannot do without (uniform lengths; ragged ones hold three quarters)."""
    c = case
    part = 0.75 if c["ragged"] else 1.0
    units, d = c["L"] * c["B"] * c["Hkv"], c["d"]
    if c["op"] == "append":
        rows = units * c["T"] * part * (c["G"] + (1 if c["shared"] else 2))
        return {"bytes": rows * d * 4 + 4 * c["B"] * c["T"], "flops": rows * (c["rot"] * 3 + 4 * d)}
    key = d * c.get("kb", 0) / 8 + 4
    if c["op"] == "bounds":
        recs = units * min(c["new"], c["n"] * part)
        return {"bytes": recs * (CHUNK * key + 4 * d), "flops": recs * CHUNK * d * (math.log2(d) + 3)}
    n, rows = c["n"] * part, units * c["G"] * c["T"] * part
    if c["op"] == "select":
        lists = units * _blocks(c)
        return {"bytes": units * n * 4 * d + rows * d * 2 + lists * (c["keep"] + 1) * 4, "flops": rows * n * 4 * d}
    keep, tail = min(c["keep"], n), c["tail"] * part
    distinct = min(n, keep * _blocks(c) * part)                     # a record that several lists name is read once
    kv = key + (0 if c["shared"] else d * c["vb"] / 8 + 4)
    return {"bytes": units * (distinct * CHUNK * kv + tail * d * (2 if c["shared"] else 4)) + rows * d * 4,
            "flops": rows * (keep * CHUNK + tail - c["T"] / 2) * 4 * d}


# ---------------------------------------------------------------- the definition, in 64 bits
def _exact_records(rec, codec, d):
    """Vectors [records * 128][d] of records [records][bytes], float64: bit by bit, transform by butterflies."""
    bits = codec["bits"]
    row = d * bits // 8
    by = rec[:, : CHUNK * row].reshape(-1, row)
    bit = ((by[:, :, None] >> torch.arange(8, device=DEV, dtype=torch.uint8)) & 1).reshape(-1, d, bits)
    code = (bit.to(torch.int16) << torch.arange(bits, device=DEV, dtype=torch.int16)).sum(-1)
    scale = rec[:, CHUNK * row:].contiguous().view(torch.float32).reshape(-1).double()
    x = codec["cent"].double()[code] * scale[:, None]
    block = 1
    while block < d:
        x = x.view(-1, d // (2 * block), 2, block)
        x = torch.stack([x[:, :, 0] + x[:, :, 1], x[:, :, 0] - x[:, :, 1]], 2)
        block *= 2
    return x.reshape(-1, d) * _signs(d).double() / math.sqrt(d)


def _exact_append(s, lens):
    c = s["case"]
    q_out, k_tail = s["q_out"].double(), s["k_tail"].double()
    v_tail = None if s["v_tail"] is None else s["v_tail"].double()
    half, a, cap = c["rot"] // 2, s["rot_start"], s["k_tail"].shape[3]
    first = torch.arange(half, device=DEV) * (2 if c["adjacent"] else 1) + a
    second = first + (1 if c["adjacent"] else half)
    for b in range(c["B"]):
        m = lens[b]
        pos = s["pos"][0, b, :m].double()
        z = torch.polar(torch.ones((m, half), device=DEV, dtype=torch.float64), pos[:, None] * s["freq"].double())[:, None]
        for l in range(c["L"]):
            at = (int(s["start"][l, b]) + int(s["len"][l, b]) + torch.arange(m, device=DEV)) % cap
            for x, w, put in ((s["q"], s["wq"], None), (s["k"], s["wk"], k_tail)):
                y = x[l, b, :m].double()
                y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / c["d"] + EPS) * w.double()
                turned = torch.complex(y[..., first], y[..., second]) * z
                y[..., first], y[..., second] = turned.real, turned.imag
                if put is None:
                    q_out[l, b, :m] = y
                else:
                    put[l, b][:, at] = y.transpose(0, 1)
            if v_tail is not None:
                v_tail[l, b][:, at] = s["v"][l, b, :m].double().transpose(0, 1)
    return [q_out, k_tail, v_tail, None]


def _exact_bounds(s):
    """The minima and maxima themselves, before they are rounded outward."""
    c = s["case"]
    out = s["bounds"].double()
    for l in range(c["L"]):
        for b in range(c["B"]):
            a, z = int(s["first"][l, b]), int(s["n"][l, b])
            z = min(z, a + c["new"])
            for h in range(c["Hkv"]):
                if z > a and s["table"] is None:
                    x = _exact_records(s["k_rec"][l, b, h, a:z], s["codec"], c["d"]).view(z - a, CHUNK, -1)
                    out[l, b, h, a:z, 0], out[l, b, h, a:z, 1] = x.min(1).values, x.max(1).values
                elif z > a:
                    at = s["table"][b, a:z].long()
                    x = _exact_records(s["k_rec"][l, at, h], s["codec"], c["d"]).view(z - a, CHUNK, -1)
                    out[l, at, h, 0], out[l, at, h, 1] = x.min(1).values, x.max(1).values
    return out


def _exact_sparse(s, lens):
    c = s["case"]
    G, qb, out = c["G"], c["qb"], s["out"].double()
    for l in range(c["L"]):
        for b in range(c["B"]):
            m, ln, cap = lens[b], int(s["len"][l, b]), s["k_tail"].shape[3]
            slots = (int(s["start"][l, b]) + torch.arange(ln, device=DEV)) % cap
            for h in range(c["Hkv"]):
                ring = [s[w + "_tail"][l, b, h, slots].double() for w in "kv"]
                for j in range(-(-m // qb)):
                    at = s["list"][l, b, j, h, : int(s["count"][l, b, j, h])].long()
                    if s["table"] is None:
                        recs = [s[w + "_rec"][l, b, h, at] for w in "kv"]
                    else:
                        recs = [s[w + "_rec"][l, s["table"][b].long()[at], h] for w in "kv"]
                    k, v = (torch.cat([_exact_records(r, s[w + "_codec"], c["d"]), x])
                            for r, w, x in zip(recs, "kv", ring))
                    t0, t1 = j * qb, min(m, j * qb + qb)
                    x = torch.einsum("tgd,nd->gtn", s["q"][l, b, t0:t1, h * G:h * G + G].double(), k)
                    if c["softcap"]:
                        x = c["softcap"] * torch.tanh(x / c["softcap"])
                    place = torch.arange(k.shape[0], device=DEV) - CHUNK * len(at)  # in the ring; records come before it
                    row = torch.arange(t0, t1, device=DEV)[:, None] + ln - m
                    w = torch.softmax(x.masked_fill(place > row, -math.inf), -1)
                    out[l, b, t0:t1, h * G:h * G + G] = torch.einsum("gtn,nd->tgd", w, v)
    return out


def exact(case, seed):
    if case["op"] == "select":
        return None  # whole numbers, which the plain form already decides in 64 bits
    s = prepare(case, seed)
    lens = None
    if case["op"] != "bounds":
        lens = [case["T"]] * case["B"] if s["lens"] is None else s["lens"].tolist()
    if case["op"] == "append":
        return _exact_append(s, lens)
    return _exact_bounds(s) if case["op"] == "bounds" else _exact_sparse(s, lens)
