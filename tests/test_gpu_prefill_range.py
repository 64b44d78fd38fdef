"""GPU tests of tq_prefill_attn where one token takes nearly all of a row's weight,
and where many equal weights round alike: what the other tokens have left counts."""
import math

import numpy as np
import pytest

import synth
import tq_testlib as tl
from cache_cases import Cache, weights

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


def _bits(x):
    """float array -> bf16 bits, to nearest even."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def _scales(c, which, bits):
    """View of a one-layer, one-sequence, one-head cache's scales [n, 128]."""
    import torch
    off = 128 * c.d * bits // 8
    return c.rec[which][0, 0, 0, :, off:off + 512].view(torch.float32)


@pytest.mark.parametrize("place", ["first", "last"])
@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_one_token_takes_most_of_the_weight(tq, orc, d, place):
    """An attention sink over 32768 tokens in one split: its logit is 13 to 17 nats above a flat context,
    its value small, and the others' values have a part in common, so that the output is theirs.
    Bound: bf16's half step of the output's norm, 2^-8 (its own rounding is under 2^-9.5 of the norm; the
    sink's logit, at most 17, is off by 2^-11 of each of d products of one sign whose operands take 16
    values, 17 2^-11 / sqrt(8) = 2^-8.4 at the very most and 2^-10 in the mean)."""
    import torch
    n = 256
    c = Cache(tq, orc, B=1, Hkv=1, d=d, kb=4, vb=4, n=n, tail=4, seed=33)
    g = np.random.default_rng(d)
    x = 0.5 * g.standard_normal((1, n * 128, d)) + g.standard_normal(d)
    tq.tq_encode(c.vc, tl.to_bf16_tensor(_bits(x), "cuda"), c.rec["v"].view(1, n, -1))
    sink = 3 if place == "first" else n * 128 - 7
    ks, vs = _scales(c, "k", 4), _scales(c, "v", 4)
    ks *= torch.where(torch.arange(n * 128, device="cuda").view(n, 128) == sink, 1.0, 0.05)
    vs[sink // 128, sink % 128] *= 0.03
    c.ring["k"].mul_(0.05)
    c._host = {w: c.rec[w].cpu().numpy() for w in "kv"}
    k, v = c.vectors("k", 0, 0, 0), c.vectors("v", 0, 0, 0)
    gaps = np.array([13.0, 14.0, 15.0, 17.0])
    q = _bits((gaps[:, None] * k[sink] / (k[sink] @ k[sink]))[None, None].reshape(1, 1, 2, 2, d))
    out = torch.zeros((1, 1, 2, 2, d), dtype=torch.bfloat16, device="cuda")
    tq.prefill_attn(k_codec=c.kc, v_codec=c.vc, q=tl.to_bf16_tensor(q, "cuda"), out=out, scale=1.0, splits=1, **c.kw())
    got = synth.bf16_bits_to_f32(tl.bf16_tensor_bits(out)).astype(np.float64)
    qf = synth.bf16_bits_to_f32(q).astype(np.float64)
    for i in range(2):
        w = weights(qf[0, 0, :, i], k, 2, n * 128 + 4, True, 0.0, 1.0)
        assert w[:, sink].min() > 0.9
        want = w @ v
        e = np.linalg.norm(got[0, 0, :, i] - want, axis=-1) / np.linalg.norm(want, axis=-1)
        assert np.all(e <= 2.0 ** -8), e


@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_equal_weights_that_round_alike(tq, orc, d):
    """Ring tokens whose weights all lie just under the middle of two bf16 numbers (2^-3 (1 + 0.98 2^-8) of
    the largest): the sum they are divided by counts them as rounded.  Exactly, they hold 0.99 of the weight, so
    a common factor moves the output by a hundredth of itself: 2^-8 (the output's rounding) + 2^-10."""
    import torch
    t = math.log(0.125 * (1 + 0.98 * 2.0 ** -8))
    tail = 700
    c = Cache(tq, orc, B=1, Hkv=1, d=d, n=0, tail=tail, seed=34)
    g = np.random.default_rng(d)
    k, v = np.zeros((c.cap, d), np.float32), np.tile(g.standard_normal(d).astype(np.float32), (c.cap, 1))
    a = synth.bf16_bits_to_f32(_bits(np.float32(t)).reshape(1))[0]
    k[:, 0], k[:, 1] = a, t - a
    first = int(c.start[0, 0])
    k[first] = 0
    v[first] = 0
    c.ring["k"].copy_(tl.to_bf16_tensor(_bits(k), "cuda").view_as(c.ring["k"]))
    c.ring["v"].copy_(tl.to_bf16_tensor(_bits(v), "cuda").view_as(c.ring["v"]))
    q = np.zeros((1, 1, 1, 2, d), np.float32)
    q[..., :2] = 1
    out = torch.zeros((1, 1, 1, 2, d), dtype=torch.bfloat16, device="cuda")
    tq.prefill_attn(q=tl.to_bf16_tensor(_bits(q), "cuda"), out=out, scale=1.0, splits=1, **c.kw())
    got = synth.bf16_bits_to_f32(tl.bf16_tensor_bits(out)).astype(np.float64)
    kf, vf = c.vectors("k", 0, 0, 0), c.vectors("v", 0, 0, 0)
    want = weights(q[0, 0, :, 0].astype(np.float64), kf, 1, tail, True, 0.0, 1.0) @ vf
    for i in range(2):
        e = np.abs(got[0, 0, :, i] - want) / np.abs(want)
        assert np.all(e <= 2.0 ** -8 + 2.0 ** -10), float(e.max())


def _sinks(tq, orc, d, n, places, seed):
    """A cache of one head, n records and 4 ring tokens: at `places` one token's key, at its full length times
    a factor, and values of 0.03 of the others' norm; elsewhere keys of 0.05 and values with a part in common."""
    import torch
    c = Cache(tq, orc, B=1, Hkv=1, d=d, kb=4, vb=4, n=n, tail=4, seed=seed)
    g = np.random.default_rng(d + seed)
    x = 0.5 * g.standard_normal((1, n * 128, d)) + g.standard_normal(d)
    tq.tq_encode(c.vc, tl.to_bf16_tensor(_bits(x), "cuda"), c.rec["v"].view(1, n, -1))
    ks, vs, row = _scales(c, "k", 4), _scales(c, "v", 4), d // 2
    first, full = next(iter(places)), ks.clone()
    ks *= 0.05
    for at, factor in places.items():
        c.rec["k"][0, 0, 0, at // 128, at % 128 * row:(at % 128 + 1) * row] = c.rec["k"][0, 0, 0, first // 128, first % 128 * row:(first % 128 + 1) * row]
        ks[at // 128, at % 128] = full[first // 128, first % 128] * factor
        vs[at // 128, at % 128] *= 0.03
    c.ring["k"].mul_(0.05)
    c._host = {w: c.rec[w].cpu().numpy() for w in "kv"}
    return c, first


def _against(tq, c, at, gaps, softcap, splits):
    import torch
    d = c.d
    k, v = c.vectors("k", 0, 0, 0), c.vectors("v", 0, 0, 0)
    q = _bits((np.array(gaps)[:, None] * k[at] / (k[at] @ k[at])).reshape(1, 1, 2, 2, d))
    out = torch.zeros((1, 1, 2, 2, d), dtype=torch.bfloat16, device="cuda")
    tq.prefill_attn(k_codec=c.kc, v_codec=c.vc, q=tl.to_bf16_tensor(q, "cuda"), out=out, scale=1.0, softcap=softcap,
                    splits=splits, **c.kw())
    got = synth.bf16_bits_to_f32(tl.bf16_tensor_bits(out)).astype(np.float64)
    qf = synth.bf16_bits_to_f32(q).astype(np.float64)
    for i in range(2):
        w = weights(qf[0, 0, :, i], k, 2, len(k), True, softcap, 1.0)
        want = w @ v
        e = np.linalg.norm(got[0, 0, :, i] - want, axis=-1) / np.linalg.norm(want, axis=-1)
        assert np.all(e <= 2.0 ** -8), (e, w[:, at])


@pytest.mark.parametrize("softcap", [40.0, 400.0])
@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_one_token_takes_most_of_the_weight_under_a_cap(tq, orc, d, softcap):
    """As the first test, over 8192 tokens and with logits capped (below and above 177, two forms of the cap)."""
    c, at = _sinks(tq, orc, d, 64, {40: 1.0}, 35)
    _against(tq, c, at, [12.0, 13.0, 14.0, 16.0], softcap, 1)


@pytest.mark.parametrize("splits", [0, 1, 2])
@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_references_move_up_and_down(tq, orc, d, splits):
    """Tokens that dominate come and go: logits of 9, 12, 10 and 13 times a row's gain of 0.9 to 1.2 above 6144
    flat ones, in single records far apart and in neighbouring ones."""
    c, at = _sinks(tq, orc, d, 48, {5: 0.75, 900: 1.0, 4000: 0.83, 4001: 0.5, 4130: 1.08}, 36)
    _against(tq, c, at, [10.0, 11.0, 12.0, 13.3], 0.0, splits)
