"""GPU tests of NaN and infinities that a query does see, in the several-query attention and the
accumulated weights: the rows concerned come out NaN on every route, the others as with clean inputs."""
import math

import numpy as np
import pytest

import tq_testlib as tl
from cache_cases import Cache, queries

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


def _put_scale(c, which, bits, h, record, slot, value):
    import torch
    off = 128 * c.d * bits // 8 + 4 * slot
    c.rec[which][0, 0, h, record, off:off + 4] = torch.tensor([value], device="cuda").view(torch.uint8)


def _attend(tq, c, q, **kw):
    import torch
    out = torch.full_like(q, 5.0)
    tq.prefill_attn(k_codec=c.kc, v_codec=c.vc, q=q, out=out, scale=1.0, **kw, **c.kw())
    torch.cuda.synchronize()
    return out


T, G = 12, 3


def _cache(tq, orc, d, **kw):
    return Cache(tq, orc, **dict(dict(B=1, Hkv=2, d=d, kb=3, vb=4, n=7, tail=150, seed=51), **kw))


@pytest.mark.parametrize("splits", [0, 1, 4])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_attention_of_a_query_with_nan(tq, orc, d, softcap, splits):
    import torch
    c = _cache(tq, orc, d)
    q = tl.to_bf16_tensor(queries(1, 1, T, 2 * G, d, 5), "cuda")
    clean = _attend(tq, c, q, splits=splits, softcap=softcap)
    bad = q.clone()
    bad[0, 0, 4, 1, d // 2] = math.nan
    bad[0, 0, 9, 5, 0] = math.nan
    out = _attend(tq, c, bad, splits=splits, softcap=softcap)
    hit = torch.zeros((T, 2 * G), dtype=torch.bool, device="cuda")
    hit[4, 1] = hit[9, 5] = True
    assert torch.isnan(out[0, 0][hit]).all()
    assert torch.equal(out[0, 0][~hit], clean[0, 0][~hit])


@pytest.mark.parametrize("splits", [0, 1, 4])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_attention_over_a_scale_that_is_not_finite(tq, orc, d, value, splits):
    """One record of seven; the other kv head is untouched.  A key's scale, then a value's."""
    import torch
    c = _cache(tq, orc, d)
    q = tl.to_bf16_tensor(queries(1, 1, T, 2 * G, d, 6), "cuda")
    clean = _attend(tq, c, q, splits=splits)
    saved = {w: c.rec[w].clone() for w in "kv"}
    for which, bits in (("k", 3), ("v", 4)):
        c.rec[which].copy_(saved[which])
        _put_scale(c, which, bits, 1, 2, 77, value)
        out = _attend(tq, c, q, splits=splits)
        assert not torch.isfinite(out[0, 0, :, G:]).any()
        assert torch.isnan(out[0, 0, :, G:]).all() or which == "v"
        assert torch.equal(out[0, 0, :, :G], clean[0, 0, :, :G])
        c.rec[which].copy_(saved[which])


@pytest.mark.parametrize("splits", [0, 1])
@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_attention_over_a_ring_key_with_nan(tq, orc, d, splits):
    """The key of new token 7: queries from it on see it."""
    import torch
    c = _cache(tq, orc, d)
    q = tl.to_bf16_tensor(queries(1, 1, T, 2 * G, d, 7), "cuda")
    clean = _attend(tq, c, q, splits=splits)
    slot = (int(c.start[0, 0]) + 150 - T + 7) % c.cap
    c.ring["k"][0, 0, 0, slot, 3] = math.nan
    out = _attend(tq, c, q, splits=splits)
    assert torch.isnan(out[0, 0, 7:, :G]).all()
    assert torch.equal(out[0, 0, :7], clean[0, 0, :7]) and torch.equal(out[0, 0, :, G:], clean[0, 0, :, G:])


@pytest.mark.parametrize("d", [64, 256])
def test_attention_whose_logits_are_all_minus_infinity(tq, orc, d):
    """A row that sees tokens, but none of a finite logit, is NaN; one that sees no token is zero."""
    import torch
    c = _cache(tq, orc, d, n=0, tail=40)
    q = torch.zeros((1, 1, 50, 2, d), dtype=torch.bfloat16, device="cuda")
    q[..., 3] = -math.inf
    c.ring["k"].fill_(1.0)
    out = _attend(tq, c, q)
    assert torch.all(out[0, 0, :10] == 0) and torch.isnan(out[0, 0, 10:]).all()


# rows of a kv head: up to 8, 9 to 40, more; head dim 256 has no tcgen05 route
ROUTES = [(128, 1, 4), (128, 2, 4), (512, 1, 6), (64, 5, 4), (128, 5, 4), (256, 20, 3), (64, 30, 3), (128, 30, 3)]


def _weigh(tq, c, q, mass0, **kw):
    import torch
    mass = mass0.clone()
    tq.attn_mass(k_codec=c.kc, mass=mass, q=q, scale=1.0, decay=0.5, **kw, **c.kw(values=False))
    torch.cuda.synchronize()
    return mass


@pytest.mark.parametrize("outliers", [0.0, 2.0])
@pytest.mark.parametrize("splits", [0, 1, 4])
@pytest.mark.parametrize("d,rows_t,group", ROUTES)
def test_weights_of_what_is_not_finite(tq, orc, d, rows_t, group, splits, outliers):
    """A row without a finite softmax leaves NaN in every entry of its kv head below total, whichever way
    the rows are laid out; entries behind it and the other kv heads are as with clean inputs."""
    import torch
    c = _cache(tq, orc, d, T=outliers)
    total = 7 * 128 + 150
    g = np.random.default_rng(3)
    mass0 = torch.from_numpy(g.random((1, 1, 2, total + 9)).astype(np.float32)).cuda()
    q = tl.to_bf16_tensor(queries(1, 1, rows_t, 2 * group, d, 8), "cuda")
    clean = _weigh(tq, c, q, mass0, splits=splits)
    assert torch.isfinite(clean).all()

    def check(mass, h):
        assert torch.isnan(mass[0, 0, h, :total]).all()
        assert torch.equal(mass[0, 0, h, total:], mass0[0, 0, h, total:])
        assert torch.equal(mass[0, 0, 1 - h], clean[0, 0, 1 - h])

    bad = q.clone()
    bad[0, 0, rows_t - 1, 1, d - 1] = math.nan
    check(_weigh(tq, c, bad, mass0, splits=splits), 0)
    keys = c.rec["k"].clone()
    for value in (math.nan, math.inf, -math.inf):
        for record, slot in ((0, 0), (3, 100)):
            c.rec["k"].copy_(keys)
            _put_scale(c, "k", 3, 1, record, slot, value)
            check(_weigh(tq, c, q, mass0, splits=splits), 1)
    c.rec["k"].copy_(keys)
    c.ring["k"][0, 0, 0, (int(c.start[0, 0]) + 140) % c.cap, 1] = math.nan
    check(_weigh(tq, c, q, mass0, splits=splits), 0)


@pytest.mark.parametrize("d,rows_t,group", [(128, 1, 4), (128, 5, 4), (128, 30, 3)])
def test_weights_whose_logits_are_all_minus_infinity(tq, orc, d, rows_t, group):
    """Rows that see tokens of no finite logit leave NaN; where no row sees a token, the decay alone is applied."""
    import torch
    c = _cache(tq, orc, d, n=0, tail=40, B=2, lens=(0, [[40, 0]]))
    q = torch.zeros((1, 2, rows_t, 2 * group, d), dtype=torch.bfloat16, device="cuda")
    q[..., 3] = -math.inf
    c.ring["k"].fill_(1.0)
    mass = _weigh(tq, c, q, torch.ones((1, 2, 2, 41), device="cuda"))
    assert torch.isnan(mass[0, 0, :, :40]).all() and torch.all(mass[0, 0, :, 40:] == 1) and torch.all(mass[0, 1] == 1)


@pytest.mark.parametrize("value", [math.inf, -math.inf])
@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_a_query_with_an_infinity(tq, orc, d, value):
    """Its row is NaN in the attention, its kv head's entries in the weights (few rows and many); others as before."""
    import torch
    c = _cache(tq, orc, d)
    q = tl.to_bf16_tensor(queries(1, 1, T, 2 * G, d, 9), "cuda")
    bad = q.clone()
    bad[0, 0, T - 1, 1, 5] = value
    hit = torch.zeros((T, 2 * G), dtype=torch.bool, device="cuda")
    hit[T - 1, 1] = True
    clean, out = _attend(tq, c, q), _attend(tq, c, bad)
    assert torch.isnan(out[0, 0][hit]).all() and torch.equal(out[0, 0][~hit], clean[0, 0][~hit])
    total = 7 * 128 + 150
    mass0 = torch.ones((1, 1, 2, total + 3), device="cuda")
    for t in (2, 4, T):  # rows of a kv head: 6, 12, 36
        x, y = _weigh(tq, c, q[:, :, -t:], mass0), _weigh(tq, c, bad[:, :, -t:], mass0)
        assert torch.isnan(y[0, 0, 0, :total]).all() and torch.equal(y[0, 0, 1], x[0, 0, 1])
        assert torch.all(y[0, 0, :, total:] == 1)
