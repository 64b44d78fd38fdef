"""GPU tests of tq_attn_mass against softmax weights in 64 bits over the
oracle's decode of the same records."""
import math

import numpy as np
import pytest

import synth
import tq_testlib as tl
from cache_cases import Cache, queries, weights

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


def _check(tq, c, T, G, *, lens=None, causal=True, softcap=0.0, decay=0.5, splits=0, seed=21, gain=1.5):
    """A product's operands hold 22 bits (hi + lo halves; lo lo left out: 3 2^-22 together) and the f32
    sum of 3 d / 16 matrix instructions rounds each time at 2^-23 of what it holds (twice that where an
    instruction truncates), so a logit is off by at most 2^-22 (3 + 3 d / 16) sum |q~ c| n scale
    <= that |q||k|; a weight by twice that relative to itself; the sums' own roundings are below
    2^-20 of the sum, and the running sum's 2^-24 twice."""
    import torch
    q = queries(c.L, c.B, T, c.Hkv * G, c.d, seed, gain)
    qf = synth.bf16_bits_to_f32(q).astype(np.float64)
    cap = 128 * c.max_chunks + c.max_tail + 5
    rng = np.random.default_rng(seed)
    m0 = rng.random((c.L, c.B, c.Hkv, cap)).astype(np.float32)
    mass = torch.from_numpy(m0.copy()).cuda()
    dl = None if lens is None else torch.from_numpy(np.asarray(lens, np.int32)).cuda()
    tq.attn_mass(k_codec=c.kc, mass=mass, decay=decay, q=tl.to_bf16_tensor(q, "cuda"), scale=1.0, softcap=softcap,
                 causal=causal, q_lens=dl, splits=splits, **c.kw(values=False))
    got = mass.cpu().numpy()
    for l in range(c.L):
        for b in range(c.B):
            m = T if lens is None else int(lens[b])
            total = 128 * int(c.n[l, b]) + int(c.len[l, b])
            np.testing.assert_array_equal(got[l, b, :, total:], m0[l, b, :, total:])
            for h in range(c.Hkv):
                k = c.vectors("k", l, b, h)
                kn = np.linalg.norm(k, axis=-1).max() if total else 0.0
                want, tol = np.zeros(total), np.zeros(total)
                for i in range(G):
                    w = weights(qf[l, b, :, h * G + i], k, m, total, causal, softcap, 1.0)[:m]
                    ds = 2.0 ** -22 * (3 + 3 * c.d / 16) * np.linalg.norm(qf[l, b, :m, h * G + i], axis=-1) * kn
                    want += w.sum(0)
                    tol += (w * (np.expm1(2 * ds) + 2.0 ** -20)[:, None]).sum(0)
                want = decay * m0[l, b, h, :total].astype(np.float64) + want
                tol += 2.0 ** -23 * np.abs(want) + 1e-12
                e = np.abs(got[l, b, h, :total] - want)
                assert np.all(e <= tol), (l, b, h, float((e / tol).max()))
    return got


CASES = {
    "decode": dict(d=128, G=6, T=1, L=2, B=3),
    "decode_d64_one_bit": dict(d=64, G=8, T=1, kb=1, n=4),
    "decode_three_bits": dict(d=64, G=3, T=1, kb=3, n=4),
    "decode_d512": dict(d=512, G=8, T=1, kb=4, Hkv=1, n=2),
    "mqa_d512": dict(d=512, G=64, T=2, kb=4, Hkv=1, n=3, tail=20),
    "window": dict(d=128, G=4, T=33, n=3, tail=150, kb=3),
    "window_ragged": dict(d=128, G=5, T=40, n=2, tail=60, B=3, lens=[40, 3, 1]),
    "side_lists": dict(d=128, G=4, T=1, T_out=2.0, n=3),
    "side_lists_window": dict(d=64, G=4, T=13, T_out=1.5, kb=2, n=3),
    "side_lists_d512": dict(d=512, G=16, T=2, T_out=2.0, Hkv=1, kb=3, n=2),
    "d256": dict(d=256, G=4, T=5, kb=2, n=3),
    "paged": dict(d=128, G=4, T=3, paged=True, n=6, B=3, L=2),
    "softcap": dict(d=128, G=2, T=5, softcap=3.0),
    "not_causal": dict(d=64, G=4, T=19, causal=False),
    "records_only": dict(d=128, G=2, T=3, tail=0, n=2),
    "ring_only": dict(d=128, G=4, T=10, n=0, tail=200),
    "queries_in_the_records": dict(d=128, G=3, T=150, n=3, tail=60),
    "more_queries_than_tokens": dict(d=64, G=2, T=50, n=0, tail=20),
    "window_softcap": dict(d=128, G=4, T=12, softcap=3.0, n=3),
    "window_paged_two_bits": dict(d=64, G=3, T=50, kb=2, paged=True, n=6, B=3, L=2),
    "window_one_bit": dict(d=128, G=8, T=20, kb=1, n=5, tail=10),
    "twenty_rows": dict(d=128, G=4, T=5, n=4, kb=3),
    "nobody_asks_a_window": dict(d=64, G=8, T=9, lens=[0, 9]),
    "nobody_asks": dict(d=64, G=2, T=4, lens=[0, 0]),
}


@pytest.mark.parametrize("splits", [0, 2])
@pytest.mark.parametrize("name", CASES)
def test_mass_against_the_formula(tq, orc, name, splits):
    kw = dict(CASES[name])
    call = {k: kw.pop(k) for k in ("G", "T", "lens", "causal", "softcap") if k in kw}
    c = Cache(tq, orc, T=kw.pop("T_out", 0.0), seed=13, **kw)
    _check(tq, c, splits=splits, **call)


@pytest.mark.parametrize("T", [1, 7, 30])
def test_a_negative_scale(tq, orc, T):
    """The softmax scale's sign belongs to the logits on every route (few rows, some, many)."""
    import torch
    c = Cache(tq, orc, B=1, Hkv=1, d=128, n=3, tail=30, seed=29)
    q = queries(1, 1, T, 3, 128, 5)
    mass = torch.zeros((1, 1, 1, 128 * 3 + 30), device="cuda")
    tq.attn_mass(k_codec=c.kc, mass=mass, q=tl.to_bf16_tensor(q, "cuda"), scale=-1.0, **c.kw(values=False))
    qf = synth.bf16_bits_to_f32(q).astype(np.float64)
    want = sum(weights(qf[0, 0, :, i], c.vectors("k", 0, 0, 0), T, 128 * 3 + 30, True, 0.0, -1.0).sum(0) for i in range(3))
    assert np.abs(mass.cpu().numpy()[0, 0, 0] - want).max() <= 1e-4 * want.max()


@pytest.mark.parametrize("T", [1, 7, 30])
def test_huge_logits(tq, orc, T):
    """Logits of hundreds: one token takes each row's weight, nothing overflows."""
    import torch
    c = Cache(tq, orc, B=1, Hkv=1, d=128, n=4, tail=20, seed=30)
    q = queries(1, 1, T, 3, 128, 6, gain=100.0)
    mass = torch.zeros((1, 1, 1, 128 * 4 + 20), device="cuda")
    tq.attn_mass(k_codec=c.kc, mass=mass, q=tl.to_bf16_tensor(q, "cuda"), scale=1.0, **c.kw(values=False))
    got = mass.cpu().numpy()[0, 0, 0].astype(np.float64)
    assert np.isfinite(got).all() and abs(got.sum() / (3 * T) - 1) <= 2.0 ** -12


def test_every_query_gives_a_weight_of_one(tq, orc):
    """Rows that see a token sum to one: the total is query heads x tokens, to f32."""
    import torch
    c = Cache(tq, orc, B=1, Hkv=2, d=128, n=8, tail=200, seed=17)
    T, G = 24, 4
    mass = torch.zeros((1, 1, 2, 128 * 8 + 200), device="cuda")
    q = tl.to_bf16_tensor(queries(1, 1, T, 2 * G, 128, 3), "cuda")
    for k in range(1, 4):
        tq.attn_mass(k_codec=c.kc, mass=mass, q=q, scale=1.0, **c.kw(values=False))
        assert abs(float(mass[0, 0, 0].double().sum()) / (k * T * G) - 1) <= 2.0 ** -16


def test_decay_zero_replaces_even_nan(tq, orc):
    """decay 0 multiplies: NaN that was there stays NaN, finite entries are replaced."""
    import torch
    c = Cache(tq, orc, B=1, Hkv=1, n=1, tail=0, seed=19)
    mass = torch.full((1, 1, 1, 128), 5.0, device="cuda")
    mass[0, 0, 0, 7] = math.nan
    q = tl.to_bf16_tensor(queries(1, 1, 1, 1, 128, 3), "cuda")
    tq.attn_mass(k_codec=c.kc, mass=mass, decay=0.0, q=q, scale=1.0, **c.kw(values=False))
    assert int(torch.isnan(mass).sum()) == 1 and float(mass.nansum()) <= 1.0


def test_same_bits_every_time_and_from_a_graph(tq, orc):
    import torch
    c = Cache(tq, orc, B=2, n=9, tail=140, seed=23)
    q = tl.to_bf16_tensor(queries(1, 2, 20, 8, 128, 9), "cuda")
    one, two = (torch.zeros((1, 2, 2, 128 * 9 + 140), device="cuda") for _ in range(2))
    a = tq.make_query_args(q=q, scale=1.0, **c.kw(values=False))
    ws = torch.empty(tq.tq_attn_mass_workspace_size(a, c.kc), dtype=torch.uint8, device="cuda")
    tq.tq_attn_mass(a, c.kc, one, ws)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        tq.tq_attn_mass(a, c.kc, two, ws)
    ws.fill_(0xFF)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(one, two)


MORE = {
    "decode_d256": dict(d=256, G=5, T=1, kb=3, n=4, L=2, B=3),
    "decode_d256_side_lists": dict(d=256, G=4, T=2, T_out=2.0, n=3),
    "window_d256_paged": dict(d=256, G=4, T=21, kb=4, paged=True, n=4, B=3, L=2),
    "window_d512_side_lists": dict(d=512, G=8, T=9, T_out=2.0, Hkv=1, kb=2, n=3),
}


@pytest.mark.parametrize("splits", [0, 2])
@pytest.mark.parametrize("name", MORE)
def test_more_layouts_against_the_formula(tq, orc, name, splits):
    kw = dict(MORE[name])
    call = {k: kw.pop(k) for k in ("G", "T", "lens", "causal", "softcap") if k in kw}
    c = Cache(tq, orc, T=kw.pop("T_out", 0.0), seed=14, **kw)
    _check(tq, c, splits=splits, **call)


@pytest.mark.parametrize("T,G", [(1, 4), (6, 4), (23, 4)])
def test_runs_longer_than_a_split_may_be(tq, orc, T, G):
    """One split is asked for over 101 records: the routes that keep a split's sums in shared memory take as many as they need."""
    c = Cache(tq, orc, B=1, Hkv=1, d=64, kb=2, n=101, tail=100, seed=15)
    _check(tq, c, T, G, splits=1)
