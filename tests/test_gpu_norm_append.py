"""GPU tests of tq_norm_append against norm and rotation in 64 bits: sides that
are normalised, weights per head, pair layouts, padded batches, in-place
queries, heads of zeros, counters, capture."""
import math

import numpy as np
import pytest

import synth
import tq_testlib as tl
from test_gpu_append import _small, _turned

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


CASES = [  # d, rot, rs, adjacent, L, B, T, Hkv, G, far, scale, sides, per head, eps
    (128, 128, 0, False, 1, 1, 1, 2, 6, 1000, 1.0, "qk", False, 1e-6),
    (128, 64, 64, True, 2, 3, 5, 2, 5, 100000, 1.0, "qk", True, 1e-5),
    (64, 64, 0, False, 1, 2, 9, 3, 1, 1 << 30, 0.75, "k", True, 1e-6),
    (64, 32, 8, True, 1, 1, 3, 1, 8, 3, 1.0, "q", False, 0.5),
    (256, 256, 0, True, 1, 2, 7, 1, 4, 50000, 1.0, "qk", True, 1e-6),
    (512, 64, 448, False, 1, 2, 4, 1, 16, 70000, 1.25, "qk", False, 1e-6),
    (128, 48, 16, False, 2, 2, 130, 1, 2, 4000, 1.0, "qk", True, 1e-6),
    (64, 0, 0, False, 1, 2, 4, 2, 2, 10, 1.0, "qk", False, 1e-6),
    (64, 64, 0, False, 2, 2, 1211, 1, 2, 5000, 1.0, "qk", True, 1e-6),  # tokens enough for eight a CTA
    (128, 96, 32, True, 1, 3, 811, 2, 3, 5000, 1.0, "k", False, 1e-6),
    (256, 128, 0, False, 1, 1, 2437, 1, 1, 5000, 1.0, "q", False, 1e-6),
    (512, 64, 448, True, 1, 2, 1217, 1, 2, 5000, 1.0, "qk", False, 1e-6),
]


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("d,rot,rs,adjacent,L,B,T,Hkv,G,far,scale,sides,per_head,eps", CASES)
def test_norms_against_the_formula(tq, shared, d, rot, rs, adjacent, L, B, T, Hkv, G, far, scale, sides, per_head, eps):
    """Error of an output: half a bf16 step, and in f32: d squares summed in pairs and by shuffles (at most
    (16 + 6) 2^-24 relative, half of it after the root), the root's 2 ulp, two products (2^-23), then the
    rotation's 2^-21 of its pair: under 2^-19 (|x0| + |x1|) together."""
    import torch
    rng = np.random.default_rng(5)
    Hq, cap = Hkv * G, T + 29
    bits = synth.gaussian_bf16((L, B, T, Hq + 2 * Hkv, d), 11, scale=1.7)
    fused = tl.to_bf16_tensor(bits, "cuda")
    x = synth.bf16_bits_to_f32(bits).astype(np.float64)
    ring_bits = {w: synth.gaussian_bf16((L, B, Hkv, cap, d), 12 + i) for i, w in enumerate("kv")}
    ring = {w: tl.to_bf16_tensor(ring_bits[w], "cuda") for w in "kv"}
    start, ln = rng.integers(-3, 2 * cap, (L, B)), rng.integers(0, 29, (L, B))
    lens = rng.integers(0, T + 1, B)
    lens[0] = T
    pos = rng.integers(-far, far, (1, B, T)).astype(np.int32)
    freq = (10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)
    wt = {"q": rng.normal(1.0, 0.5, (Hq if per_head else 1, d)).astype(np.float32),
          "k": rng.normal(1.0, 0.5, (Hkv if per_head else 1, d)).astype(np.float32)}
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
    qo = torch.full((L, B, T, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    d_len, out_len = i32(ln), i32(np.full((L, B), -5))
    kw = dict(positions=i32(pos), inv_freq=torch.from_numpy(freq).cuda()) if rot else {}
    a = tq.make_append_args(q=fused[..., :Hq, :], k=fused[..., Hq:Hq + Hkv, :],
                            v=None if shared else fused[..., Hq + Hkv:, :], q_out=qo, rot_start=rs,
                            pair_adjacent=adjacent, rot_scale=scale, k_tail=ring["k"],
                            v_tail=None if shared else ring["v"], tail_start=i32(start), tail_len=d_len,
                            tail_len_out=out_len, q_lens=i32(lens), **kw)
    dev = {s: torch.from_numpy(wt[s] if per_head else wt[s][0]).cuda() for s in "qk"}
    norm = tq.make_head_norm(**{s + "_weight": dev[s] for s in sides}, eps=eps)
    tq.tq_norm_append(a, norm)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(out_len.cpu().numpy(), ln + lens[None])
    assert torch.equal(fused.view(torch.int16).cpu(), torch.from_numpy(bits.view(np.int16)))  # inputs untouched
    y = x.copy()
    eps32 = float(np.float32(eps))
    for s, at in (("q", slice(0, Hq)), ("k", slice(Hq, Hq + Hkv))):
        if s in sides:
            y[..., at, :] *= wt[s].astype(np.float64) / np.sqrt((y[..., at, :] ** 2).mean(-1, keepdims=True) + eps32)
    got_q = synth.bf16_bits_to_f32(tl.bf16_tensor_bits(qo)).astype(np.float64)
    got = {w: tl.bf16_tensor_bits(ring[w]) for w in "kv"}
    for l in range(L):
        for b in range(B):
            m = lens[b]
            z, size = _turned(y[l, b], pos[:, b], freq, [0] * (rot // 2), rs, adjacent, scale)
            tol = 2.0 ** -8 * np.abs(z) + 2.0 ** -19 * (size + np.abs(z))
            assert np.all(np.abs(got_q[l, b, :m] - z[:m, :Hq]) <= tol[:m, :Hq])
            assert np.all(got_q[l, b, m:] == 7.0)  # rows of no token
            slot = (start[l, b] + ln[l, b] + np.arange(m)) % cap
            k = synth.bf16_bits_to_f32(got["k"][l, b]).astype(np.float64)[:, slot].transpose(1, 0, 2)
            assert np.all(np.abs(k - z[:m, Hq:Hq + Hkv]) <= tol[:m, Hq:Hq + Hkv])
            rest = np.setdiff1d(np.arange(cap), slot)
            np.testing.assert_array_equal(got["k"][l, b][:, rest], ring_bits["k"][l, b][:, rest])
            if shared:
                np.testing.assert_array_equal(got["v"], ring_bits["v"])
            else:
                np.testing.assert_array_equal(got["v"][l, b][:, slot].transpose(1, 0, 2), bits[l, b, :m, Hq + Hkv:])
                np.testing.assert_array_equal(got["v"][l, b][:, rest], ring_bits["v"][l, b][:, rest])


def _ones(tq, d=64, **kw):
    import torch
    return tq.make_head_norm(q_weight=torch.ones(d, device="cuda"), k_weight=torch.ones(d, device="cuda"), **kw)


def test_heads_of_zeros_and_non_finite_ones(tq):
    """Zeros stay zeros with an eps and become NaN without one; a NaN or an infinity takes its own head and
    no other (an infinite norm leaves zeros beside the NaN of the infinity's own place)."""
    import torch
    for eps in (1e-6, 0.0):
        t = _small(tq, ln=(0, 0, 0, 0))
        t["k"][0, 0, 1, 0] = 0
        t["k"][0, 1, 2, 1, 5] = math.nan
        clean = _small(tq, ln=(0, 0, 0, 0))
        for x in (t, clean):
            tq.tq_norm_append(tq.make_append_args(**x), _ones(tq, eps=eps))
        got = t["k_tail"]
        if eps:
            assert torch.all(got[0, 0, 0, 1] == 0)
        else:
            assert torch.all(got[0, 0, 0, 1].isnan())
        assert torch.all(got[0, 1, 1, 2].isnan())
        same = got == clean["k_tail"]
        same[0, 0, 0, 1] = same[0, 1, 1, 2] = True
        assert torch.all(same)
        assert torch.equal(t["q_out"], clean["q_out"]) and torch.equal(t["v_tail"], clean["v_tail"])


def test_in_place_full_rings_and_counters(tq):
    """As the append without norms: a ring that is full keeps its tokens, queries are turned in place."""
    import torch
    t, u = _small(tq), _small(tq)
    before = t["k_tail"].clone()
    tq.tq_norm_append(tq.make_append_args(**t), _ones(tq))
    assert t["tail_len"].tolist() == [[5, 6, 3, 9]]
    assert torch.equal(before[0, 1], t["k_tail"][0, 1]) and torch.equal(before[0, 3], t["k_tail"][0, 3])
    assert not torch.equal(before[0, 0], t["k_tail"][0, 0])
    u["q_out"] = u["q"]
    tq.tq_norm_append(tq.make_append_args(**u), _ones(tq))
    assert torch.equal(u["q"], t["q_out"])


def test_many_tokens_in_place(tq):
    """Eight tokens a CTA, the queries' own buffer taking the normalised ones, counters moving in place."""
    import torch
    T, ln = 700, (0, 3, 1, 2)
    far, here = _small(tq, T=T, cap=800, ln=ln), _small(tq, T=T, cap=800, ln=ln)
    here["q_out"] = here["q"]
    for t in (far, here):
        tq.tq_norm_append(tq.make_append_args(**t), _ones(tq))
    assert torch.equal(here["q"], far["q_out"]) and torch.equal(here["k_tail"], far["k_tail"])
    assert here["tail_len"].tolist() == [[T + n for n in ln]]


def test_captured_and_replayed_on_another_stream(tq):
    import torch
    t, u = _small(tq, ln=(0, 1, 2, 3)), _small(tq, ln=(0, 1, 2, 3))
    a, norm = tq.make_append_args(**t), _ones(tq)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        tq.tq_norm_append(a, norm)
    g.replay()
    torch.cuda.synchronize()
    assert t["tail_len"].tolist() == [[3, 4, 5, 6]]
    tq.tq_norm_append(tq.make_append_args(**u), norm)
    assert torch.equal(t["k_tail"], u["k_tail"]) and torch.equal(t["q_out"], u["q_out"])


def test_weights_of_other_shapes_are_refused(tq):
    import torch
    a = tq.make_append_args(**_small(tq))
    w = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    for bad in (dict(q_weight=w(32)), dict(q_weight=w(3, 64)), dict(k_weight=w(4, 64)), dict(k_weight=w(128))):
        with pytest.raises(ValueError):
            tq.tq_norm_append(a, tq.make_head_norm(**bad))
    with pytest.raises(tq.TqError):
        tq.tq_norm_append(a, tq.make_head_norm())
    wide = w(4, 72)[:, 4:68]  # heads 72 apart, 16-byte aligned
    tq.tq_norm_append(a, tq.make_head_norm(q_weight=wide))
