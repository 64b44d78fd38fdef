"""GPU tests of tq_append against the rotation formula in 64 bits: axes, pair
layouts, partial rotation, far and negative positions, padded batches, fused
projections, in-place queries, full rings, counters and accumulated weights."""
import math

import numpy as np
import pytest

import synth
import tq_testlib as tl

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


def _turned(x, pos, freq, axis, rs, adjacent, scale):
    """x [T, heads, d] float64 -> rotated, and the size |x0| + |x1| behind each coordinate."""
    half = len(freq)
    y, size = x.copy(), np.zeros_like(x)
    for p in range(half):
        a, b = (rs + 2 * p, rs + 2 * p + 1) if adjacent else (rs + p, rs + half + p)
        ang = pos[axis[p]].astype(np.float64) * np.float64(freq[p])
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        y[..., a] = scale * (x[..., a] * c - x[..., b] * s)
        y[..., b] = scale * (x[..., b] * c + x[..., a] * s)
        size[..., a] = size[..., b] = abs(scale) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, size


CASES = [  # d, rot, rs, axes, adjacent, L, B, T, Hkv, G, far, scale
    (128, 128, 0, 3, False, 1, 1, 1, 2, 6, 1000, 1.0),
    (128, 64, 64, 1, True, 2, 3, 5, 2, 5, 100000, 1.0),
    (64, 64, 0, 2, False, 1, 2, 9, 3, 1, 1 << 30, 0.75),
    (64, 32, 8, 4, True, 1, 1, 3, 1, 8, 3, 1.0),
    (256, 256, 0, 3, True, 1, 2, 7, 1, 4, 50000, 1.0),
    (512, 64, 448, 1, False, 1, 2, 4, 1, 16, 70000, 1.25),
    (128, 48, 16, 3, False, 2, 2, 130, 1, 2, 4000, 1.0),
    (64, 0, 0, 1, False, 1, 2, 4, 2, 2, 10, 1.0),
]


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("d,rot,rs,axes,adjacent,L,B,T,Hkv,G,far,scale", CASES)
def test_append_against_the_formula(tq, shared, d, rot, rs, axes, adjacent, L, B, T, Hkv, G, far, scale):
    """Error of an output: the f32 rotation of its pair, then half a bf16 step.  The f32 part: cos
    and sin off by 2^-22 (their own 2 ulp, and 2^-23 from the angle's 24 bits), two products and a sum
    rounded at 2^-24 each: 2^-21 (|x0| + |x1|) covers them."""
    import torch
    rng = np.random.default_rng(5)
    Hq, cap = Hkv * G, T + 29
    bits = synth.gaussian_bf16((L, B, T, Hq + 2 * Hkv, d), 11)
    fused = tl.to_bf16_tensor(bits, "cuda")
    x = synth.bf16_bits_to_f32(bits).astype(np.float64)
    ring_bits = {w: synth.gaussian_bf16((L, B, Hkv, cap, d), 12 + i) for i, w in enumerate("kv")}
    ring = {w: tl.to_bf16_tensor(ring_bits[w], "cuda") for w in "kv"}
    start, ln = rng.integers(-3, 2 * cap, (L, B)), rng.integers(0, 29, (L, B))
    lens = rng.integers(0, T + 1, B)
    lens[0] = T
    pos = rng.integers(-far, far, (axes, B, T)).astype(np.int32)
    freq = (10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)
    axis = [p % axes for p in range(rot // 2)]
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
    qo = torch.full((L, B, T, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    d_len, out_len = i32(ln), i32(np.full((L, B), -5))
    kw = dict(positions=i32(pos), inv_freq=torch.from_numpy(freq).cuda(), pair_axis=axis) if rot else {}
    a = tq.make_append_args(q=fused[..., :Hq, :], k=fused[..., Hq:Hq + Hkv, :],
                            v=None if shared else fused[..., Hq + Hkv:, :], q_out=qo, rot_start=rs,
                            pair_adjacent=adjacent, rot_scale=scale, k_tail=ring["k"],
                            v_tail=None if shared else ring["v"], tail_start=i32(start), tail_len=d_len,
                            tail_len_out=out_len, q_lens=i32(lens), **kw)
    tq.tq_append(a)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(out_len.cpu().numpy(), ln + lens[None])
    np.testing.assert_array_equal(d_len.cpu().numpy(), ln)
    assert torch.equal(fused.view(torch.int16).cpu(), torch.from_numpy(bits.view(np.int16)))  # inputs untouched
    got_q = synth.bf16_bits_to_f32(tl.bf16_tensor_bits(qo)).astype(np.float64)
    got = {w: tl.bf16_tensor_bits(ring[w]) for w in "kv"}
    for l in range(L):
        for b in range(B):
            m = lens[b]
            y, size = _turned(x[l, b], pos[:, b], freq, axis, rs, adjacent, scale)
            tol = 2.0 ** -8 * np.abs(y) + 2.0 ** -20 * size
            assert np.all(np.abs(got_q[l, b, :m] - y[:m, :Hq]) <= tol[:m, :Hq])
            assert np.all(got_q[l, b, m:] == 7.0)  # rows of no token
            slot = (start[l, b] + ln[l, b] + np.arange(m)) % cap
            k = synth.bf16_bits_to_f32(got["k"][l, b]).astype(np.float64)[:, slot].transpose(1, 0, 2)
            assert np.all(np.abs(k - y[:m, Hq:Hq + Hkv]) <= tol[:m, Hq:Hq + Hkv])
            rest = np.setdiff1d(np.arange(cap), slot)
            np.testing.assert_array_equal(got["k"][l, b][:, rest], ring_bits["k"][l, b][:, rest])
            if shared:
                np.testing.assert_array_equal(got["v"], ring_bits["v"])
            else:
                np.testing.assert_array_equal(got["v"][l, b][:, slot].transpose(1, 0, 2), bits[l, b, :m, Hq + Hkv:])
                np.testing.assert_array_equal(got["v"][l, b][:, rest], ring_bits["v"][l, b][:, rest])


def _small(tq, T=3, cap=8, ln=(2, 6, 0, 9), **kw):
    import torch
    B, Hkv, G, d = len(ln), 2, 2, 64
    bf = lambda s, seed: tl.to_bf16_tensor(synth.gaussian_bf16(s, seed), "cuda")  # noqa: E731
    t = dict(q=bf((1, B, T, Hkv * G, d), 1), k=bf((1, B, T, Hkv, d), 2), v=bf((1, B, T, Hkv, d), 3),
             k_tail=bf((1, B, Hkv, cap, d), 4), v_tail=bf((1, B, Hkv, cap, d), 5),
             tail_len=torch.tensor([list(ln)], dtype=torch.int32, device="cuda"),
             positions=torch.arange(B * T, dtype=torch.int32, device="cuda").view(1, B, T),
             inv_freq=torch.linspace(1, 0.01, d // 2, device="cuda"))
    t["q_out"] = torch.empty_like(t["q"])
    t.update(kw)
    return t


def test_a_full_ring_is_left_alone_and_counters_in_place(tq):
    """Three tokens into a ring of 8: sequences of 2 and 0 take them, one of 6 does not, nor one whose
    length is out of range; queries are rotated everywhere; the counters move in place."""
    import torch
    t = _small(tq)
    before = t["k_tail"].clone()
    tq.tq_append(tq.make_append_args(**t))
    assert t["tail_len"].tolist() == [[5, 6, 3, 9]]
    assert torch.equal(before[0, 1], t["k_tail"][0, 1]) and torch.equal(before[0, 3], t["k_tail"][0, 3])
    assert not torch.equal(before[0, 0], t["k_tail"][0, 0])
    # in place: the queries' own buffer takes the rotated ones
    u = _small(tq)
    u["q_out"] = u["q"]
    tq.tq_append(tq.make_append_args(**u))
    assert torch.equal(u["q"], t["q_out"])


def test_new_tokens_start_without_weight(tq):
    import torch
    mass = torch.ones((1, 4, 2, 128 * 2 + 8), device="cuda")
    n = torch.tensor([[1, 2, 0, 1]], dtype=torch.int32, device="cuda")
    t = _small(tq, mass=mass, n_chunks=n, q_lens=torch.tensor([3, 3, 2, 3], dtype=torch.int32, device="cuda"))
    tq.tq_append(tq.make_append_args(**t))
    want = torch.ones_like(mass)
    want[0, 0, :, 130:133] = 0
    want[0, 2, :, 0:2] = 0
    assert torch.equal(mass, want)


def test_captured_and_replayed_on_another_stream(tq):
    import torch
    t, u = _small(tq, ln=(0, 1, 2, 3)), _small(tq, ln=(0, 1, 2, 3))
    a = tq.make_append_args(**t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        tq.tq_append(a)
    g.replay()
    torch.cuda.synchronize()
    assert t["tail_len"].tolist() == [[3, 4, 5, 6]]
    tq.tq_append(tq.make_append_args(**u))
    assert torch.equal(t["k_tail"], u["k_tail"]) and torch.equal(t["q_out"], u["q_out"])


def test_infinities_and_nans_pass(tq):
    """A non-finite coordinate reaches its own pair and nothing else."""
    import torch
    t = _small(tq, ln=(0, 0, 0, 0))
    clean = _small(tq, ln=(0, 0, 0, 0))
    t["k"][0, 1, 2, 1, 5] = math.inf
    t["k"][0, 1, 2, 1, 40] = math.nan
    for x in (t, clean):
        tq.tq_append(tq.make_append_args(**x))
    same = t["k_tail"] == clean["k_tail"]
    bad = torch.zeros_like(same)
    bad[0, 1, 1, 2, [5, 37, 8, 40]] = True
    assert torch.equal(~same, bad)
    assert torch.equal(t["v_tail"], clean["v_tail"])
