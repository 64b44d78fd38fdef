"""GPU tests of tq_prefill_attn against softmax attention in 64 bits over the
oracle's decode of the same records: head dims, group sizes, bit widths, side
lists, pages, ragged batches, rows that see nothing, splits, strides."""
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


def _run(tq, c, q, lens, G, *, causal=True, softcap=0.0, scale=1.0, splits=0, fill=9.0):
    import torch
    L, B, T, Hq, d = q.shape
    wide = torch.full((L, B, T, Hq + 1, d), fill, dtype=torch.bfloat16, device="cuda")  # a strided output
    out = wide[..., :Hq, :]
    dl = None if lens is None else torch.from_numpy(np.asarray(lens, np.int32)).cuda()
    tq.prefill_attn(k_codec=c.kc, v_codec=c.vc, q=tl.to_bf16_tensor(q, "cuda"), out=out, scale=scale, softcap=softcap,
                    causal=causal, q_lens=dl, splits=splits, **c.kw())
    torch.cuda.synchronize()
    assert torch.all(wide[..., Hq:, :] == fill)
    return out


def _check(c, q, lens, G, got, *, causal=True, softcap=0.0, scale=1.0, fill=9.0):
    """Elementwise: a score's operands are off by half an f16 step each (2^-11, the ring's not at all),
    so by 2^-10 sum |q~ c| n <= 2^-10 |q| |k|; a weight by twice that relative to itself and the
    weighted value by 2^-11 (weight; bf16's 2^-8 in the ring) + 2^-11 (centroid); the output by 2^-8 of
    itself.  The roundings of a record's values, 2^-11 of a centroid and 2^-11 of its product with the
    scale, are made in the rotated basis: with errors |e_r| <= 2^-10 |y_r| there, a coordinate is off by
    at most sum |e_r| / sqrt(d) <= 2^-10 |y| = 2^-10 |v|, however small it is itself.  The norm of the whole: those errors are independent, 2^-12.8 |q||k| / sqrt(d) a score and
    bf16's 2^-9.8 at the end, together under 2^-8 of the output's norm for |q||k| / sqrt(d) <= 3."""
    L, B, T, Hq, d = q.shape
    qf = synth.bf16_bits_to_f32(q).astype(np.float64)
    g = synth.bf16_bits_to_f32(tl.bf16_tensor_bits(got.contiguous())).astype(np.float64)
    err2 = ref2 = 0.0
    for l in range(L):
        for b in range(B):
            m = T if lens is None else int(lens[b])
            total = 128 * int(c.n[l, b]) + int(c.len[l, b])
            assert np.all(g[l, b, m:] == fill)
            for h in range(c.Hkv):
                k, v = c.vectors("k", l, b, h), c.vectors("v", l, b, h)
                for i in range(G):
                    hq = h * G + i
                    w = weights(qf[l, b, :, hq], k, m, total, causal, softcap, scale)[:m]
                    want = w @ v
                    size = w @ np.abs(v)
                    turned = 2.0 ** -10 * (w @ np.linalg.norm(v, axis=-1))[:, None]
                    ds = 2.0 ** -10 * scale * np.linalg.norm(qf[l, b, :m, hq], axis=-1) * (
                        np.linalg.norm(k, axis=-1).max() if len(k) else 0.0)
                    tol = 2.0 ** -8 * np.abs(want) + (np.expm1(2 * ds)[:, None] + 2.0 ** -7.5) * size * 1.01 + turned + 1e-6
                    e = np.abs(g[l, b, :m, hq] - want)
                    assert np.all(e <= tol), (l, b, hq, float((e / tol).max()))
                    err2 += float((e ** 2).sum())
                    ref2 += float((want ** 2).sum())
    assert math.sqrt(err2) <= 2.0 ** -8 * math.sqrt(ref2) + 1e-6, math.sqrt(err2 / ref2)


CASES = {
    "one_token": dict(d=128, G=6, T=1),
    "verify_d64": dict(d=64, G=7, T=5, kb=3, vb=2, B=3, lens=[5, 2, 4]),
    "rows_cross_tiles": dict(d=128, G=5, T=67, n=2, tail=131, B=3, lens=[67, 0, 31]),
    "side_lists": dict(d=128, G=4, T=9, T_out=2.0, kb=4, vb=3, n=3),
    "side_lists_d64_shared": dict(d=64, G=2, T=4, T_out=1.5, kb=2, shared=True, n=2),
    "d256_one_bit": dict(d=256, G=3, T=11, kb=1, vb=1, n=2, tail=40),
    "d512_shared": dict(d=512, G=16, T=6, kb=4, shared=True, Hkv=1, n=3, tail=33, B=3, lens=[6, 5, 1]),
    "d512_apart": dict(d=512, G=2, T=40, kb=3, vb=4, Hkv=2, n=2, tail=50),
    "paged": dict(d=128, G=3, T=7, kb=2, vb=3, paged=True, n=5, B=3, L=2),
    "softcap": dict(d=128, G=2, T=5, softcap=4.0),
    "not_causal": dict(d=64, G=4, T=19, causal=False, n=3),
    "records_only": dict(d=128, G=2, T=3, tail=0, n=2),
    "queries_in_the_records": dict(d=128, G=3, T=200, n=4, tail=60),
    "ring_only": dict(d=128, G=4, T=90, n=0, tail=200),
    "ring_only_d512": dict(d=512, G=4, T=70, n=0, tail=90, Hkv=1, shared=True),
    "more_queries_than_tokens": dict(d=64, G=2, T=50, n=0, tail=20),
}


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("name", CASES)
def test_prefill_against_the_formula(tq, orc, name, splits):
    kw = dict(CASES[name])
    G, T, lens = kw.pop("G"), kw.pop("T"), kw.pop("lens", None)
    causal, softcap, T_out = kw.pop("causal", True), kw.pop("softcap", 0.0), kw.pop("T_out", 0.0)
    c = Cache(tq, orc, T=T_out, seed=3, **kw)
    q = queries(c.L, c.B, T, c.Hkv * G, c.d, 77)
    out = _run(tq, c, q, lens, G, causal=causal, softcap=softcap, splits=splits)
    _check(c, q, lens, G, out, causal=causal, softcap=softcap)


def test_one_token_is_the_decode_attention(tq, orc):
    """t_q = 1 and tq_decode_attn (f32) agree to the bf16 output's half step and the f16 operands."""
    import torch
    c = Cache(tq, orc, B=2, Hkv=2, d=128, kb=4, vb=4, n=6, tail=100, seed=4)
    q = queries(1, 2, 1, 8, 128, 5)
    out = _run(tq, c, q, None, 4)
    ref = torch.empty((1, 2, 8, 128), device="cuda")
    kw = c.kw()
    kw.pop("block_table")
    tq.decode_attn(k_codec=c.kc, v_codec=c.vc, q=tl.to_bf16_tensor(q, "cuda")[:, :, 0].contiguous(), out=ref, scale=1.0,
                   **kw)
    e = (out[:, :, 0].float() - ref).norm() / ref.norm()
    assert float(e) <= 2.0 ** -8


def test_large_and_tiny_scales_and_zero_vectors(tq, orc):
    """Values of norms 1e-20 .. 1e20 in one stream, and zero vectors: the weights' exponent follows."""
    import torch
    c = Cache(tq, orc, B=1, Hkv=1, d=128, kb=4, vb=4, n=4, tail=5, seed=6)
    off = 128 * 128 * 4 // 8
    sc = c.rec["v"][0, 0, 0, :, off:off + 512].contiguous().view(torch.float32)
    factor = torch.tensor([1e-20, 1.0, 0.0, 1e20], device="cuda")[:, None]
    c.rec["v"][0, 0, 0, :, off:off + 512] = (sc * factor).view(torch.uint8)
    c._host["v"] = c.rec["v"].cpu().numpy()
    q = queries(1, 1, 3, 2, 128, 8)
    out = _run(tq, c, q, None, 2)
    _check(c, q, None, 2, out)
    # without the huge ones: the last record's values zero
    c.rec["v"][0, 0, 0, 3, off:off + 512] = 0
    c._host["v"] = c.rec["v"].cpu().numpy()
    _check(c, q, None, 2, _run(tq, c, q, None, 2))


def test_captured_and_replayed(tq, orc):
    import torch
    c = Cache(tq, orc, B=2, n=3, tail=64, seed=7)
    q = tl.to_bf16_tensor(queries(1, 2, 6, 8, 128, 9), "cuda")
    eager, out = torch.zeros_like(q), torch.zeros_like(q)
    tq.prefill_attn(k_codec=c.kc, v_codec=c.vc, q=q, out=eager, scale=1.0, **c.kw())
    a = tq.make_query_args(q=q, out=out, scale=1.0, **c.kw())
    ws = torch.empty(tq.tq_prefill_attn_workspace_size(a, c.kc, c.vc), dtype=torch.uint8, device="cuda")
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        tq.tq_prefill_attn(a, c.kc, c.vc, ws)
    for _ in range(2):
        out.zero_()
        ws.fill_(0xFF)  # nothing is left from the call before
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


@pytest.mark.parametrize("d,G,shared", [(64, 3, False), (128, 5, False), (512, 4, False)])
def test_keys_a_query_does_not_see_may_be_anything(tq, orc, d, G, shared):
    """Later new tokens' keys hold infinities and NaN: the queries before them are as with clean ones."""
    import torch
    c = Cache(tq, orc, B=1, Hkv=2, d=d, kb=3, vb=3, n=2, tail=50, seed=11)
    T = 20
    q = queries(1, 1, T, 2 * G, d, 3)
    clean = _run(tq, c, q, None, G)
    for back, bad in ((0, math.nan), (1, math.inf), (4, -math.inf)):
        slot = (int(c.start[0, 0]) + 50 - 1 - back) % c.cap
        c.ring["k"][0, 0, :, slot] = bad
    out = _run(tq, c, q, None, G)
    assert torch.equal(out[0, 0, : T - 5], clean[0, 0, : T - 5])


def test_broadcast_and_strided_queries(tq, orc):
    """Queries shared by the sequences (batch stride 0), a fused projection's view, one kv head."""
    import torch
    c = Cache(tq, orc, B=3, Hkv=1, d=64, kb=2, vb=2, n=2, tail=40, lens=([2, 2, 2], [40, 40, 40]), seed=12)
    wide = tl.to_bf16_tensor(queries(1, 1, 6, 9, 64, 4), "cuda")
    view = wide[:, :, :, 2:7].expand(1, 3, 6, 5, 64)
    out, ref = torch.empty((1, 3, 6, 5, 64), dtype=torch.bfloat16, device="cuda"), None
    tq.prefill_attn(k_codec=c.kc, v_codec=c.vc, q=view, out=out, scale=1.0, **c.kw())
    ref = torch.empty_like(out)
    tq.prefill_attn(k_codec=c.kc, v_codec=c.vc, q=view.contiguous(), out=ref, scale=1.0, **c.kw())
    assert torch.equal(out, ref)


@pytest.mark.parametrize("scale", [-1.0, 0.0])
@pytest.mark.parametrize("d", [64, 256])
def test_negative_and_zero_scales(tq, orc, d, scale):
    c = Cache(tq, orc, B=1, Hkv=1, d=d, kb=4, vb=2, n=2, tail=30, seed=14)
    q = queries(1, 1, 4, 3, d, 5)
    out = _run(tq, c, q, None, 3, scale=scale)
    qf = synth.bf16_bits_to_f32(q).astype(np.float64)
    got = synth.bf16_bits_to_f32(tl.bf16_tensor_bits(out.contiguous())).astype(np.float64)
    k, v = c.vectors("k", 0, 0, 0), c.vectors("v", 0, 0, 0)
    for i in range(3):
        want = weights(qf[0, 0, :, i], k, 4, 286, True, 0.0, scale) @ v
        assert np.linalg.norm(got[0, 0, :, i] - want) <= 2.0 ** -7 * np.linalg.norm(want)


def test_growing_logits_move_the_reference(tq, orc):
    """Keys whose scales grow by records: every record passes the reference of those before by far."""
    import torch
    for d, kb in ((128, 4), (512, 3)):
        c = Cache(tq, orc, B=1, Hkv=1, d=d, kb=kb, vb=4, n=6, tail=9, seed=15)
        off = 128 * d * kb // 8
        sc = c.rec["k"][0, 0, 0, :, off:off + 512].contiguous().view(torch.float32)
        c.rec["k"][0, 0, 0, :, off:off + 512] = (sc * torch.tensor([0.1, 1, 3, 6, 9, 12], device="cuda")[:, None]).view(torch.uint8)
        c._host["k"] = c.rec["k"].cpu().numpy()
        q = queries(1, 1, 7, 4, d, 16)
        out = _run(tq, c, q, None, 4, splits=1)
        qf = synth.bf16_bits_to_f32(q).astype(np.float64)
        got = synth.bf16_bits_to_f32(tl.bf16_tensor_bits(out.contiguous())).astype(np.float64)
        k, v = c.vectors("k", 0, 0, 0), c.vectors("v", 0, 0, 0)
        # a logit of up to 60 is off by 2^-12 of itself: 2^-6 of a weight, and so of the output
        for i in range(4):
            want = weights(qf[0, 0, :, i], k, 7, 6 * 128 + 9, True, 0.0, 1.0) @ v
            assert np.linalg.norm(got[0, 0, :, i] - want) <= 2.0 ** -5 * np.linalg.norm(want)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_scales_of_records_a_query_does_not_see_may_be_infinite(tq, orc, d):
    """The newest tokens already lie in records (no ring): the last one's key scale is infinite or NaN."""
    import torch
    c = Cache(tq, orc, B=1, Hkv=2, d=d, kb=3, vb=3, n=3, tail=0, seed=17)
    q = queries(1, 1, 9, 6, d, 18)
    clean = _run(tq, c, q, None, 3)
    for bad in (math.inf, math.nan):
        off = 128 * d * 3 // 8 + 4 * 127
        c.rec["k"][0, 0, :, 2, off:off + 4] = torch.tensor([bad], device="cuda").view(torch.uint8)
        out = _run(tq, c, q, None, 3)
        assert torch.equal(out[0, 0, :8], clean[0, 0, :8])


def test_two_calls_at_once(tq, orc):
    """Two streams, a workspace each, the same cache: both come out as they do alone."""
    import torch
    c = Cache(tq, orc, B=2, Hkv=2, d=128, kb=4, vb=4, n=20, tail=90, seed=19)
    qs = [tl.to_bf16_tensor(queries(1, 2, t, 8, 128, 20 + t), "cuda") for t in (40, 3)]
    mk = lambda i, out: tq.make_query_args(q=qs[i], out=out, scale=1.0, **c.kw())  # noqa: E731
    alone = []
    for i in (0, 1):
        alone.append(torch.zeros_like(qs[i]))
        tq.prefill_attn(k_codec=c.kc, v_codec=c.vc, q=qs[i], out=alone[i], scale=1.0, **c.kw())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in (0, 1)]
    both = [torch.zeros_like(x) for x in qs]
    args = [mk(i, both[i]) for i in (0, 1)]
    ws = [torch.empty(max(tq.tq_prefill_attn_workspace_size(args[i], c.kc, c.vc), 256), dtype=torch.uint8, device="cuda")
          for i in (0, 1)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                tq.tq_prefill_attn(args[i], c.kc, c.vc, ws[i])
    torch.cuda.synchronize()
    assert all(torch.equal(both[i], alone[i]) for i in (0, 1))


@pytest.mark.parametrize("raw", [False, True])
def test_a_dropped_workspace_is_not_handed_out_under_the_call(tq, orc, raw):
    """A call queued on a busy side stream; its workspace is dropped and memory of its size is filled meanwhile."""
    import torch
    c = Cache(tq, orc, B=1, Hkv=2, d=128, kb=4, vb=4, n=16, tail=10, seed=23)
    q = tl.to_bf16_tensor(queries(1, 1, 30, 8, 128, 24), "cuda")
    ref, out = torch.zeros_like(q), torch.zeros_like(q)
    need = tq.prefill_attn(k_codec=c.kc, v_codec=c.vc, q=q, out=ref, scale=1.0, **c.kw()).numel()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    tq.prefill_attn(k_codec=c.kc, v_codec=c.vc, q=q, out=out, scale=1.0, stream=side.cuda_stream if raw else side, **c.kw())
    junk = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and len(junk) == 4


@pytest.mark.parametrize("softcap", [0.25, 30.0, 170.0, 1000.0])
@pytest.mark.parametrize("d", [64, 256])
def test_caps_from_small_to_large(tq, orc, d, softcap):
    """The cap's own error, 2^-21 of it below 177 and tanhf's above, is far under an f16 weight's half step."""
    c = Cache(tq, orc, B=2, Hkv=2, d=d, kb=4, vb=3, n=5, tail=150, seed=27)
    q = queries(1, 2, 21, 6, d, 28)
    out = _run(tq, c, q, None, 3, softcap=softcap, splits=1)
    _check(c, q, None, 3, out, softcap=softcap)


MORE = {
    "side_lists_d256": dict(d=256, G=4, T=9, T_out=2.0, kb=4, vb=3, n=3),
    "side_lists_d512_shared": dict(d=512, G=8, T=5, T_out=2.0, kb=4, shared=True, Hkv=1, n=2),
    "side_lists_d512_paged": dict(d=512, G=3, T=7, T_out=1.5, kb=3, vb=2, paged=True, n=4, B=2, L=2),
    "paged_d256": dict(d=256, G=5, T=30, kb=2, vb=4, paged=True, n=5, B=3, L=2, lens=[30, 7, 19]),
    "paged_d512_shared": dict(d=512, G=16, T=9, kb=4, shared=True, Hkv=1, paged=True, n=3, B=3, L=2),
    "one_bit_side_lists": dict(d=128, G=2, T=6, T_out=1.5, kb=1, vb=1, n=3),
}


@pytest.mark.parametrize("splits", [0, 1])
@pytest.mark.parametrize("name", MORE)
def test_more_layouts_against_the_formula(tq, orc, name, splits):
    kw = dict(MORE[name])
    G, T, lens, T_out = kw.pop("G"), kw.pop("T"), kw.pop("lens", None), kw.pop("T_out", 0.0)
    c = Cache(tq, orc, T=T_out, seed=5, **kw)
    q = queries(c.L, c.B, T, c.Hkv * G, c.d, 78)
    out = _run(tq, c, q, lens, G, splits=splits)
    _check(c, q, lens, G, out)
