"""GPU tests of tq_key_bounds against the oracle's 64-bit decode of the same
records: head dims, bit widths, side lists, pages, ranges of records, scales."""
import math

import numpy as np
import pytest

import synth
import tq_testlib as tl
from cache_cases import CHUNK, Cache, ocodec

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


def place(c, value=7.0):
    """Bounds that lie as the cache's records do, of one value."""
    import torch
    lead = c.rec["k"].shape[:-1]
    return torch.full((*lead, 2, c.d), value, dtype=torch.bfloat16, device="cuda")


def at(c, bounds, l, b, h, r):
    x = bounds[l, b, h, r] if c.table is None else bounds[l, int(c.table[b, r]), h]
    return synth.bf16_bits_to_f32(tl.bf16_tensor_bits(x)).astype(np.float64)


def check(c, bounds, l, b, h, r, scale=None):
    """A decoded key's f32 error: at most 9 levels of butterflies over values whose sum is at most sqrt(d)
    norms (2^-24 of it each, over sqrt(d)), two products: under 2^-20 norms.  Then one step of bf16 outward,
    2^-7 of the value."""
    k = c.orc.decode_records(c._host["k"][l, b, h], (r + 1) * CHUNK, ocodec(c.orc, c.kc))[r * CHUNK:]
    off = 2.0 ** -20 * np.linalg.norm(k, axis=-1).max()
    lo, hi = at(c, bounds, l, b, h, r)
    kmin, kmax = k.min(0), k.max(0)
    assert np.all(lo <= kmin + off) and np.all(lo >= kmin - off - 2.0 ** -7 * np.abs(kmin))
    assert np.all(hi >= kmax - off) and np.all(hi <= kmax + off + 2.0 ** -7 * np.abs(kmax))


@pytest.mark.parametrize("T", [0.0, 1.8])
@pytest.mark.parametrize("bits", [1, 2, 3, 4])
@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_bounds_against_the_oracle(tq, orc, d, bits, T):
    c = Cache(tq, orc, L=2, B=3, Hkv=2, d=d, kb=bits, vb=1, n=4, T=T, seed=31)
    bounds = place(c)
    tq.key_bounds(k_codec=c.kc, k_rec=c.rec["k"], bounds=bounds, n_chunks=c.d_n, max_chunks=4)
    for l in range(2):
        for b in range(3):
            for h in range(2):
                for r in range(4):
                    if r < c.n[l, b]:
                        check(c, bounds, l, b, h, r)
                    else:
                        assert np.all(at(c, bounds, l, b, h, r) == 7.0)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("max_new", [1, 2, 9, None])
def test_ranges_of_records_and_pages(tq, orc, paged, max_new):
    """Records from `first` on, max_new at most, are bounded, the others left alone; first past the last record
    or below zero too."""
    import torch
    c = Cache(tq, orc, B=5, Hkv=2, d=128, kb=3, vb=2, n=6, paged=paged, seed=32,
              lens=([6, 4, 5, 2, 6], [0, 0, 0, 0, 0]))
    first = np.array([[0, 3, 5, 9, -2]])
    bounds = place(c)
    tq.key_bounds(k_codec=c.kc, k_rec=c.rec["k"], bounds=bounds, n_chunks=c.d_n, max_chunks=6, max_new=max_new,
                  first=torch.from_numpy(first.astype(np.int32)).cuda(), block_table=c.table)
    done = 0
    for b in range(5):
        f = max(int(first[0, b]), 0)
        for r in range(6):
            for h in range(2):
                if f <= r < min(int(c.n[0, b]), f + (max_new or 6)):
                    check(c, bounds, 0, b, h, r)
                    done += 1
                else:
                    assert np.all(at(c, bounds, 0, b, h, r) == 7.0)
    if paged:  # nothing but the blocks of bounded records was written
        assert int((bounds[0, :, :, 0, 0] != 7.0).sum()) == done


def test_every_record_of_a_long_cache_and_zero_vectors(tq, orc):
    """Bounds of zeros are zeros; scales of 1e-30 and 1e30 keep their precision."""
    import torch
    c = Cache(tq, orc, B=1, Hkv=1, d=64, kb=4, vb=4, n=5, seed=33)
    off = 128 * 64 * 4 // 8
    sc = c.rec["k"][0, 0, 0, :, off:off + 512].contiguous().view(torch.float32)
    factor = torch.tensor([1e-30, 1.0, 0.0, 1e30, 1.0], device="cuda")[:, None]
    c.rec["k"][0, 0, 0, :, off:off + 512] = (sc * factor).view(torch.uint8)
    c._host["k"] = c.rec["k"].cpu().numpy()
    bounds = place(c)
    tq.key_bounds(k_codec=c.kc, k_rec=c.rec["k"], bounds=bounds, n_chunks=c.d_n, max_chunks=5)
    for r in range(5):
        check(c, bounds, 0, 0, 0, r)
    assert torch.all(bounds[0, 0, 0, 2] == 0)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_scale_that_is_not_finite_leaves_nan(tq, orc, bad):
    import torch
    c = Cache(tq, orc, B=1, Hkv=2, d=128, kb=2, vb=2, n=3, seed=34)
    clean, got = place(c), place(c)
    kw = dict(k_codec=c.kc, k_rec=c.rec["k"], n_chunks=c.d_n, max_chunks=3)
    tq.key_bounds(bounds=clean, **kw)
    off = 128 * 128 * 2 // 8 + 4 * 77
    c.rec["k"][0, 0, 1, 1, off:off + 4] = torch.tensor([bad], device="cuda").view(torch.uint8)
    tq.key_bounds(bounds=got, **kw)
    assert torch.all(got[0, 0, 1, 1].isnan())
    got[0, 0, 1, 1] = clean[0, 0, 1, 1]
    assert torch.equal(got, clean)


def test_captured_and_replayed(tq, orc):
    import torch
    c = Cache(tq, orc, B=2, Hkv=2, d=128, kb=4, vb=4, n=3, seed=35)
    eager, out = place(c), place(c)
    tq.key_bounds(k_codec=c.kc, k_rec=c.rec["k"], bounds=eager, n_chunks=c.d_n, max_chunks=3)
    a = tq.make_bounds_args(k_rec=c.rec["k"], bounds=out, n_chunks=c.d_n, max_chunks=3)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        tq.tq_key_bounds(a, c.kc)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)


@pytest.mark.parametrize("d,B,n", [(64, 4, 100), (512, 3, 90)])
def test_more_records_than_warps_at_work(tq, orc, d, B, n):
    """Enough records for a warp each, and some that are left; every one as in a call of its own sequence and few
    records, every fiftieth against the oracle."""
    import torch
    Hkv = 8
    c = Cache(tq, orc, B=B, Hkv=Hkv, d=d, kb=3, vb=1, n=n, seed=37)
    bounds, few = place(c), place(c)
    tq.key_bounds(k_codec=c.kc, k_rec=c.rec["k"], bounds=bounds, n_chunks=c.d_n, max_chunks=n)
    for r in range(0, n, 30):  # 30 records of every sequence at a time
        tq.key_bounds(k_codec=c.kc, k_rec=c.rec["k"], bounds=few, n_chunks=c.d_n, max_chunks=n, max_new=30,
                      first=torch.full((1, B), r, dtype=torch.int32, device="cuda"))
    assert torch.equal(bounds.view(torch.int16), few.view(torch.int16))
    for i, (b, h, r) in enumerate(np.ndindex(B, Hkv, n)):
        if i % 50 == 0 and r < c.n[0, b]:
            check(c, bounds, 0, b, h, r)
        elif r >= c.n[0, b] and h == 0:
            assert torch.all(bounds[0, b, :, r] == 7.0)


def test_records_and_bounds_past_32_bits_of_their_pools(tq, orc):
    import torch
    c = Cache(tq, orc, B=2, Hkv=1, d=512, kb=1, vb=1, n=3, paged=True, seed=38)
    near, pool = place(c), c.rec["k"]
    kw = dict(k_codec=c.kc, n_chunks=c.d_n, max_chunks=3)
    tq.key_bounds(k_rec=pool, bounds=near, block_table=c.table, **kw)
    blocks = (1 << 32) // 2048 + 50  # a record's bounds are 2048 bytes, and it more
    far = torch.empty((1, blocks, 1, pool.shape[-1]), dtype=torch.uint8, device="cuda")
    far[:, -pool.shape[1]:] = pool
    out = torch.empty((1, blocks, 1, 2, 512), dtype=torch.bfloat16, device="cuda")
    out[:, -pool.shape[1]:] = 7.0
    tq.key_bounds(k_rec=far, bounds=out, block_table=c.table + (blocks - pool.shape[1]), **kw)
    assert torch.equal(out[:, -pool.shape[1]:], near)


def test_a_codec_of_another_size_is_refused(tq, orc):
    c = Cache(tq, orc, B=1, Hkv=1, d=128, kb=4, vb=4, n=2, seed=36)
    a = tq.make_bounds_args(k_rec=c.rec["k"], bounds=place(c), n_chunks=c.d_n, max_chunks=2)
    for codec in (tq.tq_make_codebook(3, 128), tq.tq_make_codebook(4, 64)):
        with pytest.raises(ValueError):
            tq.tq_key_bounds(a, codec)


@pytest.mark.parametrize("T", [0.0, 1.8])
@pytest.mark.parametrize("d,bits", [(64, 1), (128, 4), (256, 3), (512, 2)])
def test_bounds_of_the_largest_and_the_smallest_keys(tq, orc, d, bits, T):
    """Keys of norms near both ends of f32: their bounds are finite and as exact as any (1e-32: a bf16 of a
    coordinate near zero has a subnormal's step there, under 2^-20 norms)."""
    import torch
    c = Cache(tq, orc, B=1, Hkv=1, d=d, kb=bits, vb=1, n=3, T=T, seed=39)
    off = 128 * d * bits // 8
    sc = c.rec["k"][0, 0, 0, :, off:off + 512].contiguous().view(torch.float32)
    c.rec["k"][0, 0, 0, :, off:off + 512] = (sc * torch.tensor([1e36, 1e-32, 1.0], device="cuda")[:, None]).view(torch.uint8)
    c._host["k"] = c.rec["k"].cpu().numpy()
    bounds = place(c)
    tq.key_bounds(k_codec=c.kc, k_rec=c.rec["k"], bounds=bounds, n_chunks=c.d_n, max_chunks=3)
    assert torch.all(bounds.isfinite())
    for r in range(3):
        check(c, bounds, 0, 0, 0, r)
