"""GPU tests of what the Python calls for several tokens refuse before anything is launched: records of
another codec's size (they would be read past their end), workspaces that are not one run of memory."""
import pytest

from cache_cases import Cache, queries
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


@pytest.fixture(scope="module")
def case(tq, orc):
    import torch
    c = Cache(tq, orc, B=1, Hkv=1, d=128, kb=3, vb=2, n=3, tail=20, seed=61)
    q = tl.to_bf16_tensor(queries(1, 1, 2, 3, 128, 1), "cuda")
    return c, q, torch.zeros((1, 1, 1, 128 * 3 + 20), device="cuda")


def test_records_of_another_codec(tq, case):
    import torch
    c, q, mass = case
    four = tq.tq_make_codebook(4, 128)
    a = tq.make_query_args(q=q, out=torch.empty_like(q), scale=1.0, **c.kw())
    ws = torch.empty(tq.tq_prefill_attn_workspace_size(a, c.kc, c.vc), dtype=torch.uint8, device="cuda")
    for kc, vc in ((four, c.vc), (c.kc, four), (c.vc, c.kc)):
        with pytest.raises(ValueError):
            tq.tq_prefill_attn(a, kc, vc, ws)
        tq.tq_prefill_attn(a, c.kc, c.vc, ws)  # a call that was in order does not vouch for another's codecs
    with pytest.raises(ValueError):
        tq.prefill_attn(k_codec=four, v_codec=c.vc, q=q, out=torch.empty_like(q), scale=1.0, **c.kw())
    b = tq.make_query_args(q=q, scale=1.0, **c.kw(values=False))
    ws = torch.empty(tq.tq_attn_mass_workspace_size(b, c.kc), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        tq.tq_attn_mass(b, four, mass, ws)
    tq.tq_attn_mass(b, c.kc, mass, ws)
    e = tq.make_evict_mass_args(k_rec=c.rec["k"], v_rec=c.rec["v"], mass=mass, n_chunks=c.d_n.clone(), max_chunks=3, keep_chunks=3)
    ws = torch.empty(tq.tq_evict_mass_workspace_size(e, c.kc, c.vc), dtype=torch.uint8, device="cuda")
    for kc, vc in ((four, c.vc), (c.kc, four)):
        with pytest.raises(ValueError):
            tq.tq_evict_mass(e, kc, vc, ws)
    torch.cuda.synchronize()


def test_workspaces_that_are_not_one_run(tq, case):
    import torch
    c, q, mass = case
    a = tq.make_query_args(q=q, out=torch.empty_like(q), scale=1.0, **c.kw())
    need = tq.tq_prefill_attn_workspace_size(a, c.kc, c.vc)
    flat = torch.empty(2 * need, dtype=torch.uint8, device="cuda")
    for ws in (flat[:256].expand(need // 256 + 1, 256), flat[::2], torch.empty(need, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            tq.tq_prefill_attn(a, c.kc, c.vc, ws)
    with pytest.raises(tq.TqError):
        tq.tq_prefill_attn(a, c.kc, c.vc, flat[:need - 1])
    tq.tq_prefill_attn(a, c.kc, c.vc, flat)
    torch.cuda.synchronize()
