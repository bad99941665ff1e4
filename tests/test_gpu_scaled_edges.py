"""Attention over block-scaled 8-bit caches on the GPU where the order of the
tiles, the magnitudes and the addresses are unusual (needs a GB300)."""
import pytest
import torch

import operators_common as oc
from gpu_common import ensure_library
from paged_kv_cache_16_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_library()


def check(c, **over):
    g = oc.OnGpu(c, **over)
    out = g.run()
    ref, tol = c.reference()
    oc.assert_within(out[:c.T], ref[:c.T], tol[:c.T])
    return g


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("num_sms,q_lens,seq_lens", [(4, [276, 500], [1200, 900]), (3, [276, 500], [1200, 900]),
                                                     (2, [20, 20, 500], [1200, 700, 900]),
                                                     (3, [20, 276, 10, 500], [900, 1200, 700, 900])])
def test_tiles_with_an_empty_half_between_others(code, d, num_sms, q_lens, seq_lens):
    """CTAs that get 7 to 13 tiles, one to six of them with all tokens in the
    first 128 rows ahead of a tile with more: the second half's rows of that tile
    take its own blocks' scales."""
    c = oc.Case(hq=8, hkv=2, d=d, q_lens=q_lens, seq_lens=seq_lens, code=code, scales="any", seed=num_sms)
    g = check(c, num_sms=num_sms)
    first = g.out.clone()
    for _ in range(5):
        assert torch.equal(g.run(), first)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("scale", [2.0 ** -64, 2.0 ** -100, 0.0])
def test_zero_queries_over_keys_of_tiny_scales(code, scale):
    """Scores whose factor (the query row's power of two times the key scale)
    underflows, in last blocks that are partly masked: every key counts the same.
    2^-64 is what the append gives a block of zero keys; scales below 2^-100 count
    as 2^-100, so that all of them stand for scores of 0 here."""
    c = oc.Case(hq=8, hkv=2, d=64, q_lens=[1, 3, 8, 30], seq_lens=[21, 39, 17, 45], code=code, seed=3)
    c.q.zero_()
    c.ks.fill_(scale)
    check(c)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_tiny_softmax_scale_over_keys_of_zero_scale(code):
    """Queries of 1e20 with a softmax scale that undoes them, over keys of scale 0
    (read as 2^-100): the tiles' factor underflows too."""
    c = oc.Case(hq=8, hkv=2, d=128, q_lens=[1, 3, 20], seq_lens=[100, 37, 50], code=code, q_size=1e20, seed=4)
    c.ks.fill_(0.0)
    check(c)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_step_of_zero_queries_and_keys(code):
    """A zeroed batch, as a warm-up makes it: zero keys appended into blocks that
    stay partly filled, zero queries, whose rows are the means of the values."""
    a = oc.AppendCase(hq=8, hkv=2, d=128, q_lens=[5, 1, 20], computed=[0, 16, 0], code=code, seed=5)
    a.q.zero_()
    a.key.zero_()
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    kc, vc, ks, vs = (t.to(DEV) for t in (a.kc, a.vc, a.ks, a.vs))
    table = i32(a.table)
    q, key, value = (t.to(DEV).contiguous() for t in (a.q, a.key, a.value))
    binding.pa_append_kv(None, key, value, i32(a.qsl), i32(a.nc), table, kc, vc, key_scales=ks, value_scales=vs)
    seq = a.nc + a.q_lens
    c = oc.Case(hq=8, hkv=2, d=128, q_lens=a.q_lens, seq_lens=seq, code=code)
    c.table, c.nb = a.table, a.nb
    c.q, c.kc, c.vc, c.ks, c.vs = q.cpu(), kc.cpu(), vc.cpu(), ks.cpu(), vs.cpu()
    check(c)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("q_size", [1e-36, 1e-30, 1e30, 1e35])
def test_queries_at_the_ends_of_the_bf16_range(code, q_size):
    """Magnitudes beyond 2^100 and below 2^-100 on the split-KV kernel (the softmax
    scale undoes them)."""
    check(oc.Case(hq=8, hkv=2, d=128, q_lens=[1, 3], seq_lens=[100, 50], code=code, q_size=q_size))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("num_sms", [3, 152])
def test_value_scales_far_apart(code, num_sms):
    """Value scales of 2^-64 and 2^36 in one row: keys whose products with the small
    scales are lost still count in the sum of the weights."""
    c = oc.Case(hq=8, hkv=2, d=128, q_lens=[1, 4, 1, 60], seq_lens=[700, 90, 333, 200], code=code, seed=9)
    used = torch.isfinite(c.vs)
    small = torch.rand(c.vs.shape, generator=torch.Generator().manual_seed(1)) < 0.5
    c.vs = torch.where(used, torch.where(small, 2.0 ** -64, 2.0 ** 36), c.vs)
    check(c, num_sms=num_sms)
