"""Attention over block-scaled 8-bit caches on the GPU where the order of the
tiles, the magnitudes and the addresses are unusual (needs a GB300)."""
import pytest
import torch

import operators_common as oc
from gpu_common import ensure_library

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
