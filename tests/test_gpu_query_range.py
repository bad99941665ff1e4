"""Queries over the whole range of bf16, every cache type, against the plain
implementation in 64 bits (needs a GB300)."""
import numpy as np
import pytest
import torch

import operators_common as oc
import window_common as wc
from gpu_common import ensure_library
from paged_kv_cache_16_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_library()


def scaled_case(code, layout, q_lens, seq, powers, window=10**6):
    """Rows of head h times 2^powers[h % len]; the softmax scale takes the largest back,
    so that scores are those of ordinary queries (or nearly 0, in rows of smaller ones)."""
    hq, hkv, d = layout
    c = wc.WindowCase(hq=hq, hkv=hkv, d=d, q_lens=q_lens, seq_lens=seq, code=code, window=window, sinks=0, seed=hq)
    p = torch.tensor([powers[h % len(powers)] for h in range(hq)])
    c.q = (c.q.double() * (2.0 ** p.double())[None, :, None]).to(torch.bfloat16)
    c.scale = float(np.float32(d ** -0.5 * 2.0 ** -max(powers)))
    return c


POWERS = [(17,), (100,), (-9,), (-24,), (-100,), (18, 16, -3), (0, -20, -14)]


@pytest.mark.parametrize("code", wc.KINDS)
@pytest.mark.parametrize("powers", POWERS)
@pytest.mark.parametrize("layout", [(4, 2, 128), (32, 8, 128), (12, 1, 128)])
@pytest.mark.parametrize("q_lens,seq", [([1, 1, 1], [5, 77, 700]), ([4, 8, 2], [40, 300, 513]), ([40], [200])])
@pytest.mark.parametrize("window", [None, 60])
def test_queries_of_any_magnitude(code, powers, layout, q_lens, seq, window):
    """Single tokens, verify rows and chunks, with a window and by a plan without one."""
    c = scaled_case(code, layout, q_lens, seq, powers, window or 10**6)
    g = wc.OnGpu(c)
    if window is None:
        g.plan = binding.pa_plan(**{k: v for k, v in c.desc().items() if k not in ("window", "sink_tokens")})
        g.ws = torch.zeros(g.plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    out = g.run()
    ref, tol = c.reference()
    oc.assert_within(out[:c.T], ref[:c.T], tol[:c.T])


@pytest.mark.parametrize("code", wc.KINDS)
@pytest.mark.parametrize("q_len", [1, 4, 40])
def test_infinite_queries_are_not_finite_ones(code, q_len):
    """An infinite element makes its row NaN (infinite scores of both signs), no other."""
    c = wc.WindowCase(hq=8, hkv=2, d=128, q_lens=[q_len, q_len], seq_lens=[300, 200], code=code, window=1000, sinks=0, seed=q_len)
    c.q[0, 3, 17] = float("inf")
    out = wc.OnGpu(c).run()
    assert torch.isnan(out[0, 3]).all()
    c.q[0, 3, 17] = 0
    ref, tol = c.reference()
    rest = torch.ones(c.T, 8, dtype=torch.bool)
    rest[0, 3] = False
    oc.assert_within(out[:c.T][rest], ref[rest.numpy()], tol[rest.numpy()])
