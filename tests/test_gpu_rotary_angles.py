"""The angles of the rotation, where its results show them undiluted (needs a GB300)."""
import numpy as np
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


# positions next to odd multiples of pi (numerators of pi's continued fraction):
# the sine of a turn by one radian per position is 3e-5 to 1e-8 there
NEAR_HALF_TURNS = [355, 208341, 833719, 1146408, 5419351, 245850922, 355 * 3, 208341 * 3, -355, -208341, -1146408]


@pytest.mark.parametrize("layout", [0, 1])
def test_sines_near_half_a_turn(layout):
    """(1, 0) turned by the position: the second result is the sine, off by the
    angle's error, 2^-32 of a turn, by a rounding to bf16, and by 2^-22 of itself
    for everything in 32 bits (the sine of the rounded angle to 1 ulp, the product by
    the magnitude, and the last turn's fma)."""
    pos = np.array(NEAR_HALF_TURNS)
    x = torch.zeros(len(pos), 1, 8, dtype=torch.bfloat16)
    first, second = (0, 1) if layout else (0, 4)
    x[:, 0, first] = 1.0
    x = x.to(DEV)
    rope = binding.pa_rope_create(rotary_dim=8, layout=layout)
    out = torch.empty_like(x)
    binding.pa_rotary(rope, x, torch.as_tensor(pos, dtype=torch.int32, device=DEV), out)
    sine = oc.cos_sin(rope.frequencies()[0][:1], pos)[1][:, 0]
    assert (np.abs(sine) < 2e-4).all()
    got = out[:, 0, second].double().cpu().numpy()
    assert (np.abs(got - sine) <= (oc.BF16 + 2.0 ** -22) * np.abs(sine) + 2 * np.pi * 2.0 ** -32).all(), (got, sine)
