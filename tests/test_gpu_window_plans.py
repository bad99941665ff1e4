"""Windowed steps whose tiles the planner spreads in one way or another, on the GPU
against the plain implementation in 64 bits (needs a GB300)."""
import pytest
import torch

import window_common as wc
from gpu_common import ensure_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_library()


@pytest.mark.parametrize("code", wc.KINDS)
@pytest.mark.parametrize("n,q,seq,window,sinks,layout,num_sms", [
    (31, 18, 60, 5, 33, (32, 8, 128), 0), (24, 10, 700, 300, 0, (32, 8, 128), 0), (155, 1, 900, 800, 4, (32, 1, 128), 0),
    (6, 18, 900, 700, 20, (8, 8, 128), 20), (21, 1, 1300, 1024, 0, (40, 1, 64), 20), (11, 30, 500, 450, 16, (6, 2, 64), 20)])
def test_short_tiles_in_more_rounds_than_one(code, n, q, seq, window, sinks, layout, num_sms):
    """More tiles of at most one sub-tile of rows than CTAs: whole, split or in
    pieces, the last round's included."""
    hq, hkv, d = layout
    lens = [seq + i % 7 for i in range(n)]
    wc.check(wc.WindowCase(hq=hq, hkv=hkv, d=128 if code == "e4m3" else d, q_lens=[q] * n, seq_lens=lens, code=code,
                           window=window, sinks=sinks, seed=n), num_sms=num_sms)
