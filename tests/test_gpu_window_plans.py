"""Windowed steps whose tiles the planner spreads in one way or another, on the GPU
against the plain implementation in 64 bits (needs a GB300)."""
import pytest
import torch

import window_common as wc
from gpu_common import ensure_library
from paged_kv_cache_16_gb300 import binding

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


@pytest.mark.parametrize("q_len", [128, 256])
def test_long_windows_without_a_workspace(q_len):
    """Chunks whose pieces outgrow the library's scratch: the call without a workspace
    takes them, and gives the same bits each time."""
    c = wc.WindowCase(hq=32, hkv=8, d=128, q_lens=[q_len], seq_lens=[9000], code="bf16", window=8192, sinks=0, seed=q_len)
    g = wc.OnGpu(c)
    out = g.run().clone()
    assert g.plan.workspace_bytes > binding.NO_ALLOC_SCRATCH_BYTES
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    again = [torch.zeros_like(out) for _ in range(2)]
    for x in again:
        binding.pa_attention_no_alloc(g.plan, g.q, g.kc, g.vc, g.table, x, word)
        assert int(word) == 0
    assert torch.equal(*again)
    # both round each weight to 2^-8 of it, relative to other maxima: out by 2^-8 of sum p |v| each (|v| < 6), and half a
    # step of out each
    assert (again[0].float() - out.float()).abs().max() <= 6 * 4 * 2.0 ** -8
    assert torch.equal(g.run(), out)
