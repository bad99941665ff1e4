"""Output buffers that start on a 16-byte boundary and no larger one, for every
kind of row and cache type (needs a GB300)."""
import pytest
import torch

import operators_common as oc
from gpu_common import ensure_library
from paged_kv_cache_16_gb300 import binding, workloads
from paged_kv_cache_16_gb300.step import DeviceStep

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_library()


def shifted(out):
    """(a buffer, a view of it shaped like out that starts 16 bytes into it)"""
    buf = torch.full((out.numel() + 16,), 5.0, dtype=out.dtype, device=DEV)
    view = buf[8:8 + out.numel()].view(out.shape)
    assert view.data_ptr() % 32 == 16
    return buf, view


def untouched(buf):
    return (buf[:8] == 5).all() and (buf[-8:] == 5).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("shared", [0, 8])
def test_plain_caches(kind, shared):
    """Chunks, decode and verify rows, with and without a shared prefix."""
    b = workloads.make_batch(name="align", num_heads_q=8, num_heads_kv=2, head_dim=128, q_lens=[1, 40, 3, 300],
                             seq_lens=[190, 233, 150, 460], num_blocks=120, seed=shared, kv_cache_dtype=kind,
                             shared_prefix=[([0, 1, 2, 3], shared)] if shared else None, num_common_prefix_blocks=shared)
    st = DeviceStep(b, DEV)
    q, key, value, kc, vc = (t.to(DEV) for t in (b.q, b.key, b.value, b.key_cache, b.value_cache))
    want = st.run(q, key, value, kc, vc).clone()
    buf, st.out = shifted(st.out)
    assert torch.equal(st.attend(q, kc, vc), want)
    torch.cuda.synchronize()
    assert st.check_errors() == 0 and untouched(buf)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shared", [0, 8])
def test_block_scaled_caches(code, d, shared):
    c = oc.Case(hq=8, hkv=2, d=d, q_lens=[1, 40, 3, 300], seq_lens=[190, 233, 150, 460], code=code, seed=1, shared=shared)
    g = oc.OnGpu(c)
    want = g.run().clone()
    buf, g.out = shifted(g.out)
    assert torch.equal(g.run(), want) and untouched(buf)
    ref, tol = c.reference()
    oc.assert_within(g.out, ref, tol)
