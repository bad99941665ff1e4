"""Calls of the rotating append that are refused, on the GPU (needs a GB300)."""
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


def test_error_word_on_the_host_is_refused():
    """Before a kernel that meets a bad block would write there."""
    c = oc.AppendCase(hq=4, hkv=2, d=64, q_lens=[3, 1], computed=[5, 0], code="int8")
    i32 = lambda a: torch.as_tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    a = [t.to(DEV) for t in (c.key.contiguous(), c.value.contiguous())] + [i32(c.qsl), i32(c.nc), i32(c.table)]
    a += [t.to(DEV) for t in (c.kc, c.vc)]
    more = dict(key_scales=c.ks.to(DEV), value_scales=c.vs.to(DEV))
    with pytest.raises(ValueError, match="device_error_word"):
        binding.pa_append_kv(None, *a, **more, device_error_word=torch.zeros(1, dtype=torch.int32))
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    for w in (word, word.data_ptr(), None):
        binding.pa_append_kv(None, *a, **more, device_error_word=w)
    assert binding.pa_check_device_errors(word) == 0
