"""Numbers that the calls' 32-bit fields do not hold are refused, not wrapped (CPU)."""
import numpy as np
import pytest
import torch

from paged_kv_cache_16_gb300 import binding, build
from test_window_cpu import desc

TOO_LARGE = [2**31, 2**32 + 16, -2**32 + 16, 2**63]


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


@pytest.mark.parametrize("n", TOO_LARGE)
@pytest.mark.parametrize("name", ["window", "sink_tokens"])
def test_windows(name, n):
    kw = {**desc([1], [900]), name: n}
    assert binding.pa_plan_window_status(**kw) == binding.PA_ERR_INVALID_ARGUMENT
    with pytest.raises(binding.PaError):
        binding.pa_plan_window(**kw)


def test_windows_of_other_integer_types():
    for n in (np.int64(32), torch.tensor(32), 32.0):
        assert binding.pa_plan_window(**{**desc([1], [900]), "window": n}).window == (32, 0)


@pytest.mark.parametrize("n", TOO_LARGE)
def test_axes(n):
    ok = dict(num_axes=2, axis_of_pair=[0, 1] * 16, rotary_dim=64)
    binding.pa_rope_create_axes(**ok).destroy()
    for name in ("num_axes", "frequencies"):
        with pytest.raises(binding.PaError):
            binding.pa_rope_create_axes(**{**ok, name: n})
    axes = np.zeros(32, dtype=np.int64 if n < 2**63 else np.uint64)
    axes[3] = n
    with pytest.raises(ValueError, match="axis_of_pair"):
        binding.pa_rope_create_axes(**{**ok, "axis_of_pair": axes})


def test_axes_that_are_no_numbers_of_axes():
    for axes in ([0.5] * 32, [0, 1] * 15):
        with pytest.raises(ValueError, match="axis_of_pair"):
            binding.pa_rope_create_axes(num_axes=2, axis_of_pair=axes, rotary_dim=64)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64, torch.float32, torch.bool])
def test_graph_steps_take_whole_positions(dtype):
    """The static buffer of positions takes integers as they are, nothing that a cast would round."""
    from paged_kv_cache_16_gb300 import workloads
    from paged_kv_cache_16_gb300.step import GraphStep
    batch = workloads.tiny("1B", seed=0)
    rope = binding.pa_rope_create_axes(num_axes=2, axis_of_pair=[0, 1] * 16, rotary_dim=64)
    gs = GraphStep(num_heads_q=4, num_heads_kv=2, head_dim=64, num_blocks=64, max_blocks_per_req=8, softmax_scale=0.125,
                   max_tokens=64, max_reqs=8, max_extend_tiles=8, device="cpu", rope=rope)
    pos = torch.arange(2 * batch.num_tokens).reshape(2, -1)
    if dtype in (torch.int32, torch.int64):
        gs.stage(batch, positions=pos.to(dtype))
        assert torch.equal(gs.positions[:, :batch.num_tokens], pos.int())
    else:
        with pytest.raises(ValueError, match="positions"):
            gs.stage(batch, positions=pos.to(dtype))
