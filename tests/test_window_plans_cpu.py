"""What windowed plans hand out, read back from their metadata images on the CPU."""
import random

import pytest

import plan_image as pi
from paged_kv_cache_16_gb300 import binding, build
from test_window_cpu import desc


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


def image(kw):
    return pi.Image(binding.pa_plan_window(**kw), kw["num_heads_kv"])


@pytest.mark.parametrize("n,q,window,sinks,hq,hkv", [(31, 18, 5, 33, 32, 8), (40, 16, 1024, 0, 32, 8), (20, 24, 2048, 0, 32, 8),
                                                     (153, 1, 1024, 0, 32, 1), (160, 1, 900, 20, 32, 1)])
def test_bf16_tiles_are_split_all_or_none(n, q, window, sinks, hq, hkv):
    """More short tiles than SMs, a last round that may be spread: one side brings
    every V tile of a step over bf16 caches."""
    kw = desc([q] * n, [max(2 * window, 3000)] * n, window, sinks, hq=hq, hkv=hkv, max_blocks_per_req=300)
    assert len({t["split"] for t in image(kw).tiles}) == 1


@pytest.mark.parametrize("seed", range(40))
def test_bf16_tiles_of_drawn_steps_are_split_all_or_none(seed):
    rng = random.Random(seed)
    for _ in range(12):
        hq, hkv = rng.choice([(32, 8), (32, 1), (16, 2), (64, 8), (12, 4), (8, 8), (33, 1)])
        n, top = rng.randint(1, 220), rng.choice([16, 24, 64, 200])
        q = [rng.randint(9, top) for _ in range(n)]
        seq = [x + rng.randint(0, 4000) for x in q]
        kw = desc(q, seq, rng.choice([5, 100, 1024, 3000]), rng.choice([0, 4, 50]), hq=hq, hkv=hkv, max_blocks_per_req=300)
        assert len({t["split"] for t in image(kw).tiles}) <= 1, kw
