"""Rotary positions, the rotating append and attention over block-scaled
caches on the CPU: arguments, refusals, frequencies, plans (no kernel runs)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import operators_common as oc
from paged_kv_cache_16_gb300 import binding, build

INVALID, UNSUPPORTED, OK = binding.PA_ERR_INVALID_ARGUMENT, binding.PA_ERR_UNSUPPORTED, binding.PA_OK
FAKE = 1 << 20     # aligned, never dereferenced on the paths tested here


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


@pytest.mark.parametrize("over,status", [
    (dict(), OK), (dict(rotary_dim=256), OK), (dict(rotary_dim=8), OK),
    (dict(rotary_dim=0), INVALID), (dict(rotary_dim=-8), INVALID), (dict(rotary_dim=31), INVALID),
    (dict(rotary_dim=36), UNSUPPORTED), (dict(rotary_dim=264), UNSUPPORTED),
    (dict(layout=2), INVALID), (dict(layout=-1), INVALID), (dict(scaling=4), INVALID), (dict(scaling=-1), INVALID),
    (dict(base=0.0), INVALID), (dict(base=-1.0), INVALID), (dict(base=math.nan), INVALID), (dict(base=math.inf), INVALID),
    (dict(scaling=1, factor=0.0), INVALID), (dict(scaling=1, factor=math.nan), INVALID),
    (dict(scaling=1, factor=1e-40), INVALID), (dict(scaling=0, factor=-1.0), OK),
    (dict(scaling=2, factor=8.0), INVALID), (dict(scaling=2, factor=8.0, original_max_position=8192), OK),
    (dict(scaling=2, factor=8.0, original_max_position=8192, low=4.0, high=4.0), INVALID),
    (dict(scaling=2, factor=8.0, original_max_position=8192, low=-1.0), INVALID),
    (dict(scaling=3, factor=8.0, original_max_position=8192, low=1.0, high=32.0), OK),
    (dict(scaling=3, factor=8.0, original_max_position=8192, base=1.0), INVALID),
    (dict(scaling=3, factor=8.0, original_max_position=-1), INVALID),
    (dict(attention_factor=-0.5), INVALID), (dict(attention_factor=math.nan), INVALID), (dict(attention_factor=1e300), INVALID),
    (dict(attention_factor=1.5), OK)])
def test_rope_arguments(over, status):
    assert binding.pa_rope_status(**{"rotary_dim": 64, **over}) == status


def test_rope_null_arguments(lib):
    assert lib.pa_rope_create(None, ctypes.byref(ctypes.c_void_p())) == INVALID
    assert lib.pa_rope_create(ctypes.byref(binding.RopeDesc()), None) == INVALID
    lib.pa_rope_destroy(None)
    r = binding.pa_rope_create(rotary_dim=8)
    assert lib.pa_rope_frequencies(r.handle, None, None) == INVALID
    assert lib.pa_rope_frequencies(None, FAKE, None) == INVALID


def test_rope_frequencies():
    """The formulas, evaluated with 50 digits, to a relative 4e-16 x the few
    operations of each (pow, a product, a quotient)."""
    import decimal
    D = decimal.Decimal
    with decimal.localcontext() as c:
        c.prec = 50
        pi2 = D(oc.TWO_PI.numerator) / D(oc.TWO_PI.denominator)
        rd, base, s, L = 64, D(500000), D(8), D(8192)
        plain = [(-(D(2 * i) / rd) * base.ln()).exp() for i in range(rd // 2)]
        lo, hi = D(1), D(4)
        wave = []
        for f in plain:
            u = min(D(1), max(D(0), (L * f / pi2 - lo) / (hi - lo)))
            wave.append(f * (u + (1 - u) / s))
        at = lambda t: rd * (L / (D(t) * pi2)).ln() / (2 * base.ln())  # noqa: E731
        a, b = max(0, math.floor(at(32))), min(rd - 1, math.ceil(at(1)))
        yarn = [f * (r / s + 1 - r) for i, f in enumerate(plain) for r in [min(D(1), max(D(0), D(i - a) / D(b - a)))]]
        got = {}
        kw = dict(rotary_dim=rd, base=500000.0)
        got["plain"] = binding.pa_rope_create(**kw).frequencies()
        got["linear"] = binding.pa_rope_create(**kw, scaling=1, factor=8.0).frequencies()
        got["wave"] = binding.pa_rope_create(**kw, scaling=2, factor=8.0, original_max_position=8192, low=1.0, high=4.0).frequencies()
        got["yarn"] = binding.pa_rope_create(**kw, scaling=3, factor=8.0, original_max_position=8192, low=1.0, high=32.0).frequencies()
        want = dict(plain=plain, linear=[f / s for f in plain], wave=wave, yarn=yarn)
        for k, w in want.items():
            assert np.allclose(got[k][0], [float(x) for x in w], rtol=4e-15, atol=0), k
    assert got["plain"][1] == 1.0 and got["wave"][1] == 1.0
    assert abs(got["yarn"][1] - (0.1 * math.log(8) + 1)) < 1e-15
    assert binding.pa_rope_create(rotary_dim=8, attention_factor=0.5).frequencies()[1] == 0.5


def test_rotary_arguments(lib):
    r = binding.pa_rope_create(rotary_dim=64)
    call = lambda rope=r.handle, x=FAKE, xs=512, pos=FAKE, t=3, h=4, d=128, out=FAKE, os_=512: \
        lib.pa_rotary(rope, x, xs, pos, t, h, d, out, os_, None)  # noqa: E731
    assert call(t=0, x=None, out=None, pos=None) == OK
    for bad in (dict(rope=None), dict(t=-1), dict(h=0), dict(d=0), dict(x=None), dict(x=FAKE + 8), dict(out=FAKE + 4),
                dict(out=None), dict(pos=None), dict(pos=FAKE + 2), dict(xs=504), dict(xs=516), dict(os_=511), dict(d=56)):
        assert call(**bad) == INVALID, bad
    assert call(d=100) == UNSUPPORTED and call(d=264, xs=4096, os_=4096) == UNSUPPORTED


def append_args(**over):
    a = binding.AppendArgs()
    base = dict(num_reqs=2, num_tokens=3, num_heads_q=4, num_heads_kv=2, head_dim=64, block_size=16, num_blocks=9,
                max_blocks_per_req=4, kv_cache_dtype=binding.PA_KV_INT8_BLOCK, k_scale=1.0, v_scale=1.0, key_stride=128,
                value_stride=128, q_stride=256, q_out_stride=256)
    for f in ("query_start_loc", "num_computed_tokens", "block_table", "key", "value", "q", "q_out", "key_cache",
              "value_cache", "key_scales", "value_scales"):
        base[f] = FAKE
    base.update(over)
    for k, v in base.items():
        setattr(a, k, v)
    return a


def test_append_arguments(lib):
    rope = binding.pa_rope_create(rotary_dim=64)
    call = lambda rope=rope.handle, **over: lib.pa_append_kv(rope, ctypes.byref(append_args(**over)), None)  # noqa: E731
    assert lib.pa_append_kv(rope.handle, None, None) == INVALID
    assert call(num_tokens=0, key=None, q=None) == OK
    for bad in (dict(num_reqs=-1), dict(num_tokens=-1), dict(num_heads_kv=0), dict(head_dim=0), dict(num_blocks=0),
                dict(max_blocks_per_req=0), dict(block_size=0), dict(kv_cache_dtype=4), dict(kv_cache_dtype=-1),
                dict(rope=None), dict(num_heads_q=0), dict(num_reqs=0), dict(query_start_loc=None),
                dict(num_computed_tokens=None), dict(block_table=None), dict(block_table=FAKE + 2), dict(key=None),
                dict(value=FAKE + 8), dict(key_stride=120), dict(value_stride=132), dict(key_cache=None),
                dict(value_cache=FAKE + 4), dict(q_out=None), dict(q=FAKE + 2), dict(q_stride=248), dict(key_scales=None),
                dict(value_scales=None), dict(key_scales=FAKE + 1),
                dict(kv_cache_dtype=binding.PA_KV_FP8_E4M3, k_scale=0.0),
                dict(kv_cache_dtype=binding.PA_KV_FP8_E4M3, v_scale=math.nan)):
        assert call(**bad) == INVALID, bad
    wide = binding.pa_rope_create(rotary_dim=128)
    assert call(rope=wide.handle) == INVALID                       # more than a head
    for bad in (dict(block_size=32), dict(head_dim=32, num_tokens=0), dict(head_dim=96), dict(num_blocks=1 << 28)):
        assert call(rope=None, q=None, **bad) == UNSUPPORTED, bad


def test_append_wrapper_checks():
    c = oc.AppendCase(hq=4, hkv=2, d=64, q_lens=[3, 1], computed=[5, 0], code="int8")
    i32 = lambda a: torch.as_tensor(a, dtype=torch.int32)  # noqa: E731
    good = dict(rope=None, key=c.key, value=c.value, query_start_loc=i32(c.qsl), num_computed=i32(c.nc),
                block_table=i32(c.table), key_cache=c.kc, value_cache=c.vc, key_scales=c.ks, value_scales=c.vs)
    rope = binding.pa_rope_create(rotary_dim=64)
    for bad in (dict(key=c.key.float()), dict(key=c.key.transpose(0, 1)), dict(value=c.value[:2]),
                dict(key_scales=None), dict(value_scales=None), dict(key_scales=c.ks.double()), dict(key_scales=c.ks[:, :1]),
                dict(key_cache=c.kc.to(torch.int16)), dict(value_cache=c.vc.view(torch.uint8)), dict(key_cache=c.kc.to(torch.bfloat16)),
                dict(query_start_loc=i32(c.qsl)[:-1]), dict(num_computed=i32(c.nc).long()), dict(rope=rope, q=c.q),
                dict(block_table=i32(c.table).long()), dict(key_cache=c.kc[:, :, :1]), dict(rope=rope, q_out=c.q.contiguous()),
                dict(key_scales=None, value_scales=None), dict(rope=rope, q=c.q[:2], q_out=c.q[:2]),
                dict(rope=rope, q=c.q, q_out=torch.empty(4, 2, 64, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            binding.pa_append_kv(**{**good, **bad})
    with pytest.raises(ValueError):
        binding.pa_rotary(rope, c.q, i32(c.positions())[:-1], torch.empty_like(c.q))


def test_scaled_plans_and_refusals(lib):
    """Block-scaled plans are the E4M3 plans of the same step, at both head
    sizes; calls without scales refuse them, and the scaled calls others."""
    c = oc.Case(hq=8, hkv=2, d=128, q_lens=[1, 40, 3], seq_lens=[300, 90, 17], code="int8")
    plan = binding.pa_plan(**c.desc(num_sms=152, block_table_host=c.table.clip(min=0)))
    e4m3 = binding.pa_plan(**c.desc(num_sms=152, kv_cache_dtype=binding.PA_KV_FP8_E4M3))
    for k in ("num_decode_rows", "num_extend_tiles", "num_dequant_blocks", "decode_kv_bytes", "kernels_per_call"):
        assert plan.info()[k] == e4m3.info()[k], k
    d64 = oc.Case(hq=8, hkv=2, d=64, q_lens=[1, 40], seq_lens=[300, 90], code="e4m3")
    assert binding.pa_plan_status(**d64.desc(num_sms=152)) == OK
    assert binding.pa_plan_status(**d64.desc(num_sms=152, kv_cache_dtype=4)) == INVALID
    assert binding.pa_plan_status(**c.desc(num_sms=152, k_scale=0.0, v_scale=math.nan)) == OK     # not theirs
    big = 1 << 40
    eight = (FAKE,) * 5
    assert lib.pa_attention(plan.handle, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, big, None) == INVALID
    assert lib.pa_attention_launch(plan.handle, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, big, None) == INVALID
    for f in (lib.pa_attention_with_kv_update, lib.pa_attention_with_kv_update_launch):
        assert f(plan.handle, *eight, FAKE, None, FAKE, FAKE, big, None) == INVALID
    assert lib.pa_attention_no_alloc(plan.handle, FAKE, FAKE, FAKE, FAKE, FAKE, None, None) == INVALID
    for f in (lib.pa_attention_scaled, lib.pa_attention_scaled_launch):
        call = lambda p=plan.handle, q=FAKE, ks=FAKE, vs=FAKE, ws=FAKE, n=big: \
            f(p, q, FAKE, FAKE, ks, vs, FAKE, FAKE, ws, n, None)  # noqa: E731, B023
        assert call(p=None) == INVALID and call(p=e4m3.handle) == INVALID
        for bad in (dict(q=None), dict(q=FAKE + 8), dict(ks=None), dict(vs=None), dict(ks=FAKE + 2), dict(ws=FAKE + 16)):
            assert call(**bad) == INVALID, bad
        assert call(n=16) == binding.PA_ERR_WORKSPACE_TOO_SMALL
    empty = oc.Case(hq=4, hkv=2, d=64, q_lens=[0], seq_lens=[5], code="int8")
    p0 = binding.pa_plan(**empty.desc(num_sms=4))
    assert lib.pa_attention_scaled(p0.handle, None, None, None, None, None, None, None, None, 0, None) == OK
    assert lib.pa_attention(p0.handle, None, None, None, None, None, None, 0, None) == INVALID
    shape = dict(max_tokens=64, max_reqs=4, max_extend_tiles=8)
    assert binding.pa_plan_fixed_status(**shape, **c.desc(num_sms=152)) == INVALID                 # tiles need copies
    assert binding.pa_plan_fixed_status(**shape, max_dequant_blocks=64, **c.desc(num_sms=152)) == OK


def test_zero_blocks_of_scaled_caches(lib):
    for kind in (binding.PA_KV_FP8_E4M3_BLOCK, binding.PA_KV_INT8_BLOCK):
        assert lib.pa_zero_blocks(None, 0, 10, 2, 64, kind, None, None, None, None) == OK


def test_native_graph_refuses_scaled(lib):
    c = oc.Case(hq=4, hkv=2, d=64, q_lens=[1], seq_lens=[5], code="int8")
    d, keep = binding.make_desc(**c.desc(num_sms=4))
    fs = binding.FixedShape()
    fs.max_tokens = fs.max_reqs = 4
    b = binding.GraphBuffers()
    for f in ("q", "key", "value", "out", "query_start_loc", "num_computed", "block_table", "key_cache", "value_cache"):
        setattr(b, f, FAKE)
    h = ctypes.c_void_p()
    assert lib.pa_graph_create(ctypes.byref(d), ctypes.byref(fs), ctypes.byref(b), ctypes.byref(h)) == UNSUPPORTED


@pytest.mark.parametrize("call", ["pa_attention_scaled", "pa_attention_scaled_launch"])
@pytest.mark.parametrize("change, message", [
    (dict(q=torch.zeros(3, 4, 64)), "bf16"),
    (dict(q=torch.zeros(3, 64, 4, dtype=torch.bfloat16).transpose(1, 2)), "contiguous bf16"),
    (dict(out=torch.zeros(6, 4, 64, dtype=torch.bfloat16)[::2]), "contiguous bf16"),
    (dict(table=torch.zeros(1, 2, dtype=torch.int64)), "int32"),
    (dict(table=torch.zeros(2, 4, dtype=torch.int32)[:, ::2]), "contiguous int32"),
    (dict(kc=torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)), "codes"),
    (dict(vc=torch.zeros(2, 16, 2, 64, dtype=torch.uint8)), "one shape"),
    (dict(vc=torch.zeros(3, 16, 2, 64, dtype=torch.int8)), "one shape"),
    (dict(kc=torch.zeros(2, 16, 4, 64, dtype=torch.int8)[:, :, ::2]), "contiguous codes"),
    (dict(ks=torch.ones(2, 3)), "scales"),
    (dict(vs=torch.ones(2, 2, dtype=torch.float64)), "scales"),
    (dict(vs=torch.ones(2, 4)[:, ::2]), "scales"),
    (dict(), "current CUDA device"),
])
def test_attention_wrappers_refuse(call, change, message):
    a = dict(q=torch.zeros(3, 4, 64, dtype=torch.bfloat16), kc=torch.zeros(2, 16, 2, 64, dtype=torch.int8),
             vc=torch.zeros(2, 16, 2, 64, dtype=torch.int8), ks=torch.ones(2, 2), vs=torch.ones(2, 2),
             table=torch.zeros(1, 2, dtype=torch.int32), out=torch.zeros(3, 4, 64, dtype=torch.bfloat16),
             workspace=torch.zeros(4096, dtype=torch.uint8))
    with pytest.raises(ValueError, match=message):
        getattr(binding, call)(None, *(a | change).values())
