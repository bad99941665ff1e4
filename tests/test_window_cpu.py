"""Plans with a sliding window and first tokens, and rotations with several axes,
on the CPU: arguments, refusals, what the plans read (no kernel runs)."""
import ctypes

import numpy as np
import pytest
import torch

import window_common as wc
from paged_kv_cache_16_gb300 import binding, build

INVALID, UNSUPPORTED, OK = binding.PA_ERR_INVALID_ARGUMENT, binding.PA_ERR_UNSUPPORTED, binding.PA_OK
CAPACITY = binding.PA_ERR_CAPACITY
FAKE = 1 << 20     # aligned, never dereferenced on the paths tested here


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


def desc(q_lens, seq, window=32, sinks=0, code=0, hq=8, hkv=2, d=128, table=None, **over):
    qsl = np.concatenate([[0], np.cumsum(q_lens)])
    seq = np.asarray(seq)
    kw = dict(num_heads_q=hq, num_heads_kv=hkv, head_dim=d, num_blocks=1000, query_start_loc=qsl, seq_lens=seq,
              num_computed_tokens=seq - np.asarray(q_lens), max_blocks_per_req=200, softmax_scale=0.1, num_sms=152,
              kv_cache_dtype=code, block_table_host=table, window=window, sink_tokens=sinks)
    kw.update(over)
    return kw


@pytest.mark.parametrize("over,status", [
    (dict(), OK), (dict(window=1), OK), (dict(window=2**31 - 1), OK), (dict(sink_tokens=2**31 - 1), OK),
    (dict(window=2**31 - 1, sink_tokens=2**31 - 1), OK), (dict(window=0), INVALID), (dict(window=-5), INVALID),
    (dict(sink_tokens=-1), INVALID), (dict(num_common_prefix_blocks=1), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED),
    (dict(kv_cache_dtype=7), INVALID), (dict(softmax_scale=0.0), INVALID), (dict(block_size=32), UNSUPPORTED)])
@pytest.mark.parametrize("q_len", [1, 4, 300])
def test_window_arguments(over, status, q_len):
    assert binding.pa_plan_window_status(**{**desc([q_len], [900]), **over}) == status


def test_contexts_longer_than_the_pool():
    """A context may outgrow the pool, and 32 bits of rounded positions are kept."""
    for n, status in ((2**31 - 257, OK), (2**31 - 256, UNSUPPORTED), (2**31 - 1, UNSUPPORTED)):
        for q in (1, 4, 300):
            kw = desc([q], [n], 512, 20, max_blocks_per_req=2**27)
            assert binding.pa_plan_window_status(**kw) == status, (n, q)
    info = binding.pa_plan_window(**desc([1], [2**31 - 257], 512, 20, max_blocks_per_req=2**27)).info()
    assert info["decode_kv_bytes"] == (512 + 20) * 2 * 2 * 128 * 2


def test_window_null_arguments(lib):
    d, _keep = binding.make_desc(**{k: v for k, v in desc([1], [9]).items() if k not in ("window", "sink_tokens")})
    w, p, n = binding.WindowDesc(4, 0), ctypes.c_void_p(), ctypes.c_size_t()
    call = lambda *a: lib.pa_plan_window(*a)  # noqa: E731
    r = ctypes.byref
    assert call(None, r(w), None, r(p), r(n)) == INVALID
    assert call(r(d), None, None, r(p), r(n)) == INVALID
    assert call(r(d), r(w), None, None, r(n)) == INVALID
    assert call(r(d), r(w), None, r(p), None) == INVALID and p.value is None


@pytest.mark.parametrize("code", range(4))
@pytest.mark.parametrize("q_lens,seq", [([1, 1, 1], [1, 100, 1600]), ([3, 8], [500, 40]), ([200, 70], [1500, 70]),
                                        ([1, 5, 90, 0], [700, 300, 800, 1000])])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 0), (17, 3), (100, 20), (64, 200), (5000, 4)])
def test_what_a_plan_reads(code, q_lens, seq, window, sinks):
    """Pairs, bytes and copied blocks are those of the seen keys."""
    info = binding.pa_plan_window(**desc(q_lens, seq, window, sinks, code)).info()
    pairs = nbytes = blocks = 0
    for q, n in zip(q_lens, seq):
        rows = [wc.seen(p, window, sinks) for p in range(n - q, n)]
        if q > 8:
            pairs += sum(int(r.sum()) for r in rows)
            some = np.zeros(n, bool)
            for r in rows:
                some[:len(r)] |= r
            blocks += len(np.unique(np.flatnonzero(some) // 16))
        elif q > 0:
            for j in range(0, q, 4):          # units of 16 / G tokens
                some = np.zeros(n, bool)
                for r in rows[j:j + 4]:
                    some[:len(r)] |= r
                nbytes += int(some.sum()) * 2 * 2 * 128 * (1 if code else 2)
    assert info["extend_flops"] == 4 * 128 * 8 * pairs
    assert info["decode_kv_bytes"] == nbytes
    assert info["num_dequant_blocks"] == (blocks if code else 0)


def test_block_ids_that_no_query_sees_are_not_checked():
    """Request 0 sees blocks 0, 1 (20 first tokens) and 5 .. 9 (positions 119 ..
    of a window of 32 before 150), request 1 none."""
    table = np.full((2, 200), -7, dtype=np.int32)
    table[0, :2] = 3
    table[0, 5:10] = 4
    kw = desc([1, 0], [151, 400], 64, 20, table=table)
    assert (151 - 64) // 16 == 5 and binding.pa_plan_window_status(**kw) == OK
    for bad in (0, 1, 5, 9):
        t = table.copy()
        t[0, bad] = 1000
        assert binding.pa_plan_window_status(**{**kw, "block_table_host": t}) == INVALID, bad
    del kw["window"], kw["sink_tokens"]
    assert binding.pa_plan_status(**kw) == INVALID


def test_a_window_without_effect_is_the_plain_plan():
    for q_lens, seq in (([1, 4, 300], [900, 77, 301]), ([1] * 64, list(range(10, 650, 10)))):
        kw = desc(q_lens, seq, 5000, 3)
        a = binding.pa_plan_window(**kw).info()
        del kw["window"], kw["sink_tokens"]
        assert a == binding.pa_plan(**kw).info()


@pytest.mark.parametrize("code", range(4))
def test_fixed_shapes_with_a_window(code):
    """Sizes depend on the shape; capacities are checked, blocks counted as seen."""
    shape = dict(max_tokens=400, max_reqs=8, max_extend_tiles=40, max_dequant_blocks=40 if code else 0)
    sizes = {binding.pa_plan_window(shape=shape, **desc(q, s, 64, 4, code)).workspace_bytes
             for q, s in (([1], [900]), ([200, 1], [1500, 3000]), ([1] * 8, [70] * 8))}
    assert len(sizes) == 1
    assert binding.pa_plan_window_status(shape=shape, **desc([390], [3000], 300, 4, code)) == (CAPACITY if code else OK)
    assert binding.pa_plan_window_status(shape=shape, **desc([401], [3000], 64, 4, code)) == CAPACITY
    assert binding.pa_plan_window_status(shape=dict(shape, max_tokens=0), **desc([1], [3], 64, 4, code)) == INVALID


@pytest.mark.parametrize("code", range(4))
def test_tiles_that_leave_sms_idle_are_cut(code):
    """Few tiles: cut into pieces for the SMs, joined by merge rows; a shape without
    room for the pieces keeps them whole, and so does one with a decode prefix."""
    kw = desc([40], [5000], 4000, 20, code, max_blocks_per_req=400)      # one tile of 33 steps per kv head
    info = binding.pa_plan_window(**kw).info()
    assert info["num_extend_tiles"] > 8 and info["num_merge_rows"] == 40 and info["num_extend_ctas"] == info["num_extend_tiles"]
    n, d = info["num_extend_tiles"], 500 if code else 0
    assert binding.pa_plan_window(**{**kw, "window": 200}).info()["num_extend_tiles"] == 2
    assert binding.pa_plan_window(**{**kw, "num_sms": 1}).info()["num_extend_tiles"] == 2
    shape = dict(max_tokens=100, max_reqs=4, max_extend_tiles=n, max_dequant_blocks=d, max_partial_slots=5000)
    assert binding.pa_plan_window(shape=shape, **kw).info()["num_extend_tiles"] == n
    for small in (dict(max_extend_tiles=n - 1), dict(max_partial_slots=10), dict(decode_prefix_tokens=1)):
        whole = binding.pa_plan_window(shape={**shape, **small}, **kw).info()
        assert whole["num_extend_tiles"] == 2 and whole["num_merge_rows"] == 0
    # a last round of a few tiles: 8 kv heads x 20 blocks of 64 tokens on 152 SMs
    wide = dict(hq=32, hkv=8, max_blocks_per_req=700)
    assert binding.pa_plan_window(**desc([1280], [9000], 8000, 0, code, **wide)).info()["num_extend_tiles"] > 160
    assert binding.pa_plan_window(**desc([1216], [9000], 8000, 0, code, **wide)).info()["num_extend_tiles"] == 152


@pytest.mark.parametrize("num_sms", [1, 3, 20, 152])
@pytest.mark.parametrize("code", range(4))
def test_more_runs_than_ctas_and_fewer(num_sms, code):
    """Every block of every row once, however many rows a CTA gets."""
    for n in (1, 2, 7, 40, 500):
        for d, hkv in ((128, 2), (128, 3)):
            kw = desc([1] * n, [100 + 3 * i for i in range(n)], 64, 4, code, hq=4 * hkv, hkv=hkv, d=d, num_sms=num_sms)
            info = binding.pa_plan_window(**kw).info()
            assert info["num_decode_rows"] == n and info["num_decode_items"] >= n
            assert binding.pa_plan_window(**{**kw, "window": 1}).info()["num_decode_items"] >= n
            shape = dict(max_tokens=600, max_reqs=600)
            assert binding.pa_plan_window(shape=shape, **kw).info()["num_decode_items"] == info["num_decode_items"]


def test_windowed_plans_refuse_the_wrong_calls(lib):
    """The attention calls go by the cache type, windows or not."""
    plain = binding.pa_plan_window(**desc([1], [40], code=0))
    scaled = binding.pa_plan_window(**desc([1], [40], code=3))
    assert lib.pa_attention(scaled.handle, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30, None) == INVALID
    assert lib.pa_attention_scaled(plain.handle, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30, None) == INVALID
    assert lib.pa_attention_launch(plain.handle, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1, None) == binding.PA_ERR_WORKSPACE_TOO_SMALL


@pytest.mark.parametrize("call", ["pa_attention", "pa_attention_launch", "pa_attention_with_kv_update",
                                  "pa_attention_with_kv_update_launch", "pa_attention_no_alloc"])
@pytest.mark.parametrize("fault", ["type", "heads", "pool", "rows", "table", "out", "host", "new rows"])
def test_wrappers_hold_tensors_against_a_windowed_plan(call, fault):
    plan = binding.pa_plan_window(**desc([1, 1], [40, 9], hq=4, hkv=2, d=64, num_blocks=9, max_blocks_per_req=4))
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
    a = dict(q=z(2, 4, 64), key=z(2, 2, 64), value=z(2, 2, 64), key_cache=z(9, 16, 2, 64), value_cache=z(9, 16, 2, 64),
             block_table=z(2, 4, t=torch.int32), out=z(2, 4, 64), workspace=z(plan.workspace_bytes, t=torch.uint8))
    if "update" not in call:
        del a["key"], a["value"]
        if fault == "new rows":
            return
    if call == "pa_attention_no_alloc":
        del a["workspace"]
    wrong = {"type": dict(key_cache=z(9, 16, 2, 64, t=torch.uint8), value_cache=z(9, 16, 2, 64, t=torch.uint8)),
             "heads": dict(key_cache=z(9, 16, 4, 64), value_cache=z(9, 16, 4, 64)),
             "pool": dict(key_cache=z(8, 16, 2, 64), value_cache=z(8, 16, 2, 64)), "rows": dict(q=z(1, 4, 64)),
             "table": dict(block_table=z(2, 5, t=torch.int32)), "out": dict(out=z(2, 4, 64, t=torch.float16)),
             "host": {}, "new rows": dict(key=z(1, 2, 64))}[fault]
    with pytest.raises(ValueError):
        getattr(binding, call)(plan, **{**a, **wrong})


# --------------------------------------------------------------------- axes --
def axes_status(lib, num_axes, axis, frequencies=0, **over):
    kw = dict(rotary_dim=2 * len(axis), layout=0, base=10000.0, scaling=0, factor=1.0, original_max_position=0, low=1.0,
              high=4.0, attention_factor=0.0)
    kw.update(over)
    d = binding._rope_desc(**kw)
    a = np.asarray(axis, dtype=np.int32)
    h = ctypes.c_void_p()
    st = lib.pa_rope_create_axes(ctypes.byref(d), ctypes.byref(binding.RopeAxesDesc(num_axes, frequencies, a.ctypes.data)),
                                 ctypes.byref(h))
    if st == OK:
        lib.pa_rope_destroy(h)
    return st


def test_axes_arguments(lib):
    ax = [0, 1, 2, 0] * 8
    assert axes_status(lib, 3, ax) == OK and axes_status(lib, 3, ax, 1) == OK and axes_status(lib, 4, ax) == OK
    assert axes_status(lib, 1, [0] * 4) == OK and axes_status(lib, 2, [1] * 4, 1) == OK       # an axis without pairs
    for bad in (dict(num_axes=0), dict(num_axes=-1), dict(num_axes=2), dict(frequencies=2), dict(frequencies=-1),
                dict(axis=[-1] + ax[1:]), dict(base=0.0), dict(layout=2), dict(scaling=1, factor=0.0)):
        assert axes_status(lib, **{**dict(num_axes=3, axis=ax), **bad}) == INVALID, bad
    assert axes_status(lib, 5, ax) == UNSUPPORTED and axes_status(lib, 3, [0] * 6) == UNSUPPORTED
    assert axes_status(lib, 3, [0] * 132) == UNSUPPORTED
    h = ctypes.c_void_p()
    assert lib.pa_rope_create_axes(ctypes.byref(binding.RopeDesc(32, 0, 0, 0, 10000.0)), None, ctypes.byref(h)) == INVALID
    assert lib.pa_rope_create_axes(None, ctypes.byref(binding.RopeAxesDesc(1, 0, FAKE)), ctypes.byref(h)) == INVALID
    assert lib.pa_rope_create_axes(ctypes.byref(binding.RopeDesc(32, 0, 0, 0, 10000.0)),
                                   ctypes.byref(binding.RopeAxesDesc(1, 0, None)), ctypes.byref(h)) == INVALID
    with pytest.raises(ValueError):
        binding.pa_rope_create_axes(num_axes=2, axis_of_pair=[0, 1], rotary_dim=8)


@pytest.mark.parametrize("scaling", [dict(), dict(scaling=1, factor=4.0),
                                     dict(scaling=2, factor=8.0, original_max_position=8192),
                                     dict(scaling=3, factor=8.0, original_max_position=8192, low=1.0, high=32.0)])
def test_axes_frequencies(scaling):
    """Shared: those of the whole rotation; own: of a rotation as wide as the axis."""
    axis = [0] * 8 + [1, 2] * 10 + [2] * 4
    kw = dict(rotary_dim=64, base=500000.0, **scaling)
    whole = binding.pa_rope_create(**kw).frequencies()
    assert np.array_equal(binding.pa_rope_create_axes(num_axes=3, axis_of_pair=axis, **kw).frequencies()[0], whole[0])
    own, m = binding.pa_rope_create_axes(num_axes=3, axis_of_pair=axis, frequencies=1, **kw).frequencies()
    assert m == whole[1]
    for a, n in enumerate((8, 10, 14)):
        mine = own[np.asarray(axis) == a]
        if n % 4 == 0:
            assert np.array_equal(mine, binding.pa_rope_create(**{**kw, "rotary_dim": 2 * n}).frequencies()[0])
        elif not scaling:
            assert np.allclose(mine, 500000.0 ** (-np.arange(n) / n), rtol=4e-15, atol=0)


def test_calls_without_axes_refuse_rotations_of_several(lib):
    r = binding.pa_rope_create_axes(num_axes=2, axis_of_pair=[0, 1] * 16, rotary_dim=64)
    one = binding.pa_rope_create(rotary_dim=64)
    assert lib.pa_rotary(r.handle, FAKE, 512, FAKE, 3, 4, 128, FAKE, 512, None) == INVALID
    a = binding.AppendArgs(2, 0, 4, 2, 64, 16, 9, 4, 3, 1.0, 1.0)
    assert lib.pa_append_kv(r.handle, ctypes.byref(a), None) == INVALID
    assert lib.pa_append_kv(one.handle, ctypes.byref(a), None) == OK
    assert lib.pa_append_kv_axes(r.handle, ctypes.byref(a), FAKE, 0, None) == OK
    assert lib.pa_append_kv_axes(one.handle, ctypes.byref(a), None, 0, None) == OK          # no tokens
    assert lib.pa_append_kv_axes(None, ctypes.byref(a), FAKE, 0, None) == INVALID


def test_rotary_axes_arguments(lib):
    r = binding.pa_rope_create_axes(num_axes=2, axis_of_pair=[0, 1] * 16, rotary_dim=64)
    call = lambda rope=r.handle, x=FAKE, xs=512, pos=FAKE, ps=3, t=3, h=4, d=128, out=FAKE, os_=512: \
        lib.pa_rotary_axes(rope, x, xs, pos, ps, t, h, d, out, os_, None)  # noqa: E731
    assert call(t=0, x=None, out=None, pos=None, ps=0) == OK
    for bad in (dict(rope=None), dict(t=-1), dict(h=0), dict(x=None), dict(x=FAKE + 8), dict(out=None), dict(pos=None),
                dict(pos=FAKE + 2), dict(ps=2), dict(ps=-1), dict(xs=504), dict(d=56)):
        assert call(**bad) == INVALID, bad
    assert call(d=100) == UNSUPPORTED


def test_append_axes_arguments(lib):
    from test_operators_cpu import append_args
    r = binding.pa_rope_create_axes(num_axes=3, axis_of_pair=[0, 1, 2, 1] * 8, rotary_dim=64)
    call = lambda pos=FAKE, ps=3, rope=r.handle, **over: \
        lib.pa_append_kv_axes(rope, ctypes.byref(append_args(**over)), pos, ps, None)  # noqa: E731
    for bad in (dict(pos=None), dict(pos=FAKE + 1), dict(ps=2), dict(ps=-3), dict(rope=None), dict(key=None),
                dict(num_reqs=-1), dict(q_out=None), dict(key_scales=None)):
        assert call(**bad) == INVALID, bad
    assert call(block_size=32) == UNSUPPORTED
    assert lib.pa_append_kv_axes(r.handle, None, FAKE, 3, None) == INVALID


def test_wrappers_check_positions():
    r = binding.pa_rope_create_axes(num_axes=3, axis_of_pair=[0, 1, 2, 1] * 8, rotary_dim=64)
    x = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    p = torch.zeros(3, 5, dtype=torch.int32)
    for bad in (p.long(), p[:2], p[:, :4], torch.zeros(5, 3, dtype=torch.int32).T, p[0]):
        with pytest.raises(ValueError, match="positions"):
            binding.pa_rotary_axes(r, x, bad, x)
    with pytest.raises(ValueError, match="current CUDA device"):
        binding.pa_rotary_axes(r, x, p, x)
