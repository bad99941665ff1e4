"""Rotary positions on several axes, the append with them, and steps of that append
and windowed attention, on the GPU against 64 bits (needs a GB300)."""
import numpy as np
import pytest
import torch

import operators_common as oc
import window_common as wc
from gpu_common import ensure_library
from paged_kv_cache_16_gb300 import binding
from paged_kv_cache_16_gb300.step import DeviceStep, GraphStep
from test_gpu_rotary_append import SHAPES, check_scaled
from test_gpu_window import batch_of

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_library()


def i32(a):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32, device=DEV)


PLAIN_COS_SIN = oc.cos_sin


def cos_sin(freq, axis, positions):
    """cos and sin of every pair at its own axis's positions [axes, T]."""
    c, s = np.empty((positions.shape[1], len(freq))), np.empty((positions.shape[1], len(freq)))
    for a in set(axis):
        mine = [i for i, x in enumerate(axis) if x == a]
        c[:, mine], s[:, mine] = PLAIN_COS_SIN(np.asarray(freq)[mine], positions[a])
    return c, s


def check_rotated(out, x, positions, rope, axis, layout):
    f, m = rope.frequencies()
    ref, size = oc.rotate(x.double().cpu().numpy(), cos_sin(f, axis, positions), rope.rotary_dim, layout == 1, m)
    oc.assert_within(out, ref, oc.BF16 * np.abs(ref) + oc.ROTATED * size)


def sections(rd, axes, kind):
    n = rd // 2
    return [i % axes for i in range(n)] if kind == "turn" else [i * axes // n for i in range(n)]


@pytest.mark.parametrize("tokens", [1, 2, 5, 17, 130])
@pytest.mark.parametrize("axes,kind,own", [(3, "sections", 0), (2, "sections", 1), (3, "turn", 0), (4, "turn", 1), (1, "turn", 0)])
@pytest.mark.parametrize("heads,d,rd,layout", [(5, 128, 128, 0), (40, 128, 128, 1), (3, 64, 16, 1), (2, 128, 24, 0), (9, 80, 40, 1),
                                               (1, 256, 256, 0), (2, 8, 8, 1)])
def test_rotary_axes(tokens, axes, kind, own, heads, d, rd, layout):
    rng = np.random.default_rng(tokens + rd)
    axis = sections(rd, axes, kind)
    x = torch.randn(tokens, heads + 2, d, generator=torch.Generator().manual_seed(rd)).to(torch.bfloat16).to(DEV)[:, 1:1 + heads]
    pos = rng.integers(-1000, 200000, (axes, tokens))
    pos[:, 0] = [2**31 - 1, 0, -2**31, 1][:axes]
    rope = binding.pa_rope_create_axes(num_axes=axes, axis_of_pair=axis, rotary_dim=rd, frequencies=own, layout=layout)
    out = torch.full((tokens, heads, d), 9.0, dtype=torch.bfloat16, device=DEV)
    # a buffer of a larger capacity, read through a view
    wide = torch.full((axes, tokens + 3), 77, dtype=torch.int32, device=DEV)
    wide[:, :tokens] = i32(pos)
    binding.pa_rotary_axes(rope, x, wide[:, :tokens], out)
    check_rotated(out, x, pos, rope, axis, layout)
    assert torch.equal(out[..., rd:], x[..., rd:])


@pytest.mark.parametrize("scaling", [0, 1, 2, 3])
def test_one_position_on_every_axis_is_the_plain_rotation(scaling):
    """Shared frequencies: bit for bit, also with one row of positions for all axes."""
    kw = dict(rotary_dim=64, base=500000.0, scaling=scaling, factor=8.0, original_max_position=8192, low=1.0, high=32.0)
    x = torch.randn(40, 3, 64, generator=torch.Generator().manual_seed(scaling)).to(torch.bfloat16).to(DEV)
    pos = i32(np.random.default_rng(1).integers(0, 100000, 40))
    plain, a, b = (torch.empty_like(x) for _ in range(3))
    binding.pa_rotary(binding.pa_rope_create(**kw), x, pos, plain)
    rope = binding.pa_rope_create_axes(num_axes=3, axis_of_pair=[0, 1, 1, 2] * 8, **kw)
    binding.pa_rotary_axes(rope, x, pos.repeat(3, 1), a)
    binding.pa_rotary_axes(rope, x, pos[None].expand(3, -1), b)
    assert torch.equal(a, plain) and torch.equal(b, plain)


def test_rotary_axes_in_place_and_gradient():
    """In place in a packed projection, its neighbours untouched; by negated
    positions the gradient: <R x, y> = <x, R^T y>."""
    g = torch.Generator().manual_seed(5)
    packed = torch.randn(40, 8, 128, generator=g).to(torch.bfloat16).to(DEV)
    y = torch.randn(40, 3, 128, generator=g).to(torch.bfloat16).to(DEV)
    before, axis = packed.clone(), [0] * 16 + [1] * 24 + [2] * 24
    pos = np.random.default_rng(1).integers(0, 100000, (3, 40))
    rope = binding.pa_rope_create_axes(num_axes=3, axis_of_pair=axis, rotary_dim=128)
    rx, ry = packed[:, 2:5], torch.empty_like(y)
    binding.pa_rotary_axes(rope, rx, i32(pos), rx)
    check_rotated(rx, before[:, 2:5], pos, rope, axis, 0)
    assert torch.equal(packed[:, :2], before[:, :2]) and torch.equal(packed[:, 5:], before[:, 5:])
    binding.pa_rotary_axes(rope, y, -i32(pos), ry)
    a, b = rx.double() * y.double(), before[:, 2:5].double() * ry.double()
    # each rotated element is off by half a step of itself at most
    assert (a.sum() - b.sum()).abs() <= oc.BF16 * (a.abs().sum() + b.abs().sum()) * 1.01


def run_append(c, rope, pos, fn=None, pad=0):
    """The case on the GPU: (q_out, key_cache, value_cache, key_scales, value_scales)."""
    def rows(t):
        t = t.to(DEV)
        return t if not pad else torch.cat([t, torch.full((pad,) + tuple(t.shape[1:]), float("nan"), dtype=t.dtype, device=DEV)])
    q, k, v = (rows(t[:max(c.T, 1)]) for t in (c.q, c.key, c.value))
    q_out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device=DEV)
    kc, vc, ks, vs = (t.to(DEV) for t in (c.kc, c.vc, c.ks, c.vs))
    more = dict(key_scales=ks, value_scales=vs) if c.scaled else {}
    if c.code == "fp8":
        more.update(k_scale=0.031, v_scale=0.007)
    p = torch.full((len(pos), q.shape[0]), -2**31, dtype=torch.int32, device=DEV)
    p[:, :c.T] = i32(pos)
    binding.pa_append_kv_axes(rope, k, v, p, i32(c.qsl), i32(c.nc), i32(c.table), kc, vc, q=q, q_out=q_out, **more)
    torch.cuda.synchronize()
    return q_out, kc, vc, ks, vs


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("q_lens,computed", SHAPES)
@pytest.mark.parametrize("hq,hkv,d,rd,layout,axes,kind", [(4, 2, 64, 64, 0, 3, "sections"), (6, 3, 128, 32, 1, 2, "turn"),
                                                          (32, 16, 64, 24, 0, 4, "turn")])
def test_append_axes_scaled(code, q_lens, computed, hq, hkv, d, rd, layout, axes, kind, monkeypatch):
    c = oc.AppendCase(hq=hq, hkv=hkv, d=d, q_lens=q_lens, computed=computed, code=code, seed=len(q_lens) + rd)
    axis = sections(rd, axes, kind)
    pos = np.random.default_rng(c.T).integers(-50, 5000, (axes, c.T))
    rope = binding.pa_rope_create_axes(num_axes=axes, axis_of_pair=axis, rotary_dim=rd, layout=layout)
    got = run_append(c, rope, pos)
    monkeypatch.setattr(oc, "cos_sin", lambda f, _: cos_sin(f, axis, pos))
    check_scaled(c, got, rope, layout)
    check_rotated(got[0][:c.T], c.q[:c.T], pos, rope, axis, layout)


@pytest.mark.parametrize("code", ["bf16", "fp8", "int8", "e4m3"])
def test_append_axes_at_the_slots_positions_is_the_plain_append(code):
    c = oc.AppendCase(hq=4, hkv=2, d=128, q_lens=[1, 37, 0, 2, 16], computed=[40, 3, 7, 15, 32], seed=1,
                      code="bf16" if code == "fp8" else code)
    if code == "fp8":
        c.code = code
        c.kc, c.vc = (torch.randint(0, 120, c.kc.shape, dtype=torch.uint8) for _ in range(2))
    kw = dict(rotary_dim=128, layout=1, base=500000.0)
    rope = binding.pa_rope_create_axes(num_axes=3, axis_of_pair=[0, 1, 2, 1] * 16, **kw)
    one = binding.pa_rope_create(**kw)
    pos = c.positions()
    a, b = run_append(c, rope, np.tile(pos, (3, 1))), run_append(c, one, pos[None])
    from test_gpu_rotary_append import run_append as plain
    for x, y, z in zip(a, b, plain(c, one)):
        assert torch.equal(x, z) and torch.equal(y, z)


@pytest.mark.parametrize("code", ["bf16", "fp8"])
def test_append_axes_plain_caches(code):
    """bf16: pa_rotary_axes' keys; E4M3: the code of the key rotated in 32 bits."""
    c = oc.AppendCase(hq=2, hkv=2, d=128, q_lens=[21, 1, 40], computed=[11, 77, 0], code="bf16", seed=12)
    if code == "fp8":
        c.code = code
        c.kc, c.vc = (torch.randint(0, 120, c.kc.shape, dtype=torch.uint8) for _ in range(2))
    axis = sections(128, 3, "sections")
    pos = np.random.default_rng(2).integers(0, 3000, (3, c.T))
    rope = binding.pa_rope_create_axes(num_axes=3, axis_of_pair=axis, rotary_dim=128)
    got = run_append(c, rope, pos)
    rot = torch.empty(c.T, 2, 128, dtype=torch.bfloat16, device=DEV)
    binding.pa_rotary_axes(rope, c.key.to(DEV).contiguous(), i32(pos), rot)
    f, m = rope.frequencies()
    k, size = oc.rotate(c.key.double().numpy(), cos_sin(f, axis, pos), 128, False, m)
    for b, first, t0, cnt in c.segments():
        g = got[1][b, first:first + cnt]
        if code == "bf16":
            assert torch.equal(g, rot[t0:t0 + cnt]) and torch.equal(got[2][b, first:first + cnt].cpu(), c.value[t0:t0 + cnt])
            continue
        g, y = oc.values(g.cpu().numpy(), "e4m3"), k[t0:t0 + cnt] / float(np.float32(0.031))
        e = oc.ROTATED * size[t0:t0 + cnt] / 0.031 + 2.0 ** -24 * np.abs(y)
        assert (np.abs(g - y) <= oc.half_step(np.maximum(np.abs(y), np.abs(g)), "e4m3") + e).all()


@pytest.mark.parametrize("code", ["int8", "bf16"])
def test_append_axes_padded_launch(code):
    """Rows behind the last token are neither read (NaN, positions at the range's end)
    nor written."""
    c = oc.AppendCase(hq=4, hkv=2, d=64, q_lens=[5, 1, 0, 0], computed=[3, 16, 0, 0], code=code, seed=1)
    rope = binding.pa_rope_create_axes(num_axes=2, axis_of_pair=[0, 1] * 16, rotary_dim=64)
    pos = np.random.default_rng(2).integers(0, 3000, (2, c.T))
    a, b = run_append(c, rope, pos), run_append(c, rope, pos, pad=50)
    assert (b[0][c.T:] == 5).all() and torch.equal(a[0], b[0][:c.T])
    for x, y in zip(a[1:], b[1:]):
        assert torch.equal(x, y)


def test_captured_on_another_stream_follows_its_positions():
    c = oc.AppendCase(hq=4, hkv=2, d=64, q_lens=[4, 1], computed=[14, 3], code="int8", seed=5)
    axis = [0, 1] * 16
    rope = binding.pa_rope_create_axes(num_axes=2, axis_of_pair=axis, rotary_dim=64)
    q, k, v = (t.to(DEV).contiguous() for t in (c.q, c.key, c.value))
    q_out, rot = torch.zeros_like(q), torch.zeros_like(q)
    kc, vc, ks, vs = (t.to(DEV) for t in (c.kc, c.vc, c.ks, c.vs))
    pos = torch.zeros(2, c.T, dtype=torch.int32, device=DEV)
    args = (i32(c.qsl), i32(c.nc), i32(c.table))

    def call():
        binding.pa_append_kv_axes(rope, k, v, pos, *args, kc, vc, key_scales=ks, value_scales=vs, q=q, q_out=q_out)
        binding.pa_rotary_axes(rope, q, pos, rot)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    new = np.random.default_rng(2).integers(0, 3000, (2, c.T))
    pos.copy_(i32(new))
    for t, src in ((kc, c.kc), (vc, c.vc), (ks, c.ks), (vs, c.vs)):
        t.copy_(src)
    graph.replay()
    torch.cuda.synchronize()
    check_rotated(q_out, c.q, new, rope, axis, 0)
    assert torch.equal(q_out, rot)
    want = run_append(c, rope, new)
    for x, y in zip((kc, vc, ks, vs), want[1:]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("left", ["positions", "x", "out", "key", "block_table"])
def test_one_tensor_left_on_the_host_is_refused(left):
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    rope = binding.pa_rope_create_axes(num_axes=2, axis_of_pair=[0, 1] * 16, rotary_dim=64)
    a = dict(x=x, positions=i32([[0, 1, 2]] * 2), out=x.clone(), key=x, block_table=i32([[0]]))
    a[left] = a[left].cpu()
    cache = torch.zeros(1, 16, 2, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="current CUDA device"):
        if left in ("x", "out"):
            binding.pa_rotary_axes(rope, a["x"], a["positions"], a["out"])
        else:
            binding.pa_append_kv_axes(rope, a["key"], x, a["positions"], i32([0, 3]), i32([0]), a["block_table"], cache,
                                      cache.clone())


# ----------------------------------------------------------------- together --
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp8_block", "int8_block"])
def test_steps_of_append_and_windowed_attention(kind):
    """A prompt with a grid of patches in chunks, then single tokens, through
    DeviceStep and GraphStep: keys turned by positions on three axes, appended, and
    attended to through the window.  Against attention in 64 bits over the cache as
    it then is, with queries rotated in 64 bits; blocks behind the window are given
    back (zeroed, their entries invalid) as the steps go."""
    window, sinks, hq, hkv, d = 40, 5, 8, 2, 128
    code = {"bf16": "bf16", "fp8": "e4m3"}.get(kind, "e4m3_block" if kind == "fp8_block" else kind)
    total = 230
    grid = np.stack(np.unravel_index(np.arange(2 * 6 * 8), (2, 6, 8)))
    pos = np.concatenate([np.tile(np.arange(30), (3, 1)), grid + 30, np.tile(np.arange(38, 38 + total - 126), (3, 1))], 1)
    axis = sections(128, 3, "sections")
    rope = binding.pa_rope_create_axes(num_axes=3, axis_of_pair=axis, rotary_dim=128, base=500000.0)
    f, m = rope.frequencies()
    g = torch.Generator().manual_seed(1)
    q, key, value = (torch.randn(total, n, d, generator=g).to(torch.bfloat16).to(DEV) for n in (hq, hkv, hkv))
    nb = 20
    dtype = dict(bf16=torch.bfloat16, int8_block=torch.int8).get(code, torch.uint8)
    eager, graphed = ([torch.zeros(nb, 16, hkv, d, dtype=dtype, device=DEV) for _ in range(2)] +
                      ([torch.ones(nb, hkv, device=DEV) for _ in range(2)] if code in wc.SCALED else []) for _ in range(2))
    gs = GraphStep(num_heads_q=hq, num_heads_kv=hkv, head_dim=d, num_blocks=nb, max_blocks_per_req=16, softmax_scale=d ** -0.5,
                   max_tokens=100, max_reqs=2, max_extend_tiles=8, max_dequant_blocks=20, kv_cache_dtype=kind,
                   k_scale=wc.K_SCALE, v_scale=wc.V_SCALE, rope=rope, window=(window, sinks))
    ids = np.random.default_rng(3).permutation(nb)
    table = np.full(16, -1, dtype=np.int32)
    table[:15] = ids[:15]
    done = 0
    for n in (70, 3, 100, 1, 5, 1, 1, 20, 1, 1, 12, 1):
        low = max(0, done - window + 1) // 16
        table[1:low] = -1                       # behind every window; block 0 holds the first tokens
        c = wc.WindowCase(hq=hq, hkv=hkv, d=d, q_lens=[n], seq_lens=[done + n], code=code, window=window, sinks=sinks)
        c.table, c.nb = np.ascontiguousarray(table[None]), nb
        b = batch_of(c, kind)
        st = DeviceStep(b, "cuda", rope=rope, window=(window, sinks))
        now = i32(pos[:, done:done + n])
        rows = [t[done:done + n] for t in (q, key, value)]
        out = st.run_append(*rows, *eager, positions=now)
        again = gs.run(b, *rows, *graphed, positions=now)
        torch.cuda.synchronize()
        assert st.check_errors() == 0 and gs.check_errors() == 0
        assert torch.equal(out, again)
        for x, y in zip(eager, graphed):
            assert torch.equal(x, y)
        check_rotated(st.q_rot, rows[0], pos[:, done:done + n], rope, axis, 0)
        c.q = st.q_rot.cpu()
        c.kc, c.vc = eager[0].cpu(), eager[1].cpu()
        if c.scaled:
            c.ks, c.vs = eager[2].cpu(), eager[3].cpu()
        ref, tol = c.reference()
        oc.assert_within(out, ref, tol, f"{done} + {n}")
        if code == "bf16":                       # the cache holds the keys turned by their own positions
            blk, off = table[np.arange(done, done + n) // 16], np.arange(done, done + n) % 16
            check_rotated(eager[0][blk, off], rows[1], pos[:, done:done + n], rope, axis, 0)
        done += n


def test_step_classes_refuse_missing_or_spare_positions():
    rope = binding.pa_rope_create_axes(num_axes=2, axis_of_pair=[0, 1] * 32, rotary_dim=128)
    one = binding.pa_rope_create(rotary_dim=128)
    c = wc.WindowCase(hq=8, hkv=2, d=128, q_lens=[2], seq_lens=[30], code="bf16", window=9, sinks=0, pad=0, hidden=False)
    b = batch_of(c, "bf16")
    kc, vc = c.kc.to(DEV), c.vc.to(DEV)
    q, new = c.q.to(DEV), torch.zeros(2, 2, 128, dtype=torch.bfloat16, device=DEV)
    pos = i32([[1, 2], [3, 4]])
    for r, p in ((rope, None), (None, pos), (one, pos), (rope, pos[:1])):
        with pytest.raises(ValueError):
            DeviceStep(b, "cuda", rope=r).run_append(q, new, new, kc, vc, positions=p)
    DeviceStep(b, "cuda", rope=one).run_append(q, new, new, kc, vc, positions=pos[:1])
    kw = dict(num_heads_q=8, num_heads_kv=2, head_dim=128, num_blocks=c.nb, max_blocks_per_req=8, softmax_scale=0.1, max_tokens=8,
              max_reqs=2)
    for r, p in ((rope, None), (None, pos), (one, pos[:1]), (rope, pos[:, :1])):
        with pytest.raises(ValueError):
            GraphStep(rope=r, **kw).run(b, q, new, new, kc, vc, positions=p)
    with pytest.raises(ValueError):
        GraphStep(rope=rope, host_io=True, **kw)
