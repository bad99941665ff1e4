"""Rotary positions and the rotating append on the GPU, against the plain
implementations in 64 bits (needs a GB300)."""
import numpy as np
import pytest
import torch

import operators_common as oc
from gpu_common import ensure_library
from paged_kv_cache_16_gb300 import binding
from paged_kv_cache_16_gb300.workloads import bf16_bits

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_library()


def gpu(a, dtype=None):
    return torch.as_tensor(a, dtype=dtype, device=DEV)


def i32(a):
    return gpu(np.ascontiguousarray(a), torch.int32)


def check_rotated(out, x, positions, rope, layout, what=""):
    f, m = rope.frequencies()
    ref, size = oc.rotate(x.double().cpu().numpy(), oc.cos_sin(f, positions), rope.rotary_dim, layout == 1, m)
    oc.assert_within(out, ref, oc.BF16 * np.abs(ref) + oc.ROTATED * size, what)


@pytest.mark.parametrize("tokens", [1, 2, 5, 17, 300, 513])
@pytest.mark.parametrize("heads,d,rd,layout", [(5, 128, 128, 0), (40, 128, 128, 1), (3, 64, 16, 1), (17, 64, 64, 0),
                                               (2, 128, 24, 0), (9, 80, 40, 1), (1, 256, 256, 0), (33, 96, 8, 0),
                                               (2, 8, 8, 1)])
def test_rotary(tokens, heads, d, rd, layout):
    if tokens > 20 and heads * d > 2000:
        tokens = tokens // 4 + 1
    g = torch.Generator().manual_seed(tokens * 7 + rd)
    x = torch.randn(tokens, heads + 2, d, generator=g).to(torch.bfloat16).to(DEV)[:, 1:1 + heads]
    pos = np.random.default_rng(tokens).integers(0, 200000, tokens)
    pos[0] = 0 if tokens > 1 else 131071
    rope = binding.pa_rope_create(rotary_dim=rd, layout=layout, base=10000.0)
    out = torch.full((tokens, heads, d), 9.0, dtype=torch.bfloat16, device=DEV)
    binding.pa_rotary(rope, x, i32(pos), out)
    check_rotated(out, x, pos, rope, layout)
    assert torch.equal(out[..., rd:], x[..., rd:])


@pytest.mark.parametrize("scaling", [0, 1, 2, 3])
@pytest.mark.parametrize("layout", [0, 1])
def test_rotary_far_positions(scaling, layout):
    """Scaled frequencies, at the ends of the position range and negative."""
    rope = binding.pa_rope_create(rotary_dim=64, layout=layout, base=500000.0, scaling=scaling, factor=8.0,
                                  original_max_position=8192, low=1.0, high=32.0)
    pos = np.array([0, 1, -1, 2**31 - 1, -2**31, 123456789, 1 << 24, (1 << 24) + 1, -77777, 8192])
    x = torch.randn(10, 2, 64, generator=torch.Generator().manual_seed(scaling)).to(torch.bfloat16).to(DEV)
    out = torch.empty_like(x)
    binding.pa_rotary(rope, x, i32(pos), out)
    check_rotated(out, x, pos, rope, layout)


def test_rotary_in_place_strides_and_neighbours():
    """In place on the query and key heads of a packed projection; the rest of
    each row, and rows behind the last, stay as they were."""
    packed = torch.randn(21, 10, 64, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(DEV)
    before = packed.clone()
    rope = binding.pa_rope_create(rotary_dim=32)
    pos = np.arange(100, 119)
    view = packed[:19, :7]
    binding.pa_rotary(rope, view, i32(pos), view)
    check_rotated(view, before[:19, :7], pos, rope, 0)
    assert torch.equal(packed[19:], before[19:]) and torch.equal(packed[:, 7:], before[:, 7:])
    # out of place into a strided output
    wide = torch.zeros(19, 9, 64, dtype=torch.bfloat16, device=DEV)
    binding.pa_rotary(rope, before[:19, :7], i32(pos), wide[:, 1:8])
    assert torch.equal(wide[:, 1:8], view) and not wide[:, 0].any() and not wide[:, 8].any()


def test_rotary_inverse_and_gradient():
    """Rotating by the negated positions undoes the rotation, and is its
    gradient: <R x, y> = <x, R^T y>."""
    g = torch.Generator().manual_seed(5)
    x, y = (torch.randn(40, 3, 128, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    pos = i32(np.random.default_rng(1).integers(0, 100000, 40))
    rope = binding.pa_rope_create(rotary_dim=128, layout=1)
    rx, back, ry = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    binding.pa_rotary(rope, x, pos, rx)
    binding.pa_rotary(rope, rx, -pos, back)
    binding.pa_rotary(rope, y, -pos, ry)
    # two roundings to bf16 of rows whose norm the rotation keeps
    assert ((back - x).double().norm() / x.double().norm()).item() <= 2 * oc.BF16
    # each output element is off by 2^-8 of itself at most
    a, b = (rx.double() * y.double()).sum(), (x.double() * ry.double()).sum()
    bound = oc.BF16 * ((rx.double() * y.double()).abs().sum() + (x.double() * ry.double()).abs().sum()) * 1.01
    assert (a - b).abs() <= bound


def test_rotary_nan_and_infinity_stay_in_their_pairs():
    x = torch.ones(2, 1, 64, dtype=torch.bfloat16, device=DEV)
    x[0, 0, 3], x[1, 0, 40] = float("nan"), float("inf")
    rope = binding.pa_rope_create(rotary_dim=32)
    out = torch.empty_like(x)
    binding.pa_rotary(rope, x, i32([7, 7]), out)
    bad = ~torch.isfinite(out)
    assert bad.nonzero().tolist() == [[0, 0, 3], [0, 0, 19], [1, 0, 40]] and out[1, 0, 40] == float("inf")


# ------------------------------------------------------------------ append --
def run_append(c, rope=None, with_q=True, pad=0, err=None, table=None):
    """The case on the GPU: (q_out, key_cache, value_cache, key_scales, value_scales)."""
    def cap(t):      # rows of a launch sized for a capacity
        if not pad:
            return t.to(DEV) if t.is_contiguous() else strided(t)
        return torch.cat([t.to(DEV), torch.full((pad,) + tuple(t.shape[1:]), float("nan"), dtype=t.dtype, device=DEV)])

    def strided(t):
        base = torch.empty(t.shape[0], t.shape[1] + 3, t.shape[2], dtype=t.dtype, device=DEV)
        v = base[:, 1:1 + t.shape[1]]
        v.copy_(t)
        return v
    T = max(c.T, 0)
    q, k, v = (cap(t[:max(T, 1)]) for t in (c.q, c.key, c.value))
    q_out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device=DEV)
    kc, vc, ks, vs = (t.to(DEV) for t in (c.kc, c.vc, c.ks, c.vs))
    more = dict(key_scales=ks, value_scales=vs) if c.scaled else {}
    if rope is not None and with_q:
        more.update(q=q, q_out=q_out)
    if c.code == "fp8":
        more.update(k_scale=0.031, v_scale=0.007)
    binding.pa_append_kv(rope, k, v, i32(c.qsl), i32(c.nc), i32(c.table if table is None else table), kc, vc,
                         device_error_word=err, **more)
    torch.cuda.synchronize()
    return q_out, kc, vc, ks, vs


def check_scaled(c, got, rope, layout=0):
    """Codes and scales of the whole pool against the definition in 64 bits: new
    codes within half a step (plus the rotation's error in 32 bits) of the
    value, re-coded ones and all others exactly."""
    _, kc, vc, ks, vs = got
    x = {"k": c.key.double().numpy(), "v": c.value.double().numpy()}
    err = {"k": np.zeros_like(x["k"]), "v": np.zeros_like(x["v"])}
    if rope is not None and c.T:
        f, m = rope.frequencies()
        x["k"], size = oc.rotate(x["k"][:c.T], oc.cos_sin(f, c.positions()), rope.rotary_dim, layout == 1, m)
        err["k"] = oc.ROTATED * size
    for n, cache0, cache1, sc0, sc1 in (("k", c.kc, kc, c.ks, ks), ("v", c.vc, vc, c.vs, vs)):
        want = oc.values(cache0.numpy(), c.code)
        got_v = oc.values(cache1.cpu().numpy(), c.code)
        scale = sc0.double().numpy().copy()
        new = np.zeros(want.shape, bool)
        for b, first, t0, cnt in c.segments():
            for h in range(c.hkv):
                rows = x[n][t0:t0 + cnt, h]
                fine = np.abs(rows[np.isfinite(rows)])
                s = oc.power_scale(fine.max(initial=0.0), c.code)
                if c.code == "int8" and np.isnan(rows).any():
                    s = np.nan
                old = scale[b, h]
                if first and not np.isnan(s):
                    s = old if np.isnan(old) else max(s, old)
                if first and s > old:
                    want[b, :first, h] = oc.nearest(want[b, :first, h] * (old / s), c.code)
                scale[b, h] = s
                new[b, first:first + cnt, h] = True
                if np.isnan(s):
                    continue
                g = got_v[b, first:first + cnt, h]
                e = err[n][t0:t0 + cnt, h] / s
                y = np.clip(rows / s, -oc.QMAX[c.code], oc.QMAX[c.code])
                ok = np.abs(g - y) <= oc.half_step(np.maximum(np.abs(y), np.abs(g)), c.code) + e
                ok |= np.isnan(rows) & np.isnan(g)
                assert ok.all(), (n, b, h, first, cnt)
                exact = e == 0
                assert np.array_equal(g[exact], oc.nearest(y, c.code)[exact], equal_nan=True)
        assert np.array_equal(sc1.double().cpu().numpy(), scale, equal_nan=True), n
        assert np.array_equal(got_v[~new], want[~new], equal_nan=True), n


SHAPES = [([1], [0]), ([1], [15]), ([1], [16]), ([1, 1, 1, 1, 1], [3, 31, 7, 0, 100]), ([17], [0]), ([16], [16]),
          ([33, 1, 0, 5, 40], [5, 30, 9, 0, 70]), ([0, 0, 3], [0, 4, 14]), ([100], [1]), ([2] * 40, list(range(40)))]


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("q_lens,computed", SHAPES)
@pytest.mark.parametrize("hq,hkv,d,rd,layout", [(4, 2, 64, 64, 0), (6, 3, 128, 32, 1), (32, 16, 64, 24, 0), (9, 9, 128, 128, 0)])
def test_append_scaled(code, q_lens, computed, hq, hkv, d, rd, layout):
    c = oc.AppendCase(hq=hq, hkv=hkv, d=d, q_lens=q_lens, computed=computed, code=code, seed=len(q_lens) + rd)
    rope = binding.pa_rope_create(rotary_dim=rd, layout=layout, base=10000.0)
    got = run_append(c, rope)
    check_scaled(c, got, rope, layout)
    check_rotated(got[0], c.q, c.positions(), rope, layout)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("new_size,old_exp", [(1e-30, (-70, -60)), (1e30, (60, 70)), (300.0, (-9, -5)), (0.0, (-64, -60)),
                                              (1e-3, (-3, 3))])
def test_append_scaled_magnitudes(code, new_size, old_exp):
    """Values of every size next to old scales far below, near and above theirs:
    zeros, growth by many powers of two, scales at the 2^-64 floor."""
    c = oc.AppendCase(hq=4, hkv=2, d=64, q_lens=[1, 5, 20, 1], computed=[5, 11, 3, 16], code=code, seed=2,
                      new_size=new_size, old_exp=old_exp)
    check_scaled(c, run_append(c), None)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_append_scaled_nan_and_infinity(code):
    c = oc.AppendCase(hq=4, hkv=2, d=64, q_lens=[3, 1, 18], computed=[5, 11, 0], code=code, seed=4)
    for t in (c.key, c.value):
        t[0, 0, 5], t[1, 1, 7], t[3, 0, 9], t[5, 1, 0] = float("inf"), float("nan"), float("-inf"), float("nan")
        t[4, 0] = 0.0
    check_scaled(c, run_append(c), None)


def test_append_int8_nan_scale_lasts_until_the_block_starts_anew():
    c = oc.AppendCase(hq=2, hkv=2, d=64, q_lens=[2, 2, 2], computed=[4, 30, 16], code="int8", seed=1)
    c.ks[c.table[0, 0], 1] = float("nan")       # joined: stays
    c.vs[c.table[1, 1], 0] = float("nan")       # the first of its two blocks: stays
    c.ks[c.table[2, 1], 0] = float("nan")       # starts anew at slot 0: gone
    got = run_append(c)
    check_scaled(c, got, None)
    assert torch.isnan(got[3][c.table[0, 0], 1]) and torch.isnan(got[4][c.table[1, 1], 0])
    assert torch.isfinite(got[3][c.table[2, 1], 0])


def test_append_in_place_in_the_packed_projection():
    """q rotated in place beside the keys and values that are being stored."""
    c = oc.AppendCase(hq=4, hkv=2, d=64, q_lens=[19, 1], computed=[3, 40], code="int8", seed=2)
    rope = binding.pa_rope_create(rotary_dim=64)
    want = run_append(c, rope)
    rows = torch.cat([c.q, c.key, c.value], 1).to(DEV)
    before = rows.clone()
    q, k, v = rows[:, :4], rows[:, 4:6], rows[:, 6:]
    kc, vc, ks, vs = (t.to(DEV) for t in (c.kc, c.vc, c.ks, c.vs))
    binding.pa_append_kv(rope, k, v, i32(c.qsl), i32(c.nc), i32(c.table), kc, vc, key_scales=ks, value_scales=vs, q=q, q_out=q)
    torch.cuda.synchronize()
    for x, y in zip((q, kc, vc, ks, vs), want):
        assert torch.equal(x, y)
    assert torch.equal(rows[:, 4:], before[:, 4:])


def test_wrappers_refuse_tensors_of_other_devices():
    rope = binding.pa_rope_create(rotary_dim=64)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.pa_rotary(rope, x, torch.zeros(3, dtype=torch.int32), x)


@pytest.mark.parametrize("left", ["positions", "out", "key", "query_start_loc", "num_computed", "block_table", "key_scales",
                                  "q"])
def test_wrappers_refuse_one_tensor_left_on_the_host(left):
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    rope = binding.pa_rope_create(rotary_dim=64)
    a = dict(positions=i32([0, 1, 2]), out=x.clone(), key=x, value=x, query_start_loc=i32([0, 3]), num_computed=i32([0]),
             block_table=i32([[0]]), key_cache=torch.zeros(1, 16, 2, 64, dtype=torch.int8, device=DEV),
             value_cache=torch.zeros(1, 16, 2, 64, dtype=torch.int8, device=DEV), key_scales=torch.ones(1, 2, device=DEV),
             value_scales=torch.ones(1, 2, device=DEV), q=x, q_out=x.clone())
    a[left] = a[left].cpu()
    positions, out = a.pop("positions"), a.pop("out")
    with pytest.raises(ValueError, match="current CUDA device"):
        if left in ("positions", "out"):
            binding.pa_rotary(rope, x, positions, out)
        else:
            binding.pa_append_kv(rope, **a)


def test_append_scaled_foreign_scales():
    """Old scales that are no powers of two: kept where large enough, codes
    re-coded by the true ratio where not."""
    for code in ("int8", "e4m3"):
        c = oc.AppendCase(hq=4, hkv=2, d=64, q_lens=[1] * 12, computed=list(range(1, 13)), code=code, seed=6)
        c.ks *= 1.37
        c.vs *= 0.73
        x = run_append(c)
        # the quotients are rounded to 32 bits before they become codes: the
        # same there and here unless a code is decided by the last bit
        check_codes_near(c, x)


def check_codes_near(c, got):
    for x, cache0, cache1, sc0, sc1 in ((c.key, c.kc, got[1], c.ks, got[3]), (c.value, c.vc, got[2], c.vs, got[4])):
        for b, first, t0, cnt in c.segments():
            for h in range(c.hkv):
                rows = x[t0:t0 + cnt, h].double().numpy()
                p = oc.power_scale(np.abs(rows).max(), c.code)
                old = float(sc0[b, h])
                s = float(np.float32(max(old, p)))
                assert float(sc1[b, h]) == s
                v0 = oc.values(cache0[b].numpy(), c.code)[:, h]
                v1 = oc.values(cache1[b].cpu().numpy(), c.code)[:, h]
                y = np.concatenate([v0[:first] * (old / s), rows / s])
                g = v1[:first + cnt]
                assert (np.abs(g - y) <= oc.half_step(np.maximum(np.abs(y), np.abs(g)), c.code) * (1 + 1e-6) + 1e-6 * np.abs(y)).all()


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_append_token_by_token(code):
    """One token a call: the same scales as one call for all, codes within one
    step of the values, whatever the order in which the scale grew."""
    one = oc.AppendCase(hq=4, hkv=2, d=64, q_lens=[40], computed=[0], code=code, seed=9)
    one.key *= (2.0 ** torch.linspace(-6, 2, 40))[:, None, None].to(torch.bfloat16)
    whole = run_append(one)
    kc, vc, ks, vs = (t.to(DEV) for t in (one.kc, one.vc, one.ks, one.vs))
    key, value = one.key.to(DEV).contiguous(), one.value.to(DEV).contiguous()
    for t in range(40):
        binding.pa_append_kv(None, key[t:t + 1], value[t:t + 1], i32([0, 1]), i32([t]), i32(one.table), kc, vc,
                             key_scales=ks, value_scales=vs)
    for b, _, t0, cnt in one.segments():
        for x, cache, s, s1 in ((one.key, kc, ks, whole[3]), (one.value, vc, vs, whole[4])):
            assert torch.equal(s[b], s1[b])
            v = oc.values(cache[b].cpu().numpy(), code)[:cnt] * s[b].double().cpu().numpy()[None, :, None]
            w = x[t0:t0 + cnt].double().numpy()
            # roundings to steps that at least double: below one last step
            step = 2 * oc.half_step(np.abs(w) / s[b].double().cpu().numpy()[None, :, None], code) * s[b].double().cpu().numpy()[None, :, None]
            assert (np.abs(v - w) <= step).all()


@pytest.mark.parametrize("hkv,d", [(2, 64), (8, 128), (3, 128), (17, 64)])
@pytest.mark.parametrize("packed", [True, False])
def test_append_plain_caches_equal_the_writes(hkv, d, packed):
    """Without a rotation the bf16 and E4M3 caches are pa_write_kv's and
    pa_write_kv_fp8's bit for bit; with one, the bf16 cache is pa_rotary +
    pa_write_kv's."""
    c = oc.AppendCase(hq=2 * hkv, hkv=hkv, d=d, q_lens=[1, 37, 0, 2, 16], computed=[40, 3, 7, 15, 32], code="bf16", seed=hkv,
                      packed=packed)
    c.key[0, 0, 0], c.value[1, 0, 3] = float("nan"), float("inf")
    slots = torch.empty(c.T, dtype=torch.int64, device=DEV)
    binding.pa_slot_mapping(i32(c.qsl), i32(c.nc), i32(c.table), c.T, slots)
    key, value = c.key.to(DEV).contiguous(), c.value.to(DEV).contiguous()
    rope = binding.pa_rope_create(rotary_dim=d // 2, layout=hkv % 2)
    rot = torch.empty_like(key)
    binding.pa_rotary(rope, key, i32(c.positions()), rot)
    for r, k in ((None, key), (rope, rot)):
        got = run_append(c, r)
        kc, vc = c.kc.to(DEV), c.vc.to(DEV)
        binding.pa_write_kv(k, value, slots, kc, vc)
        assert np.array_equal(bf16_bits(got[1]), bf16_bits(kc)) and np.array_equal(bf16_bits(got[2]), bf16_bits(vc))
    c.code = "fp8"
    c.kc, c.vc = (torch.randint(0, 255, (c.nb, 16, hkv, d), dtype=torch.uint8) for _ in range(2))
    got = run_append(c)
    kc, vc = c.kc.to(DEV), c.vc.to(DEV)
    binding.pa_write_kv_fp8(key, value, slots, kc, vc, 0.031, 0.007)
    assert torch.equal(got[1], kc) and torch.equal(got[2], vc)


def test_append_fp8_rotated():
    """E4M3 with one scale: the code of the key rotated in 32 bits."""
    c = oc.AppendCase(hq=2, hkv=2, d=128, q_lens=[21, 1], computed=[11, 77], code="fp8", seed=12)
    rope = binding.pa_rope_create(rotary_dim=128)
    got = run_append(c, rope)
    f, m = rope.frequencies()
    k, size = oc.rotate(c.key.double().numpy(), oc.cos_sin(f, c.positions()), 128, False, m)
    codes = oc.values(got[1].cpu().numpy(), "e4m3")
    for b, first, t0, cnt in c.segments():
        g, y = codes[b, first:first + cnt], k[t0:t0 + cnt] / float(np.float32(0.031))
        e = oc.ROTATED * size[t0:t0 + cnt] / 0.031 + 2.0 ** -24 * np.abs(y)
        assert (np.abs(g - y) <= oc.half_step(np.maximum(np.abs(y), np.abs(g)), "e4m3") + e).all()


@pytest.mark.parametrize("code", ["int8", "bf16"])
def test_append_padded_launch(code):
    """A launch sized for a capacity: rows behind the last token are neither read
    (they are NaN) nor written."""
    c = oc.AppendCase(hq=4, hkv=2, d=64, q_lens=[5, 1, 0, 0], computed=[3, 16, 0, 0], code=code, seed=1)
    rope = binding.pa_rope_create(rotary_dim=64)
    a, b = run_append(c, rope), run_append(c, rope, pad=50)
    assert (b[0][c.T:] == 5).all() and torch.equal(a[0], b[0][:c.T])
    for x, y in zip(a[1:], b[1:]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("code", ["int8", "e4m3", "bf16", "fp8"])
def test_append_bad_blocks_are_reported(code):
    """Tokens whose block id is out of range, or whose block lies past the
    table, are not stored; the rest, and every query, is."""
    c = oc.AppendCase(hq=4, hkv=2, d=64, q_lens=[20, 3, 4], computed=[0, 5, 30], code=code, seed=8)
    rope = binding.pa_rope_create(rotary_dim=64)
    good = run_append(c, rope)
    table = c.table.copy()
    table[0, 1], table[1, 0] = c.nb, -1
    table = table[:, :2]                         # request 2: tokens 32, 33 lie in block 2
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = run_append(c, rope, table=np.ascontiguousarray(table), err=err)
    assert binding.pa_check_device_errors(err) == binding.PA_DEVERR_BLOCK_RANGE
    assert torch.equal(got[0], good[0])
    kept = [c.table[0, 0], c.table[2, 1]]
    for n, x in ((1, c.kc), (2, c.vc)) + (((3, c.ks), (4, c.vs)) if c.scaled else ()):
        want = x.to(DEV)
        want[kept] = good[n][kept]
        # (bf16 compared by bits: equal values are enough, no NaN here)
        assert torch.equal(got[n], want), n


def test_append_many_requests():
    """More requests than one step of the search covers, empty ones among them."""
    rng = np.random.default_rng(0)
    q = rng.choice([0, 1, 1, 2, 19], 1500)
    c = oc.AppendCase(hq=1, hkv=1, d=64, q_lens=q, computed=rng.integers(0, 50, 1500), code="int8", seed=3)
    check_scaled(c, run_append(c), None)


def test_append_captured_and_replayed():
    """A captured append follows the metadata in its buffers, on a side stream."""
    c = oc.AppendCase(hq=4, hkv=2, d=64, q_lens=[4, 1], computed=[14, 3], code="int8", seed=5)
    rope = binding.pa_rope_create(rotary_dim=32)
    q, k, v = (t.to(DEV).contiguous() for t in (c.q, c.key, c.value))
    q_out = torch.zeros_like(q)
    kc, vc, ks, vs = (t.to(DEV) for t in (c.kc, c.vc, c.ks, c.vs))
    qsl, nc, table = i32(c.qsl), i32(c.nc), i32(c.table)
    call = lambda: binding.pa_append_kv(rope, k, v, qsl, nc, table, kc, vc, key_scales=ks, value_scales=vs, q=q, q_out=q_out)  # noqa: E731
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()                                   # also on another stream than the tensors' own
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for t, src in ((kc, c.kc), (vc, c.vc), (ks, c.ks), (vs, c.vs)):
        t.copy_(src)
    nc.copy_(i32([c.nc[0] - 2, c.nc[1] + 1]))    # other positions: the replay reads them
    g.replay()
    torch.cuda.synchronize()
    c.nc = np.array([c.nc[0] - 2, c.nc[1] + 1])
    check_scaled(c, (q_out, kc, vc, ks, vs), rope)
    check_rotated(q_out, c.q, c.positions(), rope, 0)
