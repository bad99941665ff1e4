"""Attention over block-scaled 8-bit caches on the GPU against the plain
implementation in 64 bits, and the step of append + attention (needs a GB300)."""
import numpy as np
import pytest
import torch

import operators_common as oc
from gpu_common import ensure_library
from paged_kv_cache_16_gb300 import binding, workloads
from paged_kv_cache_16_gb300.step import DeviceStep, GraphStep

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_library()


def check(c, **over):
    g = oc.OnGpu(c, **over)
    out = g.run()
    ref, tol = c.reference()
    oc.assert_within(out[:c.T], ref[:c.T], tol[:c.T])
    return g


HEADS = [(4, 2, 64), (8, 8, 128), (16, 2, 64), (28, 4, 128), (24, 8, 128), (3, 3, 64), (16, 1, 128), (48, 16, 64)]


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("scales", ["power", "any", "wild"])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_decode_rows(code, scales, hq, hkv, d):
    """One token each: contexts of one key, ends of blocks, odd lengths."""
    check(oc.Case(hq=hq, hkv=hkv, d=d, q_lens=[1] * 9, seq_lens=[1, 2, 15, 16, 17, 33, 64, 177, 500], code=code,
                  scales=scales, seed=hq + d))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_verify_rows(code, hq, hkv, d):
    """2 to 8 tokens, of whole contexts and of long ones, idle requests between."""
    check(oc.Case(hq=hq, hkv=hkv, d=d, q_lens=[2, 0, 3, 5, 8, 4, 1, 8], seq_lens=[2, 5, 40, 5, 300, 31, 90, 129], code=code,
                  seed=hq))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("scales", ["power", "any", "wild"])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (8, 2, 128), (32, 1, 128), (40, 2, 64), (28, 4, 128)])
def test_tile_rows(code, scales, hq, hkv, d):
    """Chunks on the tensor-core tiles (odd lengths, cached contexts that end
    inside a block) beside decode rows."""
    check(oc.Case(hq=hq, hkv=hkv, d=d, q_lens=[37, 1, 129, 1], seq_lens=[37, 300, 300, 1], code=code, scales=scales, seed=d))


@pytest.mark.parametrize("num_sms", [4, 5, 11])
def test_tiles_evened_out(num_sms):
    """26 tiles of 5 to 11 steps whose greedy assignment is 4% to 15% off the
    mean, so that the planner packs them anew: every row is written once."""
    check(oc.Case(hq=8, hkv=2, d=64, q_lens=[300, 500], seq_lens=[1200, 900], code="int8", seed=5), num_sms=num_sms)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_cascade(code):
    check(oc.Case(hq=8, hkv=2, d=128, q_lens=[1, 1, 3, 20], seq_lens=[600, 530, 700, 560], code=code, seed=1, shared=32))


@pytest.mark.parametrize("num_sms", [1, 3, 20, 152, 400])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_partition_count(num_sms, code):
    """Cuts at every granularity; partials of scales 2^80 apart are joined."""
    check(oc.Case(hq=8, hkv=2, d=128, q_lens=[1, 1, 4, 1], seq_lens=[900, 1, 333, 129], code=code, scales="wild", seed=3),
          num_sms=num_sms)


@pytest.mark.parametrize("q_size", [1e-20, 1e-6, 1e6, 1e20])
def test_query_magnitudes(q_size):
    """Queries far outside f16's range (the softmax scale undoes them)."""
    check(oc.Case(hq=8, hkv=2, d=128, q_lens=[1, 3], seq_lens=[100, 50], code="int8", q_size=q_size))


def test_peaked_and_flat_rows():
    """One key far above the rest (in a late block, so that the reference
    moves), and a row of zeros whose weights are equal."""
    c = oc.Case(hq=4, hkv=2, d=64, q_lens=[1, 1], seq_lens=[400, 350], code="int8", seed=2)
    c.q[1] = 0
    b = c.table[0, 20]
    c.kc[b, 5] = (torch.sign(c.q[0].view(2, 2, 64).float().sum(1)) * 127).to(torch.int8)
    c.ks[b] = 0.25
    check(c)


def test_one_key_is_its_value():
    """A context of one key returns the value: a code times its scale, exact
    in bf16 for powers of two."""
    for code in ("int8", "e4m3"):
        c = oc.Case(hq=4, hkv=2, d=64, q_lens=[1], seq_lens=[1], code=code)
        out = oc.OnGpu(c).run()
        v = oc.values(c.vc[c.table[0, 0], 0].numpy(), code) * c.vs[c.table[0, 0]].double().numpy()[:, None]
        assert np.array_equal(out[0].double().cpu().numpy(), np.repeat(v, 2, axis=0))


@pytest.mark.parametrize("left", range(8))
@pytest.mark.parametrize("call", ["pa_attention_scaled", "pa_attention_scaled_launch"])
def test_one_tensor_left_on_the_host_is_refused(left, call):
    """(q, caches, scales, block table, out, workspace)"""
    g = oc.OnGpu(oc.Case(hq=4, hkv=2, d=64, q_lens=[1], seq_lens=[20], code="int8"))
    args = list(g.args())
    args[left] = args[left].cpu()
    with pytest.raises(ValueError, match="current CUDA device"):
        getattr(binding, call)(g.plan, *args)


def test_matches_the_tensor_scale_kernel():
    """Equal scales everywhere: the E4M3 kernels with one scale per tensor on the
    same codes agree within both bounds (theirs: bf16 weights on the tiles,
    2^-8 of sum p |v|, at most the largest value)."""
    c = oc.Case(hq=8, hkv=2, d=128, q_lens=[1, 4, 1, 60], seq_lens=[700, 90, 33, 200], code="e4m3", seed=7)
    used = torch.isfinite(c.ks)
    c.ks[used], c.vs[used] = 0.03125, 0.0625
    g = check(c)
    plan = binding.pa_plan(**c.desc(kv_cache_dtype=binding.PA_KV_FP8_E4M3, k_scale=0.03125, v_scale=0.0625))
    out = torch.zeros_like(g.out)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
    binding.pa_attention(plan, g.q, g.kc, g.vc, g.table, out, ws)
    ref, tol = c.reference()
    oc.assert_within(out, ref, 2 * tol + oc.BF16 * 448 * 0.0625)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_nan_scales_reach_the_output(code):
    """A NaN scale of a block that is read makes the rows of its head NaN (also
    where the row is split over CTAs), and no others."""
    c = oc.Case(hq=8, hkv=2, d=128, q_lens=[1, 1, 30], seq_lens=[900, 400, 100], code=code, seed=3)
    c.ks[c.table[0, 40], 1] = float("nan")
    c.vs[c.table[2, 1], 0] = float("nan")
    g = oc.OnGpu(c)
    out = g.run().float().cpu()
    bad = torch.isnan(out).any(-1)
    want = torch.zeros_like(bad)
    want[0, 4:8] = True
    want[2:, 0:4] = True                 # positions 70 .. 99 all see block 1
    assert torch.equal(bad, want)


@pytest.mark.parametrize("q_len", [4, 40])
@pytest.mark.parametrize("which", ["ks", "vs"])
def test_nan_scales_of_later_blocks(q_len, which):
    """Tokens of a verify row or a chunk that stand before a block with a NaN scale
    do not see it; the others' rows of its head are NaN."""
    c = oc.Case(hq=8, hkv=2, d=128, q_lens=[q_len], seq_lens=[82], code="int8", seed=5)
    clean, tol = c.reference()
    getattr(c, which)[c.table[0, 5], 1] = float("nan")          # block 5: positions 80, 81
    out = oc.OnGpu(c).run()
    seen = np.arange(82 - q_len, 82) >= 80
    bad = torch.isnan(out.float().cpu()).any(-1).numpy()
    assert np.array_equal(bad[:, 4:], np.repeat(seen[:, None], 4, 1)) and not bad[:, :4].any()
    oc.assert_within(out[:q_len - 2], clean[:q_len - 2], tol[:q_len - 2])


def test_tiny_and_zero_scales():
    """Scales at and below the floor count as 2^-100, zero ones too."""
    c = oc.Case(hq=4, hkv=2, d=64, q_lens=[1, 1], seq_lens=[100, 40], code="int8", seed=4)
    b = c.table[0, 2]
    c.vs[b], c.ks[c.table[1, 0]] = 0.0, 0.0
    out = oc.OnGpu(c).run()
    c.vs[b], c.ks[c.table[1, 0]] = 2.0 ** -100, 2.0 ** -100
    ref, tol = c.reference()
    oc.assert_within(out, ref, tol)


def test_bad_block_is_reported():
    c = oc.Case(hq=4, hkv=2, d=64, q_lens=[1, 1, 40], seq_lens=[100, 40, 40], code="int8", seed=4)
    g = oc.OnGpu(c)
    g.table[0, 3] = c.nb + 5
    g.table[2, 1] = -7
    binding.pa_attention_scaled(g.plan, *g.args())
    torch.cuda.synchronize()
    assert binding.pa_check_device_errors(g.ws[:4].view(torch.int32)) == binding.PA_DEVERR_BLOCK_RANGE
    ref, tol = c.reference()
    oc.assert_within(g.out[1:2], ref[1:2], tol[1:2])


def test_block_ids_do_not_matter_and_runs_repeat():
    c = oc.Case(hq=8, hkv=2, d=128, q_lens=[1, 4, 50], seq_lens=[700, 90, 333], code="int8", scales="any", seed=11)
    a = oc.OnGpu(c)
    x = a.run().clone()
    assert torch.equal(x, a.run())
    perm = torch.randperm(c.nb, generator=torch.Generator().manual_seed(1))
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(c.nb)
    for n in ("kc", "vc", "ks", "vs"):
        setattr(c, n, getattr(c, n)[perm].contiguous())
    c.table = np.where(c.table >= 0, inv.numpy()[c.table.clip(min=0)], -1).astype(np.int32)
    assert torch.equal(x, oc.OnGpu(c).run())


def test_fixed_shape_graph_replays():
    """One captured launch of a fixed shape replays steps of other lengths,
    with tiles beside the decode stream, bit-equal to the eager calls."""
    shape = dict(max_tokens=96, max_reqs=6, max_extend_tiles=16, max_dequant_blocks=64)
    kw = dict(hq=8, hkv=2, d=64, code="e4m3")
    steps = [oc.Case(q_lens=[1, 1, 40, 1], seq_lens=[300, 77, 90, 5], seed=1, **kw),
             oc.Case(q_lens=[3, 1, 1, 50, 1], seq_lens=[40, 100, 200, 50, 16], seed=2, **kw),
             oc.Case(q_lens=[1], seq_lens=[444], seed=3, **kw)]
    nb, mb = max(c.nb for c in steps), max(c.table.shape[1] for c in steps)
    q = torch.zeros(96, 8, 64, dtype=torch.bfloat16, device=DEV)
    out = torch.zeros_like(q)
    kc, vc = (torch.zeros(nb, 16, 2, 64, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros(nb, 2, device=DEV) for _ in range(2))
    table = torch.zeros(6, mb, dtype=torch.int32, device=DEV)
    over = dict(num_blocks=nb, max_blocks_per_req=mb)
    plans = [binding.pa_plan_fixed(**shape, **c.desc(**over)) for c in steps]
    ws = torch.zeros(plans[0].workspace_bytes, dtype=torch.uint8, device=DEV)
    binding.pa_upload_metadata(plans[0], ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.pa_attention_scaled_launch(plans[0], q, kc, vc, ks, vs, table, out, ws)
    for c, plan in zip(steps, plans):
        q[:c.T] = c.q.to(DEV)
        for dst, src in ((kc, c.kc), (vc, c.vc), (ks, c.ks), (vs, c.vs)):
            dst[:c.nb] = src.to(DEV)
        table[:c.table.shape[0], :c.table.shape[1]] = torch.from_numpy(c.table).to(DEV)
        out.fill_(3.0)
        binding.pa_upload_metadata(plan, ws)
        g.replay()
        torch.cuda.synchronize()
        assert binding.pa_check_device_errors(ws[:4].view(torch.int32)) == 0
        assert (out[c.T:] == 3).all()            # rows behind the last sequence
        ref, tol = c.reference()
        oc.assert_within(out[:c.T], ref[:c.T], tol[:c.T])
        eager = torch.zeros_like(out)
        p = binding.pa_plan(**c.desc(**over))
        w2 = torch.zeros(p.workspace_bytes, dtype=torch.uint8, device=DEV)
        binding.pa_attention_scaled(p, q, kc, vc, ks, vs, table, eager, w2)
        assert torch.equal(eager[:c.T], out[:c.T])


def test_two_streams_at_once():
    """Two plans with workspaces of their own on two streams."""
    cs = [oc.Case(hq=8, hkv=2, d=128, q_lens=[1] * 6 + [70], seq_lens=[100 * k + 7 for k in range(1, 7)] + [150],
                  code=code, seed=k) for k, code in enumerate(("int8", "e4m3"))]
    gs = [oc.OnGpu(c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in gs]
    for _ in range(5):
        for g, s in zip(gs, streams):
            binding.pa_attention_scaled(g.plan, *g.args(), stream=s)
    torch.cuda.synchronize()
    for c, g in zip(cs, gs):
        ref, tol = c.reference()
        oc.assert_within(g.out, ref, tol)


def test_long_cache_offsets_past_32_bits():
    """A pool whose bytes pass 2^32: blocks at its end, for the append and both
    kernels."""
    hkv, d = 8, 128
    nb = (1 << 32) // (16 * hkv * d) + 300
    kc, vc = (torch.empty(nb, 16, hkv, d, dtype=torch.int8, device=DEV) for _ in range(2))
    c = oc.Case(hq=8, hkv=hkv, d=d, q_lens=[1, 20], seq_lens=[200, 40], code="int8", seed=6)
    shift = nb - c.nb
    kc[shift:], vc[shift:] = c.kc.to(DEV), c.vc.to(DEV)
    ks, vs = (torch.full((nb, hkv), float("nan"), device=DEV) for _ in range(2))
    ks[shift:], vs[shift:] = c.ks.to(DEV), c.vs.to(DEV)
    table = torch.from_numpy(np.where(c.table >= 0, c.table + shift, -1).astype(np.int32)).to(DEV)
    plan = binding.pa_plan(**c.desc(num_blocks=nb))
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
    out = torch.zeros(c.T, 8, d, dtype=torch.bfloat16, device=DEV)
    binding.pa_attention_scaled(plan, c.q.to(DEV), kc, vc, ks, vs, table, out, ws)
    ref, tol = c.reference()
    oc.assert_within(out, ref, tol)
    a = oc.AppendCase(hq=8, hkv=hkv, d=d, q_lens=[20], computed=[7], code="int8", seed=7)
    sub = [t.to(DEV) for t in (a.kc, a.vc, a.ks, a.vs)]
    big = (kc, vc, ks, vs)
    shift = nb - a.nb
    for x, y in zip(big, sub):
        x[shift:] = y
    i32 = lambda x: torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32, device=DEV)  # noqa: E731
    for caches, t in ((sub, a.table), (big, np.where(a.table >= 0, a.table + shift, -1))):
        binding.pa_append_kv(None, a.key.to(DEV).contiguous(), a.value.to(DEV).contiguous(), i32(a.qsl), i32(a.nc), i32(t),
                             caches[0], caches[1], key_scales=caches[2], value_scales=caches[3])
    torch.cuda.synchronize()
    for x, y in zip(big, sub):
        assert torch.equal(x[shift:], y)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_steps_of_append_and_attention(code):
    """A prefill and decode steps through the operators as an engine runs them:
    the append with the rotation, then attention, against 64-bit attention over
    the cache as it then stands."""
    hq, hkv, d, R = 8, 2, 128, 3
    g = torch.Generator().manual_seed(4)
    prompt, steps = [21, 40, 16], 6
    rope = binding.pa_rope_create(rotary_dim=64, base=10000.0)
    nb, mb = 40, 8
    table = np.random.default_rng(2).permutation(nb)[:R * mb].reshape(R, mb).astype(np.int32)
    dt = torch.int8 if code == "int8" else torch.uint8
    kc, vc = (torch.zeros(nb, 16, hkv, d, dtype=dt, device=DEV) for _ in range(2))
    ks, vs = (torch.full((nb, hkv), float("nan"), device=DEV) for _ in range(2))
    seen = np.zeros(R, np.int64)
    i32 = lambda a: torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32, device=DEV)  # noqa: E731
    for step in range(steps + 1):
        q_lens = np.array(prompt if step == 0 else [1, 3, 1] if step == 2 else [1, 1, 1])
        T = int(q_lens.sum())
        qsl = np.concatenate([[0], np.cumsum(q_lens)])
        rows = torch.randn(T, hq + 2 * hkv, d, generator=g).to(torch.bfloat16).to(DEV)
        q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
        q_rot = torch.empty(T, hq, d, dtype=torch.bfloat16, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        binding.pa_append_kv(rope, k, v, i32(qsl), i32(seen), i32(table), kc, vc, key_scales=ks, value_scales=vs, q=q,
                             q_out=q_rot, device_error_word=err)
        seen = seen + q_lens
        c = oc.Case(hq=hq, hkv=hkv, d=d, q_lens=q_lens, seq_lens=seen, code=code)
        c.table, c.nb = table, nb
        plan = binding.pa_plan(**c.desc())
        ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
        out = torch.empty_like(q_rot)
        binding.pa_attention_scaled(plan, q_rot, kc, vc, ks, vs, i32(table), out, ws)
        torch.cuda.synchronize()
        assert binding.pa_check_device_errors(err) == 0
        c.q, c.kc, c.vc, c.ks, c.vs = (t.cpu() for t in (q_rot, kc, vc, ks, vs))
        ref, tol = c.reference()
        oc.assert_within(out, ref, tol, f"step {step}")


def batch_case(b, q, kc, vc, ks, vs):
    """An oc.Case over a workloads batch and the device state after its append."""
    c = oc.Case.__new__(oc.Case)
    c.hq, c.hkv, c.d, c.code, c.n_common = b.num_heads_q, b.num_heads_kv, b.head_dim, \
        "int8" if b.kv_cache_dtype == "int8_block" else "e4m3", b.num_common_prefix_blocks
    c.q_lens, c.seq, c.table, c.nb, c.T = b.q_lens, b.seq_lens, b.block_table, b.num_blocks, b.num_tokens
    c.qsl, c.scale = b.query_start_loc, b.softmax_scale
    c.q, c.kc, c.vc, c.ks, c.vs = (t.cpu() for t in (q, kc, vc, ks, vs))
    return c


@pytest.mark.parametrize("kind", ["int8_block", "fp8_block"])
@pytest.mark.parametrize("d", [64, 128])
def test_device_step_run_append(kind, d):
    """DeviceStep.run_append with a rope over block-scaled caches: a mixed step
    against 64-bit attention over the cache it leaves; without a rope the queries
    are the caller's."""
    b = workloads.make_batch(name="scaled", num_heads_q=8, num_heads_kv=2, head_dim=d, q_lens=[1, 1, 40, 3, 1],
                             seq_lens=[90, 33, 100, 20, 1], num_blocks=40, seed=d, kv_cache_dtype=kind)
    for rope in (binding.pa_rope_create(rotary_dim=d), None):
        q, k, v, kc, vc, ks, vs = (t.to(DEV) for t in (b.q, b.key, b.value, b.key_cache, b.value_cache, b.key_scales,
                                                       b.value_scales))
        st = DeviceStep(b, "cuda", rope=rope)
        out = st.run_append(q, k, v, kc, vc, ks, vs)
        torch.cuda.synchronize()
        assert st.check_errors() == 0
        used = q if rope is None else st.q_rot
        if rope is not None:
            pos = np.concatenate([np.arange(n, n + m) for n, m in zip(b.num_computed, b.q_lens)])
            want = torch.empty_like(q)
            binding.pa_rotary(rope, q, torch.as_tensor(pos, dtype=torch.int32, device=DEV), want)
            assert torch.equal(st.q_rot, want)
        ref, tol = batch_case(b, used, kc, vc, ks, vs).reference()
        oc.assert_within(out, ref, tol)


@pytest.mark.parametrize("kind", ["int8_block", "bf16", "fp8"])
def test_graph_step_with_rope(kind):
    """GraphStep with a rope replays steps of changing size, bit-equal to
    DeviceStep.run_append: caches, scales and outputs."""
    rope = binding.pa_rope_create(rotary_dim=64, layout=binding.PA_ROPE_INTERLEAVED)
    mk = lambda ql, sl, seed: workloads.make_batch(name="g", num_heads_q=8, num_heads_kv=2, head_dim=128, q_lens=ql,  # noqa: E731
                                                   seq_lens=sl, num_blocks=60, seed=seed, kv_cache_dtype=kind)
    steps = [mk([1, 1, 30], [200, 17, 60], 1), mk([1, 2, 1, 1], [90, 40, 300, 16], 2), mk([50], [50], 3)]
    first = steps[0]
    pool = [t.to(DEV) for t in (first.key_cache, first.value_cache)]
    scales = [t.to(DEV) for t in (first.key_scales, first.value_scales)] if kind == "int8_block" else [None, None]
    gs = GraphStep(num_heads_q=8, num_heads_kv=2, head_dim=128, num_blocks=60, max_blocks_per_req=24,
                   softmax_scale=first.softmax_scale, max_tokens=64, max_reqs=6, max_extend_tiles=16,
                   max_dequant_blocks=0 if kind == "bf16" else 64, kv_cache_dtype=kind, k_scale=first.k_scale,
                   v_scale=first.v_scale, rope=rope)
    for b in steps:
        for t, src in zip(pool + scales, (b.key_cache, b.value_cache, b.key_scales, b.value_scales)):
            if t is not None:
                t.copy_(src)
        eager = [t.clone() if t is not None else None for t in pool + scales]
        q, k, v = (t.to(DEV) for t in (b.q, b.key, b.value))
        got = gs.run(b, q, k, v, *pool, *scales)
        st = DeviceStep(b, "cuda", rope=rope)
        want = st.run_append(q, k, v, *eager)
        torch.cuda.synchronize()
        assert gs.check_errors() == 0 and st.check_errors() == 0
        assert torch.equal(got, want)
        for x, y in zip(pool + scales, eager):
            if x is not None:
                assert x.float().nan_to_num(7e4).equal(y.float().nan_to_num(7e4))
