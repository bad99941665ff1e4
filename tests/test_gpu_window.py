"""Attention with a sliding window and first tokens that stay visible, on the GPU
against the plain implementation in 64 bits (needs a GB300)."""
import numpy as np
import pytest
import torch

import operators_common as oc
import window_common as wc
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


def heads(code, small):
    """Head layouts of a cache type (E4M3 with one scale: head_dim 128)."""
    return [(hq, hkv, d if code != "e4m3" else 128) for hq, hkv, d in small]


WINDOWS = [(1, 0), (16, 0), (17, 3), (5, 16), (100, 4), (64, 40), (33, 200), (1000, 0)]


@pytest.mark.parametrize("code", wc.KINDS)
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("layout", [(4, 2, 64), (28, 4, 128), (16, 1, 128), (3, 3, 64)])
def test_decode_rows(code, window, sinks, layout):
    """One token each: contexts of one key, of the window's length, ends of blocks."""
    hq, hkv, d = heads(code, [layout])[0]
    wc.check(wc.WindowCase(hq=hq, hkv=hkv, d=d, q_lens=[1] * 14, code=code, window=window, sinks=sinks, seed=hq + window,
                           seq_lens=[1, 2, 15, 16, 17, 18, 33, 48, 64, 65, 113, 177, 500, 1311]))


@pytest.mark.parametrize("code", wc.KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 5), (17, 0), (64, 33), (300, 4)])
@pytest.mark.parametrize("layout", [(4, 2, 64), (32, 8, 128), (8, 8, 64), (14, 1, 128)])
def test_verify_rows(code, window, sinks, layout):
    """2 to 8 tokens, each with a window of its own, idle requests between."""
    hq, hkv, d = heads(code, [layout])[0]
    wc.check(wc.WindowCase(hq=hq, hkv=hkv, d=d, q_lens=[2, 0, 3, 5, 8, 4, 1, 8], code=code, window=window, sinks=sinks,
                           seq_lens=[2, 5, 40, 5, 300, 31, 90, 513], seed=hq))


@pytest.mark.parametrize("code", wc.KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 1), (50, 0), (128, 130), (200, 17), (300, 600), (700, 4)])
@pytest.mark.parametrize("layout", [(4, 2, 64), (8, 8, 128), (32, 1, 128), (20, 4, 64)])
def test_tile_rows(code, window, sinks, layout):
    """Chunks on the tensor-core tiles, longer and shorter than the window, cached
    contexts that end inside a block, beside decode rows."""
    hq, hkv, d = heads(code, [layout])[0]
    wc.check(wc.WindowCase(hq=hq, hkv=hkv, d=d, q_lens=[37, 1, 129, 1, 300], seq_lens=[37, 300, 433, 1, 1000], code=code,
                           window=window, sinks=sinks, seed=d + window))


@pytest.mark.parametrize("code", wc.KINDS)
@pytest.mark.parametrize("q_lens,seq,window,sinks", [([9], [1500], 1400, 0), ([40], [2300], 2000, 20), ([300], [1900], 1024, 700),
                                                     ([20, 1, 130], [1200, 700, 1700], 1100, 140), ([256], [900], 2000, 0)])
@pytest.mark.parametrize("layout", [(8, 2, 128), (2, 2, 64), (32, 1, 128), (6, 2, 64)])
def test_tiles_cut_along_their_keys(code, q_lens, seq, window, sinks, layout):
    """Few tiles over long windows: pieces on idle SMs, some without a key for some
    rows, joined by the merge; and whole in a shape without room for the pieces."""
    hq, hkv, d = heads(code, [layout])[0]
    c = wc.WindowCase(hq=hq, hkv=hkv, d=d, q_lens=q_lens, seq_lens=seq, code=code, window=window, sinks=sinks, seed=hq)
    g = wc.check(c)
    G = hq // hkv
    whole = hkv * sum(-(-q // (2 * (128 // G))) for q in q_lens if q > (0 if G > 16 else max(8, 16 // G)))
    assert g.plan.info()["num_extend_tiles"] > whole or whole == 0 or q_lens == [256]
    blocks = 400 if code != "bf16" else 0
    for tiles in (300, whole):                  # room for the pieces, or for whole tiles only
        shape = dict(max_tokens=500, max_reqs=4, max_extend_tiles=tiles, max_dequant_blocks=blocks,
                     max_partial_slots=20000)
        f = wc.check(c, shape=shape)
        assert tiles != 300 or torch.equal(f.out[:c.T], g.out)


@pytest.mark.parametrize("code", wc.KINDS)
def test_nan_in_a_piece_reaches_its_rows(code):
    """A NaN key (int8: a NaN scale) in one piece makes the rows that see it NaN, and no
    other row's key: split-KV items and pieces of tiles alike."""
    for q_len, hq in ((1, 8), (40, 8), (1, 64)):
        c = wc.WindowCase(hq=hq, hkv=2, d=128, q_lens=[q_len, q_len], seq_lens=[3000, 2900], code=code, window=2500, sinks=0, seed=3)
        b = c.table[0, 2000 // 16]
        if c.scaled:
            c.ks[b] = float("nan")
        else:
            c.kc[b, 0] = float("nan") if code == "bf16" else 0x7F
        g = wc.OnGpu(c)
        out = g.run()
        assert torch.isnan(out[:q_len]).all()
        ref, tol = c.reference()
        oc.assert_within(out[q_len:2 * q_len], ref[q_len:], tol[q_len:])


@pytest.mark.parametrize("seed", range(40))
def test_drawn_steps(seed):
    """Steps of every kind of row, windows and first tokens of any size."""
    rng = np.random.default_rng(seed)
    code = wc.KINDS[seed % 4]
    hq, hkv, d = [(4, 2, 64), (12, 3, 64), (16, 2, 128), (6, 6, 128), (32, 2, 64), (40, 1, 128)][rng.integers(6)]
    q = rng.choice([0, 1, 1, 2, 7, 9, 40, 161], rng.integers(1, 7))
    past = (2.0 ** rng.uniform(0, 10, len(q))).astype(int) - 1
    wc.check(wc.WindowCase(hq=hq, hkv=hkv, d=128 if code == "e4m3" else d, q_lens=q, seq_lens=q + past, code=code,
                           window=int(2 ** rng.uniform(0, 9)), sinks=int(rng.choice([0, 1, 4, 16, 129, 400])), seed=seed,
                           pad=int(rng.choice([-1, 2**31 - 1]))),
             num_sms=int(rng.choice([0, 1, 3, 20])))


@pytest.mark.parametrize("code", wc.KINDS)
@pytest.mark.parametrize("window,sinks", [(2**31 - 1, 0), (2**31 - 1, 2**31 - 1), (1, 2**31 - 1), (5000, 3)])
def test_a_window_without_effect(code, window, sinks):
    """The plain rows' results; one and few tokens bit for bit where cut alike."""
    c = wc.WindowCase(hq=8, hkv=2, d=128, q_lens=[1, 4, 90, 1], seq_lens=[300, 70, 333, 17], code=code, window=window,
                      sinks=sinks, seed=1)
    g = wc.check(c)
    plain = wc.OnGpu(c)
    kw = c.desc()
    del kw["window"], kw["sink_tokens"]
    plain.plan = binding.pa_plan(**kw)
    ref, tol = c.reference()
    oc.assert_within(plain.run(), ref, tol)
    if plain.plan.info() == g.plan.info():      # the rows of the split-KV kernel
        rows = [*range(5), c.T - 1]
        assert torch.equal(plain.out[rows], g.out[rows])


@pytest.mark.parametrize("code", wc.KINDS)
def test_other_requests_and_later_rows_stay(code):
    """Rows of the output behind the last token are left as they were; a step
    without tokens writes nothing."""
    c = wc.WindowCase(hq=4, hkv=2, d=128, q_lens=[0, 3, 0, 20], seq_lens=[50, 90, 0, 220], code=code, window=30, sinks=2)
    g = wc.OnGpu(c)
    g.out = torch.full((c.T + 9, 4, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    g.run()
    ref, tol = c.reference()
    oc.assert_within(g.out[:c.T], ref, tol)
    assert (g.out[c.T:] == 7).all()
    none = wc.WindowCase(hq=4, hkv=2, d=128, q_lens=[0, 0], seq_lens=[50, 0], code=code, window=30, sinks=2)
    assert (wc.OnGpu(none).run() == 7).all()


@pytest.mark.parametrize("code", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_lens,seq", [([1] * 5, [1, 16, 17, 200, 555]), ([1, 5, 70, 1], [300, 44, 290, 33])])
def test_fused_update_equals_write_then_attend(code, q_lens, seq):
    """Caches, slots and output of the fused call against the separate ones."""
    c = wc.WindowCase(hq=8, hkv=2, d=128, q_lens=q_lens, seq_lens=seq, code=code, window=40, sinks=5, seed=4, hidden=False)
    g = torch.Generator().manual_seed(9)
    key, value = (torch.randn(c.T, 2, 128, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    a, b = wc.OnGpu(c), wc.OnGpu(c)
    i32 = lambda x: torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32, device=DEV)  # noqa: E731
    slots, fused = (torch.full((c.T,), -5, dtype=torch.int64, device=DEV) for _ in range(2))
    binding.pa_slot_mapping(i32(c.qsl), i32(c.seq - c.q_lens), a.table, c.T, slots)
    if code == "bf16":
        binding.pa_write_kv(key, value, slots, a.kc, a.vc)
    else:
        binding.pa_write_kv_fp8(key, value, slots, a.kc, a.vc, wc.K_SCALE, wc.V_SCALE)
    a.run()
    binding.pa_attention_with_kv_update(b.plan, b.q, key, value, b.kc, b.vc, b.table, b.out, b.ws, fused)
    torch.cuda.synchronize()
    for x, y in ((a.out, b.out), (a.kc, b.kc), (a.vc, b.vc), (slots, fused)):
        assert torch.equal(x, y)
    c.kc, c.vc = a.kc.cpu(), a.vc.cpu()
    ref, tol = c.reference()
    oc.assert_within(a.out, ref, tol)


def test_call_without_workspace():
    c = wc.WindowCase(hq=8, hkv=2, d=128, q_lens=[1, 5, 20], seq_lens=[300, 44, 90], code="bf16", window=40, sinks=5)
    g = wc.check(c)
    out = torch.zeros_like(g.out)
    binding.pa_attention_no_alloc(g.plan, g.q, g.kc, g.vc, g.table, out)
    assert torch.equal(out, g.out)


@pytest.mark.parametrize("code", wc.KINDS)
def test_fixed_shape_graph_replays_other_steps(code):
    """One capture, replayed for steps of other sizes, equals plain plans bit for bit."""
    shape = dict(max_tokens=300, max_reqs=6, max_extend_tiles=16, max_dequant_blocks=120 if code != "bf16" else 0)
    kw = dict(hq=8, hkv=2, d=128, code=code, window=70, sinks=20, spare=0)
    steps = [wc.WindowCase(q_lens=q, seq_lens=s, seed=i, **kw) for i, (q, s) in enumerate(
        [([1, 60, 3], [400, 300, 90]), ([1] * 6, [9, 80, 81, 300, 400, 64]), ([200, 1], [330, 100]), ([1], [1])])]
    nb, mb = max(c.nb for c in steps), max(c.table.shape[1] for c in steps)
    over = dict(num_blocks=nb, max_blocks_per_req=mb)

    def padded(c):
        t = np.full((6, mb), -1, dtype=np.int32)
        t[:c.table.shape[0], :c.table.shape[1]] = c.table
        return t
    pool = [torch.zeros((nb, 16) + tuple(steps[0].kc.shape[2:]), dtype=steps[0].kc.dtype, device=DEV) for _ in range(2)]
    scales = [torch.ones(nb, 2, device=DEV) for _ in range(2)]
    q = torch.zeros(300, 8, 128, dtype=torch.bfloat16, device=DEV)
    out, table = torch.zeros_like(q), torch.zeros(6, mb, dtype=torch.int32, device=DEV)
    plans = [binding.pa_plan_window(shape=shape, **c.desc(block_table_host=np.ascontiguousarray(padded(c)[:len(c.q_lens)]), **over))
             for c in steps]
    ws = torch.zeros(plans[0].workspace_bytes, dtype=torch.uint8, device=DEV)

    def launch(p):
        if steps[0].scaled:
            binding.pa_attention_scaled_launch(p, q, *pool, *scales, table, out, ws)
        else:
            binding.pa_attention_launch(p, q, *pool, table, out, ws)
    binding.pa_upload_metadata(plans[0], ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        launch(plans[0])
    for c, p in zip(steps, plans):
        for dst, src in zip(pool + scales, (c.kc, c.vc, c.ks, c.vs)):
            dst[:c.nb].copy_(src)
        q[:c.T].copy_(c.q[:c.T])
        table.copy_(torch.from_numpy(padded(c)))
        out.fill_(7.0)
        binding.pa_upload_metadata(p, ws)
        graph.replay()
        torch.cuda.synchronize()
        assert binding.pa_check_device_errors(ws[:4].view(torch.int32)) == 0
        ref, tol = c.reference()
        oc.assert_within(out[:c.T], ref[:c.T], tol[:c.T])
        assert (out[c.T:] == 7).all()
        g = wc.OnGpu(c)
        assert torch.equal(g.run()[:c.T], out[:c.T])


@pytest.mark.parametrize("code", ["bf16", "int8_block"])
def test_two_streams_at_once(code):
    """Two plans with workspaces of their own, on streams of their own."""
    cs = [wc.WindowCase(hq=8, hkv=2, d=64, q_lens=[1] * 20 + [90], seq_lens=[200 + 37 * i for i in range(21)], code=code,
                        window=w, sinks=s, seed=w) for w, s in ((64, 4), (300, 0))]
    gs = [wc.OnGpu(c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in gs]
    for _ in range(5):
        for g, st in zip(gs, streams):
            with torch.cuda.stream(st):
                g.call()
    torch.cuda.synchronize()
    for c, g in zip(cs, gs):
        ref, tol = c.reference()
        oc.assert_within(g.out, ref, tol)


@pytest.mark.parametrize("q_lens,seq", [([1, 1], [500, 70]), ([20, 1, 100], [900, 33, 260])])
def test_staged_inputs(q_lens, seq):
    """Rows from the decode prefix on behind an event: the unstaged results."""
    order = np.argsort([q > 1 for q in q_lens], kind="stable")      # decode rows first
    q_lens, seq = [q_lens[i] for i in order], [seq[i] for i in order]
    c = wc.WindowCase(hq=8, hkv=2, d=128, q_lens=q_lens, seq_lens=seq, code="bf16", window=90, sinks=5, seed=4, hidden=False)
    P = sum(q for q in q_lens if q == 1)
    shape = dict(max_tokens=200, max_reqs=4, max_extend_tiles=8, decode_prefix_tokens=P)
    g = torch.Generator().manual_seed(9)
    key, value = (torch.randn(200, 2, 128, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    a, b = wc.OnGpu(c, shape=shape, num_sms=40), wc.OnGpu(c, shape=shape, num_sms=40)
    for x in (a, b):
        binding.pa_upload_metadata(x.plan, x.ws)
    binding.pa_attention_with_kv_update_launch(a.plan, a.q, key, value, a.kc, a.vc, a.table, a.out, a.ws)
    late, ready = torch.cuda.Event(), torch.cuda.Event()
    late.record()
    binding.pa_attention_with_kv_update_launch_staged(b.plan, b.q, key, value, b.kc, b.vc, b.table, b.out, b.ws, late,
                                                      late_out_ready=ready)
    torch.cuda.synchronize()
    for x, y in ((a.out, b.out), (a.kc, b.kc), (a.vc, b.vc)):
        assert torch.equal(x, y)
    c.kc, c.vc = a.kc.cpu(), a.vc.cpu()
    ref, tol = c.reference()
    oc.assert_within(a.out[:c.T], ref, tol)


@pytest.mark.parametrize("code", wc.KINDS)
@pytest.mark.parametrize("q_len", [1, 5, 30, 200])
def test_cache_offsets_past_32_bits(code, q_len):
    """Blocks whose elements lie beyond 2^32: a pool of 9 GB (bf16) for K and for V."""
    c = wc.WindowCase(hq=16, hkv=8, d=128, q_lens=[q_len], seq_lens=[700], code=code, window=300, sinks=20, seed=q_len, spare=0)
    nb, base = 2**32 // (16 * 8 * 128) + 1000, 2**32 // (16 * 8 * 128) + 500
    big = [torch.empty((nb,) + tuple(t.shape[1:]), dtype=t.dtype, device=DEV) for t in (c.kc, c.vc)]
    for t, src in zip(big, (c.kc, c.vc)):
        t[base:base + c.nb].copy_(src)
    g = wc.OnGpu(c)
    g.kc, g.vc = big
    if c.scaled:
        g.ks, g.vs = (torch.ones(nb, 8, device=DEV) for _ in range(2))
        g.ks[base:base + c.nb], g.vs[base:base + c.nb] = c.ks.to(DEV), c.vs.to(DEV)
    table = np.where(c.table >= 0, c.table + base, c.table).astype(np.int32)
    g.table = torch.from_numpy(table).to(DEV)
    g.plan = binding.pa_plan_window(**c.desc(num_blocks=nb, block_table_host=table))
    g.ws = torch.zeros(g.plan.workspace_bytes, dtype=torch.uint8, device=DEV)
    out = g.run()
    ref, tol = c.reference()
    oc.assert_within(out[:c.T], ref[:c.T], tol[:c.T])


@pytest.mark.parametrize("code", wc.KINDS)
def test_physical_blocks_do_not_matter_and_runs_repeat(code):
    """The same logical contents elsewhere in the pool, and the same call again: the
    same bits."""
    kw = dict(hq=8, hkv=2, d=128, q_lens=[1, 4, 30, 1, 150], seq_lens=[900, 300, 1500, 40, 700], code=code, window=600, sinks=40)
    c = wc.WindowCase(seed=1, spare=30, **kw)
    g = wc.OnGpu(c)
    first = g.run().clone()
    assert torch.equal(g.run(), first)
    perm = np.random.default_rng(7).permutation(c.nb)
    p = torch.from_numpy(perm).to(DEV)
    for name in ("kc", "vc", "ks", "vs"):
        t = getattr(g, name)
        moved = torch.empty_like(t)
        moved[p] = t
        setattr(g, name, moved)
    g.table = torch.from_numpy(np.where(c.table >= 0, perm[c.table], c.table).astype(np.int32)).to(DEV)
    assert torch.equal(g.run(), first)


@pytest.mark.parametrize("code", wc.KINDS)
def test_outputs_at_16_bytes(code):
    """An output that starts 16 bytes past a 32-byte boundary."""
    c = wc.WindowCase(hq=8, hkv=2, d=128, q_lens=[1, 30, 3, 150], seq_lens=[300, 500, 99, 700], code=code, window=200, sinks=4)
    g = wc.OnGpu(c)
    want = g.run().clone()
    buf = torch.zeros(want.numel() + 64, dtype=torch.bfloat16, device=DEV)
    at = 8 if buf.data_ptr() % 32 == 0 else 0
    g.out = buf[at:at + want.numel()].view(want.shape)
    assert g.out.data_ptr() % 32 == 16
    assert torch.equal(g.run(), want)
    assert not buf[:at].any() and not buf[at + want.numel():].any()


@pytest.mark.parametrize("code", wc.KINDS)
def test_bad_block_is_reported(code):
    """A block id out of range that the host did not see, in the window or among the
    first tokens, sets the error word; the other request's rows are right."""
    for bad in (0, 14):
        c = wc.WindowCase(hq=4, hkv=2, d=128, q_lens=[1, 1], seq_lens=[230, 100], code=code, window=20, sinks=4)
        g = wc.OnGpu(c)
        g.table[0, bad] = c.nb + 5
        g.call()
        torch.cuda.synchronize()
        assert binding.pa_check_device_errors(g.ws[:4].view(torch.int32)) == binding.PA_DEVERR_BLOCK_RANGE
        ref, tol = c.reference()
        oc.assert_within(g.out[1:2], ref[1:2], tol[1:2])


@pytest.mark.parametrize("code", wc.SCALED)
@pytest.mark.parametrize("q_len", [1, 4, 100])
def test_nan_scales_of_unseen_parts_play_no_part(code, q_len):
    """The scale of a block that some rows of a request see may be NaN for the rows
    that do: those that do not are finite."""
    c = wc.WindowCase(hq=4, hkv=2, d=64, q_lens=[q_len], seq_lens=[400], code=code, window=60, sinks=3, seed=2)
    first = (400 - q_len - 60 + 1) // 16            # the block where the first row's window begins
    i = c.table[0, first]
    c.ks[i] = float("nan")
    g = wc.OnGpu(c)
    out = g.run()
    sees = np.array([wc.seen(p, 60, 3)[16 * first:16 * first + 16].any() for p in range(400 - q_len, 400)])
    bad = torch.isnan(out[:q_len].float()).any(-1).any(-1).cpu().numpy()
    assert np.array_equal(bad, sees)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp8_block", "int8_block"])
def test_device_step_and_graph_step_with_a_window(kind):
    """The step classes: equal to the calls, and the graph to the eager step."""
    rng = np.random.default_rng(5)
    code = {"bf16": "bf16", "fp8": "e4m3"}.get(kind, "e4m3_block" if kind == "fp8_block" else kind)
    gs = GraphStep(num_heads_q=8, num_heads_kv=2, head_dim=128, num_blocks=160, max_blocks_per_req=40, softmax_scale=128 ** -0.5,
                   max_tokens=120, max_reqs=5, max_extend_tiles=12, max_dequant_blocks=100, kv_cache_dtype=kind,
                   k_scale=wc.K_SCALE, v_scale=wc.V_SCALE, window=(48, 6))
    pools = None
    for q, seq in (([1, 30, 1], [200, 90, 33]), ([1, 1, 4, 60], [300, 50, 77, 200]), ([1] * 5, [600, 17, 48, 49, 90])):
        c = wc.WindowCase(hq=8, hkv=2, d=128, q_lens=q, seq_lens=seq, code=code, window=48, sinks=6, seed=int(rng.integers(99)),
                          pad=0, hidden=False, spare=0)
        b = batch_of(c, kind)
        st = DeviceStep(b, "cuda", window=(48, 6))
        g = torch.Generator().manual_seed(3)
        new = [torch.randn(c.T, 2, 128, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2)]
        dev = [t.to(DEV) for t in (c.kc, c.vc)] + ([t.to(DEV) for t in (c.ks, c.vs)] if c.scaled else [])
        if pools is None:
            pools = [torch.zeros((160,) + tuple(t.shape[1:]), dtype=t.dtype, device=DEV) for t in dev]
        for p, t in zip(pools, dev):
            p[:c.nb].copy_(t)
        out = st.run_append(c.q.to(DEV), *new, *dev) if c.scaled else st.run(c.q.to(DEV), *new, *dev)
        again = gs.run(b, c.q.to(DEV), *new, *pools)
        torch.cuda.synchronize()
        assert st.check_errors() == 0 and gs.check_errors() == 0
        assert torch.equal(out, again)
        for p, t in zip(pools, dev):
            assert torch.equal(p[:c.nb], t)
        c.kc, c.vc = dev[0].cpu(), dev[1].cpu()
        if c.scaled:
            c.ks, c.vs = dev[2].cpu(), dev[3].cpu()
        ref, tol = c.reference()
        oc.assert_within(out, ref, tol)


def batch_of(c, kind):
    """The case's metadata as a Batch."""
    z = torch.zeros(0)
    return workloads.Batch(num_common_prefix_blocks=0, poison_block=-1, name="window", num_heads_q=c.hq,
                           num_heads_kv=c.hkv, head_dim=c.d, block_size=16, num_blocks=c.nb, query_start_loc=c.qsl, seq_lens=c.seq.astype(np.int32),
                           num_computed=(c.seq - c.q_lens).astype(np.int32), block_table=c.table, q=z, key=z, value=z,
                           key_cache=z, value_cache=z, softmax_scale=c.scale, kv_cache_dtype=kind, k_scale=wc.K_SCALE,
                           v_scale=wc.V_SCALE)
