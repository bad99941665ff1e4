"""What windowed plans hand out, read back from their metadata images on the CPU."""
import random

import pytest
import torch

import plan_image as pi
from paged_kv_cache_16_gb300 import binding, build
from test_window_cpu import FAKE, desc


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


def view(first, end, window, sinks, unit):
    """(head, skip) of the blocks that query tokens at [first, end) read."""
    low, head = max(0, first - window + 1) // 16, -(-min(sinks, end) // 16)
    if low <= head:
        return 0, 0
    head = -(-head // unit) * unit
    return head, low - head


def joined(spans, parts, end):
    """Spans of one row's or tile's keys: [0, end) each once, numbered or alone."""
    spans = sorted(spans)
    assert spans[0][0] == 0 and spans[-1][1] == end
    assert all(a[1] == b[0] for a, b in zip(spans, spans[1:])) and all(a < b for a, b in spans)
    assert sorted(parts) == (list(range(len(parts))) if len(parts) > 1 else [-1])


def check_plan(kw):
    """Every block of every row, and every key tile of every chunk, handed out once;
    merge rows for what is in pieces."""
    im = image(kw)
    hq, hkv, window, sinks = kw["num_heads_q"], kw["num_heads_kv"], kw["window"], kw["sink_tokens"]
    G, per_group = hq // hkv, hkv // im.groups
    qsl, seq, done = kw["query_start_loc"], kw["seq_lens"], kw["num_computed_tokens"]
    req_of = {t: r for r in range(len(seq)) for t in range(qsl[r], qsl[r + 1])}
    pos = {t: int(done[r] + t - qsl[r]) for t, r in req_of.items()}
    assert list(im.counts[:4]) == [len(im.tiles), len(im.merges), im.info["num_dequant_blocks"], len(req_of)]
    pieces = {}                                       # (token, kv head) -> pieces of its keys
    # split-KV rows
    assert im.cta_begin[0] == 0 and im.cta_begin[-1] == len(im.items) and (im.cta_begin[1:] >= im.cta_begin[:-1]).all()
    rows = {}
    for x in im.items:
        rows.setdefault((x["token"], x["head_group"]), []).append(x)
    for (token, group), xs in rows.items():
        n, r = xs[0]["n_tok"], req_of[token]
        assert all((x["n_tok"], x["req"], x["key_end"]) == (n, r, pos[token] + n) for x in xs)
        _, skip = view(pos[token], pos[token] + n, window, sinks, 1)
        joined([(x["page_begin"], x["page_end"]) for x in xs], [x["part"] for x in xs], -(-(pos[token] + n - 16 * skip) // 16))
        for t in range(token, token + n):
            for h in range(group * per_group, (group + 1) * per_group):
                assert req_of[t] == r and pieces.setdefault((t, h), len(xs)) == len(xs)
    # tiles: sub-tiles of rows, none without a key
    sub, blocks = 128 // G, {}
    for x in im.tiles:
        blocks.setdefault((x["t0"], x["n_tok"], x["kv_head"]), []).append(x)
    for (t0, n, h), xs in blocks.items():
        head, skip = view(pos[t0], pos[t0] + n, window, sinks, 8 if kw["kv_cache_dtype"] else 1)
        p0 = pos[t0] - 16 * skip
        joined([(x["key_begin"], x["key_end"]) for x in xs], [x["part"] for x in xs], p0 + n)
        for x in xs:
            assert (x["pos0"], x["head"], x["skip"], x["causal"]) == (p0, head, skip, 1)
            assert x["key_begin"] % 128 == 0 and x["key_begin"] < p0 + min(n, sub) and n <= (sub if x["split"] else 2 * sub)
        for t in range(t0, t0 + n):
            assert req_of[t] == req_of[t0] and (t, h) not in pieces
            pieces[t, h] = len(xs)
    assert pieces.keys() == {(t, h) for t in req_of for h in range(hkv)}
    # merges
    merged = {}
    for m in im.merges:
        group = m["hq_begin"] // (per_group * G)
        assert (m["hq_begin"], m["hq_count"]) == (group * per_group * G, per_group * G)
        assert m["slot0"] == im.part_offset[m["token"] * im.groups + group]
        for h in range(group * per_group, (group + 1) * per_group):
            merged[m["token"], h] = m["count"]
    assert merged == {k: v for k, v in pieces.items() if v > 1}
    slots = sorted((m["slot0"], m["count"]) for m in im.merges)
    assert all(a + n <= b for (a, n), (b, _) in zip(slots, slots[1:]))
    assert not slots or sum(slots[-1]) <= im.info["num_partial_slots"]


@pytest.mark.parametrize("num_sms", [1, 3, 20, 152])
@pytest.mark.parametrize("code", range(4))
def test_more_rows_than_ctas_and_fewer_are_read_once(num_sms, code):
    for n in (1, 2, 7, 40, 500):
        for hkv in (2, 3, 16):
            for window in (64, 1):
                check_plan(desc([1] * n, [100 + 3 * i for i in range(n)], window, 4, code, hq=4 * hkv, hkv=hkv, num_sms=num_sms))


@pytest.mark.parametrize("code", range(4))
@pytest.mark.parametrize("seed", range(12))
def test_drawn_steps_are_read_once(seed, code):
    rng = random.Random(100 * code + seed)
    for _ in range(12):
        hq, hkv = rng.choice([(32, 8), (32, 1), (16, 2), (64, 8), (12, 4), (16, 16), (33, 1), (10, 5)])
        q = [rng.choice([0, 1, 1, 2, 5, 8, 9, 33, rng.randint(1, 700)]) for _ in range(int(2 ** rng.uniform(0, 6)))]
        seq = [x + int(2 ** rng.uniform(0, 13)) - 1 for x in q]
        check_plan(desc(q, seq, int(2 ** rng.uniform(0, 13)), int(rng.choice([0, 1, 4, 17, 130, 900])), code, hq=hq, hkv=hkv,
                        max_blocks_per_req=600, num_sms=rng.choice([1, 3, 20, 152, 152])))


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers lead nowhere")
@pytest.mark.parametrize("code", [0, 1])
@pytest.mark.parametrize("hq,hkv", [(32, 8), (64, 8), (32, 1), (48, 16)])
@pytest.mark.parametrize("rows", [[128], [256], [1300], [600], [60, 60], [9] * 5, [200, 1, 1, 2], [30], [3000]])
@pytest.mark.parametrize("window", [1500, 4096, 8192])
def test_pieces_of_tiles_do_not_outgrow_the_librarys_scratch(lib, code, hq, hkv, rows, window):
    """pa_attention_no_alloc takes every windowed step whose whole tiles fit its scratch
    (here it ends where it asks for a device), and refuses the others."""
    n, scratch = len(rows), binding.NO_ALLOC_SCRATCH_BYTES
    kw = desc(rows, [9000 - 7 * i for i in range(n)], window, 4, code, hq=hq, hkv=hkv, max_blocks_per_req=600)
    plan, whole = binding.pa_plan_window(**kw), binding.pa_plan_window(**{**kw, "num_sms": 1})
    decode = 2 * 152 * (-(-hkv // 8)) * hq * 130 * 4 * (1 in rows)      # more partials of split-KV rows on more SMs
    statuses = set()
    for _ in range(2):
        statuses.add(lib.pa_attention_no_alloc(plan.handle, FAKE, FAKE, FAKE, FAKE, FAKE, None, None))
    assert len(statuses) == 1
    status = statuses.pop()
    if whole.workspace_bytes + decode <= scratch:
        assert status == binding.PA_ERR_CUDA
    elif whole.workspace_bytes > scratch:
        assert status == binding.PA_ERR_WORKSPACE_TOO_SMALL
    else:
        assert status in (binding.PA_ERR_CUDA, binding.PA_ERR_WORKSPACE_TOO_SMALL)
