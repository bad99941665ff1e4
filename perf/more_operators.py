"""The measured cases of three operators that belong together: the rotation of
queries and keys by positions on several axes (time, height, width), the append
of new keys and values to a paged cache with that rotation on the way, and
attention with a sliding window and a few first tokens that stay visible, over
a paged cache that has given the blocks between them back.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, angles in 64) where ``own`` is false, and calls the library where it
is true.

Shapes as everywhere in this repository: q, out [T][Hq][D]; new keys and
values [T][Hkv][D]; caches [num_blocks][16][Hkv][D]; block scales
[num_blocks][Hkv]; block_table [R][max_blocks]; positions [axes][T].  New rows
come as views of the packed projection output [T][(Hq + 2 Hkv)][D], as a
model's linear layer leaves them.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
QMAX = {"int8_block": 127.0, "e4m3_block": 448.0}
MIN_EXP = -64                      # smallest block scale: 2^-64
UNIT = {"bf16": 1.0, "e4m3": 1 / 64, "e4m3_block": 1 / 64, "int8_block": 1 / 32}   # what a code of 1 stands for


def listed():
    wide = dict(heads_q=32, heads_kv=8, dim=128)
    video = dict(axes=3, assign="sections", own_freq=False, rotary_dim=128, layout="half", scaling="none", base=500000.0)
    return [
        # one token each of 64 running requests, text behind images: the smallest rotation, latency
        dict(name="axes rotary decode 64", op="rotary", tokens=64, runs=64, reach=4096, heads=40, rest=8, dim=128, **video),
        # a full token budget of prefill: frames of video between pieces of text
        dict(name="axes rotary video 8192", op="rotary", tokens=8192, runs=3, reach=131072, heads=40, rest=8, dim=128, **video),
        # the patches of an image, height and width with frequencies of their own, an odd number of tokens and heads
        dict(name="axes rotary image 1021", op="rotary", tokens=1021, runs=2, reach=1, heads=7, rest=2, dim=64, axes=2,
             assign="sections", own_freq=True, rotary_dim=64, layout="interleaved", scaling="none", base=10000.0),
        # 64 running requests, one token each, into an int8 cache
        dict(name="axes append decode int8", op="append", reqs=64, q_len=1, reach=4096, code="int8_block", **video, **wide),
        # two chunks of a video prompt over cached context that ends inside a block, into E4M3 codes with block scales
        dict(name="axes append video e4m3", op="append", reqs=2, q_len=2048, reach=4100, code="e4m3_block", **video, **wide),
        # the largest: four chunks into a bf16 cache, the axes dealt to the pairs in turn
        dict(name="axes append prefill bf16", op="append", reqs=4, q_len=2048, reach=1,
             code="bf16", **dict(video, assign="turn", rotary_dim=64, base=10000.0), **wide),
        # one request at its start, few heads: the smallest attention call
        dict(name="window 1 x 33 bf16", op="window", reqs=1, q_len=1, lo=33, hi=33, window=16, sinks=2, code="bf16", heads_q=4,
             heads_kv=2, dim=64),
        # an ordinary decode step of a layer with a window
        dict(name="window decode bf16", op="window", reqs=64, q_len=1, lo=512, hi=4096, window=1024, sinks=4, code="bf16",
             **wide),
        # a large decode step far into long contexts, of which the window alone is still in the cache
        dict(name="window decode long int8", op="window", reqs=128, q_len=1, lo=4096, hi=131072, window=4096, sinks=16,
             code="int8_block", **wide),
        # verify rows of four tokens over E4M3 codes with one scale, no first tokens kept
        dict(name="window verify e4m3", op="window", reqs=128, q_len=4, lo=1024, hi=8000, window=2048, sinks=0, code="e4m3",
             **wide),
        # two prefill chunks longer than the window
        dict(name="window chunks bf16", op="window", reqs=2, q_len=2048, lo=1024, hi=6144, window=1024, sinks=4, code="bf16",
             **wide),
        # one long chunk far into a prompt, a wide window, E4M3 codes with block scales: bound by arithmetic
        dict(name="window prefill e4m3", op="window", reqs=1, q_len=4096, lo=12288, hi=12288, window=4096, sinks=64,
             code="e4m3_block", **wide),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _rope_of(rng, dim):
    return dict(axes=rng.choice([2, 3, 3]), assign=rng.choice(["sections", "turn"]), own_freq=rng.random() < 0.3,
                rotary_dim=8 * rng.randint(1, dim // 8) if rng.random() < 0.5 else dim,
                layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "none", "linear", "yarn"]),
                base=rng.choice([10000.0, 500000.0]))


HEADS = [(32, 8, 128), (64, 8, 128), (4, 2, 64), (8, 8, 128), (16, 2, 64), (28, 4, 128), (32, 1, 128), (12, 3, 64)]


def draw(rng):
    op = rng.choice(["rotary", "append", "window", "window"])
    hq, hkv, d = rng.choice(HEADS)
    if op == "rotary":
        t = _log(rng, 1, 8192)
        return dict(op=op, tokens=t, runs=min(t, _log(rng, 1, 64)), reach=_log(rng, 1, 200000),
                    heads=min(hq + hkv, 40), rest=rng.choice([0, hkv]), dim=d, **_rope_of(rng, d))
    if op == "append":
        r = _log(rng, 1, 256)
        most = 8192 if hq + hkv <= 40 else 4096
        return dict(op=op, reqs=r, q_len=_log(rng, 1, max(1, most // r)), reach=_log(rng, 1, 20000),
                    code=rng.choice(["bf16", "int8_block", "int8_block", "e4m3_block", "e4m3"]), heads_q=hq, heads_kv=hkv,
                    dim=d, **_rope_of(rng, d))
    q = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, 2048)])
    hi = _log(rng, 1, 131072 if q <= 8 else 16384)
    window, sinks = _log(rng, 1, 8192), rng.choice([0, 4, _log(rng, 1, 300)])
    keys = min(hi + q, window + sinks + q)
    room = min(4e8 / (keys * hkv * d), 6e10 / (4 * hq * d * q * min(hi + q, window + sinks)), 128 if q <= 8 else 4)
    return dict(op=op, reqs=max(1, _log(rng, 1, max(1.0, room))), q_len=q, lo=rng.randint(1, hi), hi=hi, window=window,
                sinks=sinks, code=rng.choice(["bf16", "int8_block", "e4m3_block"] + ["e4m3"] * (d == 128)), heads_q=hq,
                heads_kv=hkv, dim=d)


# ------------------------------------------------------------------ inputs --
FACTOR, ORIGINAL, BETA_FAST, BETA_SLOW = 8.0, 8192, 32.0, 1.0       # scaling of the frequencies


def _axis_of_pair(c):
    """The axis each of the rotary_dim / 2 pairs turns with: sections one after
    the other (the first axis the smaller ones), or in turn."""
    n, a = c["rotary_dim"] // 2, c["axes"]
    if c["assign"] == "turn":
        return [i % a for i in range(n)]
    if a == 3:
        first = n // 4
        ends = [first, first + (n - first + 1) // 2]
    else:
        ends = [(n + 1) // 2]
    return [sum(i >= e for e in ends) for i in range(n)]


def _scaled(c, dim):
    """Angles per position of the dim / 2 pairs of a rotation of dim elements, and
    the factor on cos and sin."""
    n, base = dim // 2, c["base"]
    f = [base ** (-2.0 * i / dim) for i in range(n)]
    if c["scaling"] == "linear":
        return [x / FACTOR for x in f], 1.0
    if c["scaling"] == "yarn":
        at = lambda turns: dim * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0, math.floor(at(BETA_FAST))), min(dim - 1, math.ceil(at(BETA_SLOW)))
        ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3))) for i in range(n)]
        return [x / FACTOR * r + x * (1 - r) for x, r in zip(f, ramp)], 0.1 * math.log(FACTOR) + 1.0
    return f, 1.0


def _frequencies(c):
    """Angles per position of the pairs; with frequencies of its own, the k-th of
    an axis's m pairs turns as pair k of a rotation of 2 m elements does."""
    if not c["own_freq"]:
        return _scaled(c, c["rotary_dim"])
    axis = _axis_of_pair(c)
    f, mag = [0.0] * len(axis), _scaled(c, c["rotary_dim"])[1]
    for a in range(c["axes"]):
        mine = [i for i, x in enumerate(axis) if x == a]
        for k, x in enumerate(_scaled(c, 2 * len(mine))[0]):
            f[mine[k]] = x
    return f, mag


def _rope(c):
    """The library's handle of a rotation."""
    from paged_kv_cache_16_gb300 import binding
    more = {"none": {}, "linear": dict(factor=FACTOR),
            "yarn": dict(factor=FACTOR, original_max_position=ORIGINAL, low=BETA_SLOW, high=BETA_FAST)}[c["scaling"]]
    kind = {"none": binding.PA_ROPE_SCALE_NONE, "linear": binding.PA_ROPE_SCALE_LINEAR,
            "yarn": binding.PA_ROPE_SCALE_YARN}[c["scaling"]]
    return binding.pa_rope_create_axes(
        num_axes=c["axes"], axis_of_pair=_axis_of_pair(c), rotary_dim=c["rotary_dim"], base=c["base"], scaling=kind,
        frequencies=binding.PA_ROPE_AXES_OWN if c["own_freq"] else binding.PA_ROPE_AXES_SHARED,
        layout=binding.PA_ROPE_HALF if c["layout"] == "half" else binding.PA_ROPE_INTERLEAVED, **more)


def _walk(n, axes, start, rng):
    """Positions [axes][n] of a piece of a prompt: text, whose tokens stand at the
    same position on every axis, and grids of patches (frames x rows x columns)
    that start behind it; two axes: rows and columns of one image after another."""
    parts, have, at = [], 0, start
    while have < n:
        h, w = int(rng.integers(4, 33)), int(rng.integers(4, 33))
        if axes == 2:
            y, x = np.divmod(np.arange(h * w), w)
            parts.append(np.stack([y, x]) + start)
        else:
            text = int(rng.integers(1, 100))
            f = int(rng.integers(1, 5))
            parts.append(np.tile(at + np.arange(text), (axes, 1)))
            at += text
            t, rest = np.divmod(np.arange(f * h * w), h * w)
            y, x = np.divmod(rest, w)
            parts.append(np.stack([t, y, x]) + at)
            at += max(f, h, w)
        have += sum(p.shape[1] for p in parts[-2 if axes > 2 else -1:])
    return np.concatenate(parts, 1)[:, :n]


def _lens(c, rng):
    """Context lengths before the step, spread evenly over [lo, hi], in an order of the seed's."""
    n = c["reqs"]
    v = np.array([c["lo"] + int((c["hi"] - c["lo"]) * (i + 0.5) / n) for i in range(n)], dtype=np.int64)
    return rng.permutation(v)


def _new_lens(c):
    """Tokens that each request appends: from q_len down to three quarters of it."""
    return np.array([c["q_len"] - c["q_len"] // 4 * k // c["reqs"] for k in range(c["reqs"])], dtype=np.int64)


def _codes(shape, code, gen):
    """Codes of normal values, as a cache in use holds them."""
    x = torch.randn(shape, generator=gen, device="cuda")
    if code == "int8_block":
        return x.mul_(32).round_().clamp_(-127, 127).to(torch.int8)
    if code != "bf16":
        return x.mul_(64).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.to(torch.bfloat16)


def _values(cache):
    """The numbers that a cache's codes stand for, without the scale, in 32 bits."""
    return cache.view(torch.float8_e4m3fn).float() if cache.dtype == torch.uint8 else cache.float()


def _i32(a):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = case
    gen = torch.Generator("cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = dict(c=c, op=c["op"])
    if c["op"] == "window":
        return _prepare_window(c, s, gen, rng)
    f, s["mag"] = _frequencies(c)
    s["freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
    s["axis"] = torch.tensor(_axis_of_pair(c), device="cuda")
    s["rope"] = _rope(c) if own else None
    if c["op"] == "rotary":
        # pieces of prompts, each starting somewhere in the reach
        t, n = c["tokens"], c["runs"]
        begin = [t * k // n for k in range(n + 1)]
        s["pos"] = _i32(np.concatenate([_walk(begin[k + 1] - begin[k], c["axes"], int(rng.integers(0, c["reach"])), rng)
                                        for k in range(n)], 1))
        packed = torch.randn(t, c["heads"] + c["rest"], c["dim"], generator=gen, device="cuda").to(torch.bfloat16)
        s["x"] = packed[:, :c["heads"]]
        s["out"] = torch.empty(t, c["heads"], c["dim"], dtype=torch.bfloat16, device="cuda")
        return s
    hq, hkv, d, r = c["heads_q"], c["heads_kv"], c["dim"], c["reqs"]
    # earlier blocks have been given back, as layers with a window do: only the blocks of the new tokens are in the pool
    nc = rng.integers(0, c["reach"], r)
    qn = rng.permutation(_new_lens(c))
    first, last = nc // BLOCK, (nc + qn - 1) // BLOCK
    table = np.zeros((r, int(last.max()) + 1), dtype=np.int32)
    nb = 1 + int(((qn + 14) // BLOCK + 1).sum())         # enough wherever in its blocks a request stands
    ids = 1 + rng.permutation(nb - 1)
    at = np.concatenate([[0], np.cumsum(last - first + 1)])
    for k in range(r):
        table[k, first[k]:last[k] + 1] = ids[at[k]:at[k + 1]]
    qsl = np.concatenate([[0], np.cumsum(qn)])
    t = int(qsl[-1])
    s.update(qsl=_i32(qsl), nc=_i32(nc), table=_i32(table), t=t)
    # an image of many tokens takes few positions: rows stand before their index in the cache
    s["pos"] = _i32(np.concatenate([_walk(int(qn[k]), c["axes"], int(nc[k] * 3 // 4), rng) for k in range(r)], 1))
    packed = torch.randn(t, hq + 2 * hkv, d, generator=gen, device="cuda").to(torch.bfloat16)
    s.update(q=packed[:, :hq], k=packed[:, hq:hq + hkv], v=packed[:, hq + hkv:])
    s["q_out"] = torch.empty(t, hq, d, dtype=torch.bfloat16, device="cuda")
    shape = (nb, BLOCK, hkv, d)
    s.update(kc=_codes(shape, c["code"], gen), vc=_codes(shape, c["code"], gen))
    if c["code"] in QMAX:
        # scales that earlier appends left: mostly large enough for the new rows, some of them not
        e = torch.randint(-1, 2, (2, nb, hkv), generator=gen, device="cuda").float() - (4 if c["code"] == "int8_block" else 6)
        s.update(ks=torch.exp2(e[0]).contiguous(), vs=torch.exp2(e[1]).contiguous())
    if c["code"] != "bf16":
        s.update(kval=torch.empty(shape, dtype=torch.bfloat16, device="cuda"),
                 vval=torch.empty(shape, dtype=torch.bfloat16, device="cuda"))
    return s


def _prepare_window(c, s, gen, rng):
    hq, hkv, d, r, q = c["heads_q"], c["heads_kv"], c["dim"], c["reqs"], c["q_len"]
    ctx = _lens(c, rng)
    seq = ctx + q
    # the blocks that some query of the step sees; the others have been given back
    total = -(-seq // BLOCK)
    begin = np.maximum(0, ctx - c["window"] + 1) // BLOCK
    head = np.minimum(-(-np.minimum(c["sinks"], seq) // BLOCK), begin)
    need = head + total - begin
    nb = int(need.sum()) + 1
    ids = rng.permutation(nb)
    table = np.full((r, int(total.max())), -1, dtype=np.int32)
    at = np.concatenate([[0], np.cumsum(need)])
    for k in range(r):
        mine = ids[at[k]:at[k + 1]]
        table[k, :head[k]] = mine[:head[k]]
        table[k, begin[k]:total[k]] = mine[head[k]:]
    shape = (nb, BLOCK, hkv, d)
    # first keys behind the window, and how many keys the longest row of keys holds
    low = np.maximum(0, ctx - c["window"] + 1)
    s.update(table=_i32(table), ctx=torch.as_tensor(ctx, device="cuda"), scale=d ** -0.5,
             length=int((np.minimum(c["sinks"], low) + seq - low).max()))
    s.update(kc=_codes(shape, c["code"], gen), vc=_codes(shape, c["code"], gen))
    if c["code"] in QMAX:
        sc = torch.exp(0.5 * torch.randn(2, nb, hkv, generator=gen, device="cuda")) * UNIT[c["code"]]
        s.update(ks=sc[0].contiguous(), vs=sc[1].contiguous())
    s["q"] = torch.randn(r * q, hq, d, generator=gen, device="cuda").to(torch.bfloat16)
    s["out"] = torch.empty(r * q, hq, d, dtype=torch.bfloat16, device="cuda")
    if own:
        from paged_kv_cache_16_gb300 import binding
        kind = {"bf16": binding.PA_KV_BF16, "e4m3": binding.PA_KV_FP8_E4M3, "e4m3_block": binding.PA_KV_FP8_E4M3_BLOCK,
                "int8_block": binding.PA_KV_INT8_BLOCK}[c["code"]]
        s["plan"] = binding.pa_plan_window(window=c["window"], sink_tokens=c["sinks"], num_heads_q=hq, num_heads_kv=hkv,
                                           head_dim=d, num_blocks=nb, query_start_loc=np.arange(r + 1) * q, seq_lens=seq,
                                           num_computed_tokens=ctx, block_table_host=table, softmax_scale=s["scale"],
                                           kv_cache_dtype=kind, k_scale=UNIT[c["code"]], v_scale=UNIT[c["code"]])
        s["ws"] = torch.zeros(s["plan"].workspace_bytes, dtype=torch.uint8, device="cuda")
        # once per step; every layer of the step with this window then launches on it
        binding.pa_upload_metadata(s["plan"], s["ws"])
    return s


# ------------------------------------------------------------- plain forms --
def _rotated(x, s):
    """Rows [T][H][D] rotated by their positions, in 32 bits (angles in 64)."""
    rd, half = s["c"]["rotary_dim"], s["c"]["rotary_dim"] // 2
    angle = s["pos"].double()[s["axis"]].T * s["freq"]                    # [T][pairs]
    cos, sin = (s["mag"] * torch.cos(angle)).float()[:, None], (s["mag"] * torch.sin(angle)).float()[:, None]
    x = x.float()
    if s["c"]["layout"] == "half":
        a, b = x[..., :half], x[..., half:rd]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rd:]], -1)
    a, b = x[..., 0:rd:2], x[..., 1:rd:2]
    y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, x[..., rd:]], -1)


def _power(amax, qmax):
    """The smallest power of two (2^MIN_EXP at least) whose qmax-fold reaches amax."""
    m, e = torch.frexp(amax)                                # amax = m * 2^e, 0.5 <= m < 1
    mq, eq = math.frexp(qmax)
    p = e - eq + (m > mq).int()
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, p, MIN_EXP).clamp(min=MIN_EXP))


def _encode(x, code):
    """Values in units of the scale as codes: to nearest, ties to even, at most QMAX."""
    if code == "int8_block":
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _store(cache, scales, rows, blk, off, first, code):
    """Append rows [T][Hkv][D] (32 bits) at (blk, off) to codes with a scale per (block, head)."""
    nb, _, hkv, _ = cache.shape
    amax = torch.zeros(nb, hkv, device="cuda").index_reduce_(0, blk, rows.abs().amax(-1), "amax")
    old = torch.where((first == 0)[:, None], 0.0, scales)   # a block that starts anew forgets its scale
    new = torch.maximum(old, _power(amax, QMAX[code]))
    new = torch.where((first < BLOCK)[:, None], new, scales)
    ratio = torch.where((first < BLOCK)[:, None], old / new, 1.0)[:, None, :, None]
    kept = _encode(_values(cache) * ratio, code)            # the scale grew: the earlier rows' codes follow
    earlier = torch.arange(BLOCK, device="cuda")[None, :, None, None] < first[:, None, None, None]
    cache.copy_(torch.where(earlier, kept, cache))
    cache[blk, off] = _encode(rows / new[blk][..., None], code)
    scales.copy_(new)


def _plain_append(s):
    c = s["c"]
    qn = s["qsl"][1:] - s["qsl"][:-1]
    tok = torch.arange(s["t"], device="cuda")
    req = torch.repeat_interleave(torch.arange(c["reqs"], device="cuda"), qn, output_size=s["t"])
    index = s["nc"][req] + (tok - s["qsl"][req])            # where a row goes in the cache
    blk, off = s["table"][req, index // BLOCK].long(), (index % BLOCK).long()
    s["q_out"].copy_(_rotated(s["q"], s))
    k = _rotated(s["k"], s)
    if c["code"] == "bf16":
        s["kc"][blk, off] = k.to(torch.bfloat16)
        s["vc"][blk, off] = s["v"]
        return
    if c["code"] == "e4m3":
        s["kc"][blk, off] = _encode(k / UNIT["e4m3"], "e4m3")
        s["vc"][blk, off] = _encode(s["v"].float() / UNIT["e4m3"], "e4m3")
        return
    first = torch.full((s["kc"].shape[0],), BLOCK, device="cuda", dtype=torch.int64).index_reduce_(0, blk, off, "amin")
    _store(s["kc"], s["ks"], k, blk, off, first, c["code"])
    _store(s["vc"], s["vs"], s["v"].float(), blk, off, first, c["code"])


def _plain_window(s):
    c = s["c"]
    r, n, hq, hkv, d, length = c["reqs"], c["q_len"], c["heads_q"], c["heads_kv"], c["dim"], s["length"]
    # the keys that some query of a request sees: first tokens, then the window
    low = (s["ctx"] - c["window"] + 1).clamp(min=0)[:, None]
    head = low.clamp(max=c["sinks"])
    col = torch.arange(length, device="cuda")
    key = torch.where(col < head, col, low + col - head)                        # [R][length]
    last = s["ctx"][:, None] + n - 1
    at = key.minimum(last)
    page = s["table"].long().gather(1, at // BLOCK)

    def gathered(cache, name):
        x = _values(cache[page, at % BLOCK])
        x = x * s[name][page][..., None] if c["code"] in QMAX else x * UNIT[c["code"]]
        return x.transpose(1, 2)                                                # [R][Hkv][length][D]

    q = s["q"].float().view(r, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(r, hkv, -1, d)
    score = (q @ gathered(s["kc"], "ks").transpose(2, 3) * s["scale"]).view(r, hkv, hq // hkv, n, length)
    pos = s["ctx"][:, None, None] + torch.arange(n, device="cuda")[:, None]    # [R][n][1]
    key = key[:, None]
    seen = (key <= pos) & ((pos - key < c["window"]) | (key < c["sinks"]))
    score = score.masked_fill_(~seen[:, None, None], -math.inf)
    w = torch.exp(score.sub_(score.amax(-1, keepdim=True)))
    w = w.div_(w.sum(-1, keepdim=True))
    out = w.view(r, hkv, -1, length) @ gathered(s["vc"], "vs")
    s["out"].copy_(out.view(r, hkv, hq // hkv, n, d).permute(0, 3, 1, 2, 4).reshape(r * n, hq, d))


def _append_outputs(s):
    """q, and the caches as the values that they stand for."""
    code = s["c"]["code"]
    if code == "bf16":
        return dict(q=s["q_out"], k=s["kc"], v=s["vc"])
    number = (lambda x: x) if code == "int8_block" else (lambda x: x.view(torch.float8_e4m3fn).to(torch.bfloat16))
    ks, vs = (s["ks"][:, None, :, None], s["vs"][:, None, :, None]) if code in QMAX else (UNIT[code], UNIT[code])
    torch.mul(number(s["kc"]), ks, out=s["kval"])
    torch.mul(number(s["vc"]), vs, out=s["vval"])
    out = dict(q=s["q_out"], k=s["kval"], v=s["vval"])
    return dict(out, ks=s["ks"], vs=s["vs"]) if code in QMAX else out


def run(state):
    s = state
    if own:
        from paged_kv_cache_16_gb300 import binding
        if s["op"] == "rotary":
            binding.pa_rotary_axes(s["rope"], s["x"], s["pos"], s["out"])
        elif s["op"] == "append":
            binding.pa_append_kv_axes(s["rope"], s["k"], s["v"], s["pos"], s["qsl"], s["nc"], s["table"], s["kc"], s["vc"],
                                      key_scales=s.get("ks"), value_scales=s.get("vs"), k_scale=UNIT[s["c"]["code"]],
                                      v_scale=UNIT[s["c"]["code"]], q=s["q"], q_out=s["q_out"])
        elif s["c"]["code"] in QMAX:
            binding.pa_attention_scaled_launch(s["plan"], s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"],
                                               s["out"], s["ws"])
        else:
            binding.pa_attention_launch(s["plan"], s["q"], s["kc"], s["vc"], s["table"], s["out"], s["ws"])
    elif s["op"] == "rotary":
        s["out"].copy_(_rotated(s["x"], s))
    elif s["op"] == "append":
        _plain_append(s)
    else:
        _plain_window(s)
    return _append_outputs(s) if s["op"] == "append" else s["out"]


# -------------------------------------------------------------------- work --
def _seen(pos, window, sinks):
    """Keys that a query at `pos` sees (numpy)."""
    low = np.maximum(0, pos - window + 1)
    return np.minimum(sinks, low) + pos + 1 - low


def work(case):
    c = case
    if c["op"] == "rotary":
        n = c["tokens"] * c["heads"] * c["dim"]
        return {"bytes": 4 * n + 4 * c["axes"] * c["tokens"], "flops": 3 * c["tokens"] * c["heads"] * c["rotary_dim"]}
    hq, hkv, d, r, q = c["heads_q"], c["heads_kv"], c["dim"], c["reqs"], c["q_len"]
    es = 2 if c["code"] == "bf16" else 1
    if c["op"] == "append":
        t = int(_new_lens(c).sum())
        blocks = int(((_new_lens(c) + BLOCK - 1) // BLOCK).sum())
        scales = 16 * hkv if c["code"] in QMAX else 0
        return {"bytes": t * d * (4 * hq + 2 * hkv * (2 + es)) + 4 * c["axes"] * t + 8 * r + blocks * (4 + scales),
                "flops": 3 * t * (hq + hkv) * c["rotary_dim"]}
    ctx = _lens(c, np.random.default_rng(0))
    low = np.maximum(0, ctx - c["window"] + 1)
    keys = int((np.minimum(c["sinks"], low) + ctx + q - low).sum())
    pairs = int(_seen(ctx[:, None] + np.arange(q), c["window"], c["sinks"]).sum())
    scales = 8 * hkv if c["code"] in QMAX else 0
    return {"bytes": 2 * keys * hkv * d * es + (keys // BLOCK) * (4 + scales) + 4 * r * q * hq * d,
            "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------- exact --
def _turned(x, s):
    """The rotation as a product of complex numbers, in 64 bits."""
    c, rd = s["c"], s["c"]["rotary_dim"]
    x = x.double()
    part = x[..., :rd].unflatten(-1, (2, rd // 2)).transpose(-1, -2) if c["layout"] == "half" else x[..., :rd].unflatten(-1, (rd // 2, 2))
    angle = torch.stack([s["pos"][a].double() * f for a, f in zip(s["axis"].tolist(), s["freq"].tolist())], -1)[:, None]
    z = torch.view_as_complex(part.contiguous()) * torch.polar(torch.full_like(angle, s["mag"]), angle)
    y = torch.view_as_real(z)
    y = y.transpose(-1, -2).flatten(-2) if c["layout"] == "half" else y.flatten(-2)
    return torch.cat([y, x[..., rd:]], -1)


def _nearest(x, code):
    """x rounded to the codes' values, ties to even, in 64 bits."""
    if code == "int8_block":
        return torch.clamp(torch.round(x), -127, 127)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    e = e + (x.abs() >= torch.exp2(e + 1)).double() - (x.abs().clamp(min=2.0 ** -6) < torch.exp2(e)).double()
    step = torch.exp2(e - 3)
    return torch.clamp(torch.round(x / step) * step, -448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "rotary":
        return _turned(s["x"], s)
    if c["op"] == "append":
        return _exact_append(s)
    n, hq, hkv, d = c["q_len"], c["heads_q"], c["heads_kv"], c["dim"]
    out = torch.empty(c["reqs"] * n, hq, d, dtype=torch.float64, device="cuda")
    ctx, g = s["ctx"].tolist(), hq // hkv
    for r in range(c["reqs"]):
        low = max(0, ctx[r] - c["window"] + 1)
        keys = torch.cat([torch.arange(0, min(c["sinks"], low), device="cuda"), torch.arange(low, ctx[r] + n, device="cuda")])
        blocks = s["table"][r].long()[keys // BLOCK]
        pos = ctx[r] + torch.arange(n, device="cuda")[:, None]
        hidden = (keys > pos) | ((keys <= pos - c["window"]) & (keys >= c["sinks"]))
        for h in range(hkv):
            def whole(cache, name):
                x = _values(cache[blocks, keys % BLOCK, h]).double()
                return x * s[name][blocks, h].double()[:, None] if c["code"] in QMAX else x * UNIT[c["code"]]
            q = s["q"][r * n:(r + 1) * n, h * g:(h + 1) * g].double().transpose(0, 1)     # [G][n][D]
            z = torch.einsum("gnd,ld->gnl", q, whole(s["kc"], "ks")) * s["scale"]
            z = torch.softmax(z.masked_fill(hidden[None], -math.inf), -1)
            out[r * n:(r + 1) * n, h * g:(h + 1) * g] = (z @ whole(s["vc"], "vs")).transpose(0, 1)
    return out


def _exact_append(s):
    c = s["c"]
    qsl, nc, table = s["qsl"].tolist(), s["nc"].tolist(), s["table"].tolist()
    k64, v64 = _turned(s["k"], s), s["v"].double()
    code = c["code"]
    val = {n: _values(s[n + "c"]).double() * (s[n + "s"].double()[:, None, :, None] if code in QMAX else UNIT[code]) for n in "kv"}
    sc = {n: s[n + "s"].double() for n in "kv"} if code in QMAX else None
    for r in range(c["reqs"]):
        p, end_r = nc[r], nc[r] + qsl[r + 1] - qsl[r]
        while p < end_r:
            end = min((p // BLOCK + 1) * BLOCK, end_r)
            b, o = table[r][p // BLOCK], p % BLOCK
            t0 = qsl[r] + p - nc[r]
            for n, rows in (("k", k64), ("v", v64)):
                new = rows[t0:t0 + end - p]
                if code not in QMAX:
                    val[n][b, o:o + end - p] = new if code == "bf16" else _nearest(new / UNIT[code], code) * UNIT[code]
                    continue
                m = (new.abs().amax((0, 2)) / QMAX[code]).clamp(min=2.0 ** MIN_EXP)
                scale = torch.exp2(torch.ceil(torch.log2(m)))
                if o:
                    scale = torch.maximum(scale, sc[n][b])
                    val[n][b, :o] = _nearest(val[n][b, :o] / scale[:, None], code) * scale[:, None]
                val[n][b, o:o + end - p] = _nearest(new / scale[:, None], code) * scale[:, None]
                # rows behind the new ones keep their codes, under the new scale
                val[n][b, o + end - p:] = _values(s[n + "c"][b, o + end - p:]).double() * scale[:, None]
                sc[n][b] = scale
            p = end
    out = dict(q=_turned(s["q"], s), k=val["k"], v=val["v"])
    return dict(out, ks=sc["k"], vs=sc["v"]) if code in QMAX else out
