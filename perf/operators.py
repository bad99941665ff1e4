"""The measured cases of three operators that belong together: the rotation of
queries and keys by their positions, the append of new keys and values to a
paged cache with that rotation on the way, and attention over a cache of 8-bit
codes with one scale per (block of 16 tokens, kv head).

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, angles in 64) where ``own`` is false, and calls the library where it
is true.

Shapes as everywhere in this repository: q, out [T][Hq][D]; new keys and
values [T][Hkv][D]; caches [num_blocks][16][Hkv][D]; scales
[num_blocks][Hkv]; block_table [R][max_blocks].  New rows come as views of the
packed projection output [T][(Hq + 2 Hkv)][D], as a model's linear layer
leaves them.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
QMAX = {"int8": 127.0, "e4m3": 448.0}
MIN_EXP = -64                      # smallest block scale: 2^-64


def listed():
    wide = dict(heads_q=32, heads_kv=8, dim=128)
    return [
        # one token each of 64 running requests, positions anywhere in the context: the smallest call, latency
        dict(name="rotary decode 64", op="rotary", tokens=64, runs=64, reach=4096, heads=40, rest=8, dim=128,
             rotary_dim=128, layout="half", scaling="none", base=500000.0),
        # a full token budget of prefill chunks far into a long context, frequencies scaled by wavelength
        dict(name="rotary prefill 8192", op="rotary", tokens=8192, runs=3, reach=131072, heads=40, rest=8, dim=128,
             rotary_dim=128, layout="half", scaling="wavelength", base=500000.0),
        # neighbouring pairs, a quarter of a small head rotated, an odd number of tokens and heads
        dict(name="rotary part 1021", op="rotary", tokens=1021, runs=7, reach=60000, heads=7, rest=2, dim=64,
             rotary_dim=16, layout="interleaved", scaling="yarn", base=10000.0),
        # 64 running requests, one token each, into an int8 cache (most appends touch a partly filled block)
        dict(name="append decode int8", op="append", reqs=64, q_len=1, reach=4096, code="int8", rotary_dim=128,
             layout="half", scaling="none", base=500000.0, **wide),
        # two prefill chunks, one over cached context that ends inside a block, into E4M3 codes with block scales
        dict(name="append chunks e4m3", op="append", reqs=2, q_len=2048, reach=4100, code="e4m3", rotary_dim=128,
             layout="half", scaling="wavelength", base=500000.0, **wide),
        # the same budget into a bf16 cache
        dict(name="append prefill bf16", op="append", reqs=4, q_len=2048, reach=1, code="bf16", rotary_dim=64,
             layout="half", scaling="linear", base=10000.0, **wide),
        # a small step: ragged short chunks, few heads, neighbouring pairs
        dict(name="append small int8", op="append", reqs=5, q_len=37, reach=300, code="int8", rotary_dim=64,
             layout="interleaved", scaling="none", base=10000.0, heads_q=4, heads_kv=2, dim=64),
        # one request at its start, few heads: the smallest attention call
        dict(name="attend 1 x 33 int8", op="attend", reqs=1, q_len=1, lo=33, hi=33, code="int8", heads_q=4,
             heads_kv=2, dim=64),
        # an ordinary decode step
        dict(name="attend decode int8", op="attend", reqs=64, q_len=1, lo=512, hi=4096, code="int8", **wide),
        # a large decode step with verify rows of four tokens, E4M3 codes
        dict(name="attend verify e4m3", op="attend", reqs=128, q_len=4, lo=1024, hi=8000, code="e4m3", **wide),
        # few requests with a very long context: the split over keys, and the largest reads
        dict(name="attend long int8", op="attend", reqs=8, q_len=1, lo=131072, hi=131072, code="int8", heads_q=64,
             heads_kv=8, dim=128),
        # two prefill chunks over cached context: bound by arithmetic
        dict(name="attend chunks e4m3", op="attend", reqs=2, q_len=2048, lo=1024, hi=6144, code="e4m3", **wide),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _rope_of(rng, dim):
    return dict(rotary_dim=8 * rng.randint(1, dim // 8) if rng.random() < 0.5 else dim,
                layout=rng.choice(["half", "interleaved"]),
                scaling=rng.choice(["none", "linear", "wavelength", "yarn"]), base=rng.choice([10000.0, 500000.0]))


HEADS = [(32, 8, 128), (64, 8, 128), (4, 2, 64), (8, 8, 128), (16, 2, 64), (28, 4, 128), (32, 1, 128), (12, 3, 64)]


def draw(rng):
    op = rng.choice(["rotary", "append", "attend", "attend"])
    hq, hkv, d = rng.choice(HEADS)
    if op == "rotary":
        t = _log(rng, 1, 8192)
        return dict(op=op, tokens=t, runs=min(t, _log(rng, 1, 64)), reach=_log(rng, 1, 200000), heads=hq + hkv,
                    rest=rng.choice([0, hkv]), dim=d, **_rope_of(rng, d))
    if op == "append":
        r = _log(rng, 1, 256)
        return dict(op=op, reqs=r, q_len=_log(rng, 1, max(1, 8192 // r)), reach=_log(rng, 1, 20000),
                    code=rng.choice(["bf16", "int8", "int8", "e4m3", "e4m3"]), heads_q=hq, heads_kv=hkv, dim=d,
                    **_rope_of(rng, d))
    q = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, 1024)])
    hi = _log(rng, 1, 32768 if q <= 8 else 4096)
    room = min(4e8 / (hi * hkv * d), 8e8 / (hq * q * (hi + q)), 128 if q <= 8 else 4)
    return dict(op=op, reqs=max(1, _log(rng, 1, max(1.0, room))), q_len=q, lo=rng.randint(1, hi), hi=hi,
                code=rng.choice(["int8", "e4m3"]), heads_q=hq, heads_kv=hkv, dim=d)


# ------------------------------------------------------------------ inputs --
FACTOR, ORIGINAL, LOW, HIGH = 8.0, 8192, 1.0, 4.0       # wavelength scaling
BETA_FAST, BETA_SLOW = 32.0, 1.0                       # yarn


def _frequencies(c):
    """Angles per position of the rotary_dim / 2 pairs, and the factor on cos and sin."""
    n, base = c["rotary_dim"] // 2, c["base"]
    f = [base ** (-2.0 * i / c["rotary_dim"]) for i in range(n)]
    if c["scaling"] == "linear":
        return [x / FACTOR for x in f], 1.0
    if c["scaling"] == "wavelength":
        mix = [min(1.0, max(0.0, (ORIGINAL * x / (2 * math.pi) - LOW) / (HIGH - LOW))) for x in f]
        return [x / FACTOR * (1 - m) + x * m for x, m in zip(f, mix)], 1.0
    if c["scaling"] == "yarn":
        at = lambda turns: c["rotary_dim"] * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0, math.floor(at(BETA_FAST))), min(c["rotary_dim"] - 1, math.ceil(at(BETA_SLOW)))
        ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3))) for i in range(n)]
        return [x / FACTOR * r + x * (1 - r) for x, r in zip(f, ramp)], 0.1 * math.log(FACTOR) + 1.0
    return f, 1.0


def _rope(c):
    """The library's handle of a rotation."""
    from paged_kv_cache_16_gb300 import binding
    more = {"none": {}, "linear": dict(factor=FACTOR),
            "wavelength": dict(factor=FACTOR, original_max_position=ORIGINAL, low=LOW, high=HIGH),
            "yarn": dict(factor=FACTOR, original_max_position=ORIGINAL, low=BETA_SLOW, high=BETA_FAST)}[c["scaling"]]
    layout = binding.PA_ROPE_HALF if c["layout"] == "half" else binding.PA_ROPE_INTERLEAVED
    kind = {"none": binding.PA_ROPE_SCALE_NONE, "linear": binding.PA_ROPE_SCALE_LINEAR,
            "wavelength": binding.PA_ROPE_SCALE_WAVELENGTH, "yarn": binding.PA_ROPE_SCALE_YARN}[c["scaling"]]
    return binding.pa_rope_create(rotary_dim=c["rotary_dim"], layout=layout, base=c["base"], scaling=kind, **more)


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
    if code == "int8":
        return x.mul_(32).round_().clamp_(-127, 127).to(torch.int8)
    if code == "e4m3":
        return x.mul_(60).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.to(torch.bfloat16)


def _values(cache):
    """The numbers that a cache's codes stand for, without the scale, in 32 bits."""
    return cache.view(torch.float8_e4m3fn).float() if cache.dtype == torch.uint8 else cache.float()


def prepare(case, seed):
    c = case
    gen = torch.Generator("cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = dict(c=c, op=c["op"])
    i32 = lambda a: torch.as_tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    if c["op"] != "attend":
        f, s["mag"] = _frequencies(c)
        s["freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        s["rope"] = _rope(c) if own else None
    if c["op"] == "rotary":
        # rows of consecutive positions, each run starting somewhere in the reach
        t, n = c["tokens"], c["runs"]
        starts = rng.integers(0, c["reach"], n)
        begin = np.array([t * k // n for k in range(n + 1)])
        s["pos"] = i32(np.arange(t) + np.repeat(starts - begin[:-1], np.diff(begin)))
        packed = torch.randn(t, c["heads"] + c["rest"], c["dim"], generator=gen, device="cuda").to(torch.bfloat16)
        s["x"] = packed[:, :c["heads"]]
        s["out"] = torch.empty(t, c["heads"], c["dim"], dtype=torch.bfloat16, device="cuda")
        return s
    hq, hkv, d, r, q = c["heads_q"], c["heads_kv"], c["dim"], c["reqs"], c["q_len"]
    if c["op"] == "append":
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
        s.update(qsl=i32(qsl), nc=i32(nc), table=i32(table), t=t)
        packed = torch.randn(t, hq + 2 * hkv, d, generator=gen, device="cuda").to(torch.bfloat16)
        s.update(q=packed[:, :hq], k=packed[:, hq:hq + hkv], v=packed[:, hq + hkv:])
        s["q_out"] = torch.empty(t, hq, d, dtype=torch.bfloat16, device="cuda")
        shape = (nb, BLOCK, hkv, d)
        s.update(kc=_codes(shape, c["code"], gen), vc=_codes(shape, c["code"], gen))
        if c["code"] != "bf16":
            # scales that earlier appends left: mostly large enough for the new rows, some of them not
            e = torch.randint(-1, 2, (2, nb, hkv), generator=gen, device="cuda").float() - (4 if c["code"] == "int8" else 6)
            s.update(ks=torch.exp2(e[0]).contiguous(), vs=torch.exp2(e[1]).contiguous())
            s.update(kval=torch.empty(shape, dtype=torch.bfloat16, device="cuda"),
                     vval=torch.empty(shape, dtype=torch.bfloat16, device="cuda"))
        return s
    ctx = _lens(c, rng)
    seq = ctx + q
    need = -(-seq // BLOCK)
    at = np.concatenate([[0], np.cumsum(need)])
    nb = int(at[-1]) + 1
    ids = rng.permutation(nb)
    table = np.full((r, int(need.max())), ids[-1], dtype=np.int32)
    for k in range(r):
        table[k, :need[k]] = ids[at[k]:at[k + 1]]
    shape = (nb, BLOCK, hkv, d)
    s.update(table=i32(table), ctx=torch.as_tensor(ctx, device="cuda"), scale=d ** -0.5)
    s.update(kc=_codes(shape, c["code"], gen), vc=_codes(shape, c["code"], gen))
    unit = 1 / 32 if c["code"] == "int8" else 1 / 60
    sc = torch.exp(0.5 * torch.randn(2, nb, hkv, generator=gen, device="cuda")) * unit
    s.update(ks=sc[0].contiguous(), vs=sc[1].contiguous())
    s["q"] = torch.randn(r * q, hq, d, generator=gen, device="cuda").to(torch.bfloat16)
    s["out"] = torch.empty(r * q, hq, d, dtype=torch.bfloat16, device="cuda")
    if own:
        from paged_kv_cache_16_gb300 import binding
        kind = binding.PA_KV_INT8_BLOCK if c["code"] == "int8" else binding.PA_KV_FP8_E4M3_BLOCK
        s["plan"] = binding.pa_plan(num_heads_q=hq, num_heads_kv=hkv, head_dim=d, num_blocks=nb,
                                    query_start_loc=np.arange(r + 1) * q, seq_lens=seq, num_computed_tokens=ctx,
                                    block_table_host=table, softmax_scale=s["scale"], kv_cache_dtype=kind)
        s["ws"] = torch.zeros(s["plan"].workspace_bytes, dtype=torch.uint8, device="cuda")
        # once per step; every layer of the step then launches on it
        binding.pa_upload_metadata(s["plan"], s["ws"])
    return s


# ------------------------------------------------------------- plain forms --
def _rotated(x, pos, s):
    """Rows [T][H][D] rotated by their positions, in 32 bits (angles in 64)."""
    rd, half = s["c"]["rotary_dim"], s["c"]["rotary_dim"] // 2
    angle = pos.double()[:, None] * s["freq"]
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
    if code == "int8":
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
    pos = s["nc"][req] + (tok - s["qsl"][req])
    blk, off = s["table"][req, pos // BLOCK].long(), (pos % BLOCK).long()
    s["q_out"].copy_(_rotated(s["q"], pos, s))
    k = _rotated(s["k"], pos, s)
    if c["code"] == "bf16":
        s["kc"][blk, off] = k.to(torch.bfloat16)
        s["vc"][blk, off] = s["v"]
        return
    first = torch.full((s["kc"].shape[0],), BLOCK, device="cuda", dtype=torch.int64).index_reduce_(0, blk, off, "amin")
    _store(s["kc"], s["ks"], k, blk, off, first, c["code"])
    _store(s["vc"], s["vs"], s["v"].float(), blk, off, first, c["code"])


def _plain_attend(s):
    c = s["c"]
    r, n, hq, hkv, d = c["reqs"], c["q_len"], c["heads_q"], c["heads_kv"], c["dim"]
    table = s["table"].long()
    length = table.shape[1] * BLOCK

    def gathered(cache, scales):
        x = _values(cache[table]) * scales[table][:, :, None, :, None]
        return x.view(r, length, hkv, d).transpose(1, 2)                       # [R][Hkv][L][D]

    q = s["q"].float().view(r, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(r, hkv, -1, d)
    score = (q @ gathered(s["kc"], s["ks"]).transpose(2, 3) * s["scale"]).view(r, hkv, hq // hkv, n, length)
    limit = s["ctx"][:, None] + torch.arange(n, device="cuda") + 1              # token i sees keys below it
    seen = torch.arange(length, device="cuda") < limit[..., None]
    score = score.masked_fill_(~seen[:, None, None], -math.inf)
    w = torch.exp(score - score.amax(-1, keepdim=True))
    w = w / w.sum(-1, keepdim=True)
    out = w.view(r, hkv, -1, length) @ gathered(s["vc"], s["vs"])
    s["out"].copy_(out.view(r, hkv, hq // hkv, n, d).permute(0, 3, 1, 2, 4).reshape(r * n, hq, d))


def _append_outputs(s):
    """q, and the caches as the values that they stand for."""
    if s["c"]["code"] == "bf16":
        return dict(q=s["q_out"], k=s["kc"], v=s["vc"])
    number = (lambda x: x) if s["c"]["code"] == "int8" else (lambda x: x.view(torch.float8_e4m3fn).to(torch.bfloat16))
    torch.mul(number(s["kc"]), s["ks"][:, None, :, None], out=s["kval"])
    torch.mul(number(s["vc"]), s["vs"][:, None, :, None], out=s["vval"])
    return dict(q=s["q_out"], k=s["kval"], v=s["vval"], ks=s["ks"], vs=s["vs"])


def run(state):
    s = state
    if own:
        from paged_kv_cache_16_gb300 import binding
        if s["op"] == "rotary":
            binding.pa_rotary(s["rope"], s["x"], s["pos"], s["out"])
        elif s["op"] == "append":
            binding.pa_append_kv(s["rope"], s["k"], s["v"], s["qsl"], s["nc"], s["table"], s["kc"], s["vc"],
                                 key_scales=s.get("ks"), value_scales=s.get("vs"), q=s["q"], q_out=s["q_out"])
        else:
            binding.pa_attention_scaled_launch(s["plan"], s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"],
                                               s["out"], s["ws"])
    elif s["op"] == "rotary":
        s["out"].copy_(_rotated(s["x"], s["pos"], s))
    elif s["op"] == "append":
        _plain_append(s)
    else:
        _plain_attend(s)
    return _append_outputs(s) if s["op"] == "append" else s["out"]


# -------------------------------------------------------------------- work --
def work(case):
    c = case
    if c["op"] == "rotary":
        n = c["tokens"] * c["heads"] * c["dim"]
        return {"bytes": 4 * n + 4 * c["tokens"], "flops": 3 * c["tokens"] * c["heads"] * c["rotary_dim"]}
    hq, hkv, d, r, q = c["heads_q"], c["heads_kv"], c["dim"], c["reqs"], c["q_len"]
    es = 2 if c["code"] == "bf16" else 1
    if c["op"] == "append":
        t = int(_new_lens(c).sum())
        blocks = int(((_new_lens(c) + BLOCK - 1) // BLOCK).sum())
        return {"bytes": t * d * (4 * hq + 2 * hkv * (2 + es)) + 8 * r + blocks * (4 + (es == 1) * 16 * hkv),
                "flops": 3 * t * (hq + hkv) * c["rotary_dim"]}
    lens = _lens(c, np.random.default_rng(0))
    seq = int(lens.sum()) + r * q
    pairs = int(lens.sum()) * q + r * q * (q + 1) // 2
    return {"bytes": 2 * seq * hkv * d + 8 * (seq // BLOCK) * hkv + 4 * (seq // BLOCK) + 4 * r * q * hq * d,
            "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------- exact --
def _turned(x, pos, s):
    """The rotation as a product of complex numbers, in 64 bits."""
    c, rd = s["c"], s["c"]["rotary_dim"]
    x = x.double()
    part = x[..., :rd].unflatten(-1, (2, rd // 2)).transpose(-1, -2) if c["layout"] == "half" else x[..., :rd].unflatten(-1, (rd // 2, 2))
    angle = pos.double()[:, None, None] * s["freq"]
    z = torch.view_as_complex(part.contiguous()) * torch.polar(torch.full_like(angle, s["mag"]), angle)
    y = torch.view_as_real(z)
    y = y.transpose(-1, -2).flatten(-2) if c["layout"] == "half" else y.flatten(-2)
    return torch.cat([y, x[..., rd:]], -1)


def _nearest(x, code):
    """x rounded to the codes' values, ties to even, in 64 bits."""
    if code == "int8":
        return torch.clamp(torch.round(x), -127, 127)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    e = e + (x.abs() >= torch.exp2(e + 1)).double() - (x.abs().clamp(min=2.0 ** -6) < torch.exp2(e)).double()
    step = torch.exp2(e - 3)
    return torch.clamp(torch.round(x / step) * step, -448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "rotary":
        return _turned(s["x"], s["pos"], s)
    if c["op"] == "append":
        qsl, nc, table = s["qsl"].tolist(), s["nc"].tolist(), s["table"].tolist()
        pos = torch.cat([torch.arange(nc[k], nc[k] + qsl[k + 1] - qsl[k], device="cuda") for k in range(c["reqs"])])
        k64, v64 = _turned(s["k"], pos, s), s["v"].double()
        code = c["code"]
        val = {n: _values(s[n + "c"]).double() * (s[n + "s"].double()[:, None, :, None] if code != "bf16" else 1.0) for n in "kv"}
        sc = {n: s[n + "s"].double() for n in "kv"} if code != "bf16" else None
        for r in range(c["reqs"]):
            p = nc[r]
            while p < nc[r] + qsl[r + 1] - qsl[r]:
                end = min((p // BLOCK + 1) * BLOCK, nc[r] + qsl[r + 1] - qsl[r])
                b, o = table[r][p // BLOCK], p % BLOCK
                t0 = qsl[r] + p - nc[r]
                for n, rows in (("k", k64), ("v", v64)):
                    new = rows[t0:t0 + end - p]
                    if code == "bf16":
                        val[n][b, o:o + end - p] = new
                        continue
                    m = (new.abs().amax((0, 2)) / QMAX[code]).clamp(min=2.0 ** MIN_EXP)
                    scale = torch.exp2(torch.ceil(torch.log2(m)))
                    if o:
                        scale = torch.maximum(scale, sc[n][b])
                        val[n][b, :o] = _nearest(val[n][b, :o] / scale[:, None], code) * scale[:, None]
                    val[n][b, o:o + end - p] = _nearest(new / scale[:, None], code) * scale[:, None]
                    # rows behind the new ones keep their codes, under the new scale
                    rest = _values(s[n + "c"][b, o + end - p:]).double()
                    val[n][b, o + end - p:] = rest * scale[:, None]
                    sc[n][b] = scale
                p = end
        out = dict(q=_turned(s["q"], pos, s), k=val["k"], v=val["v"])
        return out if code == "bf16" else dict(out, ks=sc["k"], vs=sc["v"])
    n, hq, hkv, d = c["q_len"], c["heads_q"], c["heads_kv"], c["dim"]
    out = torch.empty(c["reqs"] * n, hq, d, dtype=torch.float64, device="cuda")
    ctx, g = s["ctx"].tolist(), hq // hkv
    for r in range(c["reqs"]):
        blocks = s["table"][r, :-(-(ctx[r] + n) // BLOCK)].long()
        for h in range(hkv):
            def whole(cache, scales):
                x = _values(cache[blocks, :, h]).double() * scales[blocks, h].double()[:, None, None]
                return x.reshape(-1, d)[:ctx[r] + n]
            k, v = whole(s["kc"], s["ks"]), whole(s["vc"], s["vs"])
            q = s["q"][r * n:(r + 1) * n, h * g:(h + 1) * g].double().transpose(0, 1)     # [G][n][D]
            z = torch.einsum("gnd,ld->gnl", q, k) * s["scale"]
            later = torch.arange(ctx[r] + n, device="cuda")[None] > ctx[r] + torch.arange(n, device="cuda")[:, None]
            z = torch.softmax(z.masked_fill(later[None], -math.inf), -1)
            out[r * n:(r + 1) * n, h * g:(h + 1) * g] = (z @ v).transpose(0, 1)
    return out
