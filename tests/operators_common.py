"""Plain implementations in 64 bits of the rotary positions, the rotating
cache append and attention over block-scaled caches, with the tolerances their
kernels are held to, and builders of small cases."""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np
import torch

BLOCK = 16
QMAX = {"int8": 127.0, "e4m3": 448.0}
TWO_PI = Fraction(62831853071795864769252867665590057683943387987502116419498891846, 10 ** 64)
BF16 = 2.0 ** -8          # half a step of bf16, relative to the value


def cos_sin(freq, positions):
    """cos and sin of position * frequency, the angle reduced exactly: [T, n]."""
    c = np.empty((len(positions), len(freq)))
    s = np.empty_like(c)
    turns = [Fraction(float(f)) / TWO_PI for f in freq]
    for t, p in enumerate(positions):
        for i, f in enumerate(turns):
            x = f * int(p)
            a = 2 * math.pi * float(x - math.floor(x))
            c[t, i], s[t, i] = math.cos(a), math.sin(a)
    return c, s


def rotate(x, cs, rd, interleaved, mag=1.0):
    """Rows [T, H, D] (float64) rotated; also the magnitudes |x| + |y| that its
    errors scale with."""
    c, s = mag * cs[0][:, None], mag * cs[1][:, None]
    y, size = x.copy(), np.zeros_like(x)
    a, b = (slice(0, rd, 2), slice(1, rd, 2)) if interleaved else (slice(0, rd // 2), slice(rd // 2, rd))
    xa, xb = x[..., a], x[..., b]
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    size[..., a] = size[..., b] = mag * (np.abs(xa) + np.abs(xb))
    return y, size


# cos and sin in 32 bits: the angle's 2^-32 of a turn and its rounding to 24
# bits (2^-25 of half a turn: 9.4e-8), sincospif's 2 ulp (2.4e-7), the product
# by m and the two roundings of the combination (2^-24 each): below 6e-7 of
# |x| + |y| together
ROTATED = 6e-7


def power_scale(amax, code):
    """Smallest power of two, 2^-64 at least, with amax <= scale * QMAX."""
    s = 2.0 ** -64
    while amax > s * QMAX[code]:
        s *= 2
    return s


def values(codes, code):
    """float64 values of codes (int8 or uint8 E4M3 arrays)."""
    if code == "int8":
        return codes.astype(np.float64)
    return torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).double().numpy()


def nearest(x, code):
    """Values in units of the scale -> the nearest code values, ties to even."""
    if code == "int8":
        return np.clip(np.rint(x), -127, 127)
    a = np.abs(x)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    e = np.where(2.0 ** (e + 1) <= a, e + 1, e)
    step = 2.0 ** (e - 3)
    with np.errstate(invalid="ignore"):
        return np.where(np.isnan(x), np.nan, np.sign(x) * np.minimum(np.rint(a / step) * step, 448.0))


def half_step(v, code):
    """Half the distance from a code value to its next larger neighbour."""
    if code == "int8":
        return np.full_like(v, 0.5)
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    return 2.0 ** (e - 4)


# ----------------------------------------------------------- attention case --
class Case:
    """A step over block-scaled caches: rows of q_lens[r] query tokens that end
    contexts of seq_lens[r] tokens."""

    def __init__(self, *, hq, hkv, d, q_lens, seq_lens, code, scales="power", seed=0, shared=0, spare=3, q_size=1.0,
                 pad=-1):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.d, self.code, self.n_common = hq, hkv, d, code, shared
        self.q_lens, self.seq = np.asarray(q_lens), np.asarray(seq_lens)
        R = len(q_lens)
        need = -(-self.seq // BLOCK)
        nb = int(need.sum()) + spare
        ids = list(rng.permutation(nb))
        mb = max(1, int(need.max(initial=0)) + 1)
        self.table = np.full((R, mb), pad, dtype=np.int32)    # entries past a context are never read
        common = [ids.pop() for _ in range(shared)]
        for r in range(R):
            if self.q_lens[r] == 0 and shared:
                continue
            for b in range(int(need[r])):
                self.table[r, b] = common[b] if b < shared else ids.pop()
        self.nb = nb
        x = torch.randn(2, nb, BLOCK, hkv, d, generator=g)
        if code == "int8":
            codes = (x * 40).round().clamp(-128, 127).to(torch.int8)
            bad = 127
        else:
            codes = (x * 80).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            bad = 0x7F                                         # NaN
        self.kc, self.vc = codes[0].contiguous(), codes[1].contiguous()
        e = torch.randint(-2, 3, (2, nb, hkv), generator=g).double()
        if scales == "power":
            sc = 2.0 ** (e - 5)
        elif scales == "any":
            sc = 2.0 ** (e * 0.37 - 5.2)
        else:                                                  # values of very different blocks
            sc = 2.0 ** (e - 5)
            sc[1] = 2.0 ** (torch.randint(-40, 41, (nb, hkv), generator=g).double())
        sc = sc.float()
        used = np.zeros(nb, bool)
        for r in range(R):
            for b in range(int(need[r])):
                if self.table[r, b] < 0:
                    continue
                used[self.table[r, b]] = True
                if b == need[r] - 1 and self.seq[r] % BLOCK:   # slots past the context: anything
                    self.kc[self.table[r, b], self.seq[r] % BLOCK:] = bad
                    self.vc[self.table[r, b], self.seq[r] % BLOCK:] = bad
        sc[:, ~torch.from_numpy(used)] = float("nan")          # scales of unread blocks: anything
        self.ks, self.vs = sc[0].contiguous(), sc[1].contiguous()
        self.T = int(self.q_lens.sum())
        self.q = (torch.randn(max(self.T, 1), hq, d, generator=g) * q_size).to(torch.bfloat16)
        self.qsl = np.concatenate([[0], np.cumsum(self.q_lens)]).astype(np.int32)
        self.scale = d ** -0.5 / q_size

    def desc(self, **over):
        from paged_kv_cache_16_gb300 import binding
        kw = dict(num_heads_q=self.hq, num_heads_kv=self.hkv, head_dim=self.d, num_blocks=self.nb,
                  query_start_loc=self.qsl, seq_lens=self.seq, num_computed_tokens=self.seq - self.q_lens,
                  num_common_prefix_blocks=self.n_common, softmax_scale=self.scale, max_blocks_per_req=self.table.shape[1],
                  kv_cache_dtype=binding.PA_KV_INT8_BLOCK if self.code == "int8" else binding.PA_KV_FP8_E4M3_BLOCK)
        kw.update(over)
        return kw

    def reference(self):
        """(out, tolerance) [T, Hq, D] in float64.

        Per row: A = sum p |v|, S = scale * max_j sum_d |q_d k_jd|.  Scores: the
        fp32 accumulation of D products and the block-wise factors stay within
        2^-20 S, exponentials and logarithms add 2^-20; a score error e changes out
        by at most 2 e A.  Weights are rounded to f16: 2^-11 each, or 2^-24 absolute
        below its normal range, the largest weight times value scale being at least
        1 (n 2^-24 M, M = max p_j vs_j QMAX).  The output: half a bf16 step."""
        T, hq, d = max(self.T, 1), self.hq, self.d
        out, tol = np.zeros((T, hq, d)), np.zeros((T, hq, d))
        kv = [(values(c.numpy(), self.code), s.double().numpy()) for c, s in ((self.kc, self.ks), (self.vc, self.vs))]
        G = hq // self.hkv
        q = self.q.double().numpy()
        for r in range(len(self.q_lens)):
            blocks = self.table[r, :-(-int(self.seq[r]) // BLOCK)]
            for i in range(int(self.q_lens[r])):
                n = int(self.seq[r]) - int(self.q_lens[r]) + i + 1
                t = int(self.qsl[r]) + i
                for h in range(self.hkv):
                    k, v = [(c[blocks, :, h] * s[blocks, h][:, None, None]).reshape(-1, d)[:n] for c, s in kv]
                    vs = np.repeat(kv[1][1][blocks, h], BLOCK)[:n]
                    rows = q[t, h * G:(h + 1) * G]
                    z = rows @ k.T * self.scale
                    S = (np.abs(rows) @ np.abs(k).T).max(1) * self.scale
                    p = np.exp(z - z.max(1, keepdims=True))
                    p /= p.sum(1, keepdims=True)
                    o, A = p @ v, p @ np.abs(v)
                    M = (p * vs).max(1) * QMAX[self.code]
                    es = S * 2.0 ** -20 + 2.0 ** -20
                    out[t, h * G:(h + 1) * G] = o
                    tol[t, h * G:(h + 1) * G] = BF16 * np.abs(o) + A * (2.0 ** -11 + 2 * es[:, None]) + (n * 2.0 ** -24 * M)[:, None]
        return out, tol


class OnGpu:
    """The case's tensors, plan and workspace on cuda:0."""

    def __init__(self, case, **over):
        from paged_kv_cache_16_gb300 import binding
        dev = torch.device("cuda")
        self.case = case
        self.q, self.kc, self.vc, self.ks, self.vs = (t.to(dev) for t in (case.q, case.kc, case.vc, case.ks, case.vs))
        self.table = torch.from_numpy(case.table).to(dev)
        self.out = torch.full_like(self.q, 7.0)
        self.plan = binding.pa_plan(**case.desc(**over))
        self.ws = torch.zeros(self.plan.workspace_bytes, dtype=torch.uint8, device=dev)

    def args(self):
        return (self.q, self.kc, self.vc, self.ks, self.vs, self.table, self.out, self.ws)

    def run(self):
        from paged_kv_cache_16_gb300 import binding
        binding.pa_attention_scaled(self.plan, *self.args())
        torch.cuda.synchronize()
        assert binding.pa_check_device_errors(self.ws[:4].view(torch.int32)) == 0
        return self.out


def assert_within(got, ref, tol, what=""):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, worst {np.nanmax(np.abs(got - ref) / np.maximum(tol, 1e-300)):.3g} "
                           f"of the tolerance, first at {np.argwhere(bad)[0]}")


# -------------------------------------------------------------- append case --
class AppendCase:
    """New tokens of requests at num_computed[r], with block-scaled codes (or bf16,
    or E4M3 with one scale) in the cache already."""

    def __init__(self, *, hq, hkv, d, q_lens, computed, code, seed=0, packed=True, new_size=1.0, old_exp=None, spare=2):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.d, self.code = hq, hkv, d, code
        self.q_lens, self.nc = np.asarray(q_lens), np.asarray(computed)
        R, T = len(q_lens), int(np.sum(q_lens))
        self.T = T
        self.qsl = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        need = [-(-(int(n) + int(q)) // BLOCK) for n, q in zip(self.nc, self.q_lens)]
        nb = sum(need) + spare
        ids = rng.permutation(nb)
        self.table = np.full((R, max(need + [1])), -1, dtype=np.int32)
        at = 0
        for r in range(R):
            self.table[r, :need[r]] = ids[at:at + need[r]]
            at += need[r]
        self.nb = nb
        width = hq + 2 * hkv if packed else hq + 2 * hkv + 0
        rows = (torch.randn(max(T, 1), width, d, generator=g) * new_size).to(torch.bfloat16)
        self.q, self.key, self.value = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
        if not packed:
            self.q, self.key, self.value = (x.contiguous() for x in (self.q, self.key, self.value))
        x = torch.randn(2, nb, BLOCK, hkv, d, generator=g)
        if code == "int8":
            c = (x * 40).round().clamp(-127, 127).to(torch.int8)
        elif code == "bf16":
            c = x.to(torch.bfloat16)
        else:
            c = (x * 80).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        self.kc, self.vc = c[0].contiguous(), c[1].contiguous()
        lo, hi = old_exp or (-7, -3)
        e = torch.randint(lo, hi + 1, (2, nb, hkv), generator=g).float()
        self.ks, self.vs = torch.exp2(e[0]).contiguous(), torch.exp2(e[1]).contiguous()

    @property
    def scaled(self):
        return self.code in ("int8", "e4m3")

    def positions(self):
        return np.concatenate([np.arange(n, n + q) for n, q in zip(self.nc, self.q_lens)] or [np.zeros(0)]).astype(np.int64)

    def segments(self):
        """(block, first slot, first token, tokens) of every block that gets tokens."""
        for r in range(len(self.q_lens)):
            p, end = int(self.nc[r]), int(self.nc[r]) + int(self.q_lens[r])
            while p < end:
                n = min(end, (p // BLOCK + 1) * BLOCK) - p
                yield int(self.table[r, p // BLOCK]), p % BLOCK, int(self.qsl[r]) + p - int(self.nc[r]), n
                p += n
