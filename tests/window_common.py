"""Steps whose queries see a sliding window and a few first tokens: small cases
over caches that hold the seen blocks alone, their plain implementation in 64
bits and the tolerance of the kernels."""
from __future__ import annotations

import numpy as np
import torch

import operators_common as oc

BLOCK = 16
KINDS = ("bf16", "e4m3", "e4m3_block", "int8_block")
SCALED = ("e4m3_block", "int8_block")
K_SCALE, V_SCALE = 0.031, 0.007          # of E4M3 caches with one scale


def seen(pos, window, sinks):
    """Which keys 0 .. pos a query at `pos` sees."""
    j = np.arange(pos + 1)
    return (pos - j < window) | (j < sinks)


class WindowCase:
    """q_lens[r] query tokens that end contexts of seq_lens[r] tokens.  Blocks that
    no query sees are not in the pool (their table entries are `pad`), and what no
    query sees of the others holds NaN (int8: the largest code)."""

    def __init__(self, *, hq, hkv, d, q_lens, seq_lens, window, sinks, code, seed=0, pad=-1, spare=3, hidden=True):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.d, self.code, self.window, self.sinks = hq, hkv, d, code, window, sinks
        self.q_lens, self.seq = np.asarray(q_lens), np.asarray(seq_lens)
        R = len(q_lens)
        keys = []                        # of each request: those that some query sees
        for r in range(R):
            s = np.zeros(max(int(self.seq[r]), 1), bool)
            for p in range(int(self.seq[r] - self.q_lens[r]), int(self.seq[r])):
                s[:p + 1] |= seen(p, window, sinks)
            keys.append(s)
        blocks = [np.unique(np.flatnonzero(s) // BLOCK) for s in keys]
        nb = sum(len(b) for b in blocks) + spare
        ids = list(rng.permutation(nb))
        mb = int((-(-self.seq // BLOCK)).max(initial=0)) + 1
        self.table = np.full((R, mb), pad, dtype=np.int32)
        self.nb = nb
        x = torch.randn(2, nb, BLOCK, hkv, d, generator=g)
        if code == "int8_block":
            c, bad = (x * 40).round().clamp(-128, 127).to(torch.int8), 127
        elif code == "bf16":
            c, bad = x.to(torch.bfloat16), float("nan")
        else:
            c, bad = (x * 80).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), 0x7F
        used = np.zeros(nb, bool)
        for r in range(R):
            for b in blocks[r]:
                i = self.table[r, b] = ids.pop()
                used[i] = True
                row = np.zeros(BLOCK, bool)
                part = keys[r][b * BLOCK:(b + 1) * BLOCK]
                row[:len(part)] = part
                if hidden:
                    c[:, i, torch.from_numpy(~row)] = bad
        if hidden:
            c[:, torch.from_numpy(~used)] = bad
        self.kc, self.vc = c[0].contiguous(), c[1].contiguous()
        sc = 2.0 ** (torch.randint(-2, 3, (2, nb, hkv), generator=g).float() * 0.37 - 5.2)
        if hidden:
            sc[:, torch.from_numpy(~used)] = float("nan")
        self.ks, self.vs = sc[0].contiguous(), sc[1].contiguous()
        self.T = int(self.q_lens.sum())
        self.q = torch.randn(max(self.T, 1), hq, d, generator=g).to(torch.bfloat16)
        self.qsl = np.concatenate([[0], np.cumsum(self.q_lens)]).astype(np.int32)
        self.scale = d ** -0.5

    @property
    def scaled(self):
        return self.code in SCALED

    def desc(self, **over):
        kw = dict(num_heads_q=self.hq, num_heads_kv=self.hkv, head_dim=self.d, num_blocks=self.nb,
                  query_start_loc=self.qsl, seq_lens=self.seq, num_computed_tokens=self.seq - self.q_lens,
                  softmax_scale=self.scale, max_blocks_per_req=self.table.shape[1], block_table_host=self.table,
                  kv_cache_dtype=KINDS.index(self.code), k_scale=K_SCALE, v_scale=V_SCALE, window=self.window,
                  sink_tokens=self.sinks)
        kw.update(over)
        return kw

    def values(self):
        """K and V of the pool in 64 bits."""
        if self.code == "bf16":
            return [c.double().numpy() for c in (self.kc, self.vc)]
        code = "int8" if self.code == "int8_block" else "e4m3"
        out = [oc.values(c.numpy(), code) for c in (self.kc, self.vc)]
        if self.scaled:
            return [v * s.double().numpy()[:, None, :, None] for v, s in zip(out, (self.ks, self.vs))]
        return [v * float(np.float32(s)) for v, s in zip(out, (K_SCALE, V_SCALE))]

    def reference(self):
        """(out, tolerance) [T, Hq, D] in 64 bits.

        Per row, with A = sum p |v| and S = scale * max_j sum_d |q_d k_jd|: a score is
        off by 2^-20 S + 2^-20 at most (fp32 sums of D products, exponentials), which
        changes out by twice that times A.  Weights are rounded to bf16 (2^-8 each,
        and as much through the sum of weights; E4M3 rows of the split-KV kernel to
        f16: less), over block scales to f16 (2^-11, or 2^-24 of the largest weight
        times value scale below f16's normal range).  The output: half a bf16 step."""
        out, tol = np.zeros((max(self.T, 1), self.hq, self.d)), np.zeros((max(self.T, 1), self.hq, self.d))
        kv = self.values()
        G = self.hq // self.hkv
        q = self.q.double().numpy()
        for r in range(len(self.q_lens)):
            for i in range(int(self.q_lens[r])):
                p = int(self.seq[r]) - int(self.q_lens[r]) + i
                keys = np.flatnonzero(seen(p, self.window, self.sinks))
                blk, off = self.table[r, keys // BLOCK], keys % BLOCK
                t = int(self.qsl[r]) + i
                for h in range(self.hkv):
                    k, v = (c[blk, off, h] for c in kv)
                    rows = q[t, h * G:(h + 1) * G]
                    z = rows @ k.T * self.scale
                    S = (np.abs(rows) @ np.abs(k).T).max(1) * self.scale
                    w = np.exp(z - z.max(1, keepdims=True))
                    w /= w.sum(1, keepdims=True)
                    o, A = w @ v, w @ np.abs(v)
                    es = (S * 2.0 ** -20 + 2.0 ** -20)[:, None]
                    e = A * ((2.0 ** -11 if self.scaled else 2.0 ** -7) + 2 * es) + oc.BF16 * np.abs(o)
                    if self.scaled:
                        vs = self.vs.double().numpy()[blk, h]
                        e = e + (len(keys) * 2.0 ** -24 * (w * vs).max(1) * 448.0)[:, None]
                    out[t, h * G:(h + 1) * G], tol[t, h * G:(h + 1) * G] = o, e
        return out, tol


class OnGpu:
    """The case's tensors, plan and workspace on cuda:0."""

    def __init__(self, case, shape=None, **over):
        from paged_kv_cache_16_gb300 import binding
        dev = torch.device("cuda")
        self.case = case
        self.q, self.kc, self.vc, self.ks, self.vs = (t.to(dev) for t in (case.q, case.kc, case.vc, case.ks, case.vs))
        if shape is not None:            # q and out hold a fixed shape's rows
            self.q = torch.cat([self.q, self.q.new_zeros(shape["max_tokens"] - self.q.shape[0], *self.q.shape[1:])])
        self.table = torch.from_numpy(case.table).to(dev)
        self.out = torch.full_like(self.q, 7.0)
        self.plan = binding.pa_plan_window(shape=shape, **case.desc(**over))
        self.ws = torch.zeros(self.plan.workspace_bytes, dtype=torch.uint8, device=dev)

    def call(self, launch=False):
        from paged_kv_cache_16_gb300 import binding
        c = self.case
        if c.scaled:
            f = binding.pa_attention_scaled_launch if launch else binding.pa_attention_scaled
            f(self.plan, self.q, self.kc, self.vc, self.ks, self.vs, self.table, self.out, self.ws)
        else:
            f = binding.pa_attention_launch if launch else binding.pa_attention
            f(self.plan, self.q, self.kc, self.vc, self.table, self.out, self.ws)

    def run(self):
        from paged_kv_cache_16_gb300 import binding
        self.call()
        torch.cuda.synchronize()
        assert binding.pa_check_device_errors(self.ws[:4].view(torch.int32)) == 0
        return self.out


def check(case, **over):
    g = OnGpu(case, **over)
    out = g.run()
    ref, tol = case.reference()
    oc.assert_within(out[:case.T], ref[:case.T], tol[:case.T])
    return g
