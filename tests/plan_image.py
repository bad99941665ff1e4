"""A plan's work lists, read back from its metadata image."""
from __future__ import annotations

import numpy as np
import torch

from paged_kv_cache_16_gb300 import binding

BLOCK, KEY_TILE = 16, 128
ITEM = ("token", "req", "page_begin", "page_end", "key_end", "head_group", "part", "n_tok")
TILE = ("t0", "n_tok", "req", "pos0", "key_begin", "key_end", "kv_head", "part", "causal", "head", "skip", "split")
MERGE = ("token", "slot0", "count", "hq_begin", "hq_count", "pad0", "pad1", "pad2")
COUNTS = 8   # work counts at the image's head: tiles, merge rows, copied blocks, tokens, ...


def head_groups(hkv):
    return hkv // next(n for n in (8, 4, 2, 1) if hkv % n == 0)


class Image:
    """The lists of a plain plan (a fixed shape's lists lie at its capacities)."""

    def __init__(self, plan, hkv):
        info = plan.info()
        self.info, self.groups = info, head_groups(hkv)
        host = torch.zeros(binding.pa_plan_metadata_bytes(plan), dtype=torch.uint8)
        binding.pa_plan_copy_metadata(plan, host)
        raw, at = host.numpy(), 0

        def take(rows, names=None):
            nonlocal at
            n = rows * (len(names) if names else 1)
            x = np.frombuffer(raw[at:at + 4 * n].tobytes(), np.int32)
            at += -(-4 * n // 16) * 16
            return [dict(zip(names, map(int, r))) for r in x.reshape(rows, len(names))] if names else x

        self.counts = take(COUNTS)
        self.part_offset = take(info["num_tokens"] * self.groups)
        self.cta_begin = take(info["num_decode_ctas"] + 1)
        self.items = take(info["num_decode_items"], ITEM)
        self.tiles = take(info["num_extend_tiles"], TILE)
        self.merges = take(info["num_merge_rows"], MERGE)
