"""Caches filled row by row with torch, for the tests of the scored and the shared-prefix attention:
every row that holds no live token is garbage (NaN; INT8: NaN scales)."""

from __future__ import annotations

import torch

from tests import plain_ops as plain

ACT = {"bf16": torch.bfloat16, "f32": torch.float32, "i8": torch.bfloat16}


class Built:
    """A one-layer cache (the last of `layers`) whose sequence b holds lens[b] tokens."""

    def __init__(self, kvc, layout, dtype, lens, H, KV, D, window=0, sinks=0, bs=16, rope="none", num_splits=0,
                 layers=2, spare=3, seed=0, tables=None, qstd=2.0, new=0, softmax_scale=0.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.kvc, self.layout, self.dtype, self.lens = kvc, layout, dtype, list(lens)
        self.H, self.KV, self.D, self.window, self.sinks, self.bs = H, KV, D, window, sinks, bs
        self.act, B = ACT[dtype], len(lens)
        self.layer = layers - 1
        self.scale = softmax_scale if softmax_scale > 0 else D ** -0.5
        maxb = blocks = 0
        if layout == "paged":
            # `tables`: logical to physical block of each sequence (list of lists); else private, shuffled blocks
            if tables is None:
                need = [-(-(n + new) // bs) for n in lens]
                perm = torch.randperm(sum(need) + spare, generator=torch.Generator().manual_seed(seed)).tolist()
                tables, at = [], 0
                for n in need:
                    tables.append(perm[at:at + n])
                    at += n
                blocks = len(perm)
            else:
                blocks = max([max(t) for t in tables if t] + [0]) + 1 + spare
            blocks += -blocks % 4
            maxb = max(max(len(t) for t in tables), 1) + 1
            self.table = torch.full((B, maxb), -1, dtype=torch.int32)
            for b, t in enumerate(tables):
                self.table[b, :len(t)] = torch.tensor(t, dtype=torch.int32)
            self.table = self.table.cuda()
        else:
            self.table = None
        self.d = kvc.make_desc(layout, rope, dtype, layers=layers, batch=B, q_heads=H, kv_heads=KV, head_dim=D,
                               window=window, sinks=sinks, block_size=bs if layout == "paged" else 0,
                               num_blocks=blocks, max_blocks_per_seq=maxb, num_splits=num_splits,
                               softmax_scale=softmax_scale)
        self.cache = kvc.alloc_cache(self.d, fill=float("nan"))
        self.values = {}      # physical row -> (k, v) [KV, D] float64, shared by the sequences that map it
        self.kv = []          # sequence -> position -> row key
        for b, n in enumerate(lens):
            live = plain.attended(layout, n - 1, window, sinks)
            keys = {}
            for p in live:
                keys[p] = (tables[b][p // bs], p % bs) if layout == "paged" else \
                    (b, plain.slot_of(layout, p, window, sinks))
            self.kv.append(keys)
        rows = sorted({k for keys in self.kv for k in keys.values()})
        if rows:
            i = torch.tensor([r[0] for r in rows], device="cuda")
            r = torch.tensor([r[1] for r in rows], device="cuda")
            vals = []
            for which in (0, 1):
                x = torch.randn(len(rows), KV, D, generator=g, device="cuda")
                if dtype == "i8":
                    codes, scales = kvc.int8_views(self.d, self.cache)
                    c = (x * 40).round().clamp(-127, 127)
                    s = (torch.rand(len(rows), KV, generator=g, device="cuda") + 0.5) / 40
                    codes[self.layer, which][i, :, r] = c.to(torch.int8)
                    scales[self.layer, which][i, :, r] = s
                    vals.append(c.double() * s.double()[..., None])
                else:
                    x = x.to(self.act)
                    self.cache[self.layer, which][i, :, r] = x
                    vals.append(x.double())
            self.index = {row: j for j, row in enumerate(rows)}
            self.k, self.v = vals
        self.q = (torch.randn(B, H, D, generator=g, device="cuda") * qstd).to(self.act)
        self.pos = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device="cuda")
        self.ws = kvc.alloc_workspace(self.d)

    def rows(self, b, ps):
        """K, V [len(ps), KV, D] float64 at positions ps of sequence b."""
        j = torch.tensor([self.index[self.kv[b][p]] for p in ps], dtype=torch.long, device="cuda")
        return self.k[j], self.v[j]

    def poison(self, b, ps):
        """Positions ps of sequence b become garbage in the cache."""
        for p in ps:
            i, r = self.kv[b][p]
            if self.dtype == "i8":
                _, scales = self.kvc.int8_views(self.d, self.cache)
                scales[self.layer, :, i, :, r] = float("nan")
            else:
                self.cache[self.layer, :, i, :, r] = float("nan")
