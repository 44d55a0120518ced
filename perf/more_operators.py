"""Cases of the operators for drafted tokens and for long caches read or kept in part, with their plain forms.

Six operators, all on the caches of include/kvc.h:

  bounds   largest and smallest key of each block, channel by channel, in 8 bits (kvc.block_bounds);
  sparse   blocks chosen by what those bounds allow a query's score to be, and decode attention
           over the chosen ones (kvc.select_blocks, kvc.decode_attention_selected);
  weighed  decode attention that adds up how much weight each block received
           (kvc.decode_attention_weighed);
  evict    the lightest blocks of each sequence given back (kvc.block_evict);
  tree     attention of a tree of drafted tokens over the cache (kvc.tree_attention);
  path     the accepted path's keys and values appended (kvc.append_path).

`run` computes them in elementary torch operations in fp32, or (own) with the library's calls.
"""

import math

import torch

own = False

ELT = {"bf16": 2, "f32": 4, "i8": 1}
ACT = {"bf16": torch.bfloat16, "f32": torch.float32, "i8": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a step of the 64-sequence paged batch: each sequence's newest block summarised again
        dict(name="bounds_step", op="bounds", layout="paged", dtype="bf16", batch=64, kv_heads=8, q_heads=32,
             head_dim=128, block_size=16, lo=256, hi=2048, n_new=1),
        # the blocks of a ragged prompt chunk, right after it was appended
        dict(name="bounds_prompt", op="bounds", layout="paged", dtype="bf16", batch=8, kv_heads=8, q_heads=32,
             head_dim=128, block_size=16, lo=0, hi=3000, n_new=8192),
        # the paged batch grown long: 2048 tokens of each sequence and kv head attended
        dict(name="sparse_batch", op="sparse", layout="paged", dtype="bf16", batch=64, kv_heads=8, q_heads=32,
             head_dim=128, block_size=16, lo=2048, hi=16384, k=128, first=1, recent=4, holes=False),
        # two very long sequences on the INT8 cache
        dict(name="sparse_long_i8", op="sparse", layout="paged", dtype="i8", batch=2, kv_heads=4, q_heads=16,
             head_dim=256, block_size=64, lo=60000, hi=131072, k=64, first=1, recent=2, holes=True),
        # the paged batch with the weight of every block kept
        dict(name="weighed_batch", op="weighed", layout="paged", dtype="bf16", batch=64, kv_heads=8, q_heads=32,
             head_dim=128, block_size=16, lo=512, hi=8192, holes=False, decay=1.0),
        # few long sequences on the INT8 cache, some of whose blocks were given back before
        dict(name="weighed_long_i8", op="weighed", layout="paged", dtype="i8", batch=3, kv_heads=4, q_heads=16,
             head_dim=256, block_size=64, lo=20000, hi=65536, holes=True, decay=0.9),
        # the paged batch cut back to 256 blocks a sequence; pairs of sequences share a prompt
        dict(name="evict_batch", op="evict", layout="paged", dtype="bf16", batch=64, kv_heads=8, q_heads=32,
             head_dim=128, block_size=16, lo=3000, hi=8192, prefix=512, keep=256, first=4, recent=8),
        # two sequences of up to a million tokens
        dict(name="evict_long", op="evict", layout="paged", dtype="bf16", batch=2, kv_heads=8, q_heads=32,
             head_dim=128, block_size=16, lo=500000, hi=1000000, prefix=0, keep=20000, first=4, recent=64),
        # drafts of 32 tokens over full sliding-window rings
        dict(name="tree_ring", op="tree", layout="ring", dtype="bf16", batch=8, kv_heads=8, q_heads=32,
             head_dim=128, window=4096, sinks=0, lo=4097, hi=65536, n_new=32, holes=False),
        # one long sequence with the widest tree
        dict(name="tree_long", op="tree", layout="paged", dtype="bf16", batch=1, kv_heads=8, q_heads=32,
             head_dim=128, block_size=16, lo=100003, hi=100003, n_new=64, holes=False),
        # the accepted paths of the paged batch
        dict(name="path_batch", op="path", layout="paged", dtype="bf16", batch=64, kv_heads=8, q_heads=32,
             head_dim=128, block_size=16, lo=512, hi=8192, n_new=32, most=8),
        # the small fp32 sink cache of the configurations
        dict(name="path_sink_f32", op="path", layout="sink_ring", dtype="f32", batch=5, kv_heads=1, q_heads=4,
             head_dim=64, window=60, sinks=4, lo=1, hi=300, n_new=7, most=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["bounds", "sparse", "weighed", "evict", "tree", "path"])
    D = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    q_heads = kv * rng.choice([g for g in (1, 2, 3, 4, 8) if g * kv <= 32])
    c = dict(op=op, layout="paged", dtype="bf16", head_dim=D, kv_heads=kv, q_heads=q_heads)
    if op in ("bounds", "path"):
        c["dtype"] = rng.choice(["bf16", "bf16", "f32", "i8"] if D >= 128 else ["bf16", "f32"])
    elif op in ("sparse", "weighed"):
        c["dtype"] = rng.choice(["bf16", "bf16", "i8"] if D >= 128 else ["bf16"])
    if op in ("tree", "path"):
        c["layout"] = rng.choice(["ring", "sink_ring", "paged", "paged"])
    if c["layout"] == "paged":
        # odd block sizes where any is taken (INT8 rows come in fours)
        c["block_size"] = rng.choice([8, 16, 32, 64] if op == "tree" else [8, 12, 16, 24, 32, 64])
    else:
        c["sinks"] = 4 if c["layout"] == "sink_ring" else 0
        c["window"] = 4 * _log(rng, 16, 1024) - c["sinks"]
    if op == "bounds":
        c["batch"] = _log(rng, 1, 64)
        c["n_new"] = rng.choice([1, _log(rng, 2, max(2, 20000 // c["batch"]))])
        c["lo"], c["hi"] = 0, _log(rng, 16, 4000)
    elif op == "evict":
        c["batch"] = _log(rng, 1, 64)
        mean = max(4, _log(rng, 64, 40000) // c["batch"])              # blocks of a sequence
        c["lo"] = c["block_size"] * max(2, int(mean * rng.uniform(0.2, 1.0))) - rng.randint(0, c["block_size"] - 1)
        c["hi"] = c["lo"] + 2 * c["block_size"] * int(mean * rng.uniform(0.0, 0.5))
        c["first"], c["recent"] = rng.randint(0, 4), rng.randint(1, 8)
        c["keep"] = c["first"] + c["recent"] + _log(rng, 1, mean)
        c["prefix"] = c["block_size"] * rng.choice([0, (c["lo"] // c["block_size"]) // 2])
    elif op == "path":
        c["batch"] = _log(rng, 1, 64)
        c["n_new"] = _log(rng, 1, 64)
        c["most"] = rng.randint(1, min(16, c["n_new"], c.get("window", 64)))
        c["lo"], c["hi"] = 0, _log(rng, 16, 4000)
    elif op == "tree":
        c["batch"] = _log(rng, 1, 32)
        c["n_new"] = min(_log(rng, 1, 64), c.get("window", 64))
        mean = max(2, _log(rng, 64, 60000) // c["batch"])
        c["lo"] = max(0, int(mean * rng.uniform(0.0, 1.0)))
        c["hi"] = 2 * mean - c["lo"]
        c["holes"] = c["layout"] == "paged" and rng.random() < 0.3
    else:
        c["batch"] = _log(rng, 1, 64)
        mean = max(2, _log(rng, 64, 120000 if op == "sparse" else 60000) // c["batch"])
        c["lo"] = max(1, int(mean * rng.uniform(0.2, 1.0)))
        c["hi"] = 2 * mean - c["lo"]
        c["holes"] = rng.random() < 0.3
        if op == "sparse":
            c["first"], c["recent"] = rng.randint(0, 2), rng.randint(1, 4)
            c["k"] = c["first"] + c["recent"] + _log(rng, 1, max(1, min(2048, mean) // c["block_size"]))
        else:
            c["decay"] = rng.choice([0.0, 0.9, 1.0])
    return c


def _lengths(case):
    """Tokens of each sequence before the call (bounds, tree, path) or with the one decoded, spread over
    [lo, hi] by the golden ratio, the same for every seed."""
    n, lo, hi = case["batch"], case["lo"], case["hi"]
    return [lo + int((hi - lo + 1) * ((i * 0.6180339887498949 + 0.37) % 1.0)) for i in range(n)]


def _news(case):
    """Ragged counts 1 .. the most of a padded batch (the most itself among them)."""
    n, most = case["batch"], case.get("most", case["n_new"])
    return [most if i == 0 else max(1, most - int(most * 0.6 * ((i * 0.6180339887498949) % 1.0))) for i in range(n)]


def _hole(case, b, lb, nb):
    """Blocks that an earlier eviction took: every fifth of every other sequence, never the first or the last."""
    return bool(case.get("holes")) and b % 2 == 0 and lb % 5 == 3 and lb < nb - 1


def _rows(case, b, L):
    """Rows that the last of L tokens of sequence b attends in a paged cache."""
    bs = case["block_size"]
    nb = -(-L // bs)
    return L - bs * sum(_hole(case, b, lb, nb) for lb in range(nb))


def work(case):
    D, H, KV, B = case["head_dim"], case["q_heads"], case["kv_heads"], case["batch"]
    e, a = ELT[case["dtype"]], 4 if case["dtype"] == "f32" else 2
    half = D * e + (4 if case["dtype"] == "i8" else 0)                # a K or V row of one kv head
    lens, op = _lengths(case), case["op"]
    bs = case.get("block_size", 0)
    if op == "bounds":
        rows = blocks = 0
        for L, n in zip(lens, _news(case)):
            first = L // bs
            rows += L + n - first * bs
            blocks += (L + n - 1) // bs - first + 1
        return {"bytes": KV * (rows * half + blocks * (2 * D + 4)), "flops": 2 * KV * rows * D}
    if op == "sparse":
        scored = chosen = 0
        for b, L in enumerate(lens):
            nb = -(-L // bs)
            live = nb - sum(_hole(case, b, lb, nb) for lb in range(nb))
            k = min(live, case["k"])
            scored += live
            chosen += k * bs - (nb * bs - L)
        return {"bytes": KV * (scored * (2 * D + 4) + chosen * 2 * half + B * case["k"] * 4) + 2 * B * H * D * a,
                "flops": H * D * (2 * scored + 4 * chosen)}
    if op == "weighed":
        rows = sum(_rows(case, b, L) for b, L in enumerate(lens))
        return {"bytes": rows * KV * 2 * half + 2 * B * H * D * a + 8 * sum(-(-L // bs) for L in lens),
                "flops": 4 * rows * H * D}
    if op == "evict":
        return {"bytes": 8 * sum(-(-L // bs) for L in lens), "flops": sum(-(-L // bs) for L in lens)}
    T = case["n_new"]
    if op == "tree":
        if case["layout"] == "paged":
            cached = sum(_rows(case, b, L) for b, L in enumerate(lens))
        else:
            cached = sum(min(L, case["window"] - 1 + case["sinks"]) for L in lens)
        return {"bytes": cached * KV * 2 * half + B * T * (2 * H * D * a + 2 * KV * D * a),
                "flops": 4 * H * D * T * (cached + B)}
    n = sum(_news(case))
    return {"bytes": n * KV * (2 * D * a + 2 * half), "flops": n * KV * D}


# ------------------------------------------------------------------ inputs
def _table(case, need, g, prefix=0):
    """Block table [batch, max blocks] over a random permutation of the physical blocks; sequences 2 i and
    2 i + 1 share the first `prefix` blocks."""
    bs, B = case["block_size"], case["batch"]
    nb = [max(1, -(-n // bs)) for n in need]
    maxb = max(nb)
    total = sum(n - (prefix if b % 2 else 0) for b, n in enumerate(nb))
    rows, at, last = [], 0, []
    for b in range(B):
        take = prefix if b % 2 else 0
        row = last[:take] + list(range(at, at + nb[b] - take))
        at += nb[b] - take
        last = row
        rows.append([-1 if _hole(case, b, lb, nb[b]) else x for lb, x in enumerate(row)] + [-1] * (maxb - nb[b]))
    table = torch.tensor(rows, dtype=torch.int64).cuda()
    perm = torch.randperm(total, generator=g, device="cuda")
    return torch.where(table >= 0, perm[table.clamp(min=0)], table).to(torch.int32), total


def _parents(case, seed):
    """Trees of drafted tokens: each token continues one of those a few places before it, some sequences a plain
    chain, a few tokens of every third sequence padding (-2)."""
    T, B = case["n_new"], case["batch"]
    g = torch.Generator().manual_seed(seed)
    back = torch.randint(1, 9, (B, T), generator=g)
    p = torch.arange(T)[None] - torch.where(torch.arange(B)[:, None] % 4 == 3, 1, back)
    p = p.clamp(min=-1)
    pad = (torch.arange(B)[:, None] % 3 == 2) & (torch.arange(T)[None] >= max(1, T - T // 4))
    return torch.where(pad, -2, p).to(torch.int32)


def _paths(case, parent):
    """One path from a root of each tree: from its first token on, always the next token that continues it."""
    B, T = parent.shape
    news = _news(case)
    rows = []
    for b in range(B):
        par, path = parent[b].tolist(), []
        for i in range(T):
            if len(path) < news[b] and par[i] == (path[-1] if path else -1):
                path.append(i)
        rows.append(path)
    n = torch.tensor([len(r) for r in rows], dtype=torch.int32)
    return torch.tensor([r + [0] * (case["most"] - len(r)) for r in rows], dtype=torch.int32), n


def _step(most):
    """The step of 8-bit codes up to `most`: a correctly rounded quotient (a division by a Python number is a product
    with its reciprocal)."""
    return most / torch.full((), 127.0, device="cuda")


def _summaries(case, cache_rows):
    """Bounds [blocks, kv heads, 2 (largest, smallest), D] as codes and scales of key rows [blocks, kv heads, bs, D]."""
    hi, lo = cache_rows.amax(2).float(), cache_rows.amin(2).float()
    scale = _step(torch.maximum(hi.abs().amax(-1), lo.abs().amax(-1)))
    s = torch.where(scale > 0, scale, 1.0)[..., None]
    codes = torch.stack([torch.ceil(hi / s).clamp(max=127), torch.floor(lo / s).clamp(min=-127)], 2)
    return codes.to(torch.int8), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    D, H, KV, B, op = case["head_dim"], case["q_heads"], case["kv_heads"], case["batch"], case["op"]
    act = ACT[case["dtype"]]
    lens = _lengths(case)

    def normal(*shape, std=1.0, dtype=act):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    s = dict(case=case)
    T = case.get("n_new", 1)
    blocks = 0
    paged = case["layout"] == "paged"
    if paged:
        more = {"bounds": T, "path": case.get("most", 0)}.get(op, 0)
        s["table"], blocks = _table(case, [n + more for n in lens], g, case.get("prefix", 0) // case["block_size"])
        shape = (1, 2, blocks, KV, case["block_size"], D)
    else:
        shape = (1, 2, B, KV, case["window"] + case["sinks"], D)
    s["pos"] = torch.tensor([n if op in ("bounds", "tree", "path") else n - 1 for n in lens], dtype=torch.int32,
                            device="cuda")
    if op == "evict":
        # the block manager's state, in one buffer so that one copy renews what a pass changes
        maxb, free = s["table"].shape[1], blocks // 8
        # weights in quarters: many blocks weigh the same
        w = (torch.rand(B, maxb, generator=g, device="cuda").pow(3) * 200.0).round() / 4
        w = torch.where(s["table"] >= 0, w, 0.0)
        ref = torch.bincount(s["table"][s["table"] >= 0].long(), minlength=blocks).to(torch.int32)
        total = blocks + free
        ref = torch.cat([ref, ref.new_zeros(free)])
        stack = torch.full((total,), -1, dtype=torch.int32, device="cuda")
        stack[:free] = torch.arange(blocks, total, dtype=torch.int32, device="cuda")
        words = (total + 31) // 32
        bits = torch.zeros(words * 32, dtype=torch.int64, device="cuda")
        bits[:blocks] = 1
        valid = (bits.view(words, 32) << torch.arange(32, device="cuda")).sum(1)
        valid = torch.where(valid >= 2 ** 31, valid - 2 ** 32, valid).to(torch.int32)
        count = torch.tensor([free], dtype=torch.int32, device="cuda")
        parts, at = [], 0
        for x in (s["table"], w.view(torch.int32), ref, stack, count, valid):
            pad = -x.numel() % 4
            parts.append(torch.cat([x.flatten(), x.new_zeros(pad)]))
        s["base"] = torch.cat(parts)
        s["work"] = s["base"].clone()
        names = ("table", "weights", "refcount", "free_list", "free_count", "valid")
        for name, x, part in zip(names, (s["table"], w, ref, stack, count, valid), parts):
            view = s["work"][at:at + x.numel()].view(x.shape)
            s[name] = view.view(torch.float32) if name == "weights" else view
            at += part.numel()
        blocks = total
    else:
        # keys of a block have something in common
        top = normal(*shape[2:4], 1, D, std=0.7, dtype=torch.float32) if paged else 0.0
        if case["dtype"] == "i8":
            # codes, then the row scales: one flat buffer, as the library lays an INT8 cache out
            n = math.prod(shape)
            s["cache"] = torch.empty(n + 4 * (n // D), dtype=torch.uint8, device="cuda")
            s["codes"] = s["cache"][:n].view(torch.int8).view(shape)
            s["scales"] = s["cache"][n:].view(torch.float32).view(shape[:-1])
            for c in (0, 1):
                x = normal(*shape[2:], std=0.7, dtype=torch.float32)
                x += top if c == 0 else 0.0
                s["codes"][0, c] = (x * 32).round_().clamp_(-127, 127).to(torch.int8)
                del x
            s["scales"].copy_((torch.rand(shape[:-1], generator=g, device="cuda") + 0.5) / 32.0)
        else:
            s["cache"] = torch.empty(shape, dtype=act, device="cuda")
            for c in (0, 1):
                x = normal(*shape[2:], std=0.7, dtype=torch.float32)
                x += top if c == 0 else 0.0
                s["cache"][0, c].copy_(x)
                del x
    if op in ("sparse", "weighed"):
        s["q"] = normal(B, H, D, std=1.5)
    if op == "sparse":
        k = s["cache"][0, 0] if case["dtype"] != "i8" else s["codes"][0, 0].float() * s["scales"][0, 0][..., None]
        codes, scale = _summaries(case, k)
        del k
        # as the library lays them out: codes, then scales
        s["bounds"] = torch.cat([codes.flatten().view(torch.uint8), scale.flatten().view(torch.uint8)])
        s["b_codes"] = s["bounds"][:codes.numel()].view(torch.int8).view(codes.shape)
        s["b_scale"] = s["bounds"][codes.numel():].view(torch.float32).view(scale.shape)
    elif op == "bounds":
        n = blocks * KV * 2 * D
        s["bounds"] = torch.zeros(n + 4 * blocks * KV, dtype=torch.uint8, device="cuda")
        s["b_codes"] = s["bounds"][:n].view(torch.int8).view(blocks, KV, 2, D)
        s["b_scale"] = s["bounds"][n:].view(torch.float32).view(blocks, KV)
        s["n_tok"] = torch.tensor(_news(case), dtype=torch.int32, device="cuda")
    elif op == "weighed":
        s["base"] = torch.rand(s["table"].shape, generator=g, device="cuda") * 8.0
        s["weights"] = torch.empty_like(s["base"])
    elif op in ("tree", "path"):
        s["k"], s["v"] = normal(B, T, KV, D), normal(B, T, KV, D)
        parent = _parents(case, seed)
        s["parent"] = parent.cuda()
        if op == "tree":
            s["q"] = normal(B, T, H, D, std=1.5)
        else:
            path, n = _paths(case, parent)
            s["path"], s["n_path"] = path.cuda(), n.cuda()
    if own:
        import sliding_window_attention_kvc_gb300 as kvc
        s["kvc"] = kvc
        d = s["d"] = kvc.make_desc(case["layout"], "none", case["dtype"], layers=1, batch=B, q_heads=H, kv_heads=KV,
                                   head_dim=D, window=case.get("window", 0), sinks=case.get("sinks", 0),
                                   block_size=case.get("block_size", 0), num_blocks=blocks,
                                   max_blocks_per_seq=s["table"].shape[1] if paged else 0)
        if op == "sparse":
            s["ws"] = kvc.alloc_select_workspace(d, case["k"])
        elif op == "weighed":
            s["ws"] = kvc.alloc_weighed_workspace(d)
        elif op == "tree":
            s["ws"] = kvc.alloc_tree_workspace(d, T)
        else:
            s["ws"] = kvc.alloc_workspace(d)
        if op == "evict":
            state = s["state"] = kvc.BlockState.__new__(kvc.BlockState)
            state.table, state.valid_bits, state.refcount = s["table"], s["valid"], s["refcount"]
            state.free_list, state.free_count = s["free_list"], s["free_count"]
    return s


# ------------------------------------------------------------------ plain forms
def _read(s, which, i, r):
    """K (0) or V (1) rows [..., KV, D] of the cache, fp32, at blocks (or sequences) i and rows r."""
    if s["case"]["dtype"] == "i8":
        return s["codes"][0, which][i, :, r].float() * s["scales"][0, which][i, :, r][..., None]
    return s["cache"][0, which][i, :, r].float()


def _softmax(z, ok):
    """exp(z - max) where ok, and its sum; rows without a key: zeros."""
    z.masked_fill_(~ok, -math.inf)
    m = z.amax(-1, keepdim=True).clamp(min=-1e30)
    z.sub_(m).exp_()
    return z, z.sum(-1, keepdim=True)


def _plain_bounds(s):
    case = s["case"]
    bs, maxb = case["block_size"], s["table"].shape[1]
    p0, end = s["pos"].long(), s["pos"].long() + s["n_tok"].long()
    # touched blocks of each sequence, padded with the first one again
    most = (case["n_new"] + bs - 1) // bs + 1
    lb = p0[:, None] // bs + torch.arange(most, device="cuda")[None]
    lb = torch.where(lb * bs < end[:, None], lb, p0[:, None] // bs).clamp(max=maxb - 1)
    phys = s["table"].gather(1, lb).long()
    k = s["cache"][0, 0] if case["dtype"] != "i8" else s["codes"][0, 0]
    k = k[phys].float()                                               # [B, most, KV, bs, D]
    if case["dtype"] == "i8":
        k = k * s["scales"][0, 0][phys][..., None]
    live = (lb[..., None] * bs + torch.arange(bs, device="cuda") < end[:, None, None])[:, :, None, :, None]
    hi = k.masked_fill(~live, -math.inf).amax(3)
    lo = k.masked_fill(~live, math.inf).amin(3)
    scale = _step(torch.maximum(hi.abs().amax(-1), lo.abs().amax(-1)))
    d = torch.where(scale > 0, scale, 1.0)[..., None]
    s["b_codes"][phys] = torch.stack([torch.ceil(hi / d).clamp(max=127), torch.floor(lo / d).clamp(min=-127)],
                                     3).to(torch.int8)
    s["b_scale"][phys] = scale
    return s["b_codes"] * s["b_scale"][..., None, None]


def _plain_select(s):
    case = s["case"]
    B, H, KV, D = case["batch"], case["q_heads"], case["kv_heads"], case["head_dim"]
    q = s["q"].float()
    sq = _step(q.abs().amax(-1))
    code = torch.round(q / torch.where(sq > 0, sq, 1.0)[..., None]).clamp(-127, 127).view(B, KV, H // KV, D)
    phys = s["table"].clamp(min=0).long()
    hi = s["b_codes"][:, :, 0][phys].float().permute(0, 2, 3, 1)       # [B, KV, D, blocks]
    lo = s["b_codes"][:, :, 1][phys].float().permute(0, 2, 3, 1)
    u = torch.matmul(code.clamp(min=0), hi) + torch.matmul(code.clamp(max=0), lo)
    scale = sq.view(B, KV, H // KV, 1) * s["b_scale"][phys].permute(0, 2, 1)[:, :, None]
    score = (u * scale).amax(2)                                        # [B, KV, blocks]
    lb = torch.arange(phys.shape[1], device="cuda")[None]
    nb = (s["pos"].long() // case["block_size"] + 1)[:, None]
    live = (s["table"] >= 0) & (lb < nb)
    forced = (lb < case["first"]) | (lb >= nb - case["recent"])
    score = torch.where(forced[:, None], math.inf, score)
    score = torch.where(live[:, None], score, -math.inf)
    value, index = torch.sort(score, dim=-1, descending=True, stable=True)
    k = min(case["k"], phys.shape[1])
    none = phys.shape[1]
    index = torch.where(value[..., :k] > -math.inf, index[..., :k], none).sort(-1).values
    index = torch.where(index < none, index, -1)
    return torch.cat([index, index.new_full((B, KV, case["k"] - k), -1)], -1).to(torch.int32)


def _plain_selected(s, blocks):
    case = s["case"]
    B, H, KV, D, bs = case["batch"], case["q_heads"], case["kv_heads"], case["head_dim"], case["block_size"]
    lb = blocks.long()
    phys = s["table"].gather(1, lb.clamp(min=0).flatten(1)).view(lb.shape).long()
    head = torch.arange(KV, device="cuda")[None, :, None].expand_as(phys)
    if case["dtype"] == "i8":
        k, v = (s["codes"][0, c][phys, head].float() * s["scales"][0, c][phys, head][..., None] for c in (0, 1))
    else:
        k, v = (s["cache"][0, c][phys, head].float() for c in (0, 1))
    p = lb[..., None] * bs + torch.arange(bs, device="cuda")
    ok = ((lb >= 0)[..., None] & (p <= s["pos"].long()[:, None, None, None])).flatten(2)
    k, v = k.flatten(2, 3), v.flatten(2, 3)                            # [B, KV, L, D]
    z = torch.matmul(s["q"].float().view(B, KV, H // KV, D), k.transpose(2, 3)) / math.sqrt(D)
    w, l = _softmax(z, ok[:, :, None])
    o = torch.matmul(w, v)
    return torch.where(l > 0, o / l.clamp(min=1e-30), 0.0).view(B, H, D).to(s["q"].dtype)


def _plain_weighed(s):
    case = s["case"]
    B, H, KV, D, bs = case["batch"], case["q_heads"], case["kv_heads"], case["head_dim"], case["block_size"]
    phys = s["table"].clamp(min=0).long()
    if case["dtype"] == "i8":
        k, v = (s["codes"][0, c][phys].float() * s["scales"][0, c][phys][..., None] for c in (0, 1))
    else:
        k, v = (s["cache"][0, c][phys].float() for c in (0, 1))       # [B, blocks, KV, bs, D]
    p = torch.arange(phys.shape[1] * bs, device="cuda")[None]
    ok = (s["table"] >= 0).repeat_interleave(bs, 1) & (p <= s["pos"].long()[:, None])
    k, v = k.transpose(1, 2).flatten(2, 3), v.transpose(1, 2).flatten(2, 3)
    z = torch.matmul(s["q"].float().view(B, KV, H // KV, D), k.transpose(2, 3)) / math.sqrt(D)
    w, l = _softmax(z, ok[:, None, None])
    w.div_(l.clamp(min=1e-30))
    o = torch.matmul(w, v).view(B, H, D).to(s["q"].dtype)
    return {"out": o, "weights": s["base"] * case["decay"] + w.sum((1, 2)).view(B, -1, bs).sum(-1)}


def _plain_evict(s):
    case = s["case"]
    s["work"].copy_(s["base"])
    table, w = s["table"], s["weights"]
    total = s["refcount"].numel()
    lb = torch.arange(table.shape[1], device="cuda")[None]
    nb = (s["pos"].long() // case["block_size"] + 1)[:, None]
    live = (table >= 0) & (lb < nb)
    loose = live & (lb >= case["first"]) & (lb < nb - case["recent"])
    over = (live.sum(1) - case["keep"]).clamp(min=0).minimum(loose.sum(1))
    order = torch.sort(torch.where(loose, w, math.inf), dim=1, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, lb.expand_as(order))
    out = loose & (rank < over[:, None])
    drop = torch.zeros(total + 1, dtype=torch.int32, device="cuda")
    drop.scatter_add_(0, torch.where(out, table, total).flatten().long(), torch.ones_like(table).flatten())
    drop = drop[:total]
    s["refcount"].sub_(drop)
    back = (drop > 0) & (s["refcount"] == 0)
    at = torch.where(back, s["free_count"] + torch.cumsum(back, 0) - 1, total)
    stack = torch.cat([s["free_list"], s["free_list"].new_zeros(1)])
    stack.scatter_(0, at.long(), torch.arange(total, dtype=torch.int32, device="cuda"))
    s["free_list"].copy_(stack[:total])
    s["free_count"].add_(back.sum().to(torch.int32))
    words = s["valid"].numel()
    bits = torch.nn.functional.pad(back.long(), (0, words * 32 - total)).view(words, 32)
    s["valid"].bitwise_and_((~(bits << torch.arange(32, device="cuda")).sum(1)).to(torch.int32))
    table.masked_fill_(out, -1)
    w.masked_fill_(out, 0.0)
    return _evict_outputs(s)


def _evict_outputs(s):
    return {n: s[n] for n in ("table", "weights", "refcount", "free_list", "free_count", "valid")}


def _ancestors(parent):
    """[B, T, T] whether j is i or one of its ancestors, and whether token i is real: a power of I + P."""
    B, T = parent.shape
    j = torch.arange(T, device=parent.device)
    step = (parent[..., None].long() == j).float()                    # i -> its parent
    step = torch.cat([step, (parent == -1).float()[..., None]], -1)   # column T: the root
    root = torch.zeros(B, 1, T + 1, device=parent.device)
    root[..., T] = 1.0
    reach = torch.cat([step, root], 1) + torch.eye(T + 1, device=parent.device)
    # six squarings reach 64 steps
    r2 = (reach @ reach > 0).float()
    r4 = (r2 @ r2 > 0).float()
    r8 = (r4 @ r4 > 0).float()
    r16 = (r8 @ r8 > 0).float()
    r32 = (r16 @ r16 > 0).float()
    r64 = r32 @ r32 > 0
    real = r64[:, :T, T]
    return r64[:, :T, :T] & real[..., None], real


def _plain_tree(s):
    case = s["case"]
    B, H, KV, D, T = case["batch"], case["q_heads"], case["kv_heads"], case["head_dim"], case["n_new"]
    n0 = s["pos"].long()
    see, real = _ancestors(s["parent"])
    t = n0[:, None] + see.sum(-1) - 1
    b = torch.arange(B, device="cuda")[:, None]
    if case["layout"] == "paged":
        bs, maxb = case["block_size"], s["table"].shape[1]
        p = torch.arange(max(_lengths(case)), device="cuda")[None].expand(B, -1)
        phys = s["table"].gather(1, (p // bs).clamp(max=maxb - 1)).long()
        i, r = phys.clamp(min=0), p % bs
        ok = (p < n0[:, None]) & (phys >= 0)
        ok = ok[:, None].expand(B, T, -1)
    else:
        S, W = case["sinks"], case["window"]
        r = torch.arange(min(S + W, max(_lengths(case))), device="cuda")[None].expand(B, -1)
        i = b.expand_as(r)
        # the latest position before n0 at each slot
        p = torch.where(r < S, r, n0[:, None] - 1 - (n0[:, None] - 1 - r) % W)
        p = torch.where(r < n0[:, None], p, -1)
        ok = (p >= 0)[:, None] & ((r < S)[:, None] | (p[:, None] > t[..., None] - W))
    k = torch.cat([_read(s, 0, i, r), s["k"].float()], 1)
    v = torch.cat([_read(s, 1, i, r), s["v"].float()], 1)
    ok = torch.cat([ok & real[..., None], see], -1)
    q = s["q"].float().view(B, T, KV, H // KV, D).permute(0, 2, 3, 1, 4).reshape(B, KV, -1, D)
    z = torch.matmul(q, k.permute(0, 2, 3, 1)).view(B, KV, H // KV, T, -1).mul_(1.0 / math.sqrt(D))
    w, l = _softmax(z, ok[:, None, None])
    o = torch.matmul(w.view(B, KV, -1, w.shape[-1]), v.permute(0, 2, 1, 3)).view(B, KV, H // KV, T, D)
    o = torch.where(l > 0, o / l.clamp(min=1e-30), 0.0)
    return o.permute(0, 3, 1, 2, 4).reshape(B, T, H, D).to(s["q"].dtype)


def _plain_path(s):
    case = s["case"]
    B, P = s["path"].shape
    n, n0 = s["n_path"].long()[:, None], s["pos"].long()[:, None]
    j = torch.arange(P, device="cuda")[None]
    b = torch.arange(B, device="cuda")[:, None]
    p = n0 + j
    keep = j < n
    if case["layout"] != "paged":
        keep = keep & ((p < case["sinks"]) | (p > n0 + n - 1 - case["window"]))
    # a token that is not kept writes the sequence's last kept one again
    at = torch.where(keep, j, (keep * (j + 1)).argmax(1, keepdim=True))
    p = n0 + at
    if case["layout"] == "paged":
        i, r = s["table"].gather(1, p // case["block_size"]).long(), p % case["block_size"]
    else:
        i, r = b.expand_as(p), torch.where(p < case["sinks"], p, case["sinks"] + (p - case["sinks"]) % case["window"])
    tok = s["path"].long().gather(1, at)
    k, v = s["k"][b, tok], s["v"][b, tok]
    if case["dtype"] == "i8":
        return {"cache": _store_i8(s, i, r, torch.stack([k, v]).float())}
    s["cache"][0, 0][i, :, r] = k
    s["cache"][0, 1][i, :, r] = v
    return {"cache": s["cache"]}


def _store_i8(s, i, r, x):
    """Rows x [2, B, P, KV, D] as codes and scales; the cache's values."""
    scale = _step(x.abs().amax(-1))
    code = torch.round(x / torch.where(scale > 0, scale, 1.0)[..., None]).clamp(-127, 127).to(torch.int8)
    s["codes"][0, 0][i, :, r], s["codes"][0, 1][i, :, r] = code[0], code[1]
    s["scales"][0, 0][i, :, r], s["scales"][0, 1][i, :, r] = scale[0], scale[1]
    return s["codes"] * s["scales"][..., None]


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        if op == "sparse":
            blocks = _plain_select(s)
            return {"blocks": blocks, "out": _plain_selected(s, blocks)}
        return {"bounds": _plain_bounds, "weighed": _plain_weighed, "evict": _plain_evict, "tree": _plain_tree,
                "path": _plain_path}[op](s)
    kvc, d, ws, table = s["kvc"], s["d"], s["ws"], s.get("table")
    if op == "bounds":
        kvc.block_bounds(d, s["cache"], 0, s["bounds"], s["pos"], case["n_new"], ws, table, n_tok=s["n_tok"])
        return s["b_codes"] * s["b_scale"][..., None, None]
    if op == "sparse":
        blocks = kvc.select_blocks(d, s["bounds"], 0, s["q"], s["pos"], case["k"], ws, table, first=case["first"],
                                   recent=case["recent"])
        return {"blocks": blocks,
                "out": kvc.decode_attention_selected(d, s["cache"], 0, s["q"], s["pos"], blocks, ws, table)}
    if op == "weighed":
        s["weights"].copy_(s["base"])
        out = kvc.decode_attention_weighed(d, s["cache"], 0, s["q"], s["pos"], s["weights"], ws, table,
                                           decay=case["decay"])
        return {"out": out, "weights": s["weights"]}
    if op == "evict":
        s["work"].copy_(s["base"])
        kvc.block_evict(d, s["state"], s["weights"], s["pos"], case["keep"], ws, first=case["first"],
                        recent=case["recent"])
        return _evict_outputs(s)
    if op == "tree":
        return kvc.tree_attention(d, s["cache"], 0, s["q"], s["k"], s["v"], s["pos"], s["parent"], ws,
                                  block_table=table)
    kvc.append_path(d, s["cache"], 0, s["k"], s["v"], s["pos"], s["path"], s["n_path"], ws, block_table=table)
    return {"cache": s["codes"] * s["scales"][..., None] if case["dtype"] == "i8" else s["cache"]}


# ------------------------------------------------------------------ 64 bits
def _key_rows(s, which, i, h, r):
    """K or V rows [L, D] of kv head h in float64 at blocks (or sequences) i and rows r (index tensors)."""
    if s["case"]["dtype"] == "i8":
        return s["codes"][0, which][i, h, r].double() * s["scales"][0, which][i, h, r].double()[:, None]
    return s["cache"][0, which][i, h, r].double()


def _mapped(s, b, L):
    """Positions below L of sequence b that are mapped, their blocks and rows."""
    bs = s["case"]["block_size"]
    p = torch.arange(L, device="cuda")
    phys = s["table"][b].long()[p // bs]
    p = p[phys >= 0]
    return p, s["table"][b].long()[p // bs], p % bs


def _exact_bounds(case, s):
    codes, scale = s["b_codes"].double(), s["b_scale"].double()
    bs = case["block_size"]
    for b, (L, n) in enumerate(zip(_lengths(case), _news(case))):
        row = s["table"][b].tolist()
        whole = torch.tensor([row[x] for x in range(L // bs, (L + n) // bs)], dtype=torch.long, device="cuda")
        part = (L + n) % bs
        last = torch.tensor([row[(L + n) // bs]] if part else [], dtype=torch.long, device="cuda")
        for phys, rows in ((whole, bs), (last, part)):
            if not phys.numel():
                continue
            if case["dtype"] == "i8":
                k = s["codes"][0, 0][phys, :, :rows].double() * s["scales"][0, 0][phys, :, :rows].double()[..., None]
                k = k.float().double()
            else:
                k = s["cache"][0, 0][phys, :, :rows].double()
            ends = torch.stack([k.max(2).values, k.min(2).values], 2)
            # a step and a quotient are kept in 32 bits: two roundings of the same number
            step = (ends.abs().flatten(2).max(-1).values / 127.0).float().double()
            x = (ends / step.clamp(min=1e-300)[..., None, None]).float().double()
            codes[phys] = torch.stack([x[:, :, 0].ceil().clamp(max=127), x[:, :, 1].floor().clamp(min=-127)], 2)
            scale[phys] = step
    return codes * scale[..., None, None]


def _exact_sparse(case, s):
    B, H, KV, D, bs = case["batch"], case["q_heads"], case["kv_heads"], case["head_dim"], case["block_size"]
    out = torch.zeros(B, H, D, dtype=torch.float64, device="cuda")
    ids = torch.full((B, KV, case["k"]), -1, dtype=torch.int32, device="cuda")
    q = s["q"].double()
    sq = (q.abs().max(-1).values / 127.0).float().double()
    code = (q / sq[..., None]).float().double().round().clamp(-127, 127)
    G = H // KV
    for b, L in enumerate(_lengths(case)):
        nb = -(-L // bs)
        lb = torch.arange(nb, device="cuda")[s["table"][b, :nb] >= 0]
        phys = s["table"][b].long()[lb]
        for h in range(KV):
            ends, step = s["b_codes"][phys, h].double(), s["b_scale"][phys, h].double()
            best = torch.full((lb.numel(),), -math.inf, dtype=torch.float64, device="cuda")
            for x in range(h * G, h * G + G):
                u = torch.maximum(ends[:, 0] * code[b, x], ends[:, 1] * code[b, x]).sum(-1)
                best = torch.maximum(best, (u * (sq[b, x] * step).float().double()).float().double())
            best[(lb < case["first"]) | (lb >= nb - case["recent"])] = math.inf
            top = torch.sort(best, descending=True, stable=True).indices[:case["k"]]
            chosen = lb[top].sort().values
            ids[b, h, :chosen.numel()] = chosen.to(torch.int32)
            p = (chosen[:, None] * bs + torch.arange(bs, device="cuda")).flatten()
            p = p[p < L]
            i, r = s["table"][b].long()[p // bs], p % bs
            w = torch.softmax(q[b, h * G:h * G + G] @ _key_rows(s, 0, i, h, r).T / math.sqrt(D), -1)
            out[b, h * G:h * G + G] = w @ _key_rows(s, 1, i, h, r)
    return {"blocks": ids, "out": out}


def _exact_weighed(case, s):
    B, H, KV, D, bs = case["batch"], case["q_heads"], case["kv_heads"], case["head_dim"], case["block_size"]
    out = torch.zeros(B, H, D, dtype=torch.float64, device="cuda")
    weights = s["base"].double() * case["decay"]
    G = H // KV
    for b, L in enumerate(_lengths(case)):
        p, i, r = _mapped(s, b, L)
        for h in range(KV):
            w = torch.softmax(s["q"][b, h * G:h * G + G].double() @ _key_rows(s, 0, i, h, r).T / math.sqrt(D), -1)
            out[b, h * G:h * G + G] = w @ _key_rows(s, 1, i, h, r)
            weights[b].index_add_(0, p // bs, w.sum(0))
    return {"out": out, "weights": weights}


def _exact_tree(case, s):
    B, H, KV, D, T = case["batch"], case["q_heads"], case["kv_heads"], case["head_dim"], case["n_new"]
    out = torch.zeros(B, T, H, D, dtype=torch.float64, device="cuda")
    G = H // KV
    parent = s["parent"].tolist()
    for b, L in enumerate(_lengths(case)):
        lines = []
        for i, p in enumerate(parent[b]):
            above = [] if p == -1 else lines[p] if p >= 0 else None
            lines.append(None if above is None else above + [i])
        if case["layout"] == "paged":
            pos, i, r = _mapped(s, b, L)
        else:
            S, W = case["sinks"], case["window"]
            pos = torch.tensor([x for x in range(L) if x < S or x >= max(S, L - W)], dtype=torch.long, device="cuda")
            i, r = torch.full_like(pos, b), torch.where(pos < S, pos, S + (pos - S) % W)
        hide = torch.ones(T, pos.numel() + T, dtype=torch.bool)
        for x, line in enumerate(lines):
            if line is not None:
                t = L + len(line) - 1
                ok = torch.ones(pos.numel(), dtype=torch.bool, device="cuda")
                if case["layout"] != "paged":
                    ok = (pos < case["sinks"]) | (pos > t - case["window"])
                hide[x, :pos.numel()] = ~ok.cpu()
                hide[x, [pos.numel() + y for y in line]] = False
        hide = hide.cuda()
        gone = torch.tensor([line is None for line in lines], device="cuda")
        for h in range(KV):
            k = torch.cat([_key_rows(s, 0, i, h, r), s["k"][b, :, h].double()])
            v = torch.cat([_key_rows(s, 1, i, h, r), s["v"][b, :, h].double()])
            for x in range(h * G, h * G + G):
                w = torch.softmax((s["q"][b, :, x].double() @ k.T / math.sqrt(D)).masked_fill(hide, -math.inf), -1)
                out[b, :, x] = torch.where(gone[:, None], 0.0, w) @ v
    return out


def _exact_path(case, s):
    if case["dtype"] == "i8":
        cache = s["codes"].double() * s["scales"].double()[..., None]
    else:
        cache = s["cache"].double()
    path, count = s["path"].tolist(), s["n_path"].tolist()
    for b, L in enumerate(_lengths(case)):
        row = s["table"][b].tolist() if case["layout"] == "paged" else None
        for j in range(count[b]):
            p = L + j
            for which, x in enumerate((s["k"], s["v"])):
                new = x[b, path[b][j]].double()
                if case["dtype"] == "i8":
                    step = (new.abs().max(-1).values / 127.0).float().double()[:, None]
                    new = (new / step).float().double().round().clamp(-127, 127) * step
                if row is not None:
                    cache[0, which, row[p // case["block_size"]], :, p % case["block_size"]] = new
                else:
                    S = case["sinks"]
                    cache[0, which, b, :, p if p < S else S + (p - S) % case["window"]] = new
    return {"cache": cache}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "evict":
        # whole numbers throughout, and weights that are copied
        w, table, lens = s["weights"].double().cpu(), s["table"].cpu(), _lengths(case)
        for b, L in enumerate(lens):
            nb = -(-L // case["block_size"])
            live = [x for x, p in enumerate(table[b, :nb].tolist()) if p >= 0]
            row = w[b].tolist()
            loose = sorted((row[x], x) for x in live if case["first"] <= x < nb - case["recent"])
            for _, x in loose[:max(0, len(live) - case["keep"])]:
                w[b, x] = 0.0
        return {"table": None, "weights": w, "refcount": None, "free_list": None, "free_count": None, "valid": None}
    return {"bounds": _exact_bounds, "sparse": _exact_sparse, "weighed": _exact_weighed, "tree": _exact_tree,
            "path": _exact_path}[case["op"]](case, s)
