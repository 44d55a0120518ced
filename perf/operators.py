"""Cases of the serving-step operators around the KV cache, with their plain forms.

Four operators, all on the caches of include/kvc.h:

  append   norms of queries and keys for each head, rotary positions (pairs of halves or
           neighbours, part of the head, scaled for long contexts) and the append of keys
           and values to the cache, in one pass (kvc.append_qk);
  decode   single-token attention with capped scores, a distance bias and a document start
           (kvc.decode_attention_scored);
  prefill  the same for a chunk of tokens of each sequence (kvc.prefill_scored);
  shared   single-token attention of a batch whose groups share a long prefix
           (kvc.decode_attention_shared).

`run` computes them in elementary torch operations in fp32, or (own) with the library's calls.
"""

import math

import torch

own = False

ELT = {"bf16": 2, "f32": 4, "i8": 1}
ACT = {"bf16": torch.bfloat16, "f32": torch.float32, "i8": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token each for the 64 sequences of the paged batch: q/k norms, positions scaled to 4x
        dict(name="append_step_paged", op="append", layout="paged", dtype="bf16", batch=64, q_heads=32, kv_heads=8,
             head_dim=128, block_size=16, lo=512, hi=8192, n_new=1, norm=True, pairs="half", rot=128, scaling="yarn"),
        # a prompt chunk of ragged sequences out of one packed projection, neighbour pairs on half of the head
        dict(name="append_prompt_paged", op="append", layout="paged", dtype="bf16", batch=8, q_heads=32, kv_heads=8,
             head_dim=128, block_size=16, lo=0, hi=3000, n_new=2048, norm=True, pairs="interleaved", rot=64,
             scaling="none"),
        # the small fp32 sink cache of the configurations: one sequence, a few heads, no norm
        dict(name="append_sink_f32", op="append", layout="sink_ring", dtype="f32", batch=5, q_heads=4, kv_heads=1,
             head_dim=64, window=60, sinks=4, lo=1, hi=300, n_new=7, norm=False, pairs="half", rot=64,
             scaling="linear"),
        # the sliding-window ring with capped scores: every slot of 8 x 4096 read once
        dict(name="decode_ring_cap", op="decode", layout="ring", dtype="bf16", batch=8, q_heads=32, kv_heads=8,
             head_dim=128, window=4096, lo=4097, hi=65536, cap=20.0, bias=False, start=False),
        # the paged batch with a distance bias for each head and documents that begin inside the cache
        dict(name="decode_paged_bias_doc", op="decode", layout="paged", dtype="bf16", batch=64, q_heads=32, kv_heads=8,
             head_dim=128, block_size=16, lo=512, hi=8192, cap=0.0, bias=True, start=True),
        # few long sequences on the INT8 cache, capped and biased
        dict(name="decode_paged_i8", op="decode", layout="paged", dtype="i8", batch=3, q_heads=16, kv_heads=4,
             head_dim=256, block_size=64, lo=20000, hi=65536, cap=30.0, bias=True, start=False),
        # the smallest decode: fp32 sink cache, one sequence, nothing but latency
        dict(name="decode_sink_f32", op="decode", layout="sink_ring", dtype="f32", batch=1, q_heads=4, kv_heads=1,
             head_dim=64, window=60, sinks=4, lo=257, hi=257, cap=15.0, bias=True, start=False),
        # chunked prefill over full rings, capped scores
        dict(name="prefill_ring_cap", op="prefill", layout="ring", dtype="bf16", batch=8, q_heads=32, kv_heads=8,
             head_dim=128, window=4096, n_new=256, lo=4096, hi=20000, cap=20.0, bias=False, start=False),
        # a long packed prompt from the start: documents in one sequence, distance bias
        dict(name="prefill_paged_docs", op="prefill", layout="paged", dtype="bf16", batch=1, q_heads=32, kv_heads=8,
             head_dim=128, block_size=16, n_new=6000, lo=0, hi=0, cap=0.0, bias=True, start=True),
        # the paged batch with 2048-token prefixes shared by groups of 8
        dict(name="shared_groups_of_8", op="shared", layout="paged", dtype="bf16", batch=64, q_heads=32, kv_heads=8,
             head_dim=128, block_size=16, groups=8, prefix=2048, lo=2049, hi=8192),
        # one long document asked by 96 readers at once, short turns behind it
        dict(name="shared_one_document", op="shared", layout="paged", dtype="bf16", batch=96, q_heads=32, kv_heads=8,
             head_dim=128, block_size=64, groups=1, prefix=32768, lo=32790, hi=34000),
        # a few readers of a middling prefix, head_dim 64
        dict(name="shared_small", op="shared", layout="paged", dtype="bf16", batch=6, q_heads=16, kv_heads=8,
             head_dim=64, block_size=16, groups=2, prefix=1008, lo=1030, hi=1500),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefill", "shared"])
    D = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    q_heads = kv * rng.choice([g for g in (1, 2, 3, 4, 8) if g * kv <= 32])
    c = dict(op=op, dtype="bf16", head_dim=D, kv_heads=kv, q_heads=q_heads)
    if op == "append":
        c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
    elif op == "decode":
        c["dtype"] = rng.choice(["bf16", "bf16", "f32", "i8"] if D >= 128 else ["bf16", "f32"])
    c["layout"] = "paged" if op == "shared" else rng.choice(["ring", "sink_ring", "paged"])
    if c["layout"] == "paged":
        c["block_size"] = rng.choice([8, 16, 32, 64])
    else:
        c["sinks"] = 4 if c["layout"] == "sink_ring" else 0
        # the INT8 cache's rows come in fours
        c["window"] = 4 * _log(rng, 16, 1024) - c["sinks"]
    if op == "append":
        c["batch"] = _log(rng, 1, 64)
        c["n_new"] = rng.choice([1, _log(rng, 2, max(2, 10000 // c["batch"]))])
        c["lo"], c["hi"] = 0, _log(rng, 16, 4000)
        c["norm"] = rng.random() < 0.7
        c["pairs"] = rng.choice(["half", "interleaved"])
        c["rot"] = rng.choice([D, D // 2, 2 * rng.randint(1, D // 2)])
        c["scaling"] = rng.choice(["none", "linear", "yarn", "bands"])
    elif op == "decode":
        c["batch"] = _log(rng, 1, 64)
        mean = max(2, _log(rng, 64, 60000) // c["batch"])
        c["lo"] = max(1, int(mean * rng.uniform(0.2, 1.0)))
        c["hi"] = 2 * mean - c["lo"]
    elif op == "prefill":
        c["batch"] = rng.choice([1, 1, 2])
        c["n_new"] = _log(rng, 1, 700)
        if c["layout"] != "paged":
            c["n_new"] = min(c["n_new"], c["window"])
        c["lo"] = 0
        c["hi"] = _log(rng, 1, 2500)
    else:
        c["groups"] = _log(rng, 1, 8)
        c["batch"] = c["groups"] * _log(rng, 2, 16)
        c["prefix"] = c["block_size"] * _log(rng, 4, 50000 // (64 * c["groups"]))
        c["lo"] = c["prefix"] + 1
        c["hi"] = c["lo"] + _log(rng, 1, 900)
    if op in ("decode", "prefill"):
        c["cap"] = rng.choice([0.0, 15.0, 30.0])
        c["bias"] = rng.random() < 0.5
        c["start"] = rng.random() < 0.5
    return c


def _lengths(case):
    """Tokens of each sequence before the call (append, prefill) or with the one decoded (decode,
    shared): spread over [lo, hi] by the golden ratio, the same for every seed."""
    n, lo, hi = case["batch"], case["lo"], case["hi"]
    return [lo + int((hi - lo + 1) * ((i * 0.6180339887498949 + 0.37) % 1.0)) for i in range(n)]


def _news(case):
    """append: ragged token counts 1 .. n_new of a padded batch (n_new itself among them)."""
    n, most = case["batch"], case["n_new"]
    return [most if i == 0 else max(1, most - int(most * 0.6 * ((i * 0.6180339887498949) % 1.0))) for i in range(n)]


def _live(case, t):
    """How many tokens the token at position t attends, itself included."""
    if case["layout"] == "paged":
        return t + 1
    return min(t + 1, case["window"] + case.get("sinks", 0))


def _starts(case, i):
    """Document starts of a decode case: about a quarter of the sequences carry earlier documents."""
    t = _lengths(case)[i] - 1
    return 0 if i % 4 else int(t * 0.45)


def _docs(case, b):
    """First token (chunk index, may be negative: before the chunk) of the document of each chunk token."""
    T, L0 = case["n_new"], _lengths(case)[b]
    size = max(1, T // 3 + 7)
    first = -(L0 // 2) if L0 else 0
    return [first if i < size else (i // size) * size for i in range(T)]


def work(case):
    D, H, KV, B = case["head_dim"], case["q_heads"], case["kv_heads"], case["batch"]
    e, a = ELT[case["dtype"]], 4 if case["dtype"] == "f32" else 2
    row = KV * 2 * (D * e + (4 if case["dtype"] == "i8" else 0))      # K and V of one token in the cache
    if case["op"] == "append":
        n = sum(_news(case))
        return {"bytes": n * (2 * H * D * a + 2 * KV * D * a + row), "flops": n * (H + KV) * D * 8}
    if case["op"] == "decode":
        keys = 0
        for i, L in enumerate(_lengths(case)):
            n = _live(case, L - 1)
            if case["start"]:
                n = min(n, L - _starts(case, i))
            keys += n
        return {"bytes": keys * row + 2 * B * H * D * a, "flops": 4 * keys * H * D}
    if case["op"] == "prefill":
        T, pairs, cached = case["n_new"], 0, 0
        for b, L0 in enumerate(_lengths(case)):
            first = _docs(case, b) if case["start"] else [-L0] * T
            low = 0
            for i in range(T):
                n = min(_live(case, L0 + i), i - first[i] + 1)
                pairs += n
                low = max(low, n - 1 - i)
            cached += min(low, L0)
        return {"bytes": cached * row + B * T * (2 * H * D * a + 2 * KV * D * a + row), "flops": 4 * pairs * H * D}
    keys = sum(_lengths(case))
    unique = keys - (B - case["groups"]) * case["prefix"]
    return {"bytes": unique * row + 2 * B * H * D * a, "flops": 4 * keys * H * D}


# ------------------------------------------------------------------ inputs
def _frequencies(case, device):
    """Angle for each position step of each pair, float64, and what multiplies the rotated values."""
    n, base, factor, orig = case["rot"], 10000.0, 4.0, 4096
    i = torch.arange(n // 2, dtype=torch.float64, device=device)
    f = base ** (-2.0 * i / n)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "yarn":
        def dim_of(turns):
            return n * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(dim_of(32.0)), 0), min(math.ceil(dim_of(1.0)), n - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    if case["scaling"] == "bands":
        turns = orig * f / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return f / factor * (1 - keep) + f * keep, 1.0
    return f, 1.0


def _paged_table(case, need, g, shared=None):
    """Block table [batch, max blocks] over a random permutation of the physical blocks; `shared`:
    (groups, blocks) of prefixes that the sequences of a group (b mod groups) hold in common."""
    bs, B = case["block_size"], case["batch"]
    nb = [-(-n // bs) for n in need]
    maxb = max(nb)
    groups, pre = shared or (0, 0)
    total = sum(n - pre for n in nb) + groups * pre
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, maxb), -1, dtype=torch.int32, device="cuda")
    at = groups * pre
    for b in range(B):
        if pre:
            k = b % groups
            table[b, :pre] = perm[k * pre:(k + 1) * pre]
        table[b, pre:nb[b]] = perm[at:at + nb[b] - pre]
        at += nb[b] - pre
    return table, total


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
    if case["layout"] == "paged":
        need = [n + (T if op in ("append", "prefill") else 0) for n in lens]
        shared = (case["groups"], case["prefix"] // case["block_size"]) if op == "shared" else None
        s["table"], blocks = _paged_table(case, need, g, shared)
        shape = (1, 2, blocks, KV, case["block_size"], D)
    else:
        shape = (1, 2, B, KV, case["window"] + case.get("sinks", 0), D)
    if case["dtype"] == "i8":
        # codes, then the row scales: one flat buffer, as the library lays an INT8 cache out
        n = math.prod(shape)
        s["cache"] = torch.empty(n + 4 * (n // D), dtype=torch.uint8, device="cuda")
        s["codes"] = s["cache"][:n].view(torch.int8).view(shape)
        s["scales"] = s["cache"][n:].view(torch.float32).view(shape[:-1])
        for c in (0, 1):
            s["codes"][0, c] = normal(*shape[2:], std=32.0, dtype=torch.float32).round_().clamp_(-127, 127).to(torch.int8)
        s["scales"].copy_((torch.rand(shape[:-1], generator=g, device="cuda") + 0.5) / 32.0)
    else:
        s["cache"] = torch.empty(shape, dtype=act, device="cuda")
        for c in (0, 1):
            s["cache"][0, c].copy_(normal(*shape[2:]))
    if op in ("append", "prefill"):
        s["pos"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    else:
        s["pos"] = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device="cuda")
    if op == "append":
        # q, k and v side by side, as one projection writes them
        qkv = normal(B, T, (H + 2 * KV) * D)
        s["q"] = qkv[..., :H * D].unflatten(-1, (H, D))
        s["k"] = qkv[..., H * D:(H + KV) * D].unflatten(-1, (KV, D))
        s["v"] = qkv[..., (H + KV) * D:].unflatten(-1, (KV, D))
        s["n_tok"] = torch.tensor(_news(case), dtype=torch.int32, device="cuda")
        s["q_out"] = torch.zeros(B, T, H, D, dtype=act, device="cuda")
        s["qw"] = s["kw"] = None
        if case["norm"]:
            s["qw"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(act)
            s["kw"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(act)
        s["freq"], s["mul"] = _frequencies(case, "cuda")
    elif op == "prefill":
        s["q"] = normal(B, T, H, D, std=2.0)
        s["k"], s["v"] = normal(B, T, KV, D), normal(B, T, KV, D)
    else:
        s["q"] = normal(B, H, D, std=2.0)
    if op in ("decode", "prefill"):
        s["slopes"] = s["start"] = None
        if case["bias"]:
            s["slopes"] = (2.0 ** (-8.0 * torch.arange(1, H + 1, device="cuda") / H)).float()
        if case["start"] and op == "decode":
            s["start"] = torch.tensor([_starts(case, i) for i in range(B)], dtype=torch.int32, device="cuda")
        elif case["start"]:
            s["start"] = torch.tensor([[max(0, lens[b] + i) for i in _docs(case, b)] for b in range(B)],
                                      dtype=torch.int32, device="cuda")
    if op == "shared":
        s["group"] = torch.tensor([b % case["groups"] for b in range(B)], dtype=torch.int32, device="cuda")
    if own:
        import sliding_window_attention_kvc_gb300 as kvc
        s["kvc"] = kvc
        d = s["d"] = kvc.make_desc(case["layout"], "none", case["dtype"], layers=1, batch=B, q_heads=H, kv_heads=KV,
                                   head_dim=D, window=case.get("window", 0), sinks=case.get("sinks", 0),
                                   block_size=case.get("block_size", 0), num_blocks=blocks,
                                   max_blocks_per_seq=s["table"].shape[1] if blocks else 0)
        if op == "append":
            rotary = kvc.make_rotary(case["pairs"], dim=case["rot"], base=10000.0, scaling=case["scaling"], factor=4.0,
                                     original_len=4096, fast=4.0 if case["scaling"] == "bands" else 32.0, slow=1.0)
            s["qk"] = kvc.make_qk(d, rotary=rotary, q_weight=s["qw"], k_weight=s["kw"], eps=EPS)
            s["ws"] = kvc.alloc_workspace(d)
        elif op == "decode":
            s["score"] = kvc.make_score(softcap=case["cap"], slopes=s["slopes"], start=s["start"])
            s["ws"] = kvc.alloc_workspace(d)
        elif op == "prefill":
            s["score"] = kvc.make_score(softcap=case["cap"], slopes=s["slopes"], start=s["start"])
            s["ws"] = kvc.alloc_prefill_workspace(d, T)
        else:
            s["ws"] = kvc.alloc_shared_workspace(d)
    return s


# ------------------------------------------------------------------ plain forms
def _rows(s, p):
    """Indices (block or sequence, row) [B, L] of positions p [B, L] (in range)."""
    case = s["case"]
    if case["layout"] == "paged":
        bs = case["block_size"]
        return s["table"].gather(1, p // bs).long(), p % bs
    S, W = case.get("sinks", 0), case["window"]
    return torch.arange(p.shape[0], device=p.device)[:, None].expand_as(p), torch.where(p < S, p, S + (p - S) % W)


def _read(s, which, at):
    """K (0) or V (1) rows [B, L, KV, D] of the cache at indices of _rows, fp32."""
    i, r = at
    if s["case"]["dtype"] == "i8":
        return s["codes"][0, which][i, :, r].float() * s["scales"][0, which][i, :, r][..., None]
    return s["cache"][0, which][i, :, r].float()


def _positions(s, t):
    """Positions [B, L] that a token at t [B] can attend in the cache, and which are real."""
    case = s["case"]
    lens = _lengths(case)
    if case["layout"] == "paged":
        most = max(lens)
        p = torch.arange(most, device="cuda")[None].expand(t.shape[0], most)
        return p, p <= t[:, None]
    S, W = case.get("sinks", 0), case["window"]
    n = min(max(lens), S + W)
    j = torch.arange(n, device="cuda")[None]
    shift = (t[:, None] + 1 - (S + W)).clamp(min=0)
    p = torch.where(j < S, j, j + shift)
    return p, p <= t[:, None]


def _attend(q, k, v, dist, ok, case, slopes):
    """q [B, T, H, D], k, v [B, L, KV, D] fp32; dist, ok [B, T, L]; rows that see nothing give 0."""
    B, T, H, D = q.shape
    KV = k.shape[2]
    q = q.view(B, T, KV, H // KV, D).permute(0, 2, 3, 1, 4).reshape(B, KV, -1, D)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)).view(B, KV, H // KV, T, -1)
    s.mul_(1.0 / math.sqrt(D))
    if case.get("cap"):
        s.div_(case["cap"]).tanh_().mul_(case["cap"])
    if slopes is not None:
        s.sub_(slopes.view(1, KV, H // KV, 1, 1) * dist[:, None, None].float())
    s.masked_fill_(~ok[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    s.sub_(m).exp_()
    z = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(B, KV, -1, s.shape[-1]), v.permute(0, 2, 1, 3)).view(B, KV, H // KV, T, D)
    o = torch.where(z > 0, o / z.clamp(min=1e-30), 0.0)
    return o.permute(0, 3, 1, 2, 4).reshape(B, T, H, D)


def _write(s, p, keep, new):
    """Rows new [B, T, KV, D] (two: K, V) to positions p where `keep`; a token that is not kept writes
    its sequence's last kept token again."""
    last = (keep * torch.arange(1, keep.shape[1] + 1, device=keep.device)).argmax(1, keepdim=True)
    at = torch.where(keep, torch.arange(keep.shape[1], device=keep.device)[None], last)
    i, r = _rows(s, p.gather(1, at))
    b = torch.arange(p.shape[0], device=p.device)[:, None]
    for which, x in enumerate(new):
        x = x[b, at]
        s["cache"][0, which][i, :, r] = x.to(s["cache"].dtype)


def _kept(case, p, n):
    """Tokens of a chunk (positions p [B, T], the first n [B] real) that are in the cache after it."""
    j = torch.arange(p.shape[1], device=p.device)[None]
    keep = j < n[:, None]
    if case["layout"] != "paged":
        end = (p[:, :1] + n[:, None] - 1)
        keep = keep & ((p < case.get("sinks", 0)) | (p > end - case["window"]))
    return keep


def _rotate(x, cos, sin, case):
    n = case["rot"]
    if case["pairs"] == "half":
        a, b = x[..., :n // 2], x[..., n // 2:n]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0:n:2], x[..., 1:n:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([y, x[..., n:]], -1)


def _plain_append(s):
    case = s["case"]
    T = case["n_new"]
    p = s["pos"].long()[:, None] + torch.arange(T, device="cuda")[None]
    ang = p.double()[..., None] * s["freq"]
    cos, sin = (ang.cos() * s["mul"]).float()[:, :, None], (ang.sin() * s["mul"]).float()[:, :, None]
    out = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        out.append(_rotate(x, cos, sin, case))
    real = torch.arange(T, device="cuda")[None] < s["n_tok"][:, None]
    s["q_out"].copy_(torch.where(real[..., None, None], out[0].to(s["q_out"].dtype), s["q_out"]))
    _write(s, p, _kept(case, p, s["n_tok"].long()), (out[1], s["v"].float()))
    return {"q": s["q_out"], "cache": s["cache"]}


def _plain_decode(s):
    t = s["pos"].long()
    p, ok = _positions(s, t)
    if s.get("start") is not None:
        ok = ok & (p >= s["start"].long()[:, None])
    at = _rows(s, torch.minimum(p, t[:, None]))
    dist = t[:, None, None] - p[:, None]
    o = _attend(s["q"].float()[:, None], _read(s, 0, at), _read(s, 1, at), dist, ok[:, None], s["case"], s.get("slopes"))
    return o[:, 0].to(s["q"].dtype)


def _plain_prefill(s):
    case = s["case"]
    T = case["n_new"]
    n0 = s["pos"].long()
    t = n0[:, None] + torch.arange(T, device="cuda")[None]
    k, v, p, ok = s["k"].float(), s["v"].float(), t, torch.ones_like(t, dtype=torch.bool)
    if max(_lengths(case)) > 0:
        pc, okc = _positions(s, n0 - 1)
        at = _rows(s, torch.minimum(pc, (n0 - 1).clamp(min=0)[:, None]))
        zero = okc[..., None, None]
        k = torch.cat([torch.where(zero, _read(s, 0, at), 0.0), k], 1)
        v = torch.cat([torch.where(zero, _read(s, 1, at), 0.0), v], 1)
        p, ok = torch.cat([pc, t], 1), torch.cat([okc, ok], 1)
    see = ok[:, None] & (p[:, None] <= t[..., None])
    if case["layout"] != "paged":
        see = see & ((p[:, None] < case.get("sinks", 0)) | (p[:, None] > t[..., None] - case["window"]))
    if s["start"] is not None:
        see = see & (p[:, None] >= s["start"].long()[..., None])
    o = _attend(s["q"].float(), k, v, t[..., None] - p[:, None], see, case, s["slopes"])
    _write(s, t, _kept(case, t, torch.full_like(n0, T)), (s["k"].float(), s["v"].float()))
    return {"out": o.to(s["q"].dtype), "cache": s["cache"]}


def run(s):
    op = s["case"]["op"]
    if not own:
        if op == "append":
            return _plain_append(s)
        if op == "prefill":
            return _plain_prefill(s)
        return _plain_decode(s)
    kvc, d, table = s["kvc"], s["d"], s.get("table")
    if op == "append":
        kvc.append_qk(d, s["cache"], 0, s["q"], s["k"], s["v"], s["pos"], s["ws"], s["qk"], n_tok=s["n_tok"],
                      block_table=table, q_out=s["q_out"])
        return {"q": s["q_out"], "cache": s["cache"]}
    if op == "decode":
        return kvc.decode_attention_scored(d, s["cache"], 0, s["q"], s["pos"], s["ws"], s["score"], block_table=table)
    if op == "prefill":
        out = kvc.prefill_scored(d, s["cache"], 0, s["q"], s["k"], s["v"], s["pos"], s["ws"], s["score"],
                                 block_table=table)
        return {"out": out, "cache": s["cache"]}
    return kvc.decode_attention_shared(d, s["cache"], 0, s["q"], s["pos"], s["group"], s["ws"], block_table=table)


# ------------------------------------------------------------------ 64 bits
def _slot(case, p):
    S, W = case.get("sinks", 0), case["window"]
    return p if p < S else S + (p - S) % W


def _attended(case, t):
    if case["layout"] == "paged":
        return list(range(t + 1))
    S, W = case.get("sinks", 0), case["window"]
    return [p for p in range(min(S, t + 1))] + [p for p in range(max(S, t - W + 1), t + 1)]


def _exact_rows(s, b, p):
    """K and V [KV, L, D] in float64 of the cached positions p of sequence b."""
    case = s["case"]
    if case["layout"] == "paged":
        row = s["table"][b].tolist()
        i = torch.tensor([row[x // case["block_size"]] for x in p], device="cuda")
        r = torch.tensor([x % case["block_size"] for x in p], device="cuda")
    else:
        i = torch.full((len(p),), b, device="cuda")
        r = torch.tensor([_slot(case, x) for x in p], device="cuda")
    out = []
    for which in (0, 1):
        if case["dtype"] == "i8":
            x = s["codes"][0, which][i, :, r].double() * s["scales"][0, which][i, :, r].double()[..., None]
        else:
            x = s["cache"][0, which][i, :, r].double()
        out.append(x.transpose(0, 1))
    return out


def _exact_attend(case, s, q, t, k, v, p, start):
    """One sequence: q [T, H, D] at positions t [T], keys at positions p [L]; out [T, H, D]."""
    T, H, D = q.shape
    KV = case["kv_heads"]
    out = torch.empty(T, H, D, dtype=torch.float64, device="cuda")
    see = p[None] <= t[:, None]
    if case["layout"] != "paged":
        see &= (p[None] < case.get("sinks", 0)) | (t[:, None] - p[None] < case["window"])
    if start is not None:
        see &= p[None] >= start[:, None]
    some = see.any(1)
    for h in range(H):
        z = q[:, h].double() @ k[h * KV // H].T / math.sqrt(D)
        if case.get("cap"):
            z = case["cap"] * torch.tanh(z / case["cap"])
        if s.get("slopes") is not None:
            z = z + s["slopes"][h].double() * (p[None] - t[:, None]).double()
        w = torch.softmax(z.masked_fill(~see, -math.inf), -1)
        out[:, h] = torch.where(some[:, None], w, 0.0).nan_to_num() @ v[h * KV // H]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    lens, op, B = _lengths(case), case["op"], case["batch"]
    if op in ("decode", "shared"):
        out = torch.empty(B, case["q_heads"], case["head_dim"], dtype=torch.float64, device="cuda")
        for b in range(B):
            t = lens[b] - 1
            lo = int(s["start"][b]) if s.get("start") is not None else 0
            p = [x for x in _attended(case, t) if x >= lo]
            if not p:
                out[b] = 0
                continue
            k, v = _exact_rows(s, b, p)
            out[b] = _exact_attend(case, s, s["q"][b][None], torch.tensor([t], device="cuda"), k, v,
                                   torch.tensor(p, device="cuda"), None)[0]
        return out
    T = case["n_new"]
    cache = s["cache"].double()
    news = _news(case) if op == "append" else [T] * B
    if op == "append":
        res = s["q_out"].double().clone()
        f, mul = _frequencies(case, "cpu")
        f, n = f.cuda(), case["rot"]
        kk = torch.empty(B, T, case["kv_heads"], case["head_dim"], dtype=torch.float64, device="cuda")
        for b in range(B):
            ang = torch.arange(lens[b], lens[b] + T, dtype=torch.float64, device="cuda")[:, None] * f
            turn = torch.polar(torch.full_like(ang, mul), ang)[:, None]
            for x, w, to in ((s["q"], s["qw"], res), (s["k"], s["kw"], kk)):
                y = x[b].double()
                if w is not None:
                    y = y / (y.pow(2).sum(-1, keepdim=True) / y.shape[-1] + EPS).sqrt() * w.double()
                y = y.clone()
                if case["pairs"] == "half":
                    z = torch.complex(y[..., :n // 2], y[..., n // 2:n]) * turn
                    y[..., :n // 2], y[..., n // 2:n] = z.real, z.imag
                else:
                    z = torch.view_as_complex(y[..., :n].reshape(T, -1, n // 2, 2)) * turn
                    y[..., :n] = torch.view_as_real(z).reshape(T, -1, n)
                to[b, :news[b]] = y[:news[b]]
        new = (kk, s["v"].double())
        name = "q"
    else:
        res = torch.empty(B, T, case["q_heads"], case["head_dim"], dtype=torch.float64, device="cuda")
        for b in range(B):
            old = _attended(case, lens[b] - 1) if lens[b] else []
            k, v = s["k"][b].double().transpose(0, 1), s["v"][b].double().transpose(0, 1)
            if old:
                kc, vc = _exact_rows(s, b, old)
                k, v = torch.cat([kc, k], 1), torch.cat([vc, v], 1)
            t = torch.arange(lens[b], lens[b] + T, device="cuda")
            p = torch.cat([torch.tensor(old, dtype=torch.long, device="cuda"), t])
            start = s["start"][b].long() if s["start"] is not None else None
            res[b] = _exact_attend(case, s, s["q"][b], t, k, v, p, start)
        new = (s["k"].double(), s["v"].double())
        name = "out"
    # the rows that each sequence's tokens leave in the cache
    for b in range(B):
        end = lens[b] + news[b]
        kept = [x for x in range(lens[b], end)
                if case["layout"] == "paged" or x < case.get("sinks", 0) or x >= end - case["window"]]
        tok = torch.tensor([x - lens[b] for x in kept], device="cuda")
        if case["layout"] == "paged":
            row = s["table"][b].tolist()
            i = torch.tensor([row[x // case["block_size"]] for x in kept], device="cuda")
            r = torch.tensor([x % case["block_size"] for x in kept], device="cuda")
        else:
            i = torch.full((len(kept),), b, device="cuda")
            r = torch.tensor([_slot(case, x) for x in kept], device="cuda")
        for which in (0, 1):
            cache[0, which][i, :, r] = new[which][b][tok]
    return {name: res, "cache": cache}
