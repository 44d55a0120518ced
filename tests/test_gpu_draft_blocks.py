"""Drafts verified over the block manager, by the README's own example: paths that cross blocks' ends, and paths that
begin inside a block that another sequence maps too."""

import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import sliding_window_attention_kvc_gb300 as m
    return m


def _example():
    with open(os.path.join(ROOT, "README.md")) as f:
        text = f.read().split("- **Drafted tokens.**", 1)[1]
    code = re.search(r"```python\n(.*?)```", text, re.S).group(1)
    return compile("\n".join(line[2:] for line in code.splitlines()), "README.md", "exec")


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("bs", [8, 16, 64])
def test_readme_example(kvc, bs):
    B, L, H, KV, D, T, P, rounds = 4, 2, 4, 2, 64, 12, 10, 20
    prompt = bs + 5                                          # its second block part full
    maxb = (prompt + rounds * P) // bs + 2
    d = kvc.make_desc("paged", "none", "bf16", layers=L, batch=B, q_heads=H, kv_heads=KV, head_dim=D, block_size=bs,
                      num_blocks=B * maxb, max_blocks_per_seq=maxb)
    cache, ws, state = kvc.alloc_cache(d, fill=0.0), kvc.alloc_workspace(d), kvc.BlockState(d)
    g = torch.Generator(device="cuda").manual_seed(bs)

    def rows(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    # sequence 0 takes the prompt in, 1 and 2 share its blocks, the part-full one too; 3 is idle
    want = [[[] for _ in range(L)] for _ in range(B)]        # sequence, layer -> (k, v) of each position
    for p in range(prompt):
        at = _i32(p, -1, -1, -1)
        kvc.block_prepare(d, cache, at, state, ws)
        for layer in range(L):
            k, v = rows(B, KV, D), rows(B, KV, D)
            kvc.append(d, cache, layer, k, v, at, ws, block_table=state.table)
            for b in range(3):
                want[b][layer].append((k[0], v[0]))
    kvc.block_share(d, state, _i32(0, 0), _i32(1, 2), _i32(2, 2), ws)
    pos0 = _i32(prompt, prompt, prompt, -1)
    parent = _i32(*range(-1, T - 1)).repeat(B, 1)
    run, pick = _example(), torch.Generator().manual_seed(bs)
    for r in range(rounds):
        n = torch.randint(0, P + 1, (B,), generator=pick).tolist()
        q, k, v = ([rows(B, T, x, D) for _ in range(L)] for x in (H, KV, KV))
        path = torch.stack([torch.randperm(T, generator=pick)[:P].sort().values for _ in range(B)]).to(torch.int32).cuda()
        names = dict(kvc=kvc, torch=torch, d=d, cache=cache, L=L, T=T, P=P, q=q, k=k, v=v, pos0=pos0, parent=parent, path=path,
                     n_path=_i32(*n), state=state)
        exec(run, names)
        assert kvc.get_error(names["tws"]) == 0, r
        for b in range(3):
            for layer in range(L):
                for j in range(n[b]):
                    t = int(path[b, j])
                    want[b][layer].append((k[layer][b, t], v[layer][b, t]))
        pos0 = torch.where(pos0 >= 0, pos0 + _i32(*n), -1)
        table = state.table.tolist()
        for b in range(3):
            for layer in range(L):
                ks, vs = (torch.stack(x) for x in zip(*want[b][layer]))
                blocks = torch.tensor([table[b][p // bs] for p in range(len(ks))], device="cuda")
                at = torch.arange(len(ks), device="cuda") % bs
                assert int(blocks.min()) >= 0
                assert torch.equal(cache[layer, 0][blocks, :, at], ks) and torch.equal(cache[layer, 1][blocks, :, at], vs), (r, b)
        assert all(x == -1 for x in table[3])
    counts = torch.bincount(state.table[state.table >= 0].long(), minlength=d.num_blocks)
    assert torch.equal(counts.to(torch.int32), state.refcount)
    assert int(state.free_count) == d.num_blocks - int((counts > 0).sum())
