"""Groups with members that have nothing to share -- idle slots, sequences shorter than a block, a stale group
id -- are shared by the others all the same: their results are bit for bit those of the call in which these
members are alone, and not those of a call without groups (another order of sums)."""

import pytest
import torch

from tests.cache_builder import Built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import sliding_window_attention_kvc_gb300 as m
    return m


def _tables(lens, shares, blocks, bs):
    tables, at = [], blocks
    for b, n in enumerate(lens):
        need = -(-n // bs)
        t = list(range(min(blocks, need))) if b in shares else []
        t += list(range(at, at + need - len(t)))
        at += need
        tables.append(t)
    return tables


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,out", [
    ((0, 200, 190, 230), (0,)),             # an idle slot, the group's first
    ((200, 0, 190, 230), (1,)),
    ((200, 190, 230, 0), (3,)),
    ((9, 200, 5, 190, 230), (0, 2)),        # shorter than a block
    ((0, 200, 300, 190, 0), (0, 2, 4)),     # and one on blocks of its own, under the group's id
])
def test_members_with_nothing_to_share(kvc, D, lens, out):
    bs, blocks = 16, 10
    shares = [b for b in range(len(lens)) if b not in out]
    c = Built(kvc, "paged", "bf16", lens, 8, 2, D, bs=bs, tables=_tables(lens, shares, blocks, bs))
    ws = kvc.alloc_shared_workspace(c.d)
    B = len(lens)

    def call(group):
        g = torch.tensor(group, dtype=torch.int32, device="cuda")
        return kvc.decode_attention_shared(c.d, c.cache, c.layer, c.q, c.pos, g, ws, c.table)

    want = call([-1 if b in out else 2 for b in range(B)])
    alone = call([-1] * B)
    got = call([2] * B)
    assert not torch.equal(want[shares], alone[shares])       # the shared form rounds differently
    assert torch.equal(got, want)


def test_only_one_member_with_blocks(kvc):
    """Nothing is shared with nobody: the results of the call without groups."""
    lens = (0, 200, 9)
    c = Built(kvc, "paged", "bf16", lens, 8, 2, 128)
    ws = kvc.alloc_shared_workspace(c.d)
    outs = [kvc.decode_attention_shared(c.d, c.cache, c.layer, c.q, c.pos,
                                        torch.tensor(g, dtype=torch.int32, device="cuda"), ws, c.table)
            for g in ([1, 1, 1], [-1, -1, -1])]
    assert torch.equal(*outs)


def test_idle_members_of_many_groups(kvc):
    """More sequences than the plan's thread block is wide, an idle one in every group."""
    n, bs = 300, 16
    lens = [0 if i < 30 else 40 + (i * 13) % 50 for i in range(n)]
    tables, at = [], 30 * 2
    for i, m in enumerate(lens):
        need = -(-m // bs)
        t = [2 * (i % 30), 2 * (i % 30) + 1][:need]
        t += list(range(at, at + need - len(t)))
        at += need
        tables.append(t)
    c = Built(kvc, "paged", "bf16", lens, 4, 1, 64, bs=bs, tables=tables)
    ws = kvc.alloc_shared_workspace(c.d)
    call = lambda g: kvc.decode_attention_shared(c.d, c.cache, c.layer, c.q, c.pos,
                                                 torch.tensor(g, dtype=torch.int32, device="cuda"), ws, c.table)
    got = call([i % 30 for i in range(n)])
    want = call([-1 if i < 30 else i % 30 for i in range(n)])
    assert torch.equal(got, want) and not torch.equal(got, call([-1] * n))


def test_thousands_of_sequences(kvc):
    """A batch far wider than the plan's thread block, against the formula for some of its sequences and
    against plain decode for all: two roundings of the weights and of the output, and plain decode's query
    rounded after its scale (2^-8 sum |q_i k_i| scale, under 8 here, twice in a weight)."""
    from tests import test_gpu_shared as shared

    n, ng, bs = 4096, 500, 8
    lens = [17 + (i * 13) % 23 for i in range(n)]
    tables, at = [], 2 * ng
    for i, m in enumerate(lens):
        need = -(-m // bs)
        g = i % ng
        tables.append([2 * g, 2 * g + 1] + list(range(at, at + need - 2)))
        at += need - 2
    c = Built(kvc, "paged", "bf16", lens, 4, 1, 64, bs=bs, tables=tables, qstd=1.0)
    ws = kvc.alloc_shared_workspace(c.d)
    group = torch.tensor([i % ng for i in range(n)], dtype=torch.int32, device="cuda")
    out = kvc.decode_attention_shared(c.d, c.cache, c.layer, c.q, c.pos, group, ws, c.table)
    again = kvc.decode_attention_shared(c.d, c.cache, c.layer, c.q, c.pos, group, ws, c.table)
    assert torch.equal(out, again) and kvc.get_error(ws) == 0
    shared._check(c, out, skip=[b for b in range(n) if b % 97], rel=2.0 ** -8 + 1e-3)
    ref = kvc.decode_attention(c.d, c.cache, c.layer, c.q, c.pos, c.ws, block_table=c.table)
    vmax = float(c.v.abs().max())
    rel = 2 * (2.0 ** -8 + 1e-3) + 2 * 8 * 2.0 ** -8
    assert ((out.float() - ref.float()).abs() <= rel * vmax + 2.0 ** -7 * ref.float().abs()).all()
