"""Page calls and row calls past one round of their kernels' loops: lists of thousands of sequences, pools of
20000 pages, rows that no tensor map describes."""
import random

import pytest
import torch

import decode_attention_11_b200 as tq

from test_gpu_paged import check_rows, params
from test_gpu_pages import ARRAYS, Model, copied, ints, make, raw, same_tables

pytestmark = pytest.mark.gpu


def test_lists_of_thousands_of_sequences():
    """Three rounds of 1024 entries: prefix sums carried between rounds, entries that need nothing in between."""
    r = random.Random(4)
    n_seq, ps = 5200, 16
    pt, pools = make(n_seq, 4, 9000, ps, layers=1, Hkv=1, bits=(2, 2), qjl=0)
    m = Model(n_seq, 4, 9000, ps)
    for grow in (lambda: r.choice([0, 0, 1, 15, 16, 17, 20]), lambda: r.choice([0, 1, 3])):
        seqs = r.sample(range(2500), 2500)
        add = [grow() for _ in seqs]
        slots = tq.pages_reserve(pt, ints(seqs), ints(add), sum(add) + 3)
        assert slots.tolist() == m.reserve(seqs, add) + [-1] * 3
        same_tables(pt, m)
    dst = r.sample(range(2600, 5200), 2600)
    src = [r.randrange(2500) for _ in dst]
    before = raw(pools)
    tq.pages_fork(pt, ints(src), ints(dst), pools)
    copied(before, pools, m.fork(src, dst))
    same_tables(pt, m)
    gone = r.sample(range(n_seq), 3000)
    tq.pages_free(pt, ints(gone))
    m.free(gone)
    same_tables(pt, m)
    pt.check()
    # a repeat past the first round is found, and nothing changes
    seqs = list(range(1500)) + [3]
    tq.pages_reserve(pt, ints(seqs), ints([1] * 1501), 1501)
    with pytest.raises(ValueError, match="listed twice"):
        pt.check()
    same_tables(pt, m)


def test_pools_of_20000_pages():
    """A plan's warp walks more than eight rounds of 32 pages: holes over the whole range, then compact."""
    r = random.Random(5)
    n_seq, ps, P = 64, 16, 20011
    pt, pools = make(n_seq, 400, P, ps, layers=1, Hkv=1, bits=(2, 2), qjl=0)
    m = Model(n_seq, 400, P, ps)
    for step in range(3):
        empty = [s for s in range(n_seq) if m.lens[s] == 0]
        room, seqs, add = len(m.free_pages()), [], []
        for s in r.sample(empty, len(empty)):
            a = r.randint(1, 400 * ps)
            if room < -(-a // ps):
                continue
            room -= -(-a // ps)
            seqs.append(s)
            add.append(a)
        slots = tq.pages_reserve(pt, ints(seqs), ints(add), sum(add))
        assert slots.tolist() == m.reserve(seqs, add)
        gone = r.sample([s for s in range(n_seq) if m.lens[s]], 25)
        tq.pages_free(pt, ints(gone))
        m.free(gone)
        same_tables(pt, m)
        if step:
            before = raw(pools)
            tq.pages_compact(pt, pools)
            moved = m.compact()
            assert len(moved) > 1000
            copied(before, pools, moved)
            same_tables(pt, m)
    pt.check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [30, 2000])
@pytest.mark.parametrize("shared", ["heads", "tokens"])
def test_quantize_of_expanded_rows(dtype, N, shared):
    """Rows with a stride of 0: all kv-heads of a token alike, or all tokens (no tensor map describes them, so
    many bf16 rows take the general kernel too)."""
    torch.manual_seed(N)
    H = 4
    shape = (N, 1, 128) if shared == "heads" else (1, H, 128)
    K, V = ((torch.randn(*shape, device="cuda") * 3).to(dtype).expand(N, H, 128) for _ in range(2))
    pool = tq.Cache.allocate(-(-N // 16) + 1, H, 16, 3, 4)
    for n in ARRAYS:
        getattr(pool, n).view(torch.uint8).fill_(0x5A)
    slots = torch.randperm(pool.B * 16, device="cuda")[:N].to(torch.int32)
    slots[1] = -1
    tq.paged_quantize(params(3, 4), K, V, pool, slots)
    check_rows(pool, slots, K, V, 3, 4, True)
    used = torch.zeros(pool.B * 16, dtype=torch.bool, device="cuda")
    used[slots[slots >= 0].long()] = True
    rest = ~used.view(pool.B, 1, 16).expand(-1, H, -1)
    for n in ARRAYS:
        a = getattr(pool, n).view(torch.uint8).view(pool.B, H, 16, -1)
        assert (a[rest] == 0x5A).all(), n
    assert tq.quantize_device_errors() == 0
