"""Page management (tq_pages_*) on the GPU against a plain model of the same rules in Python: every
table, length, count and slot, and every byte of the pools, exactly."""
import random

import pytest
import torch

import decode_attention_11_b200 as tq

pytestmark = pytest.mark.gpu

ARRAYS = ("k_codes", "k_signs", "k_norm", "k_rnorm", "v_codes", "v_norm")


class Model:
    """The rules in lists: lowest free page first; fork shares full pages and copies the last."""

    def __init__(self, n_seq, max_pages, num_pages, ps):
        self.ps, self.max_pages, self.num_pages = ps, max_pages, num_pages
        self.table = [[] for _ in range(n_seq)]
        self.lens = [0] * n_seq
        self.refs = [0] * num_pages

    def free_pages(self):
        return [p for p in range(self.num_pages) if self.refs[p] == 0]

    def reserve(self, seqs, grow):
        room, slots = self.free_pages(), []
        for s, a in zip(seqs, grow):
            for t in range(self.lens[s], self.lens[s] + a):
                if t // self.ps == len(self.table[s]):
                    p = room.pop(0)
                    self.refs[p] = 1
                    self.table[s].append(p)
                slots.append(self.table[s][t // self.ps] * self.ps + t % self.ps)
            self.lens[s] += a
        return slots

    def fork(self, src, dst):
        room, copies = self.free_pages(), []
        for s, d in zip(src, dst):
            full = self.lens[s] // self.ps
            self.table[d] = self.table[s][:full]
            if self.lens[s] % self.ps:
                p = room.pop(0)
                copies.append((self.table[s][full], p))
                self.table[d].append(p)
        for s, d in zip(src, dst):
            self.lens[d] = self.lens[s]
            for p in self.table[d]:
                self.refs[p] += 1
        return copies

    def free(self, seqs):
        for s in seqs:
            for p in self.table[s]:
                self.refs[p] -= 1
            self.table[s], self.lens[s] = [], 0

    def compact(self):
        used = [p for p in range(self.num_pages) if self.refs[p]]
        live = len(used)
        holes = [p for p in range(live) if not self.refs[p]]
        movers = [p for p in used if p >= live]
        new = dict(zip(movers, holes))
        for s, d in new.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
        self.table = [[new.get(p, p) for p in row] for row in self.table]
        return list(new.items())


def make(n_seq, max_pages, num_pages, ps, layers=2, Hkv=2, bits=(4, 3), qjl=128):
    pt = tq.PageTable.allocate(n_seq, max_pages, num_pages, ps)
    pools = [tq.Cache.allocate(num_pages, Hkv, ps, *bits, qjl_m=qjl) for _ in range(layers)]
    g = torch.Generator(device="cuda").manual_seed(1)
    for c in pools:
        for n in ARRAYS:
            a = getattr(c, n)
            if a is not None:
                a.view(torch.uint8).random_(0, 256, generator=g)  # any bits, NaN among them
    return pt, pools


def raw(pools):
    return [[None if getattr(c, n) is None else getattr(c, n).view(torch.uint8).clone() for n in ARRAYS] for c in pools]


def same_tables(pt, m):
    torch.cuda.synchronize()
    assert pt.seq_lens.tolist() == m.lens
    assert pt.refs.tolist() == m.refs
    want = [row + [-1] * (m.max_pages - len(row)) for row in m.table]
    assert pt.table.tolist() == want


def copied(before, pools, pairs):
    for arrs, c in zip(before, pools):
        for a, n in zip(arrs, ARRAYS):
            if a is None:
                continue
            want = a.clone()
            for s, d in pairs:
                want[d] = a[s]
            assert torch.equal(getattr(c, n).view(torch.uint8), want), n


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("ps,num_pages,n_seq,seed", [(16, 40, 6, 0), (64, 23, 9, 1), (16, 5003, 40, 2), (48, 300, 17, 3)])
def test_random_life(ps, num_pages, n_seq, seed):
    r = random.Random(seed)
    max_pages = max(4, num_pages // 4)
    pt, pools = make(n_seq, max_pages, num_pages, ps)
    m = Model(n_seq, max_pages, num_pages, ps)
    for step in range(60):
        op = r.choice(["reserve", "reserve", "fork", "free", "compact"])
        before = raw(pools)
        if op == "reserve":
            seqs = r.sample(range(n_seq), r.randint(0, n_seq))
            grow = [r.choice([0, 1, ps - 1, ps, ps + 1, r.randint(0, 3 * ps)]) for _ in seqs]
            need = sum(-(-(m.lens[s] + a) // ps) - -(-m.lens[s] // ps) for s, a in zip(seqs, grow))
            # (a partly filled last page is this sequence's alone: fork copies it)
            if need > len(m.free_pages()) or any(m.lens[s] + a > max_pages * ps for s, a in zip(seqs, grow)):
                continue
            pad = r.randint(0, 5)
            slots = tq.pages_reserve(pt, ints(seqs), ints(grow), sum(grow) + pad)
            assert slots.tolist() == m.reserve(seqs, grow) + [-1] * pad
        elif op == "fork":
            empty = [s for s in range(n_seq) if m.lens[s] == 0]
            dst = r.sample(empty, r.randint(0, len(empty)))
            src = [s for s in range(n_seq) if s not in dst]
            if not src:
                continue
            src = [r.choice(src) for _ in dst]
            if sum(m.lens[s] % ps != 0 for s in src) > len(m.free_pages()):
                continue
            tq.pages_fork(pt, ints(src), ints(dst), pools)
            copied(before, pools, m.fork(src, dst))
        elif op == "free":
            seqs = r.sample(range(n_seq), r.randint(0, n_seq // 2))
            m.free(seqs)
            tq.pages_free(pt, ints(seqs + seqs[:1]))  # the first listed twice: the second is left as it is
        else:
            tq.pages_compact(pt, pools)
            copied(before, pools, m.compact())
        same_tables(pt, m)
        pt.check()


def test_refused_requests_change_nothing():
    ps, P = 16, 12
    pt, pools = make(5, 6, P, ps, layers=1)
    tq.pages_reserve(pt, ints([0, 1]), ints([40, 50]), 90)  # 3 + 4 pages
    tq.pages_fork(pt, ints([1]), ints([2]), pools)          # one more
    pt.check()
    state = lambda: [t.clone() for t in (pt.table, pt.seq_lens, pt.refs)] + [a for l in raw(pools) for a in l]
    before = state()

    def refused(call, text):
        out = call()
        torch.cuda.synchronize()
        with pytest.raises(ValueError, match=text):
            pt.check()
        pt.check()
        if isinstance(out, torch.Tensor):
            assert (out == -1).all()
        for a, b in zip(before, state()):
            assert torch.equal(a, b)

    refused(lambda: tq.pages_reserve(pt, ints([0, 3]), ints([8, 81]), 100), "not enough free pages")  # needs 6 of 4
    refused(lambda: tq.pages_reserve(pt, ints([0, 5]), ints([1, 1]), 4), "out of range")
    refused(lambda: tq.pages_reserve(pt, ints([0, -1]), ints([1, 1]), 4), "out of range")
    refused(lambda: tq.pages_reserve(pt, ints([0, 0]), ints([1, 1]), 4), "listed twice")
    refused(lambda: tq.pages_reserve(pt, ints([0]), ints([-1]), 4), "bad length")
    refused(lambda: tq.pages_reserve(pt, ints([0]), ints([57]), 99), "bad length")     # past six pages
    refused(lambda: tq.pages_reserve(pt, ints([0]), ints([5]), 4), "bad length")       # more tokens than slots
    refused(lambda: tq.pages_fork(pt, ints([0]), ints([1]), pools), "not empty")
    refused(lambda: tq.pages_fork(pt, ints([0, 0]), ints([3, 3]), pools), "listed twice")
    refused(lambda: tq.pages_fork(pt, ints([0, 3]), ints([3, 4]), pools), "not empty")  # a source is a target
    refused(lambda: tq.pages_fork(pt, ints([7]), ints([3]), pools), "out of range")
    refused(lambda: tq.pages_free(pt, ints([9, -3])), "out of range")
    # a page shared by hand: growth inside it is refused
    last = pt.table[0, 2].item()
    pt.refs[last] = 2
    before = state()
    refused(lambda: tq.pages_reserve(pt, ints([0]), ints([1]), 4), "shared page")


def test_more_layers_than_one_launch_takes_and_no_layers():
    pt, pools = make(4, 4, 9, 16, layers=67, Hkv=1, bits=(2, 2), qjl=0)
    m = Model(4, 4, 9, 16)
    assert tq.pages_reserve(pt, ints([2]), ints([20]), 20).tolist() == m.reserve([2], [20])
    before = raw(pools)
    tq.pages_fork(pt, ints([2, 2]), ints([0, 3]), pools)
    copied(before, pools, m.fork([2, 2], [0, 3]))
    m.free([2])
    tq.pages_free(pt, ints([2]))
    before = raw(pools)
    tq.pages_compact(pt, pools)
    copied(before, pools, m.compact())
    same_tables(pt, m)
    tq.pages_fork(pt, ints([0]), ints([1]), [])
    m.fork([0], [1])
    same_tables(pt, m)


def test_copy_list():
    _, pools = make(1, 1, 30, 32, layers=3)
    before = raw(pools)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pairs = [(3, 7), (4, 8), (5, 5), (3, 29), (0, 1)]
    tq.pages_copy(pools, ints([s for s, _ in pairs]), ints([d for _, d in pairs]), status=status)
    copied(before, pools, pairs)
    assert status.item() == 0
    before = raw(pools)
    tq.pages_copy(pools, ints([2, 30, -1, 6]), ints([9, 0, 0, 10]), status=status)
    copied(before, pools, [(2, 9), (6, 10)])
    assert status.item() == tq.TQ_PAGES_BAD_INDEX
    tq.pages_copy(pools, ints([]), ints([]))


def test_captured_step_replays():
    """free + fork captured once: each replay reads the table as it is then."""
    pt, pools = make(8, 8, 40, 16)
    m = Model(8, 8, 40, 16)
    m.reserve([0, 1], [37, 60])
    tq.pages_reserve(pt, ints([0, 1]), ints([37, 60]), 97)
    src, dst, fives = ints([0, 1, 0]), ints([4, 5, 6]), ints([5, 5, 5])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        tq.pages_free(pt, dst)
        tq.pages_fork(pt, src, dst, pools)
        slots = tq.pages_reserve(pt, dst, fives, 15)
    for _ in range(3):
        g.replay()
        m.free([4, 5, 6])
        m.fork([0, 1, 0], [4, 5, 6])
        want = m.reserve([4, 5, 6], [5, 5, 5])
        torch.cuda.synchronize()
        assert slots.tolist() == want
        same_tables(pt, m)
        m.reserve([0], [3])
        tq.pages_reserve(pt, ints([0]), ints([3]), 3)
    pt.check()
