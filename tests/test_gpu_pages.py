"""The pages of a cache (kda_pages_resize, kda_pages_fork, kda_pages_compact) against a plain form."""
import random

import pytest
import torch

import cache8_ref as ref
from gated_delta_rule_46_gb300 import KDAError, check_device_status, kda, pages_compact, pages_fork, pages_resize
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
ARG, PAGES = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_NO_PAGES


class Both:
    """The plain form and the device's state side by side."""

    def __init__(self, rows, cols, pages, ps, dev, pools=True):
        self.m, self.dev, self.ps = ref.Pages(rows, cols, pages, ps), dev, ps
        g = torch.Generator().manual_seed(rows + pages)
        # a page of 16-byte multiples, of 4, of an odd number of bytes, of more than one copy unit, and of none
        self.host = [torch.randint(0, 255, s, dtype=torch.uint8, generator=g) if t is torch.uint8 else
                     torch.randn(s, generator=g).to(t) for s, t in
                     (((pages, 2, ps, 32), torch.uint8), ((pages, 3), torch.float32), ((pages, 7), torch.uint8),
                      ((pages, 5000), torch.float32), ((pages, 0), torch.float32))] if pools else []
        self.pools = [t.to(dev) for t in self.host]
        self.lens = [0] * rows
        self.status = torch.zeros(4, dtype=torch.int32, device=dev)
        self.load()

    def load(self):
        """The device's state from the plain one."""
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=self.dev)  # noqa: E731
        m = self.m
        self.table = i32(m.table).reshape(len(m.table), m.cols)
        self.held, self.refs, self.dlens = i32(m.held), i32(m.refs), i32(self.lens)

    def check(self):
        m = self.m
        assert self.table.tolist() == m.table
        assert self.held.tolist() == m.held
        assert self.refs.tolist() == m.refs
        assert self.dlens.tolist() == self.lens
        for i, (a, b) in enumerate(zip(self.pools, self.host)):
            assert torch.equal(a.cpu(), b), f"pool {i}"
        st, want = check_device_status(self.status), {{"arg": ARG, "pages": PAGES}[e] for e in m.errors}
        assert st in want if want else st == kda.KDA_OK, (st, m.errors)
        m.errors.clear()
        self.status.zero_()

    def resize(self, tokens, check=True):
        pages_resize(self.table, self.held, self.refs, torch.tensor(tokens, dtype=torch.int32, device=self.dev), self.ps,
                     status=self.status)
        self.m.resize(tokens)
        if check:
            self.check()

    def fork(self, src, dst):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=self.dev)  # noqa: E731
        pages_fork(self.pools, self.table, self.held, self.refs, self.dlens, i32(src), i32(dst), self.ps, status=self.status)
        self.m.fork(self.host, self.lens, src, dst)
        self.check()

    def set_lens(self, lens):
        self.lens[:] = lens
        self.dlens.copy_(torch.tensor(lens, dtype=torch.int32))

    def compact(self):
        to, live = pages_compact(self.pools, self.table, self.refs, status=self.status)
        want = self.m.compact(self.host)
        assert to.tolist() == want[0] and live.tolist() == [want[1]]
        self.check()


def test_resize_small():
    dev = need_gpu()
    b = Both(4, 5, 12, 16, dev)
    b.resize([1, 16, 17, 0])
    b.resize([33, -1, 0, 80])
    b.resize([0, 1, 0, 0])
    b.resize([0, 0, 0, 0])
    assert not b.refs.any()


def test_resize_out_of_pages():
    """What is left goes to the first rows; a later call serves the others."""
    dev = need_gpu()
    b = Both(5, 8, 10, 16, dev)
    b.resize([16 * 4, 16 * 3, 16 * 5, 16, 0])
    assert b.held.tolist() == [4, 3, 3, 0, 0]
    b.resize([16, -1, 16 * 5, 16, 16])
    assert b.held.tolist() == [1, 3, 5, 1, 0]
    b.resize([16, 0, 0, 16, 16])


def test_resize_malformed():
    dev = need_gpu()
    b = Both(5, 4, 20, 16, dev)
    b.resize([64, 64, 64, 64, 0])
    b.resize([65, 64, -9, 2 ** 31 - 1, 16])                              # past the table: left as they are
    b.m.held[1], b.m.held[2] = 7, -1                                     # no such rows
    b.m.table[0][1], b.m.table[0][2], b.m.table[0][3] = 99, -5, b.m.free()[-1]
    b.load()
    b.resize([0, 0, 16, 0, 32])
    b.m.refs[3] = -1                                                     # kept from use
    b.m.held[1] = b.m.held[2] = 0
    b.load()
    b.resize([64, 0, 0, 0, 0])
    assert 3 not in b.table[0].tolist()


def test_pages_kept_from_use_are_shared():
    """A negative count stays what it is: rows that share such a page give it back, and it is never handed out."""
    dev = need_gpu()
    b = Both(6, 4, 14, 16, dev)
    b.m.refs[2] = b.m.refs[5] = -1
    b.m.refs[7] = -2 ** 31
    b.m.table[0][:3], b.m.held[0] = [2, 7, 5], 3
    b.lens[0] = 40
    b.load()
    b.fork([0, 0, 0], [1, 2, 3])
    b.resize([-1, 0, 60, 16, 64, 64])
    b.resize([0] * 6)
    assert b.refs.tolist() == [0, 0, -1, 0, 0, -1, 0, -2 ** 31] + [0] * 6
    b.resize([64] * 6)
    assert not {2, 5, 7} & set(b.table.flatten().tolist())


@pytest.mark.parametrize("rows,cols,pages,ps", [(1, 1, 1, 1), (3000, 3, 5000, 64), (17, 5000, 70001, 1), (9000, 20, 140000, 1024)])
def test_resize_sizes(rows, cols, pages, ps):
    """More rows and pages than one round of the kernel takes, rows of thousands of pages, pages of one token."""
    dev = need_gpu()
    b = Both(rows, cols, pages, ps, dev, pools=False)
    r = random.Random(rows)
    for _ in range(3):
        b.resize([r.choice([-1, 0, r.randrange(cols * ps + 1)]) for _ in range(rows)])


def test_fork():
    dev = need_gpu()
    b = Both(8, 5, 24, 16, dev)
    lens = [40, 48, 0, 7, 0, 0, 0, 0]
    b.resize(lens)
    b.set_lens(lens)
    b.fork([0, 1, -1, 2], [4, 5, 3, 6])                                  # a copy, none, padding, an empty row
    assert b.held.tolist()[4:] == [3, 3, 0, 0]
    b.resize([0, -1, -1, -1, -1, -1, -1, -1])                            # the source ends, what it shared stays
    b.fork([4, 4], [0, 7])
    b.resize([0] * 8)
    assert not b.refs.any()


def test_fork_pairs_that_do_not_hold():
    dev = need_gpu()
    b = Both(10, 5, 30, 16, dev)
    lens = [40, 48, 16, 7, 0, 0, 0, 0, 0, 0]
    b.resize(lens)
    b.set_lens(lens)
    b.fork([0, 1, 0], [4, 4, 5])                                         # one destination twice: the first
    b.fork([0, 6], [6, 7])                                               # a destination that is a source
    b.fork([0, 3], [0, 8])                                               # itself
    b.fork([0, 1], [1, 9])                                               # holds pages
    b.fork([10, 0, -3], [5, 10, 77])                                     # outside the table
    b.resize([0] * 10)
    b.resize(lens)
    for bad in (49, -1, 2 ** 31 - 1):                                    # more tokens than pages
        b.set_lens([40, bad, 16, 7, 0, 0, 0, 0, 0, 0])
        b.fork([1], [5])
    b.set_lens([40, 47, 33, 7, 0, 0, 0, 0, 0, 0])
    b.m.table[0][1], b.m.table[1][2], b.m.held[2] = 1 << 20, -1, 9       # no pages of the cache
    b.load()
    b.fork([0, 1, 2], [5, 6, 7])
    assert b.table[5].tolist()[1] == -1


def test_fork_out_of_pages():
    dev = need_gpu()
    b = Both(8, 3, 6, 16, dev)
    lens = [30, 16, 20, 0, 0, 0, 0, 0]
    b.resize(lens)
    b.set_lens(lens)
    b.fork([0, 1, 2, 2], [4, 5, 6, 7])
    assert b.held.tolist() == [2, 1, 2, 0, 2, 1, 0, 0]


def test_compact():
    dev = need_gpu()
    b = Both(6, 6, 25, 16, dev)
    b.resize([50, 60, 16, 90, 1, 0])
    b.compact()                                                          # nothing to do
    b.resize([0, -1, 0, -1, -1, -1])
    b.compact()
    assert b.refs.tolist() == sorted(b.refs.tolist(), reverse=True)
    b.resize([16, 0, 33, 0, 0, 5])
    b.set_lens([16, 0, 33, 0, 0, 5])
    b.fork([2, 5], [1, 3])
    b.resize([0, -1, 0, -1, -1, -1])
    b.compact()
    b.resize([0] * 6)
    b.compact()                                                          # no page in use
    b.m.refs[20], b.m.refs[24] = -1, 3                                   # pages of other holders move too
    b.load()
    b.compact()


def test_compact_malformed_table():
    dev = need_gpu()
    b = Both(3, 4, 10, 16, dev)
    b.resize([64, 48, 16])
    b.m.table[0][1], b.m.table[1][0], b.m.table[2][0] = 10, 9, -8
    b.load()
    b.compact()


def test_compact_without_table_and_pools():
    dev = need_gpu()
    refs = torch.tensor([0, 2, 0, 1], dtype=torch.int32, device=dev)
    to, live = pages_compact([], None, refs)
    assert to.tolist() == [-1, 1, -1, 0] and live.tolist() == [2] and refs.tolist() == [1, 2, 0, 0]
    to, live = pages_compact([], None, refs[:0])
    assert to.numel() == 0 and live.tolist() == [0]


@pytest.mark.parametrize("pages", [300, 70001])
def test_compact_many_pages(pages):
    dev = need_gpu()
    r = random.Random(pages)
    b = Both(40, pages // 20, pages, 16, dev, pools=False)
    b.host = [torch.randint(0, 255, (pages, 48), dtype=torch.uint8)]
    b.pools = [b.host[0].to(dev)]
    for _ in range(2):
        b.resize([r.choice([0, r.randrange(pages // 20 * 16)]) for _ in range(40)])
        b.resize([r.choice([-1, 0]) for _ in range(40)])
        b.compact()


def test_many_pools():
    """More pools than one launch takes."""
    dev = need_gpu()
    b = Both(4, 3, 9, 16, dev, pools=False)
    b.host = [torch.randn(9, 1 + i % 9) for i in range(300)]
    b.pools = [t.to(dev) for t in b.host]
    b.resize([40, 20, 0, 0])
    b.set_lens([40, 20, 0, 0])
    b.fork([0, 1], [2, 3])
    b.resize([0, -1, -1, -1])
    b.compact()


def test_random_runs():
    dev = need_gpu()
    r = random.Random(1)
    b = Both(30, 12, 160, 16, dev)
    for _ in range(12):
        tokens = [r.choice([-1, -1, 0, r.randrange(16 * 12)]) for _ in range(30)]
        b.resize(tokens)
        b.set_lens([r.randrange(16 * h + 1) for h in b.m.held])
        empty = [i for i in range(30) if b.m.held[i] == 0]
        used = [i for i in range(30) if b.m.held[i]]
        if used and empty:
            dst = r.sample(empty, r.randrange(len(empty) + 1))
            b.fork([r.choice(used) for _ in dst], dst)
        b.compact()


def test_many_forks():
    """More pairs than one round takes, sources shared by many."""
    dev = need_gpu()
    rows, ps = 5000, 16
    b = Both(rows, 4, 9000, ps, dev, pools=False)
    b.host = [torch.randn(9000, 4)]
    b.pools = [b.host[0].to(dev)]
    lens = [(i * 7) % 64 for i in range(500)] + [0] * (rows - 500)
    b.resize(lens)
    b.set_lens(lens)
    r = random.Random(3)
    dst = list(range(500, rows))
    r.shuffle(dst)
    b.fork([r.randrange(-1, 500) for _ in dst], dst)
    b.resize([0] * 500 + [-1] * (rows - 500))
    b.compact()


def test_no_rows():
    dev = need_gpu()
    e = torch.zeros(0, dtype=torch.int32, device=dev)
    pages_resize(e.reshape(0, 3), e, torch.zeros(4, dtype=torch.int32, device=dev), e, 16)
    pages_fork([], torch.zeros(2, 3, dtype=torch.int32, device=dev), e.new_zeros(2), e.new_zeros(4), e.new_zeros(2), e, e, 16)


def test_refusals():
    dev = need_gpu()
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
    table, held, refs = i(3, 4), i(3), i(9)
    with pytest.raises(KDAError):
        pages_resize(table, held, refs, i(3), 24)
    with pytest.raises(ValueError):
        pages_resize(table, held, refs, i(2), 16)
    with pytest.raises(TypeError):
        pages_resize(table, held.long(), refs, i(3), 16)
    with pytest.raises(ValueError):
        pages_resize(table.t(), i(4), refs, i(4), 16)
    with pytest.raises(KDAError):
        pages_resize(table, held, i(70000), i(3), 16, workspace=torch.zeros(8, dtype=torch.uint8, device=dev))
    pool = torch.zeros(9, 4, device=dev)
    for bad in (pool[:8], pool.cpu(), pool.t().contiguous().t()):
        with pytest.raises(ValueError):
            pages_fork([pool, bad], table, held, refs, i(3), i(1), i(1), 16)
        with pytest.raises(ValueError):
            pages_compact([bad], table, refs)
    with pytest.raises(ValueError):
        pages_fork([pool], table, held, refs, i(3), i(1), i(2), 16)
    with pytest.raises(TypeError):
        pages_fork([None], table, held, refs, i(3), i(1), i(1), 16)
