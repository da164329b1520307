"""The pages of a cache (include/kda_pages.h) against plain lists
(oracle/attn.Pool): whole numbers and moved bits, so everything is equal."""
import random

import numpy as np
import pytest

from oracle.attn import Pool

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU-only container
    pytest.skip("no GPU", allow_module_level=True)

import gated_delta_rule_amd as kda  # noqa: E402


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Both:
    """A pool on the device beside the same one as lists."""

    def __init__(self, n_slots, max_pages, n_pages, page, shape=(2, 24), dtype=torch.float32, tensors=1):
        self.page = page
        self.plain = Pool([[-1] * max_pages for _ in range(n_slots)], [0] * n_slots, [0] * n_pages, page,
                          list(range(n_pages)))
        self.table = torch.full((n_slots, max_pages), -1, dtype=torch.int32, device="cuda")
        self.lengths, self.refs = ints([0] * n_slots), ints([0] * n_pages)
        self.pages = []
        for t in range(tensors):   # every page holds its first number
            x = torch.empty((n_pages,) + tuple(shape), dtype=dtype, device="cuda")
            x[:] = torch.arange(n_pages, device="cuda").view((-1,) + (1,) * len(shape)).to(dtype) + 1000 * t
            self.pages.append(x)

    def resize(self, want):
        ok = kda.kv_resize(self.table, self.lengths, self.refs, ints(want), self.page)
        assert ok.tolist() == self.plain.resize(want)
        self.same()

    def fork(self, src, dst):
        ok = kda.kv_fork(self.table, self.lengths, self.refs, ints(src), ints(dst), self.pages, self.page)
        assert ok.tolist() == self.plain.fork(src, dst)
        self.same()

    def compact(self, in_place=False):
        out = dict(table_out=self.table, refs_out=self.refs) if in_place else {}
        table, refs, n_live = kda.kv_compact(self.table, self.lengths, self.refs, self.pages, self.page, **out)
        if not in_place:
            self.same(data=False)   # (the inputs stay)
        want_table, want_refs, want_live = self.plain.compact()
        assert (table.tolist(), refs.tolist(), n_live.tolist()) == (want_table, want_refs, [want_live])
        self.table, self.refs, self.plain.table, self.plain.refs = table, refs, want_table, want_refs
        self.same()

    def same(self, data=True):
        assert self.table.tolist() == self.plain.table
        assert self.lengths.tolist() == self.plain.lengths
        assert self.refs.tolist() == self.plain.refs
        for t, x in enumerate(self.pages if data else []):
            first = x.flatten(1)
            assert (first == first[:, :1]).all()
            assert first[:, 0].tolist() == [p + 1000 * t for p in self.plain.data]


def test_by_hand():
    b = Both(4, 4, 8, 16)
    b.resize([33, 0, 16, 1])            # pages 0 1 2 | | 3 | 4
    assert b.plain.table[:3] == [[0, 1, 2, -1], [-1] * 4, [3, -1, -1, -1]]
    b.fork([0], [1])                    # shares 0 and 1, copies 2 into 5
    assert b.plain.table[1] == [0, 1, 5, -1] and b.plain.refs[:6] == [2, 2, 1, 1, 1, 1] and b.plain.data[5] == 2
    b.resize([0, 33, 64, 1])            # frees the source; slot 2 takes pages 2, 6, 7
    assert b.plain.table[2] == [3, 2, 6, 7]
    b.resize([17, 33, 64, 1])           # nothing is left
    assert b.plain.lengths[0] == 0
    b.resize([0, 16, 16, 0])
    b.compact()


def test_cut_back_into_a_shared_page():
    b = Both(3, 4, 8, 16)
    b.resize([32, 0, 0])
    b.fork([0], [1])                    # both pages are shared
    b.resize([32, 30, 0])               # the second one is open in the branch, and shared
    assert b.plain.table[1][:2] == [0, 1] and b.plain.refs[1] == 2
    b.fork([1], [2])                    # a branch of it has a copy
    assert b.plain.table[2][:2] == [0, 2] and b.plain.data[2] == 1 and b.plain.refs[:3] == [3, 2, 1]
    b.resize([32, 0, 40])


@pytest.mark.parametrize("seed", range(6))
def test_random_steps(seed):
    r = random.Random(seed)
    page = r.choice([16, 32, 256])
    n_slots, max_pages = r.randint(1, 40), r.randint(1, 12)
    b = Both(n_slots, max_pages, r.randint(1, n_slots * max_pages), page, shape=(r.choice([4, 4096, 5000]),),
             tensors=r.choice([1, 1, 3]))
    for _ in range(30):
        what = r.choice(["resize", "resize", "fork", "fork", "compact"])
        if what == "resize":
            b.resize([r.choice([w, w, 0, w + r.randint(-20, 40), r.randint(-5, max_pages * page + 40)])
                      for w in b.plain.lengths])
        elif what == "fork":
            n = r.randint(1, 2 * n_slots)
            b.fork([r.randint(-1, n_slots) for _ in range(n)], [r.randint(-1, n_slots) for _ in range(n)])
        else:
            b.compact(in_place=r.random() < 0.5)


def test_slots_change_places():
    b = Both(3, 3, 12, 16)
    b.resize([20, 35, 48])
    b.fork([1, 2, 0], [0, 1, 2])        # each from the one behind it, as they were
    assert b.plain.lengths == [35, 48, 20]
    b.fork([0, 0, 0], [0, 1, 2])
    assert b.plain.lengths == [35] * 3


def test_entries_that_are_no_pages():
    b = Both(3, 4, 6, 16)
    b.resize([40, 20, 0])
    for slot, col, bad in ((0, 1, 6), (0, 2, -9), (1, 0, 2 ** 31 - 1)):
        b.table[slot, col] = bad
        b.plain.table[slot][col] = bad
    b.fork([0, 1], [2, 0])
    b.compact()
    b.resize([0, 5, 0])


def test_many_slots_and_pages():
    # more slots than threads, counts past one step of the search
    r = random.Random(11)
    b = Both(2500, 20, 60000, 16, shape=(4,))
    b.resize([r.randint(0, 320) for _ in range(2500)])
    b.resize([r.randint(0, 320) for _ in range(2500)])
    b.fork([r.randrange(2500) for _ in range(2400)], r.sample(range(2500), 2400))
    b.compact()
    b.resize([320] * 2500)
    b.compact(in_place=True)


def test_too_few_pages_refuse_in_order():
    b = Both(5, 8, 10, 16)
    b.resize([16 * 4, 16 * 3, 16 * 8, 16, 0])     # the third finds 3 left, and so does the fourth
    assert b.plain.lengths == [64, 48, 0, 0, 0]
    b.resize([64, 33, 0, 16, 0])
    b.fork([1, 1, 1], [2, 4, 2])
    b.fork([1, 1], [4, 3])
    b.resize([16 * 8] * 5)


def test_no_slots_no_pages():
    table = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    none = ints([])
    assert kda.kv_resize(table, none, none, none, 16).shape == (0,)
    pages = torch.empty((0, 4), device="cuda")
    t, refs, n_live = kda.kv_compact(table, none, none, pages, 16)
    assert t.shape == (0, 4) and refs.shape == (0,) and n_live.tolist() == [0]
    wide = torch.full((2, 0), 0, dtype=torch.int32, device="cuda")
    lengths, refs = ints([5, 0]), ints([0, 0])
    assert kda.kv_resize(wide, lengths, refs, ints([7, 0]), 16).tolist() == [1, 1] and lengths.tolist() == [0, 0]
    assert kda.kv_fork(wide, lengths, refs, ints([0]), ints([1]), torch.zeros(2, 4, device="cuda"), 16).tolist() == [1]


def test_data_with_strides_and_odd_sizes():
    # a page of a wider pool, 16-byte pieces that do not fill the last step
    pool = torch.arange(6 * 3 * 4108, device="cuda", dtype=torch.float32).view(6, 3, 4108)
    want = pool.clone()
    table, lengths, refs = ints([[3, 4], [-1, -1]]), ints([20, 0]), ints([0, 0, 0, 1, 1, 0])
    assert kda.kv_fork(table, lengths, refs, ints([0]), ints([1]), pool[:, 1], 16).tolist() == [1]
    want[0, 1] = want[4, 1]
    assert torch.equal(pool, want) and table.tolist() == [[3, 4], [3, 0]] and refs.tolist() == [1, 0, 0, 2, 1, 0]
    t, r, n = kda.kv_compact(table, lengths, refs, [pool[:, 0], pool[:, 1, :4104]], 16)
    for p, h in ((3, 1), (4, 2)):
        want[h, 0] = want[p, 0]
        want[h, 1, :4104] = want[p, 1, :4104]
    assert torch.equal(pool, want) and t.tolist() == [[1, 2], [1, 0]] and r.tolist() == [1, 2, 1, 0, 0, 0]


def test_pairs_that_copy_nothing_need_no_page():
    # all pages are held: one open source, one that ends with its page, one without tokens
    table = ints([[0, -1], [1, -1], [2, 3], [-1, -1], [-1, -1], [4, 5]])
    lengths, refs = ints([10, 16, 32, 0, 0, 20]), ints([1] * 6)
    pages = torch.arange(6 * 4, device="cuda", dtype=torch.float32).view(6, 4)
    before = pages.clone()
    ok = kda.kv_fork(table, lengths, refs, ints([0, 1, 0, 5, 3]), ints([3, 4, 5, 5, 2]), pages, 16)
    # the copy of page 0 finds none left, twice (the second time for slot 5); the full page is shared; slot 2 becomes empty
    assert ok.tolist() == [0, 1, 0, 0, 1]
    assert table.tolist() == [[0, -1], [1, -1], [-1, -1], [-1, -1], [1, -1], [4, 5]]
    assert lengths.tolist() == [10, 16, 0, 0, 16, 20] and refs.tolist() == [1, 2, 0, 0, 1, 1]
    assert torch.equal(pages, before)
    # two pages are free now: one copy, a slot onto itself behind the one that finds none
    ok = kda.kv_fork(table, lengths, refs, ints([0, 5, 0, 5, 1]), ints([2, 3, 4, 5, 1]), pages, 16)
    assert ok.tolist() == [1, 1, 0, 1, 1]
    assert table.tolist() == [[0, -1], [1, -1], [2, -1], [4, 3], [1, -1], [4, 5]]
    assert lengths.tolist() == [10, 16, 10, 20, 16, 20] and refs.tolist() == [1, 2, 1, 1, 2, 1]
    before[2], before[3] = before[0], before[5]
    assert torch.equal(pages, before)


@pytest.mark.parametrize("n", [20, 45])
def test_rows_of_several_column_blocks(n):
    # 600 columns: counts and rows in blocks of 256; 12000 and 27000 entries, counted by one workgroup and by many
    r = random.Random(n)
    b = Both(60, 600, 12000, 16, shape=(4,))
    b.resize([r.choice([0, 255 * 16, 256 * 16, 256 * 16 + 1, 512 * 16, 513 * 16, r.randint(4100, 9600), 9599, 9600]) if s < 20 else
              r.randint(0, 600) for s in range(60)])
    b.fork([r.randrange(20) for _ in range(n)], r.sample(range(60), n))
    b.resize([r.choice([w, w // 2, 0]) for w in b.plain.lengths])
    b.fork([r.randrange(60) for _ in range(n)], [r.randrange(60) for _ in range(n)])
    b.compact()


def test_more_slots_than_lds_holds():
    r = random.Random(5)
    b = Both(9000, 3, 24000, 16, shape=(4,))
    b.resize([r.randint(0, 40) for _ in range(9000)])
    n = 10000   # destinations twice and thrice, no slots among them
    b.fork([r.randint(-1, 9000) for _ in range(n)], [r.choice([0, 4095, 8191, 8192, 8999, -1, 9000, r.randrange(9000)]) for _ in range(n)])
    b.resize([r.randint(0, 48) for _ in range(9000)])
    b.fork(list(range(9000)), [(i * 7 + 1) % 9000 for i in range(9000)])
    b.compact(in_place=True)


def test_pages_above_a_megabyte():
    # 66 pieces of 16 KB and a rest, more than the workgroups that share a copy
    b = Both(4, 3, 10, 16, shape=(270340,), tensors=2)
    b.resize([20, 5, 48, 0])
    b.fork([0, 1, 0], [3, 2, 1])
    b.resize([0, 20, 5, 20])
    b.compact()
