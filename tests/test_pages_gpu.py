"""GPU page lists against the token-by-token oracle: every value exactly."""
import numpy as np
import pytest

from oracle.paged4 import Lists

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def attn():
    import exact_io_aware_09_gb300 as m

    return m


class Device:
    """The same lists on the GPU."""

    def __init__(self, attn, B, free, page, width):
        import torch

        self.attn, self.page = attn, page
        i32 = lambda x: torch.as_tensor(np.asarray(x, dtype=np.int32), device="cuda")
        self.table = i32(np.full((B, width), -7))
        self.len, self.free, self.n_free = i32(np.zeros(B)), i32(free), i32([len(free)])
        self.i32 = i32

    def extend(self, n, total=None, first=0, **kw):
        cu = first + np.concatenate([[0], np.cumsum(n)])
        return self.attn.attn_pages_extend(self.table, self.len, self.i32(cu), self.free, self.n_free,
                                           self.page, int(cu[-1]) if total is None else total, **kw)

    def trim(self, keep):
        self.attn.attn_pages_trim(self.table, self.len, self.i32(keep), self.free, self.n_free, self.page)

    def state(self):
        return [x.cpu().numpy().copy() for x in (self.table, self.len, self.free, self.n_free)]

    def same_as(self, lists):
        table, length, free, n_free = self.state()
        assert length.tolist() == lists.len
        assert n_free[0] == len(lists.free) and free[:n_free[0]].tolist() == lists.free
        for row, pages in zip(table, lists.table):
            assert row[:len(pages)].tolist() == pages
        return table


def both(attn, B, n_pages, page, width, seed):
    free = np.random.default_rng(seed).permutation(n_pages).tolist()
    return Lists(B, free, page), Device(attn, B, free, page, width)


# one sequence, a serving batch, more than the sequences of one pass of the kernel (2,048)
@pytest.mark.parametrize("B,page,steps,most", [(1, 16, 12, 90), (5, 16, 12, 40), (64, 64, 10, 300),
                                               (300, 32, 4, 200), (2048, 16, 3, 12),
                                               (2049, 256, 3, 20), (5000, 16, 3, 9)])
def test_growing_and_shrinking(attn, B, page, steps, most):
    rng = np.random.default_rng(B * 31 + page)
    width = -(-steps * most // page) + 1
    a, d = both(attn, B, B * width, page, width, seed=B)
    for step in range(steps):
        n = rng.integers(0, most, size=B, endpoint=True)
        if step % 3 == 1:
            n = np.ones(B, dtype=np.int64)      # a decode step
        elif step % 3 == 2:
            n[rng.random(B) < 0.7] = 0          # most sequences wait
        want = a.extend(n.tolist())
        assert d.extend(n).cpu().tolist() == want
        table = d.same_as(a)
        for b in range(min(B, 50)):             # nothing past a sequence's pages is touched
            assert set(table[b][len(a.table[b]):].tolist()) <= {-7, -1}
        keep = np.array(a.len)
        cut = rng.random(B)
        keep = np.where(cut < 0.4, keep, np.where(cut < 0.9, rng.integers(0, keep, endpoint=True), 0))
        gone = [len(p) for p in a.table]
        a.trim(keep.tolist())
        d.trim(keep)
        table = d.same_as(a)
        for b in range(min(B, 50)):
            assert (table[b][len(a.table[b]):gone[b]] == -1).all()
    assert attn.attn_poll_status() == 0


@pytest.mark.parametrize("B,most,pages", [(3, 70000, 9000), (40, 4000, 6000), (2500, 60, 12000), (40, 4000, 20)])
def test_many_rows(attn, B, most, pages):
    """Whole prompts, whose slots take a launch of their own; the last list is too short for them."""
    rng = np.random.default_rng(B)
    a, d = both(attn, B, pages, 16, most // 16 + 3, seed=2)
    first = rng.integers(0, 20, size=B)
    if pages > 20:
        a.extend(first.tolist())
        d.extend(first)
    n = rng.integers(most // 2, most, size=B)
    total = int(n.sum())
    assert total >= 1 << 16
    before = d.state()
    want = a.extend(n.tolist())
    got = d.extend(n, total=total + 9, first=5).cpu().numpy()
    if want is None:
        assert attn.attn_poll_status() == -9 and (got == -1).all()
        assert all(np.array_equal(x, y) for x, y in zip(before, d.state()))
        return
    assert got[:5].tolist() == [-1] * 5 and got[5 + total:].tolist() == [-1] * 4
    assert np.array_equal(got[5:5 + total], want)
    d.same_as(a)
    keep = np.where(rng.random(B) < 0.5, first, 0)
    a.trim(keep.tolist())
    d.trim(keep)
    d.same_as(a)
    assert attn.attn_poll_status() == 0


def test_trim_undoes_an_extension(attn):
    rng = np.random.default_rng(3)
    _, d = both(attn, 40, 700, 16, 30, seed=9)
    first = rng.integers(0, 100, size=40)
    d.extend(first)
    before = d.state()
    d.extend(rng.integers(0, 150, size=40))
    d.trim(first)
    after = d.state()
    assert all(np.array_equal(x, y) for x, y in zip(before[1:], after[1:]))
    assert np.array_equal(np.maximum(before[0], -1), np.maximum(after[0], -1))
    assert attn.attn_poll_status() == 0


@pytest.mark.parametrize("first,behind", [(0, 7), (3, 0), (5, 4098)])
def test_rows_of_no_sequence(attn, first, behind):
    a, d = both(attn, 3, 60, 16, 20, seed=1)
    n = [20, 0, 33]
    slots = d.extend(n, total=first + 53 + behind, first=first).cpu().tolist()
    assert slots == [-1] * first + a.extend(n) + [-1] * behind
    d.same_as(a)
    assert attn.attn_poll_status() == 0


def test_no_sequences_and_no_tokens(attn):
    import torch

    a, d = both(attn, 4, 9, 16, 2, seed=1)
    assert d.extend([0, 0, 0, 0]).numel() == 0
    d.trim([0, 0, 0, 0])
    d.same_as(a)
    none = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = attn.attn_pages_extend(none, cu[:0], cu, d.free, d.n_free, 16, 5)
    assert got.cpu().tolist() == [-1] * 5
    assert attn.attn_poll_status() == 0


@pytest.mark.parametrize("many", [3, 4096])
def test_too_few_pages_change_nothing(attn, many):
    B = many
    _, d = both(attn, B, B + 2, 16, 8, seed=4)
    d.extend([16] * B)                       # two pages are left
    before = d.state()
    slots = d.extend([1, 20, 1] + [0] * (B - 3))   # four are wanted
    assert attn.attn_poll_status() == -9
    assert (slots == -1).all()
    assert all(np.array_equal(x, y) for x, y in zip(before, d.state()))
    assert (d.extend([1, 16, 0] + [0] * (B - 3)) >= 0).all()    # two do
    assert attn.attn_poll_status() == 0 and d.state()[3][0] == 0


def test_bad_lengths_change_nothing(attn):
    import torch

    _, d = both(attn, 3, 40, 16, 4, seed=4)
    d.extend([5, 16, 40])

    def refused(call):
        before = d.state()
        out = call()
        assert attn.attn_poll_status() == -8
        assert all(np.array_equal(x, y) for x, y in zip(before, d.state()))
        assert out is None or (out == -1).all()

    refused(lambda: d.extend([1, 49, 1]))              # past the table's four pages
    refused(lambda: d.extend([3, -1, 3]))
    refused(lambda: d.extend([3, 3, 3], total=8))      # past the packed rows
    refused(lambda: d.extend([1, 1, 1], first=-1))
    refused(lambda: d.trim([5, 17, 40]))               # longer than it is
    refused(lambda: d.trim([5, -1, 40]))
    for wrong in (-1, 41):
        was = d.n_free.clone()
        d.n_free.fill_(wrong)
        refused(lambda: d.extend([1, 1, 1]))
        refused(lambda: d.trim([5, 16, 40]))
        d.n_free.copy_(was)
    was = d.n_free.clone()
    d.n_free.fill_(40)                                 # no room on the list
    refused(lambda: d.trim([0, 0, 0]))
    d.n_free.copy_(was)
    was = d.len.clone()
    d.len[1] = -5
    refused(lambda: d.extend([1, 1, 1]))
    refused(lambda: d.trim([5, 0, 40]))
    d.len.copy_(was)
    d.extend([1, 1, 1])
    assert attn.attn_poll_status() == 0
    assert torch.equal(d.len.cpu(), torch.tensor([6, 17, 41], dtype=torch.int32))


def test_a_bad_entry_of_the_list(attn):
    _, d = both(attn, 2, 8, 16, 4, seed=4)
    d.free[7] = 8                                # the pool has pages 0 .. 7
    slots = d.extend([17, 3]).cpu().numpy()
    assert attn.attn_poll_status() == -8
    good = d.free.cpu().numpy()[[6, 5]]
    assert (slots[:16] == -1).all() and slots[16] == good[0] * 16 and slots[17] == good[1] * 16


def test_captured_steps(attn):
    """A captured decode step allocates its own pages, and a captured trim returns drafted tokens'."""
    import torch

    a, d = both(attn, 6, 64, 16, 10, seed=8)
    a.extend([3, 15, 16, 17, 0, 30])
    d.extend([3, 15, 16, 17, 0, 30])
    cu = d.i32(np.arange(7) * 4)
    slots = torch.empty(24, dtype=torch.int32, device="cuda")
    keep = torch.empty(6, dtype=torch.int32, device="cuda")

    def step():
        keep.copy_(d.len)
        attn.attn_pages_extend(d.table, d.len, cu, d.free, d.n_free, 16, 24, slots=slots)
        keep.add_(1)                              # one of four drafted tokens is accepted
        attn.attn_pages_trim(d.table, d.len, keep, d.free, d.n_free, 16)

    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        step()
    d.same_as(a)                                  # capturing ran nothing
    for _ in range(40):
        g.replay()
        length = list(a.len)
        assert slots.cpu().tolist() == a.extend([4] * 6)
        a.trim([x + 1 for x in length])
        d.same_as(a)
    assert attn.attn_poll_status() == 0


def test_another_stream(attn):
    import torch

    a, d = both(attn, 50, 400, 16, 40, seed=8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    rng = np.random.default_rng(0)
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    n = rng.integers(0, 60, size=50)
    slots = d.extend(n, stream=side)
    side.synchronize()
    assert slots.cpu().tolist() == a.extend(n.tolist())
    assert attn.attn_poll_status(side) == 0


@pytest.mark.parametrize("B,most", [(3, 60), (70, 1500)])   # one block, a cluster of eight
def test_trim_of_entries_outside_the_pool(attn, B, most):
    """They are reported, go onto the list as they are, and come off it again as an extension reports them."""
    rng = np.random.default_rng(B)
    for wrong in (-1, B * 100, 2147483647, -2147483648):
        a, d = both(attn, B, B * 100, 16, 100, seed=5)
        n = rng.integers(most // 2, most, size=B)
        a.extend(n.tolist())
        d.extend(n)
        first = n // 3
        at = len(a.table[1]) - 1                 # the last page of sequence 1
        a.table[1][at] = wrong
        d.table[1, at] = wrong
        d.trim(n)                                # nothing goes back: the entry is not looked at
        assert attn.attn_poll_status() == 0
        a.trim(first.tolist())
        d.trim(first)
        assert attn.attn_poll_status() == -8
        d.same_as(a)
        assert wrong in a.free
        slots = d.extend(n - first).cpu().numpy()
        assert attn.attn_poll_status() == -8
        want = np.array(a.extend((n - first).tolist()))
        bad = np.concatenate([np.isin(np.repeat(a.table[b], 16)[first[b]:n[b]], [wrong]) for b in range(B)])
        assert bad.any() and (slots[bad] == -1).all() and np.array_equal(slots[~bad], want[~bad])
        d.same_as(a)


@pytest.mark.parametrize("n,pages", [(5, 120), (400_000, 120), (400_000, 3)])
def test_the_most_rows(attn, n, pages):
    """2^31 - 1 packed rows, a sequence's tokens the last of them (the last list is too short)."""
    import torch

    T, page = (1 << 31) - 1, 4096
    a, d = both(attn, 1, pages, page, 130, seed=3)
    slots = torch.zeros(T, dtype=torch.int32, device="cuda")
    got = attn.attn_pages_extend(d.table, d.len, d.i32([T - n, T]), d.free, d.n_free, page, T, slots=slots)
    assert got is slots
    want = a.extend([n])
    assert attn.attn_poll_status() == (-9 if want is None else 0)
    assert bool((slots[:T - n] == -1).all())
    tail = slots[T - n:].cpu().numpy()
    assert np.array_equal(tail, np.full(n, -1) if want is None else want)
    d.same_as(a)
