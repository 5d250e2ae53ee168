"""update_pages on the GPU against the same on Python lists (tests/blocks_reference.py): every array,
exactly."""
import random

import pytest

from tests import blocks_reference as ref

pytestmark = pytest.mark.gpu

BOUNDS, NO_PAGES = 6, 8


@pytest.fixture(scope="module")
def mla():
    import mla_latent_kv_paged_gb300 as m
    m.build()
    return m


@pytest.fixture()
def err():
    import torch
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def cum(v):
    return [sum(v[:i]) for i in range(len(v) + 1)]


class State:
    """The GPU's arrays and the same on lists; all pages free, in a shuffled order."""

    def __init__(self, B, max_pages, num_pages, page, seed=0):
        import torch
        self.rng = random.Random(seed)
        free = list(range(num_pages))
        self.rng.shuffle(free)
        self.want = ref.Pages([[-1] * max_pages for _ in range(B)], [0] * B, free, page)
        self.i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
        self.table, self.held, self.free = self.i(self.want.table), self.i([0] * B), self.i(free)
        self.count, self.num_pages, self.page = self.i([num_pages]), num_pages, page

    def update(self, mla, lens, new=None, pad=0, err=None, **kw):
        import torch
        slots = cu = None
        if new is not None:
            slots = torch.full((max(1, sum(new) + pad),), 12345, dtype=torch.int64, device="cuda")
            cu = self.i(cum(new))
        got = mla.update_pages(self.table, self.held, self.i(lens), self.free, self.count, page_size=self.page, cu=cu,
                               slots=slots, err_word=err, **kw)
        want = self.want.update(lens, new, 0 if slots is None else slots.numel())
        torch.cuda.synchronize()
        assert got is slots
        self.check()
        if slots is not None:
            assert slots.tolist() == want

    def check(self):
        assert self.count.item() == len(self.want.free)
        assert self.free[:len(self.want.free)].tolist() == self.want.free
        assert self.held.tolist() == self.want.held
        assert self.table.tolist() == self.want.table


def test_many_pages_and_no_rows(mla, err):
    """All the pages of a large batch taken, most given back, taken again: no slots, so one launch does it."""
    s = State(1000, 40, 41000, 64, seed=4)
    s.update(mla, [40 * 64 - b % 64 for b in range(1000)], err=err)
    s.update(mla, [0 if b % 3 else 100 + b for b in range(1000)], err=err)
    s.update(mla, [64 * (b % 41) for b in range(1000)], err=err)
    assert int(err.item()) == 0


@pytest.mark.parametrize("B,page,steps", [(1, 64, 12), (7, 128, 12), (33, 64, 8), (500, 64, 4), (1024, 128, 3),
                                          (1025, 64, 3), (4096, 128, 3)])
def test_serving_loop(mla, err, B, page, steps):
    """Sequences start, grow by a token, shrink (rejected drafts) and finish."""
    s = State(B, 9, 6 * B + 9, page, seed=B)
    r, lens = s.rng, [0] * B
    for step in range(steps):
        new = [0] * B
        for b in range(B):
            what = r.randrange(6)
            if lens[b] == 0 and what < 4:
                lens[b] = new[b] = r.randint(1, 3 * page + 5)
            elif lens[b] and what == 0:
                lens[b] = 0
            elif lens[b] and what == 1:
                lens[b] -= r.randint(0, min(lens[b] - 1, 5))
            elif lens[b] and lens[b] < 5 * page:
                lens[b] += 1
                new[b] = 1
        s.update(mla, lens, new, pad=step % 3, err=err)
        assert s.want.refused == [] and int(err.item()) == 0
    s.update(mla, [0] * B, err=err)
    assert sorted(s.want.free) == list(range(s.num_pages)) and (s.table == -1).all() and int(err.item()) == 0


@pytest.mark.parametrize("B,scale", [(3, 1), (40, 1), (40, 60), (1500, 2)])
def test_a_step_and_back(mla, err, B, scale):
    s = State(B, 8 * scale + 2, 6 * B * scale + 30, 64, seed=3)
    a = [s.rng.randint(0, 300 * scale) for _ in range(B)]
    b = [s.rng.choice([0, x, s.rng.randint(0, 400 * scale)]) for x in a]
    s.update(mla, a, a, err=err)
    n = s.count.item()  # (what lies past the top of the stack is not part of it)
    start = [t.clone() for t in (s.table, s.held, s.free[:n], s.count)]
    s.update(mla, b, [max(0, y - x) for x, y in zip(a, b)], err=err)
    s.update(mla, a, err=err)
    assert all((x == y).all() for x, y in zip(start, (s.table, s.held, s.free[:n], s.count))) and int(err.item()) == 0


def test_chunk_boundaries_and_single_tokens(mla, err):
    """Lengths around page borders, new tokens that begin inside a held page, pages taken ahead of the tokens."""
    s = State(6, 5, 25, 64)
    s.update(mla, [63, 64, 65, 1, 0, 128], [63, 64, 65, 1, 0, 128], err=err)
    s.update(mla, [64, 65, 66, 2, 1, 129], [1, 1, 1, 1, 1, 1], pad=5, err=err)
    s.update(mla, [65, 200, 66, 130, 64, 320], [1, 135, 0, 128, 63, 191], err=err)
    s.update(mla, [320, 0, 66, 130, 64, 320], [1, 0, 0, 0, 0, 320], err=err)  # one token on four new pages
    assert int(err.item()) == 0 and s.want.refused == []


@pytest.mark.parametrize("B", [5, 1300])
def test_too_few_pages(mla, err, B):
    """Served whole and in order; a sequence that misses nothing is served behind one that is refused."""
    s = State(B, 6, 2 * B, 64, seed=1)
    lens = [130 if b % 5 == 1 else 64 for b in range(B)]
    lens[B // 2] = 64 * 6
    s.update(mla, lens, lens, pad=2, err=err)
    more = [L + 64 * (b % 3) if L + 64 * (b % 3) <= 384 else L for b, L in enumerate(lens)]
    s.update(mla, more, [1] * B, err=err)
    assert s.want.refused and int(err.item()) == NO_PAGES
    err.zero_()
    less = [0 if b < B // 2 else L for b, L in enumerate(more)]  # the pages of the first half
    s.update(mla, less, [0] * (B // 2) + [1] * (B - B // 2), err=err)
    assert s.want.refused == [] and int(err.item()) == 0


def test_no_free_page_at_all(mla, err):
    s = State(2, 2, 2, 64)
    s.update(mla, [128, 0], [128, 0], err=err)
    assert s.count.item() == 0
    s.update(mla, [128, 1], [0, 1], err=err)
    assert int(err.item()) == NO_PAGES
    err.zero_()
    s.update(mla, [64, 1], [0, 1], err=err)  # the page given back is the page taken
    assert int(err.item()) == 0 and s.count.item() == 0


@pytest.mark.parametrize("lens,cu,held", [
    ([-1, 70], [0, 0, 70], None), ([64 * 4 + 1, 70], [0, 0, 70], None),  # lengths out of range
    ([3, 70], [0, 5, 75], None),                                        # more new tokens than the length
    ([3, 70], [0, 0, 70], [-2, 0]), ([3, 70], [0, 0, 70], [5, 0]),      # pages held out of range
    ([64, 70], [0, -4, 66], None), ([64, 70], [0, 64, 900], None),      # rows outside the array
])
def test_bad_numbers_are_reported(mla, err, lens, cu, held):
    """A sequence whose numbers are out of range is left as it is, the others are served."""
    import torch
    s = State(2, 4, 9, 64)
    i = s.i
    h = i(held or [0, 0])
    slots = torch.full((80,), 12345, dtype=torch.int64, device="cuda")
    mla.update_pages(s.table, h, i(lens), s.free, s.count, page_size=64, cu=i(cu), slots=slots, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == BOUNDS
    bad = [b for b in range(2) if not (0 <= lens[b] <= 256 and 0 <= (held or [0, 0])[b] <= 4
                                       and 0 <= cu[b] <= cu[b + 1] <= 80 and cu[b + 1] - cu[b] <= lens[b])]
    taken = 0
    for b in range(2):
        if b in bad:
            assert h[b].item() == (held or [0, 0])[b] and (s.table[b] == -1).all()
        else:
            taken += -(-lens[b] // 64)
            assert h[b].item() == -(-lens[b] // 64)
    assert s.count.item() == 9 - taken
    got = slots.tolist()
    assert all(v == -1 or v == 12345 or 0 <= v < 9 * 64 for v in got)


def test_pages_that_are_there_twice_are_not_moved(mla, err):
    """More pages free and given back than there are: nothing moves."""
    import torch
    s = State(2, 4, 5, 64)
    s.update(mla, [130, 64], [130, 64], err=err)
    s.count.fill_(4)
    before = [t.clone() for t in (s.table, s.held, s.free, s.count)]
    slots = torch.full((3,), 5, dtype=torch.int64, device="cuda")
    mla.update_pages(s.table, s.held, s.i([0, 65]), s.free, s.count, cu=s.i([0, 0, 1]), slots=slots, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == BOUNDS and slots.tolist() == [-1, -1, -1]
    assert all((x == y).all() for x, y in zip(before, (s.table, s.held, s.free, s.count)))
    for count in (-1, 6):
        err.zero_()
        s.count.fill_(count)
        mla.update_pages(s.table, s.held, s.i([130, 64]), s.free, s.count, err_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == BOUNDS


def test_page_ids_outside_the_pool_are_reported(mla, err):
    import torch
    s = State(2, 4, 5, 64)
    s.free[4] = 77  # the top of the stack
    slots = torch.empty(70, dtype=torch.int64, device="cuda")
    mla.update_pages(s.table, s.held, s.i([70, 0]), s.free, s.count, cu=s.i([0, 70, 70]), slots=slots, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == BOUNDS and s.table[0, 0].item() == 77
    assert (slots[:64] == -1).all() and slots[64:].tolist() == [s.free[3].item() * 64 + k for k in range(6)]


@pytest.mark.parametrize("n_rows", [300, 5000])  # one launch, two launches
def test_replayed_with_other_lengths(mla, err, n_rows):
    """One captured call serves every step: lengths, cu and the arrays change in place."""
    import torch
    s = State(5, 4, 17, 64)
    lens, cu = s.i([0] * 5), s.i([0] * 6)
    slots = torch.zeros(n_rows, dtype=torch.int64, device="cuda")

    def call():
        mla.update_pages(s.table, s.held, lens, s.free, s.count, cu=cu, slots=slots, err_word=err)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for L, n in (([70, 0, 64, 1, 0], [70, 0, 64, 1, 0]), ([71, 200, 0, 2, 0], [1, 200, 0, 1, 0]), ([0] * 5, [0] * 5)):
        lens.copy_(s.i(L))
        cu.copy_(s.i(cum(n)))
        graph.replay()
        want = s.want.update(L, n, n_rows)
        torch.cuda.synchronize()
        s.check()
        assert slots.tolist() == want and int(err.item()) == 0


def test_on_another_stream_and_two_calls_at_once(mla, err):
    import torch
    states, streams = [State(300, 9, 2000, 64, seed=k) for k in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    plans = [[s.rng.randint(0, 400) for _ in range(300)] for s in states]
    args = [(s.i(p), s.i(cum(p)), torch.empty(sum(p), dtype=torch.int64, device="cuda")) for s, p in zip(states, plans)]
    torch.cuda.synchronize()
    for s, (lens, cu, slots), st in zip(states, args, streams):
        mla.update_pages(s.table, s.held, lens, s.free, s.count, cu=cu, slots=slots, err_word=err, stream=st)
    torch.cuda.synchronize()
    for s, p, (_, _, slots) in zip(states, plans, args):
        assert slots.tolist() == s.want.update(p, p, sum(p))
        s.check()
    assert int(err.item()) == 0


def test_python_checks(mla):
    import torch
    s = State(2, 4, 5, 64)
    lens = s.i([1, 1])
    good = dict(block_table=s.table, held=s.held, seq_lens=lens, free_pages=s.free, free_count=s.count)
    for name, bad in (("held", s.i([0] * 3)), ("seq_lens", lens.long()), ("free_pages", s.free[::2]),
                      ("free_count", s.i([5, 5])), ("block_table", s.table.t()), ("held", s.held.cpu())):
        with pytest.raises(ValueError):
            mla.update_pages(**{**good, name: bad})
    with pytest.raises(ValueError, match="both or neither"):
        mla.update_pages(**good, cu=s.i([0, 1, 2]))
    with pytest.raises(ValueError, match="slots"):
        mla.update_pages(**good, cu=s.i([0, 1, 2]), slots=s.i([0, 0]))
    with pytest.raises(mla.MlaError, match="INVALID_ARG"):
        mla.update_pages(**good, cu=s.i([0, 1, 2]), slots=torch.zeros(0, dtype=torch.int64, device="cuda"))
