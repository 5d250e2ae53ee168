"""update_pages told two things wrong in one call: the code that it reports does not depend on timing."""
import pytest

from tests.test_gpu_pages import BOUNDS, NO_PAGES, State

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    import mla_latent_kv_paged_gb300 as m
    m.build()
    return m


@pytest.mark.parametrize("B,n_rows", [(5, 1), (1000, 1000), (700, 5000), (1300, 1300)])  # one launch, two launches
@pytest.mark.parametrize("what", ["length", "rows", "page", "page and length"])
def test_numbers_out_of_range_are_told_before_missing_pages(mla, B, n_rows, what):
    """The first sequence misses pages; the last one's length or the rows are out of range, or a sequence's page is
    (which only the thread that meets it knows)."""
    import torch
    s = State(B, 4, B + 2, 64)
    lens = [64] * B
    s.update(mla, lens)
    start = [t.clone() for t in (s.table, s.held, s.free, s.count)]
    lens[0] = 256
    cu = [0] * B + [1]
    if "length" in what:
        lens[B // 2] = 64 * 4 + 1
    if what == "rows":
        cu[B] = n_rows + 1
    lens, cu = s.i(lens), s.i(cu)
    slots = torch.empty(n_rows, dtype=torch.int64, device="cuda")
    for want in [NO_PAGES if what == "page" else BOUNDS] + [BOUNDS] * 20:
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        for t, v in zip((s.table, s.held, s.free, s.count), start):
            t.copy_(v)
        if want == BOUNDS and "page" in what:
            s.table[B - 1, 0] = 1 << 20  # the page of the one new token
        mla.update_pages(s.table, s.held, lens, s.free, s.count, page_size=64, cu=cu, slots=slots, err_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == want and s.held[0].item() == 1
