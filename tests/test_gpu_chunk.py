"""The chunk operators (append_chunk, read_kv, attend_chunk, chunk_step) on the GPU,
against a plain 64-bit implementation (tests/chunk_reference.py), element by element
within bounds derived from the roundings of each form."""
import pytest

from tests import chunk_reference as ref

pytestmark = pytest.mark.gpu

BOUNDS, RANGE = 6, 7


@pytest.fixture(scope="module")
def mla():
    import mla_latent_kv_paged_gb300 as m
    m.build()
    return m


@pytest.fixture()
def err():
    import torch
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def hidden(T, d_model, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.randn(T, d_model, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(576, d_model, generator=g, device="cuda") * d_model ** -0.5).to(torch.bfloat16)
    return h, w


def bits(t):
    import torch
    return t.view(torch.uint8) if t.dtype == torch.uint8 else t.view(torch.int16)


# ------------------------------------------------------------------ read_kv
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page,lens,first,count", [
    (64, [1], [0], [1]),
    (64, [70, 1, 129, 64], [0, 0, 3, 63], [70, 1, 126, 1]),
    (128, [300, 5, 128], [299, 0, 0], [1, 5, 128]),
    (64, [100, 40], [90, 40], [30, 7]),              # past the end: zeros
    (128, [1000, 777, 0, 513], [1, 0, 0, 500], [999, 0, 0, 13]),
])
def test_read_rows(mla, err, fp8, page, lens, first, count):
    import torch
    c = ref.Chunk(count, lens, page=page, fp8=fp8, seed=3)
    n_rows = c.total + 5
    out = torch.full((n_rows, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    f = torch.tensor(first, dtype=torch.int32, device="cuda")
    got = mla.read_kv(*c.paged(), n_rows=n_rows, first=f, fp8_scales=c.scales, out=out, err_word=err)
    torch.cuda.synchronize()
    assert got is out and int(err.item()) == 0
    want = []
    for b in range(len(lens)):
        hi = min(first[b] + count[b], lens[b])
        x = c.cache.view(-1, 576)[c.rows(b, first[b], hi)] if hi > first[b] else c.cache.view(-1, 576)[:0]
        if fp8:  # one fp32 product, one rounding to bf16
            x = (x.view(torch.float8_e4m3fn).float() * c.scales).to(torch.bfloat16)
        want.append(torch.cat([x, torch.zeros(count[b] - len(x), 576, dtype=torch.bfloat16, device="cuda")]))
    assert torch.equal(got[:c.total], torch.cat(want))
    assert (got[c.total:] == 7.0).all()


def test_read_reports_bad_pages_and_starts(mla, err):
    import torch
    c = ref.Chunk([5, 70], [5, 70], seed=4)
    c.table[1, 0] = c.num_pages  # outside the pool: those rows read as zeros
    got = mla.read_kv(*c.paged(), n_rows=75, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == BOUNDS
    assert torch.equal(got[:5], c.cache.view(-1, 576)[c.rows(0)])
    assert (got[5:69] == 0).all() and torch.isfinite(got[69:]).all()
    err.zero_()
    f = torch.tensor([-1, 0], dtype=torch.int32, device="cuda")
    c = ref.Chunk([5, 70], [5, 70], seed=4)
    got = mla.read_kv(*c.paged(), n_rows=75, first=f, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == BOUNDS and (got[0] == 0).all()
    assert torch.equal(got[1:5], c.cache.view(-1, 576)[c.rows(0, 0, 4)])


# ------------------------------------------------------------------ append_chunk
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,lens,d_model,page,pad", [
    ([1], [1], 64, 64, 0),
    ([3, 0, 70], [3, 9, 200], 128, 64, 4),            # one split: the GEMM's own epilogue writes the rows
    ([130, 1, 257], [1000, 64, 257], 192, 128, 0),
    ([1] * 33, list(range(1, 331, 10)), 512, 64, 0),  # decode-like, split over d_model
    ([200, 0, 57], [70000, 3, 57], 1024, 64, 130),    # far positions, a padded tile
    ([1700, 1650], [1700, 1650], 512, 128, 1),        # many row tiles
])
def test_append_rows(mla, err, fp8, new, lens, d_model, page, pad):
    import torch
    c = ref.Chunk(new, lens, H=1, page=page, fp8=fp8, seed=5, pad_rows=pad)
    h, w = hidden(c.T, d_model, 6)
    before = c.cache.clone()
    rows, want, slack = ref.append(c, h, w)
    mla.append_chunk(h, w, *c.paged(), fp8_scales=c.scales, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    got = c.cache.view(-1, 576)[rows]
    if fp8:
        # e4m3: half a step is 2^-4 of the value, 2^-10 below 2^-6; then the sum's own error
        s = c.scales.double()
        got = got.view(torch.float8_e4m3fn).double()
        want, slack = (want / s).clamp(-448, 448), slack / s
        assert ((got - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -10 + 1.1 * slack).all()
    else:
        assert ((got.double() - want).abs() <= ref.U_BF16 * want.abs() + 1.1 * slack).all()
    other = torch.ones(c.num_pages * page, dtype=torch.bool, device="cuda")
    other[rows] = False
    assert torch.equal(bits(c.cache).view(-1, 576)[other], bits(before).view(-1, 576)[other])
    first = c.cache.clone()
    mla.append_chunk(h, w, *c.paged(), fp8_scales=c.scales, err_word=err)
    assert torch.equal(bits(first), bits(c.cache))


def test_append_fp8_saturates_and_keeps_nan(mla, err):
    import torch
    c = ref.Chunk([2], [2], H=1, fp8=True, seed=7)
    h = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(576, 64, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = 1.0
    h[0, 0], h[1, 0] = 1e6, float("nan")
    mla.append_chunk(h, w, *c.paged(), fp8_scales=c.scales, err_word=err)
    got = c.cache.view(-1, 576)[c.rows(0)].view(torch.float8_e4m3fn).float()
    assert (got[0, :512] == 448).all() and torch.isnan(got[1]).all()


def test_append_reports_and_skips_bad_targets(mla, err):
    import torch
    for split in (64, 1024):  # one split, many splits
        c = ref.Chunk([4, 3, 2], [70, 3, 2], H=1, seed=8)
        h, w = hidden(9, split, 9)
        rows, want, slack = ref.append(c, h, w)
        c.table[0, 1] = -5           # tokens 66..69 of sequence 0
        c.seq_lens[1] = 2            # fewer tokens than new rows
        before = c.cache.clone()
        err.zero_()
        mla.append_chunk(h, w, *c.paged(), err_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == BOUNDS
        got = c.cache.view(-1, 576)[rows[7:]].double()
        assert ((got - want[7:]).abs() <= ref.U_BF16 * want[7:].abs() + 1.1 * slack[7:]).all()
        assert torch.equal(bits(c.cache).view(-1, 576)[rows[:4]], bits(before).view(-1, 576)[rows[:4]])


# ------------------------------------------------------------------ attend_chunk
# The roundings of a form are independent, so over many outputs they add in squares. Half
# a bf16 step (2^-8) each: absorbed on a bf16 cache the query, the weights and the output,
# sqrt(3) 2^-8 < 1.75 x 2^-8 of the norm; else the output alone, beside at most eight in
# fp16 (2^-11): sqrt(1 + 8 / 64) 2^-8 < 1.1 x 2^-8.
REL = 1.75 * ref.U_BF16
REL_F16 = 1.1 * ref.U_BF16


def check(got, want, bound, what, rel_max=REL):
    import torch
    assert torch.isfinite(got).all(), what
    off = (got.double() - want).abs()
    worst = (off / bound).max().item()
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound, max |diff| {off.max().item():.3e}"
    rel = (off.norm() / want.norm()).item()
    assert rel <= rel_max, f"{what}: {rel:.2e} of the norm"


SHAPES = [
    # new, lens, H, page, pad
    ([1], [1], 1, 64, 0),
    ([1, 2, 5], [1, 64, 65], 4, 64, 0),
    ([3, 0, 4], [200, 7, 130], 16, 128, 5),
    ([127, 128], [127, 500], 3, 64, 0),
    ([129, 1], [129, 300], 2, 64, 2),
    ([257, 255, 256], [257, 1000, 256], 2, 128, 0),
    ([1, 700], [2000, 700], 3, 64, 1),
    ([40] * 5, [41, 400, 40, 127, 129], 5, 64, 0),
    ([6], [5000], 128, 64, 0),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("form", ["expanded", "absorbed"])
@pytest.mark.parametrize("new,lens,H,page,pad", SHAPES)
def test_attend(mla, err, fp8, form, new, lens, H, page, pad):
    import torch
    c = ref.Chunk(new, lens, H=H, page=page, fp8=fp8, seed=10 + len(new), pad_rows=pad)
    want, lse_want, bound = ref.attend(c)
    out = torch.full((c.T, H, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.T, H), 5.0, device="cuda")
    got = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=sum(lens), fp8_scales=c.scales,
                           form=form, out=out, lse=lse, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(got[:c.total], want, bound[form], form, REL_F16 if fp8 or form == "expanded" else REL)
    # an lse moves by at most the largest score error of its row
    assert (lse[:c.total].double() - lse_want).abs().max().item() <= (0.12 if form == "absorbed" and not fp8 else 0.02)
    assert (out[c.total:] == 3.0).all() and (lse[c.total:] == 5.0).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("form", ["expanded", "absorbed"])
def test_attend_values_whose_products_cancel(mla, err, form, fp8):
    """A row that sees one key answers with that key's value. Among 128 x 128 values a few
    are 1e-5 of the products they sum: off by the fp32 sum's 2^-24 of the absolute products
    per term (measured: about 1 x 2^-24 of a sum of 14), not by a fraction of themselves."""
    c = ref.Chunk([1, 2, 1, 1], [1, 2, 1, 1], H=128, fp8=fp8, seed=0)
    want, _, bound = ref.attend(c)
    got = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=5, fp8_scales=c.scales,
                           form=form, err_word=err)
    assert int(err.item()) == 0
    assert want.abs().min().item() < 2.0 ** -14
    check(got, want, bound[form], form, REL_F16 if fp8 or form == "expanded" else REL)


def test_attend_auto_equals_the_form_it_chooses(mla):
    import torch
    for new, form in (([4, 4], "absorbed"), ([600], "expanded")):
        c = ref.Chunk(new, [700] * len(new), H=16, seed=11)
        a = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=sum(c.lens))
        b = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=sum(c.lens), form=form)
        assert torch.equal(a, b)


@pytest.mark.parametrize("form", ["expanded", "absorbed"])
def test_attend_rising_scores(mla, err, form):
    """Scores that grow along the context: the running maximum keeps rising by far more
    than the rescale threshold, and the largest weights come last."""
    import torch
    c = ref.Chunk([200, 3], [900, 640], H=2, seed=12)
    pool = c.cache.view(-1, 576)
    for b in range(2):
        s = torch.arange(c.lens[b], device="cuda", dtype=torch.float32)
        pool[c.rows(b), 512] = (s * (64.0 / c.lens[b])).to(torch.bfloat16)
    c.q_rope[..., 0] = 32.0
    want, _, bound = ref.attend(c)
    got = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=1540, form=form, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(got, want, bound[form], form)


def test_attend_falling_scores(mla, err):
    """The first token carries nearly all the weight: later weights underflow quietly."""
    import torch
    c = ref.Chunk([150], [1000], H=2, seed=13)
    c.cache.view(-1, 576)[c.rows(0), 512] = -8.0
    c.cache.view(-1, 576)[c.rows(0, 0, 1), 512] = 8.0
    c.q_rope[..., 0] = 32.0
    want, _, bound = ref.attend(c)
    got = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=1000, form="expanded",
                           err_word=err)
    check(got, want, bound["expanded"], "falling")


@pytest.mark.parametrize("form", ["expanded", "absorbed"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attend_nonfinite_token_reaches_only_the_rows_that_see_it(mla, err, form, bad):
    import torch
    c = ref.Chunk([300, 20], [420, 20], H=2, seed=14)
    want, _, bound = ref.attend(c)
    c.cache.view(-1, 576)[c.rows(0, 200, 201), :512] = bad  # row 80 of sequence 0
    got = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=440, form=form, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) in (0, RANGE)
    keep = torch.ones(320, dtype=torch.bool, device="cuda")
    keep[80:300] = False
    check(got[keep], want[keep], bound[form][keep], form)
    assert torch.isnan(got[80:300]).all()


def test_attend_reports_expanded_values_outside_fp16(mla, err):
    c = ref.Chunk([130], [130], H=1, seed=15)
    c.cache.view(-1, 576)[c.rows(0, 50, 51), :512] = 3e6
    import torch
    got = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=130, form="expanded",
                           err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == RANGE
    assert torch.isfinite(got[:50]).all()


def test_attend_large_queries_on_small_scales(mla, err):
    """Queries beyond fp16 on an FP8 cache of small values, absorbed: the query is scaled
    by the cache's columns before it is rounded."""
    c = ref.Chunk([3, 2], [200, 66], H=3, fp8=True, seed=19)
    c.scales *= 2.0 ** -7
    c.q_nope *= 2.0 ** 17
    c.q_rope *= 2.0 ** 17
    want, _, bound = ref.attend(c, ref.SCALE * 2.0 ** -10)
    got = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=266, fp8_scales=c.scales,
                           softmax_scale=ref.SCALE * 2.0 ** -10, form="absorbed", err_word=err)
    assert int(err.item()) == 0
    check(got, want, bound["absorbed"], "large queries", REL_F16)


@pytest.mark.parametrize("form,part", [(f, p) for f in ("expanded", "absorbed") for p in ("nope", "rope")])
def test_attend_reports_queries_outside_fp16(mla, err, form, part):
    import torch
    c = ref.Chunk([5, 2], [200, 66], H=3, fp8=True, seed=20, pad_rows=2)
    want, _, bound = ref.attend(c)
    (c.q_nope if part == "nope" else c.q_rope)[4, 1] = 1e9
    got = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=266, fp8_scales=c.scales,
                           form=form, err_word=err)
    assert int(err.item()) == RANGE
    keep = torch.ones(7, 3, dtype=torch.bool, device="cuda")
    keep[4, 1] = False
    check(got[:7][keep], want[keep], bound[form][keep], form, REL_F16)


def test_attend_reports_a_query_outside_fp16_beside_a_nan(mla, err):
    import torch
    c = ref.Chunk([100], [100], H=1, seed=21)
    want, _, bound = ref.attend(c)
    c.q_nope[3] = float("nan")
    c.q_nope[35] = 1e9  # rows 32 apart are one thread's
    got = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=100, form="expanded",
                           err_word=err)
    assert int(err.item()) == RANGE
    keep = torch.ones(100, dtype=torch.bool, device="cuda")
    keep[[3, 35]] = False
    check(got[keep], want[keep], bound["expanded"][keep], "expanded", REL_F16)


@pytest.mark.parametrize("form,fp8", [("expanded", True), ("absorbed", False), ("absorbed", True)])
def test_attend_reports_weights_outside_fp16_beside_nans(mla, err, form, fp8):
    import torch
    c = ref.Chunk([2], [70], H=3, fp8=fp8, seed=22)
    want, _, bound = ref.attend(c)
    c.w_uv[0] = float("nan")
    c.w_uv[2] = 1e6
    got = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=70, fp8_scales=c.scales,
                           form=form, err_word=err)
    assert int(err.item()) == RANGE
    assert torch.isnan(got[:, 0]).all()
    check(got[:, 1], want[:, 1], bound[form][:, 1], form)


@pytest.mark.parametrize("form", ["expanded", "absorbed"])
def test_attend_reports_bad_lengths_pages_and_rows(mla, err, form):
    import torch
    c = ref.Chunk([130, 5], [200, 70], H=2, seed=16)
    want, _, bound = ref.attend(c)

    def run(**kw):
        err.zero_()
        out = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), form=form, err_word=err, **kw)
        torch.cuda.synchronize()
        return out, int(err.item())

    out, e = run(max_tokens=270)
    assert e == 0
    good = c.table.clone()
    c.table[0, 1] = c.num_pages + 9
    out, e = run(max_tokens=270)
    assert e == BOUNDS
    check(out[130:], want[130:], bound[form][130:], "the other sequence")
    c.table.copy_(good)
    c.seq_lens[0] = 1 << 30
    assert run(max_tokens=270)[1] == BOUNDS
    c.seq_lens[0] = 100
    assert run(max_tokens=270)[1] == BOUNDS
    c.seq_lens[0] = 200
    c.cu[2] = 1000
    assert run(max_tokens=270)[1] == BOUNDS
    c.cu[2] = 135
    if form == "expanded":  # the second sequence does not fit what was announced
        out, e = run(max_tokens=120)
        assert e == BOUNDS
    out, e = run(max_tokens=270)
    assert e == 0
    check(out, want, bound[form], "afterwards")


@pytest.mark.parametrize("form", ["expanded", "absorbed"])
def test_attend_without_any_new_row(mla, err, form):
    import torch
    c = ref.Chunk([0, 0], [9, 0], H=3, seed=17, pad_rows=4)
    out = torch.full((4, 3, 128), 2.0, dtype=torch.bfloat16, device="cuda")
    mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=9, form=form, out=out, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and (out == 2.0).all()


def test_attend_shared_pages(mla, err):
    """Two sequences whose first pages are the same physical pages (a shared prefix)."""
    import torch
    c = ref.Chunk([30, 140], [200, 300], H=2, seed=18)
    c.table[1, :3] = c.table[0, :3]
    c.host_table = c.table.cpu().tolist()
    c.table[1, 3] = c.host_table[1][3]
    want, _, bound = ref.attend(c)
    for form in ("expanded", "absorbed"):
        got = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=500, form=form, err_word=err)
        check(got, want, bound[form], form)


@pytest.mark.parametrize("form", ["expanded", "absorbed"])
def test_attend_workspace_is_the_stated_size_at_any_16_bytes(mla, form):
    import torch
    c = ref.Chunk([70, 3], [300, 200], H=3, seed=19)
    need = mla.attend_chunk_workspace_bytes(2, 73, 3, 500, form)
    room = torch.full((need + 48,), 0xA5, dtype=torch.uint8, device="cuda")
    want, _, bound = ref.attend(c)
    got = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=500, form=form,
                           workspace=room[16:16 + need])
    check(got, want, bound[form], form)
    assert (room[:16] == 0xA5).all() and (room[16 + need:] == 0xA5).all()


def test_attend_in_head_groups(mla, err):
    """A context whose keys and values are expanded a few heads at a time."""
    c = ref.Chunk([300], [70000], H=128, seed=20)
    import torch
    got = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=70000, form="expanded",
                           err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    few = [0, 63, 64, 127]
    c.H = 4
    c.q_nope, c.q_rope, c.w_uk, c.w_uv = (c.q_nope[:, few].contiguous(), c.q_rope[:, few].contiguous(),
                                          c.w_uk[few].contiguous(), c.w_uv[few].contiguous())
    want, _, bound = ref.attend(c)
    check(got[:, few], want, bound["expanded"], "head groups")


# ------------------------------------------------------------------ together, as they are used
@pytest.mark.parametrize("fp8", [False, True])
def test_prompt_in_pieces_then_decode(mla, err, fp8):
    """Two prompts written and attended in ragged pieces, then one decode step on the same
    cache, all against the 64-bit reference on the final cache."""
    import torch
    H, d_model, page = 4, 512, 64
    lens = [333, 150]
    c = ref.Chunk(lens, lens, H=H, page=page, fp8=fp8, seed=21)
    h, w = hidden(c.T, d_model, 22)
    pieces = [([128, 1], [128, 1]), ([5, 149], [133, 150]), ([200, 0], [333, 150])]
    rows, want_rows, slack = ref.append(c, h, w)
    c.cache.view(-1, 576)[rows] = ref.NAN_CODE if fp8 else float("nan")
    got = torch.empty(c.T, H, 128, dtype=torch.bfloat16, device="cuda")
    for new, upto in pieces:
        pick = torch.cat([torch.arange(u - n, u) + sum(lens[:b]) for b, (n, u) in enumerate(zip(new, upto))]).cuda()
        cu = torch.tensor([0, new[0], sum(new)], dtype=torch.int32, device="cuda")
        sl = torch.tensor(upto, dtype=torch.int32, device="cuda")
        got[pick] = mla.chunk_step(h[pick], c.q_nope[pick], c.q_rope[pick], w, c.w_uk, c.w_uv, c.cache, c.table, sl, cu,
                                   max_tokens=sum(upto), fp8_scales=c.scales, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    want, _, bound = ref.attend(c)  # on the cache as it was written
    check(got, want, torch.maximum(bound["expanded"], bound["absorbed"]), "pieces")
    vals = torch.cat([c.values(b) for b in range(2)])
    tol = (2.0 ** -4 if fp8 else ref.U_BF16) * want_rows.abs() + 1.1 * slack
    if fp8:
        tol += 2.0 ** -10 * c.scales.double()
    inside = (want_rows / c.scales.double()).abs() <= 440 if fp8 else torch.ones_like(tol, dtype=torch.bool)
    assert ((vals - want_rows).abs() <= tol)[inside].all()
    last = torch.tensor([332, 482], device="cuda")
    step = mla.decode_step(c.q_nope[last], c.q_rope[last], c.w_uk, c.w_uv, c.cache, c.table, c.seq_lens, n_q=1,
                           fp8_scales=c.scales, err_word=err)
    torch.cuda.synchronize()
    check(step["out"], want[last], bound["absorbed"][last], "decode")


@pytest.mark.parametrize("form", ["expanded", "absorbed"])
def test_captured_chunk_follows_its_lengths(mla, err, form):
    """One graph of append + attend, replayed with other lengths, tables and fewer rows."""
    import torch
    H, d_model = 2, 256
    c = ref.Chunk([60, 80], [160, 280], H=H, seed=23, pad_rows=0)
    h, w = hidden(c.T, d_model, 24)
    out = torch.zeros(c.T, H, 128, dtype=torch.bfloat16, device="cuda")
    kw = dict(max_tokens=600, form=form, out=out, err_word=err)
    kw["bufs"] = dict(append_workspace=torch.empty(mla.append_chunk_workspace_bytes(c.T, d_model), dtype=torch.uint8,
                                                   device="cuda"),
                      attend_workspace=torch.empty(mla.attend_chunk_workspace_bytes(2, c.T, H, 600, form),
                                                   dtype=torch.uint8, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mla.chunk_step(h, c.q_nope, c.q_rope, w, c.w_uk, c.w_uv, *c.paged(), **kw)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mla.chunk_step(h, c.q_nope, c.q_rope, w, c.w_uk, c.w_uv, *c.paged(), **kw)
    for seed, (new, lens) in enumerate([([60, 80], [160, 280]), ([1, 3], [200, 77]), ([0, 130], [50, 130])]):
        d = ref.Chunk(new, lens, H=H, seed=30 + seed, spare=c.num_pages - sum(-(-L // 64) for L in lens),
                      pad_rows=c.T - sum(new))
        c.cache.copy_(d.cache)
        c.table.fill_(-1)
        k = min(c.table.shape[1], d.table.shape[1])
        c.table[:, :k] = d.table[:, :k]
        c.seq_lens.copy_(d.seq_lens)
        c.cu.copy_(d.cu)
        c.q_nope.copy_(d.q_nope)
        c.q_rope.copy_(d.q_rope)
        c.w_uk.copy_(d.w_uk)
        c.w_uv.copy_(d.w_uv)
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        d.cache = c.cache.clone()
        want, _, bound = ref.attend(d)
        check(out[:d.total], want, bound[form], (form, seed))
        assert (out[d.total:] == 9.0).all()


def test_calls_on_another_stream(mla):
    import torch
    c = ref.Chunk([140, 3], [200, 90], H=2, seed=25)
    want, _, bound = ref.attend(c)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = {f: mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=290, form=f, stream=s)
           for f in ("expanded", "absorbed")}
    s.synchronize()
    for f, g in got.items():
        check(g, want, bound[f], f)


def test_memory_of_a_call_on_another_stream_is_that_streams(mla, monkeypatch):
    """What a call allocates for itself must not be handed out again on the current stream
    while the other stream's kernels use it."""
    import torch
    c = ref.Chunk([140, 3], [200, 90], H=2, seed=25)
    h, w = hidden(c.T, 512, 26)
    seen = []
    real = mla._call
    monkeypatch.setattr(mla, "_call", lambda name, fn, dev, stream, *a: (seen.append(a), real(name, fn, dev, stream, *a)))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    need = mla.attend_chunk_workspace_bytes(2, c.T, 2, 290, "expanded")
    mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=290, form="expanded", stream=s)
    mla.append_chunk(h, w, *c.paged(), stream=s)
    mla.read_kv(*c.paged(), n_rows=50, stream=s)
    again = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in
             (need, mla.append_chunk_workspace_bytes(c.T, 512), 50 * 576 * 2, c.T * 2 * 128 * 2)]
    s.synchronize()
    for t in again:
        lo, hi = t.data_ptr(), t.data_ptr() + t.numel()
        inputs = {x.data_ptr() for x in (c.cache, c.table, c.seq_lens, c.cu, c.q_nope, c.q_rope, c.w_uk, c.w_uv, h, w)}
        assert not any(lo <= v < hi for a in seen for v in a if isinstance(v, int) and v > 1 << 32 and v not in inputs)


def test_back_to_back_calls_share_a_workspace(mla):
    import torch
    cs = [ref.Chunk(n, L, H=3, seed=40 + i) for i, (n, L) in
          enumerate([([200, 3], [300, 90]), ([5], [700]), ([129], [129]), ([1, 1, 1], [5, 6, 400])])]
    need = max(mla.attend_chunk_workspace_bytes(len(c.new), c.T, 3, sum(c.lens), f)
               for c in cs for f in ("expanded", "absorbed"))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    got = [(f, c, mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=sum(c.lens), form=f,
                                   workspace=ws)) for _ in range(2) for c in cs for f in ("expanded", "absorbed")]
    for f, c, g in got:
        want, _, bound = ref.attend(c)
        check(g, want, bound[f], f)


@pytest.mark.parametrize("new,lens,H", [([5], [4000], 1), ([200, 3, 300], [3000, 2500, 300], 2),
                                        ([300], [20000], 3), ([1, 1], [128, 129], 1), ([513], [1300], 5)])
def test_attend_cut_over_the_keys(mla, err, new, lens, H):
    """Few heads and rows on long contexts: the items are cut over the keys and joined."""
    import torch
    c = ref.Chunk(new, lens, H=H, seed=50, pad_rows=3)
    want, lse_want, bound = ref.attend(c)
    out = torch.full((c.T, H, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.T, H), 5.0, device="cuda")
    kw = dict(max_tokens=sum(lens), form="expanded", lse=lse, err_word=err)
    mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), out=out, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(out[:c.total], want, bound["expanded"], "cut")
    assert (lse[:c.total].double() - lse_want).abs().max().item() <= 0.02
    assert (out[c.total:] == 3.0).all() and (lse[c.total:] == 5.0).all()
    again = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), **kw)
    assert torch.equal(again[:c.total], out[:c.total])


def test_attend_cut_rising_scores(mla, err):
    """Pieces whose references lie far apart."""
    import torch
    c = ref.Chunk([40], [6000], H=1, seed=51)
    s = torch.arange(6000, device="cuda", dtype=torch.float32)
    c.cache.view(-1, 576)[c.rows(0), 512] = (s * (64.0 / 6000)).to(torch.bfloat16)
    c.q_rope[::2, :, 0], c.q_rope[1::2, :, 0] = 32.0, -32.0
    want, _, bound = ref.attend(c)
    got = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=6000, form="expanded",
                           err_word=err)
    check(got, want, bound["expanded"], "rising")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("form", ["expanded", "absorbed"])
def test_rows_of_no_sequence_report_nothing(mla, err, form, fp8):
    """Padding rows with any bits in their queries, and a pool whose first page holds any
    bits: nothing of it reaches the outputs or the error word."""
    import torch
    c = ref.Chunk([3, 2], [100, 66], H=2, fp8=fp8, seed=60, pad_rows=150)
    used = torch.unique(c.table[c.table >= 0])
    free = [p for p in range(c.num_pages) if p not in used.tolist()]
    assert free
    # the free page first in the pool: swap it with page 0 in place
    order = torch.arange(c.num_pages, device="cuda")
    order[0], order[free[0]] = free[0], 0
    c.cache = c.cache[order].contiguous()
    c.table = torch.where(c.table < 0, c.table, torch.argsort(order).to(torch.int32)[c.table.clamp(min=0).long()])
    c.host_table = c.table.cpu().tolist()
    c.cache[0] = 0x7E if fp8 else 3e38
    c.q_nope[c.total:] = 1e38
    c.q_rope[c.total:] = float("nan")
    want, _, bound = ref.attend(c)
    got = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=166, fp8_scales=c.scales,
                           form=form, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(got[:c.total], want, bound[form], form)


def test_first_row_offset_is_reported(mla, err):
    import torch
    c = ref.Chunk([3, 2], [100, 66], H=2, seed=61, pad_rows=4)
    c.cu += 1
    for form in ("expanded", "absorbed"):
        err.zero_()
        mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=166, form=form, err_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == BOUNDS


@pytest.mark.parametrize("fp8", [False, True])
def test_pool_beyond_32_bit_offsets(mla, err, fp8):
    """Rows in pages whose element offsets (and, bf16, byte offsets / 2) pass 2^32."""
    import torch
    pages = 120000  # x 64 x 576 = 4.4e9 elements
    c = ref.Chunk([70, 3], [300, 130], H=2, fp8=fp8, seed=62)
    pool = torch.zeros(pages, 64, 576, dtype=c.cache.dtype, device="cuda")
    shift = pages - c.num_pages
    pool[shift:] = c.cache
    c.cache, c.num_pages = pool, pages
    c.table = torch.where(c.table < 0, c.table, c.table + shift)
    c.host_table = c.table.cpu().tolist()
    h, w = hidden(c.T, 128, 63)
    rows, want_rows, slack = ref.append(c, h, w)
    mla.append_chunk(h, w, *c.paged(), fp8_scales=c.scales, err_word=err)
    got = c.cache.view(-1, 576)[rows]
    got = got.view(torch.float8_e4m3fn).double() * c.scales.double() if fp8 else got.double()
    tol = (2.0 ** -4 if fp8 else ref.U_BF16) * want_rows.abs() + 1.1 * slack
    if fp8:
        tol += 2.0 ** -10 * c.scales.double()
    inside = (want_rows / c.scales.double()).abs() <= 440 if fp8 else torch.ones_like(tol, dtype=torch.bool)
    assert ((got - want_rows).abs() <= tol)[inside].all()
    back = mla.read_kv(*c.paged(), n_rows=73, first=torch.tensor([230, 127], dtype=torch.int32, device="cuda"),
                       fp8_scales=c.scales, err_word=err)
    assert ((back.double() - got).abs() <= ref.U_BF16 * got.abs()).all()
    want, _, bound = ref.attend(c)
    for form in ("expanded", "absorbed"):
        o = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=430, fp8_scales=c.scales,
                             form=form, err_word=err)
        check(o, want, bound[form], form)
    assert int(err.item()) == 0


def test_many_sequences_and_the_largest_batch(mla, err):
    """4096 sequences, most of one token; the batch limit of every call."""
    import torch
    B = 4096
    new = [1] * B
    new[7], new[4000] = 0, 30
    lens = [1 + (b % 3) for b in range(B)]
    lens[4000], lens[100] = 700, 130
    c = ref.Chunk(new, lens, H=1, seed=64)
    back = mla.read_kv(c.cache, c.table, c.seq_lens, c.cu, n_rows=c.total, err_word=err)
    assert torch.equal(back[1], c.cache.view(-1, 576)[c.rows(1, 0, 1)][0])
    got = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=sum(lens), form="expanded",
                           err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    pick = [0, 1, 99, 100, 3999, 4000, 4095]
    d = ref.Chunk([new[b] for b in pick], [lens[b] for b in pick], H=1, seed=65)
    d.w_uk, d.w_uv = c.w_uk, c.w_uv
    rows = []
    for i, b in enumerate(pick):
        d.cache.view(-1, 576)[d.rows(i)] = c.cache.view(-1, 576)[c.rows(b)]
        rows += list(range(int(c.cu[b]), int(c.cu[b + 1])))
    d.q_nope, d.q_rope = c.q_nope[rows].contiguous(), c.q_rope[rows].contiguous()
    want, _, bound = ref.attend(d)
    check(got[rows], want, bound["expanded"], "many sequences")
    with pytest.raises(mla.MlaError):
        mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=sum(lens), form="absorbed")


def test_two_calls_at_once_on_two_streams(mla):
    """Calls that overlap on the GPU, each with its own workspace and outputs."""
    import torch
    cs = [ref.Chunk([300, 40], [900, 500], H=4, seed=70), ref.Chunk([130], [2000], H=3, seed=71)]
    hw = [hidden(c.T, 512, 72) for c in cs]
    wants = []
    for c, (h, w) in zip(cs, hw):
        rows, _, _ = ref.append(c, h, w)
        mla.append_chunk(h, w, *c.paged())
        wants.append(ref.attend(c))
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [[] for _ in cs]
    torch.cuda.synchronize()
    for _ in range(6):
        for i, (c, (h, w), s) in enumerate(zip(cs, hw, streams)):
            for form in ("expanded", "absorbed"):
                outs[i].append((form, mla.chunk_step(h, c.q_nope, c.q_rope, w, c.w_uk, c.w_uv, *c.paged(), form=form,
                                                     max_tokens=sum(c.lens), stream=s)))
    torch.cuda.synchronize()
    for (want, _, bound), got in zip(wants, outs):
        for form, g in got:
            check(g, want, bound[form], form)
