"""The chunk operators where their inputs leave the ordinary: bad lengths and row ranges,
quotients next to a tie, angles next to a quarter turn, two rows for one cache row, values
below fp16's normal range, scores far beyond fp32's integers. On the GPU, against 64 bits."""
import pytest

from tests import chunk_reference as ref

pytestmark = pytest.mark.gpu

OK, BOUNDS, RANGE = 0, 6, 7


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


def ints(v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ append_chunk: what is written
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d_model", [64, 1024])  # one split, many
@pytest.mark.parametrize("bad", ["short", "zero", "negative", "beyond the table", "huge"])
def test_append_writes_no_row_of_a_bad_length(mla, err, bad, d_model, fp8):
    """A length that does not hold the new rows, or passes the block table: none of the
    sequence's rows goes anywhere (its cached rows are not replaced by rows rotated for
    another position), the others are written."""
    import torch
    c = ref.Chunk([4, 3, 2], [70, 100, 20], H=1, fp8=fp8, seed=80)
    h, w = hidden(c.T, d_model, 81)
    rows, want, slack = ref.append(c, h, w)
    table = c.table.clone()
    table[1, 2:] = table[1, 1]  # every entry of the row is a page of its own
    c.table = table
    c.seq_lens[1] = {"short": 2, "zero": 0, "negative": -7, "beyond the table": c.max_pages * c.page + 1,
                     "huge": 2 ** 31 - 1}[bad]
    before = c.cache.clone()
    mla.append_chunk(h, w, *c.paged(), fp8_scales=c.scales, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == BOUNDS
    kept = torch.ones(c.num_pages * c.page, dtype=torch.bool, device="cuda")
    kept[rows[:4]] = kept[rows[7:]] = False
    assert torch.equal(bits(c.cache).view(-1, 576)[kept], bits(before).view(-1, 576)[kept])
    for part in (slice(0, 4), slice(7, 9)):
        got, y, s = c.cache.view(-1, 576)[rows[part]], want[part], slack[part]
        if fp8:
            got, y, s = got.view(torch.float8_e4m3fn), y / c.scales.double(), s / c.scales.double()
            tol = 2.0 ** -4 * y.abs() + 2.0 ** -10 + 1.1 * s
            y = y.clamp(-448, 448)
        else:
            tol = ref.U_BF16 * y.abs() + 1.1 * s
        assert ((got.double() - y).abs() <= tol).all()


CUTS = [[1, 5, 9], [0, 4, 12], [0, 6, 4], [-2, 4, 9], [0, 20, 9]]  # of 9 rows


@pytest.mark.parametrize("d_model", [64, 1024])
@pytest.mark.parametrize("cu", CUTS)
def test_append_reports_rows_outside_the_array(mla, err, cu, d_model):
    import torch
    c = ref.Chunk([4, 5], [70, 100], H=1, seed=82)
    h, w = hidden(c.T, d_model, 83)
    c.cu = ints(cu)
    allowed = torch.cat([c.rows(0), c.rows(1)])
    before = c.cache.clone()
    mla.append_chunk(h, w, *c.paged(), err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == BOUNDS
    other = torch.ones(c.num_pages * c.page, dtype=torch.bool, device="cuda")
    other[allowed] = False
    assert torch.equal(bits(c.cache).view(-1, 576)[other], bits(before).view(-1, 576)[other])


def test_append_writes_no_row_of_a_sequence_cut_short(mla, err):
    """Rows cu[1] .. cu[2]-1 of which the array holds the first only: attention would place
    that one last, its own count places it first, so it is not written at all."""
    import torch
    for d_model in (64, 1024):
        c = ref.Chunk([4, 5], [70, 100], H=1, seed=84)
        h, w = hidden(5, d_model, 85)
        rows = c.rows(0, 66, 70)
        before = c.cache.clone()
        err.zero_()
        mla.append_chunk(h, w, *c.paged(), err_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == BOUNDS
        kept = torch.ones(c.num_pages * c.page, dtype=torch.bool, device="cuda")
        kept[rows] = False
        assert torch.equal(bits(c.cache).view(-1, 576)[kept], bits(before).view(-1, 576)[kept])
        assert not torch.equal(bits(c.cache).view(-1, 576)[rows], bits(before).view(-1, 576)[rows])


def test_append_with_room_behind_the_last_row_reports_nothing(mla, err):
    import torch
    for d_model in (64, 1024):
        c = ref.Chunk([0, 4, 0, 5, 0], [0, 70, 3, 100, 0], H=1, seed=86, pad_rows=300)
        h, w = hidden(c.T, d_model, 87)
        mla.append_chunk(h, w, *c.paged(), err_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == OK


# ------------------------------------------------------------------ append_chunk: the values
@pytest.mark.parametrize("d_model", [64, 1024])
@pytest.mark.parametrize("seed", [90, 91, 92])
def test_append_quotients_next_to_ties(mla, err, seed, d_model):
    """The codes are those of the fp32 quotient, as mla_quantize_fp8's: columns whose
    quotient lies on or beside the middle of two codes, scales from 2^-110 to 2^127."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = ref.Chunk([1] * 8, [1] * 8, H=1, fp8=True, seed=seed)  # position 0: nothing is rotated
    h = torch.zeros(8, d_model, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(576, d_model, dtype=torch.bfloat16, device="cuda")
    h[:, 0] = 2.0 ** -torch.arange(8, device="cuda")
    w[:, 0] = torch.randn(576, generator=g, device="cuda").to(torch.bfloat16)
    low = torch.arange(1, 126, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    high = torch.arange(2, 127, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    pick = ((low + high) / 2)[torch.randint(0, 125, (576,), generator=g, device="cuda")]
    c.scales = (w[:, 0].float().abs() / pick).clamp(min=2.0 ** -100)  # row 0 on the ties, half of it in row 1, ...
    wide = torch.arange(0, 576, 9, device="cuda")
    e = torch.linspace(-110, 127, len(wide), device="cuda").round()
    c.scales[wide] = 2.0 ** e
    w[wide, 0] = (1.5 * 2.0 ** e.clamp(max=126)).to(torch.bfloat16)
    x = h[:, :1] * w[:, 0]  # exact: by powers of two; every other product is zero
    mla.append_chunk(h, w, *c.paged(), fp8_scales=c.scales, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == OK
    rows = torch.cat([c.rows(b) for b in range(8)])
    got = c.cache.view(-1, 576)[rows]
    assert torch.equal(got, (x.float() / c.scales).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    assert torch.equal(got, mla.quantize_fp8(x.contiguous(), c.scales))


@pytest.mark.parametrize("d_model", [64, 1024])
@pytest.mark.parametrize("last", [2000, 130000])
def test_append_rotation_keeps_small_sines(mla, err, last, d_model):
    """Rows whose pairs are (1, 0) before the rotation: the cosine and the sine themselves.
    A value is rounded to bf16 (2^-8 of it), after an angle within 2^-32 of a turn
    (below 2^-29) and a sine or cosine within 2^-22 of itself."""
    import torch
    n = 2000
    c = ref.Chunk([n], [last], H=1, seed=93)
    h = torch.zeros(n, d_model, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(576, d_model, dtype=torch.bfloat16, device="cuda")
    h[:, 0] = 1.0
    w[512::2, 0] = 1.0
    mla.append_chunk(h, w, *c.paged(), err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == OK
    got = c.cache.view(-1, 576)[c.rows(0, last - n, last), 512:].double()
    pos = torch.arange(last - n, last, dtype=torch.float64, device="cuda")
    ang = pos[:, None] * torch.tensor([10000.0 ** (-i / 32) for i in range(32)], dtype=torch.float64, device="cuda")
    want = torch.stack([ang.cos(), ang.sin()], -1).reshape(n, 64)
    assert (want.abs() < 1e-3).sum() > 20
    off = (got - want).abs()
    assert (off <= (ref.U_BF16 + 2.0 ** -21) * want.abs() + 2.0 ** -29).all(), (off / want.abs()).max().item()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d_model", [64, 1024])
def test_append_two_rows_for_one_cache_row(mla, err, d_model, fp8):
    """Two sequences whose new tokens fall on the same cache rows: each value is one of the
    two, and the rest of the pool is untouched."""
    import torch
    c = ref.Chunk([3, 3], [40, 40], H=1, fp8=fp8, seed=94)
    h, w = hidden(6, d_model, 95)
    mla.append_chunk(h, w, *c.paged(), fp8_scales=c.scales, err_word=err)
    one, two = (c.cache.view(-1, 576)[c.rows(b, 37, 40)].clone() for b in (0, 1))
    d = ref.Chunk([3, 3], [40, 40], H=1, fp8=fp8, seed=94)
    before = d.cache.clone()
    d.table[1] = d.table[0]
    rows = d.rows(0, 37, 40)
    mla.append_chunk(h, w, *d.paged(), fp8_scales=d.scales, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == OK
    got = bits(d.cache.view(-1, 576)[rows])
    assert ((got == bits(one)) | (got == bits(two))).all()
    other = torch.ones(d.num_pages * d.page, dtype=torch.bool, device="cuda")
    other[rows] = False
    assert torch.equal(bits(d.cache).view(-1, 576)[other], bits(before).view(-1, 576)[other])


# ------------------------------------------------------------------ read_kv
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cu", CUTS)
def test_read_reports_rows_outside_the_array(mla, err, cu, fp8):
    import torch
    c = ref.Chunk([4, 5], [70, 100], H=1, fp8=fp8, seed=96)
    c.cu = ints(cu)
    room = torch.full((9 + 20, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    mla.read_kv(*c.paged(), n_rows=9, fp8_scales=c.scales, out=room[:9], err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == BOUNDS
    assert (room[9:] == 7.0).all()
    if cu == [0, 4, 12]:  # the rows that are there are right
        for b, lo, n in ((0, 0, 4), (1, 4, 5)):
            x = c.values(b, 0, n)
            assert ((room[lo:lo + n].double() - x).abs() <= ref.U_BF16 * x.abs()).all()


# ------------------------------------------------------------------ attend_chunk
@pytest.mark.parametrize("form", ["expanded", "absorbed"])
@pytest.mark.parametrize("pad", [0, 60])  # up to 32 rows, more
@pytest.mark.parametrize("cu", CUTS + [[3, 3, 9], [9, 9, 9], [0, 0, -1]])
def test_attend_reports_rows_outside_the_array(mla, err, cu, pad, form):
    """Also where no row of the array belongs to the sequence that is out of range."""
    import torch
    c = ref.Chunk([4, 5], [70, 100], H=2, seed=101, pad_rows=pad)
    c.cu = ints(cu if pad == 0 else [v + pad if v > 9 else v for v in cu])
    room = torch.full((c.T + 4, 2, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=170, form=form, out=room[:c.T],
                     err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == BOUNDS
    assert (room[c.T:] == 3.0).all()


def scored(c, q, kr):
    """Scores of position alone, on the first positional column: exact products."""
    c.q_nope.zero_()
    c.q_rope.zero_()
    c.q_rope[:c.total, :, 0] = q
    pool = c.cache.view(-1, 576)
    for b in range(len(c.lens)):
        pool[c.rows(b), 512] = kr[b]


@pytest.mark.parametrize("size", [10, 20, 28, 30, 60, 100])
@pytest.mark.parametrize("sign", [1, -1])
def test_attend_scores_of_any_size(mla, err, sign, size):
    """Scores of up to 2^103: the tokens of the largest share the weight equally, whatever
    fp32 cannot tell of the scores themselves. (Score differences are 2^10 / 14 at least:
    every other weight is below 2^-100.)"""
    import torch
    c = ref.Chunk([300, 3], [900, 5000], H=2, seed=97)
    kr = [torch.arange(L, device="cuda") % 7 + 1 for L in c.lens]
    scored(c, sign * 2.0 ** size, [k.to(torch.bfloat16) for k in kr])
    got = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=5900, form="expanded",
                           err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == OK
    at = 0
    for b, (n, L) in enumerate(zip(c.new, c.lens)):
        lat = c.values(b)[:, :512]
        seen = torch.arange(L, device="cuda")[None] <= torch.arange(L - n, L, device="cuda")[:, None]
        k = (sign * kr[b]).double()[None].masked_fill(~seen, float("-inf"))
        p = (k == k.amax(-1, keepdim=True)).double()
        p /= p.sum(-1, keepdim=True)
        for h in range(2):
            uv = c.w_uv[h].double()
            v, vabs = lat @ uv.t(), lat.abs() @ uv.abs().t()
            want = p @ v
            tol = ref.U_BF16 * want.abs() + 4 * ref.U_F16 * (p @ v.abs()) + ref.TINY_F16 + 512 * ref.U_F32 * (p @ vabs)
            assert ((got[at:at + n, h].double() - want).abs() <= tol).all(), (b, h)
        at += n


def test_attend_scores_a_rounding_apart(mla, err):
    """Two scores that differ by two units in fp32's last place, which at this size are 296
    (2^12 / sqrt(192)): all the weight is the larger one's, also between pieces cut over
    the keys."""
    import torch
    c = ref.Chunk([2], [6000], H=1, seed=98)
    kr = torch.full((6000,), -1.0, device="cuda")
    scored(c, 2.0 ** 34, [kr.to(torch.bfloat16)])
    pool = c.cache.view(-1, 576)
    first, second = c.rows(0, 10, 11), c.rows(0, 5500, 5501)
    pool[first, 512], pool[second, 512] = 1.0, 1.0
    c.q_rope[:, :, 1] = 2.0 ** 12  # 2^34 + 2^12 against 2^34
    pool[c.rows(0), 513] = 0.0
    for high, low in ((second, first), (first, second)):
        pool[high, 513], pool[low, 513] = 1.0, 0.0
        got = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=6000, form="expanded",
                               err_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == OK
        lat = pool[high, :512].double()
        v, vabs = lat @ c.w_uv[0].double().t(), lat.abs() @ c.w_uv[0].double().abs().t()
        tol = (ref.U_BF16 + 4 * ref.U_F16) * v.abs() + ref.TINY_F16 + 512 * ref.U_F32 * vabs
        assert ((got[:, 0].double() - v).abs() <= tol).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_absorbed_reports_scores_too_far_apart(mla, err, fp8):
    """The absorbed form exchanges partial scores as fp16 offsets: beyond them, a report."""
    import torch
    c = ref.Chunk([3, 2], [200, 66], H=3, fp8=fp8, seed=99)
    c.q_nope.zero_()
    c.q_rope.zero_()
    c.q_rope[:, :, 0] = 2.0 ** 14

    def run(scale):
        err.zero_()
        out = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=266, fp8_scales=c.scales,
                               softmax_scale=scale, form="absorbed", err_word=err)
        torch.cuda.synchronize()
        return out, int(err.item())

    out, e = run(2.0 ** -2)   # scores of about +-2^13
    assert e == OK and torch.isfinite(out).all()
    out, e = run(2.0 ** 6)    # ... of +-2^21
    assert e == RANGE


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("form", ["expanded", "absorbed"])
@pytest.mark.parametrize("what", ["values", "queries", "keys"])
def test_attend_below_the_normal_range_of_fp16(mla, err, what, form, fp8):
    """Weights or queries that bring keys, values or queries below 2^-14: the resolution is
    2^-25 there, whatever the value. (Where a weight itself falls below it, each of the 512
    products of a value is off by 2^-25 of its latent.)"""
    import torch
    c = ref.Chunk([30, 150], [200, 170], H=2, fp8=fp8, seed=100)
    if what == "values":
        c.w_uv *= 2.0 ** -15
    elif what == "keys":
        c.w_uk *= 2.0 ** -15
        c.q_nope *= 2.0 ** 8
    else:
        c.q_nope *= 2.0 ** -17
    want, _, bound = ref.attend(c)
    got = mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=370, fp8_scales=c.scales,
                           form=form, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == OK
    extra = torch.zeros((), dtype=torch.float64, device="cuda")
    lat = max(c.values(b)[:, :512].abs().sum(-1).max().item() for b in range(2))
    if what == "values":
        extra = ref.TINY_F16 * lat
    elif what == "keys" and form == "expanded" and fp8:
        # a key off by 2^-25 of the latents' sum: scores by q times that
        qn = c.q_nope[:c.total].double().abs().sum(-1, keepdim=True)
        v = max((c.values(b)[:, :512].abs() @ c.w_uv.double().abs().transpose(1, 2)).max().item() for b in range(2))
        extra = torch.expm1(2 * ref.SCALE * ref.TINY_F16 * lat * qn) * v
    assert ((got.double() - want).abs() <= bound[form] + extra).all()
