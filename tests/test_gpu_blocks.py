"""The block-scaled 8-bit cache on the GPU. What is written is compared exactly with loops over the
definition (tests/blocks_reference.py). A value of such a cache is a bf16 number exactly, so reading it
back and the expanded attention are compared bit for bit with the same calls on a bf16 cache that holds the
values. The decode and the absorbed attention, whose products take fp16 operands, are compared with
64 bits, element by element, within bounds derived from their roundings."""
import numpy as np
import pytest

from tests import blocks_reference as blk
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


def bits(t):
    import torch
    return t.view(torch.int16) if t.element_size() == 2 else t.view(torch.int32)


class Blocks(ref.Chunk):
    """ref.Chunk, its cache as codes and entries (``codes``, ``entries``) and as the bf16 cache that holds
    the same values (``cache``). Spare pages and slack hold NaN codes, entries of what is not written 127."""

    def __init__(self, new, lens, *, block=32, spread=1.0, powers=(0, 0), **kw):
        import torch
        super().__init__(new, lens, **kw)
        page, n = self.page, self.num_pages
        g = torch.Generator(device=self.dev).manual_seed(kw.get("seed", 0) + 1)
        x = torch.nan_to_num(self.cache.double().cpu()).numpy().reshape(n, page, 576)
        # blocks and groups of unequal size
        size = torch.randn(n, page // block, 5, generator=g, device=self.dev).mul_(spread).round_()
        size += torch.randint(powers[0], powers[1] + 1, size.shape, generator=g, device=self.dev)
        size = size.long().cpu().numpy().repeat(block, 1)
        for k, (c0, c1) in enumerate(blk.GROUPS):
            x[:, :, c0:c1] = np.ldexp(x[:, :, c0:c1], size[:, :, k:k + 1])
        codes, entries = np.full((n, page, 576), blk.NAN_CODE, np.uint8), np.full((n, page // block, 8), 127, np.uint8)
        rows = np.concatenate([x.reshape(-1, 576)[self.rows(b).cpu().numpy()] for b in range(len(lens))] or [x[0, :0]])
        blk.write(codes, entries, rows, self.host_table, self.lens, self.lens, page, block)
        self.block = block
        self.codes, self.entries = torch.from_numpy(codes).to(self.dev), torch.from_numpy(entries).to(self.dev)
        self.cache = torch.from_numpy(blk.values(codes, entries)).to(self.dev).to(torch.bfloat16)

    def paged8(self):
        return self.codes, self.table, self.seq_lens, self.cu


# ------------------------------------------------------------------ write_kv
def written(mla, c, rows, err=None):
    """write_kv of the chunk's rows; returns (codes, entries) wanted."""
    codes, entries = c.codes.cpu().numpy().copy(), c.entries.cpu().numpy().copy()
    blk.write(codes, entries, rows.double().cpu().numpy(), c.host_table, c.lens, c.new, c.page, c.block)
    mla.write_kv(rows, *c.paged8(), fp8_scales=c.entries, err_word=err)
    return codes, entries


def draw_rows(c, seed, spread=2.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(c.T, 576, generator=g, device="cuda")
    x *= torch.exp2((torch.randn(c.T, 1, generator=g, device="cuda") * spread).round())
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("block", [16, 32, 64])
@pytest.mark.parametrize("new,lens,page,pad", [
    ([1], [1], 64, 0),
    ([1] * 33, list(range(1, 331, 10)), 64, 0),             # a decode step
    ([3, 0, 70], [3, 9, 200], 64, 4),
    ([63, 64, 65, 1, 128], [127, 64, 130, 65, 128], 64, 0),  # around tiles
    ([200, 2, 57, 0], [300, 129, 57, 3], 128, 130),
    ([1700, 1650], [1717, 1650], 128, 1),
    ([0, 0, 5], [100, 7, 64], 64, 3),
])
def test_rows_written(mla, err, block, new, lens, page, pad):
    c = Blocks(new, lens, H=1, page=page, block=block, seed=5, pad_rows=pad)
    rows = draw_rows(c, 6)
    codes, entries = written(mla, c, rows, err)
    assert (c.codes.cpu().numpy() == codes).all() and (c.entries.cpu().numpy() == entries).all()
    mla.write_kv(rows, *c.paged8(), fp8_scales=c.entries, err_word=err)  # the same again changes nothing
    assert (c.codes.cpu().numpy() == codes).all() and (c.entries.cpu().numpy() == entries).all()
    assert int(err.item()) == 0


@pytest.mark.parametrize("B", [31, 100, 1100, 4096])
def test_many_sequences(mla, err, B):
    """No row to three for each of many sequences, a page each: the search for a CTA's sequence at every depth."""
    import torch
    new = [(7 * b) % 4 for b in range(B)]
    lens = [n + (13 * b) % 61 for b, n in enumerate(new)]
    i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(B)
    codes = torch.randint(0, 127, (B, 64, 576), dtype=torch.uint8, generator=g, device="cuda")
    entries = torch.randint(120, 124, (B, 4, 8), dtype=torch.uint8, generator=g, device="cuda")
    rows = torch.randn(sum(new) + 2, 576, generator=g, device="cuda").to(torch.bfloat16)
    table = [[B - 1 - b] for b in range(B)]
    want = codes.cpu().numpy(), entries.cpu().numpy()
    blk.write(*want, rows.double().cpu().numpy(), table, lens, new, 64, 16)
    cu = i([0] + np.cumsum(new).tolist())
    mla.write_kv(rows, codes, i(table), i(lens), cu, fp8_scales=entries, err_word=err)
    assert (codes.cpu().numpy() == want[0]).all() and (entries.cpu().numpy() == want[1]).all() and int(err.item()) == 0


@pytest.mark.parametrize("block", [16, 64])
def test_token_by_token(mla, err, block):
    """A sequence grown a token at a time, the rows' size rising and falling: powers grow with it and older
    codes are requantised each time."""
    import torch
    c = Blocks([1], [1], H=1, block=block, seed=9, spare=1)
    c.table[0, 0] = 1
    c.host_table[0][0] = 1
    want = [c.codes.cpu().numpy(), c.entries.cpu().numpy()]
    g = torch.Generator(device="cuda").manual_seed(3)
    for L in range(1, 65):
        row = (torch.randn(1, 576, generator=g, device="cuda") * 2.0 ** ((L * 5) % 23 - 11)).to(torch.bfloat16)
        c.seq_lens.fill_(L)
        mla.write_kv(row, *c.paged8(), fp8_scales=c.entries, err_word=err)
        blk.write(*want, row.double().cpu().numpy(), c.host_table, [L], [1], 64, block)
    assert (c.codes.cpu().numpy() == want[0]).all() and (c.entries.cpu().numpy() == want[1]).all()
    assert int(err.item()) == 0


@pytest.mark.parametrize("block", [16, 32])
def test_special_values(mla, err, block):
    """Zeros, signed zeros, infinities, NaNs, subnormals, the largest and values on both sides of a power."""
    import torch
    c = Blocks([40], [45], H=1, block=block, seed=2)
    rows = torch.zeros(40, 576, dtype=torch.bfloat16, device="cuda")
    rows[3, 0:128] = float("inf")
    rows[4, 5] = float("nan")
    rows[4, 6] = -float("nan")
    rows[5, 128:256] = 2.0 ** -130
    rows[6, 256] = 448.0 * 2 ** 20
    rows[7, 256] = 450.0
    rows[8, 300:310] = -2.0 ** 126
    rows[9, 511] = 2.0 ** -133
    rows[10, 512:] = torch.linspace(-448, 448, 64).to(torch.bfloat16)
    rows[11, 512] = -float("inf")
    rows[20, :] = -0.0
    rows[30, 100] = 448.0
    rows[31, 200] = 450.0  # the next bf16 number
    codes, entries = written(mla, c, rows, err)
    assert (c.codes.cpu().numpy() == codes).all() and (c.entries.cpu().numpy() == entries).all()
    assert int(err.item()) == 0


def test_bad_rows_lengths_and_pages_write_nothing(mla, err):
    import torch
    def fresh():
        c = Blocks([5, 70, 9], [5, 130, 40], H=1, seed=4)
        return c, draw_rows(c, 1), c.codes.clone(), c.entries.clone()

    c, rows, codes, entries = fresh()
    c.table[1, 1] = c.num_pages  # positions 64 .. 127 of sequence 1
    mla.write_kv(rows, *c.paged8(), fp8_scales=c.entries, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == BOUNDS
    same = (c.codes == codes).all(-1).view(-1)
    wrote = torch.cat([c.rows(0), c.rows(1, 60, 64), c.rows(2, 31, 40)])
    kept = torch.ones_like(same)
    kept[wrote] = False
    kept[c.host_table[1][2] * 64:][:64] = False  # the third page, and the first one's older tokens
    kept[c.host_table[1][0] * 64:][:64] = False
    kept[c.host_table[2][0] * 64:][:64] = False
    assert same[kept].all() and not same[wrote].any()
    for lens, cu in (([5, 69, 40], [0, 5, 75, 84]), ([5, 64 * c.max_pages + 1, 40], [0, 5, 75, 84]),
                     ([5, 130, 40], [0, 5, 4, 84]), ([5, 130, 90], [0, 5, 75, 160]), ([5, 130, 40], [-1, 5, 75, 84])):
        c, rows, codes, entries = fresh()
        err.zero_()
        c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        c.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        mla.write_kv(rows, *c.paged8(), fp8_scales=c.entries, err_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == BOUNDS, (lens, cu)
        for b in range(3):
            n = cu[b + 1] - cu[b]
            if cu[b] < 0 or n < 0 or cu[b + 1] > 84 or lens[b] < n or lens[b] > 64 * c.max_pages:
                assert torch.equal(c.codes.view(-1, 576)[c.rows(b)], codes.view(-1, 576)[c.rows(b)]), (lens, cu, b)


# ------------------------------------------------------------------ read_kv
@pytest.mark.parametrize("block", [16, 32, 64])
@pytest.mark.parametrize("page,lens,first,count", [
    (64, [1], [0], [1]),
    (64, [70, 1, 129, 64], [0, 0, 3, 63], [70, 1, 126, 1]),
    (128, [300, 5, 128], [299, 0, 0], [1, 5, 128]),
    (64, [100, 40], [90, 40], [30, 7]),              # past the end: zeros
    (128, [1000, 777, 0, 513], [1, 0, 0, 500], [999, 0, 0, 13]),
])
def test_read_rows(mla, err, block, page, lens, first, count):
    import torch
    c = Blocks(count, lens, H=1, page=page, block=block, seed=3, spread=3.0, powers=(-100, 100))
    f = torch.tensor(first, dtype=torch.int32, device="cuda")
    out = [torch.full((c.total + 5, 576), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    got = mla.read_kv(*c.paged8(), n_rows=c.total + 5, first=f, fp8_scales=c.entries, out=out[0], err_word=err)
    mla.read_kv(*c.paged(), n_rows=c.total + 5, first=f, out=out[1])
    torch.cuda.synchronize()
    assert got is out[0] and torch.equal(bits(out[0]), bits(out[1])) and int(err.item()) == 0


def test_read_gives_nan_for_nan_codes(mla):
    import torch
    c = Blocks([70], [70], H=1, seed=3)
    c.codes.view(-1, 576)[c.rows(0)[10], 5] = 0xFF
    got = mla.read_kv(*c.paged8(), n_rows=70, fp8_scales=c.entries)
    assert torch.isnan(got[10, 5]) and torch.isnan(got).sum() == 1


# ------------------------------------------------------------------ decode
def decode(mla, c, cache, scales, n_q, err=None, scale=ref.SCALE):
    return mla.decode_step(c.q_nope, c.q_rope, c.w_uk, c.w_uv, cache, c.table, c.seq_lens, n_q=n_q, fp8_scales=scales,
                           err_word=err, softmax_scale=scale)


def check_decode(c, r, n_q, scale=ref.SCALE, skip=()):
    """A step's q_abs, u, lse and out within the bounds of its roundings, each given those before it.

    q_abs is a sum of 128 products in fp32, rounded to fp16. A score is off by dz: values in fp16 are exact from
    2^-14 on and off by 2^-25 below, the
    sums of 576 products are in fp32, the half of them that comes from the other CTA goes through fp16 as an
    offset of at most half the half's spread (2^-11 relative), and scaling and shifting round a few times
    in fp32. That moves weights by a factor exp(+-2 dz). A weight is rounded to fp16 (2^-11, below 2^-14 of the largest
    by 2^-25 of it), ex2 and the fp32 sums are off by less than 2^-16; the partial is rounded to fp16 and the
    merged u to bf16. out is W^UV times that u, in fp32, rounded to bf16."""
    import torch
    tiny, f16, bf = ref.TINY_F16, ref.U_F16, ref.U_BF16
    qn, wk = c.q_nope.double(), c.w_uk.double()
    qa = torch.cat([torch.einsum("thd,hdc->thc", qn, wk), c.q_rope.double()], 2)
    bound = 1.01 * f16 * qa.abs() + tiny
    bound[..., :512] += 128 * ref.U_F32 * torch.einsum("thd,hdc->thc", qn.abs(), wk.abs())
    assert r["q_abs"].dtype == torch.float16
    rows = [b * n_q + j for b in range(len(c.lens)) if b not in skip for j in range(n_q)]
    assert ((r["q_abs"].double() - qa).abs() <= bound)[rows].all()
    for b, L in enumerate(c.lens):
        if b in skip:
            continue
        x = c.values(b)
        for j in range(n_q):
            t, n = b * n_q + j, L - n_q + j + 1
            qa, xs = r["q_abs"][t].double(), x[:n]
            lat = xs[:, :512]
            cta = [torch.cat([torch.arange(256 * k, 256 * k + 256), torch.arange(512 + 32 * k, 544 + 32 * k)])
                   for k in range(2)]
            half = [qa[:, i] @ xs[:, i].t() * scale for i in (i.to(c.dev) for i in cta)]
            z = half[0] + half[1]
            spread = torch.stack([h.amax(-1) - h.amin(-1) for h in half]).amax(0)
            dz = scale * (tiny * (qa.abs().sum(-1) + xs.abs().sum(-1).max())
                          + 576 * ref.U_F32 * (qa.abs() @ xs.abs().t()).amax(-1))
            dz += f16 * spread / 2 + 2.0 ** -20 * z.abs().amax(-1)
            p = torch.softmax(z, -1)
            u, lse = p @ lat, torch.logsumexp(z, -1)
            du = (p @ lat.abs()) * (torch.expm1(2 * dz) + f16 + 2.0 ** -15)[:, None] + 2 * tiny * lat.abs().sum(0)
            du += (f16 + bf) * 1.01 * u.abs() + 2 * tiny
            assert ((r["u"][t].double() - u).abs() <= du).all(), (b, j)
            assert ((r["lse"][t].double() - lse).abs() <= dz + 2.0 ** -15 + 2.0 ** -20 * lse.abs()).all(), (b, j)
            gu, w = r["u"][t].double(), c.w_uv.double()
            out = torch.einsum("hc,hvc->hv", gu, w)
            bound = 1.01 * bf * out.abs() + 512 * ref.U_F32 * torch.einsum("hc,hvc->hv", gu.abs(), w.abs())
            assert ((r["out"][t].double() - out).abs() <= bound).all(), (b, j)


@pytest.mark.parametrize("H,n_q,page,block,lens", [
    (128, 1, 64, 64, [4096, 64, 1]),
    (16, 2, 64, 16, [256, 2, 65]),
    (128, 2, 128, 32, [130, 1000, 129]),
    (1, 1, 128, 16, [1]),
    (40, 1, 128, 64, [300, 127, 128, 3000]),
    (97, 1, 64, 32, [int(7 + 61 * b) for b in range(40)]),
    (128, 1, 64, 16, [9000]),
    (128, 1, 64, 64, [63] * 90),
])
def test_decode(mla, err, H, n_q, page, block, lens):
    import torch
    c = Blocks([n_q] * len(lens), lens, H=H, page=page, block=block, seed=8)
    got = decode(mla, c, c.codes, c.entries, n_q, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check_decode(c, got, n_q)
    again = decode(mla, c, c.codes, c.entries, n_q, err)
    for k in ("u", "lse", "out"):
        assert torch.equal(bits(got[k]), bits(again[k])), k


@pytest.mark.parametrize("powers,top", [((-40, -30), -110), ((-20, -8), -110), ((-6, 6), 0), ((8, 12), 12)])
def test_decode_at_small_and_large_powers(mla, err, powers, top):
    """Powers below 2^-24, where the widening takes a second step, around fp16's subnormals, and up to values
    of some 20000; the scale brings the largest scores to ordinary size. The positional group of the large ones
    is kept at ordinary size (its own scores would pass any range)."""
    import torch
    c = Blocks([1, 1], [700, 64], H=128, block=16, seed=8, powers=powers, spread=0.0)
    got = decode(mla, c, c.codes, c.entries, 1, err, ref.SCALE * 2.0 ** -max(top, 0))
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check_decode(c, got, 1, ref.SCALE * 2.0 ** -max(top, 0))


def test_values_outside_fp16_are_reported(mla, err):
    """A value of the context of 65520 or more, in a latent or positional column; one behind the context is not."""
    import torch
    for row, col, code, entry, want in ((60, 300, 0x7E, 127 + 8, RANGE), (60, 300, 0x7E, 127 + 7, 0),
                                        (60, 540, 0xFE, 127 + 20, RANGE), (3, 5, 0x38, 127 + 15, 0),
                                        (3, 5, 0x38, 127 + 16, RANGE)):
        c = Blocks([1], [70], H=16, block=16, seed=8)
        group = min(col // 128, 4)
        for at, expect in ((row, want), (75, 0)):
            codes, entries = c.codes.clone(), c.entries.clone()
            pool = c.rows(0)[at].item() if at < 70 else c.host_table[0][1] * 64 + at - 64
            rows = slice(pool // 16 * 16, pool // 16 * 16 + 16)
            cols = slice(*blk.GROUPS[group])
            codes.view(-1, 576)[rows, cols] = 0  # the block's group holds nothing else
            codes.view(-1, 576)[pool, col] = code
            entries.view(-1, 8)[pool // 16, group] = entry
            err.zero_()
            decode(mla, c, codes, entries, 1, err, 2.0 ** -20)
            torch.cuda.synchronize()
            # (a lone positional key of 2^27, or a latent of 57344, may pass the partial's range as well)
            assert int(err.item()) == expect, (row, col, code, entry, at)


def test_queries_outside_fp16_are_reported(mla, err):
    import torch
    for pos in (False, True):
        c = Blocks([1, 1], [70, 70], H=16, seed=8)
        if pos:
            c.q_rope[1, 3, 40] = 65536.0
        else:
            c.q_nope[1, 3] = 3.0e5
        err.zero_()
        got = decode(mla, c, c.codes, c.entries, 1, err)
        torch.cuda.synchronize()
        assert int(err.item()) == RANGE
        assert torch.isfinite(got["out"][0].float()).all()


def test_nan_code_in_the_context_and_behind_it(mla, err):
    """A NaN code behind the context changes nothing (Blocks puts them there); one inside gives NaN to its
    sequence and to no other."""
    import torch
    c = Blocks([1, 1, 1], [100, 200, 65], H=16, block=32, seed=8)
    c.codes.view(-1, 576)[c.rows(1)[150], 77] = 0x7F
    got = decode(mla, c, c.codes, c.entries, 1, err)
    torch.cuda.synchronize()
    assert torch.isnan(got["u"][1, :, 77].float()).all() and torch.isfinite(got["out"][0].float()).all()
    check_decode(c, got, 1, skip=(1,))


def test_decode_calls_without_the_step(mla, err):
    """decode_paged_fp8 with block scales, planned and not, is the step's decode."""
    import torch
    c = Blocks([1, 1], [500, 70], H=24, page=128, block=16, seed=8)
    want = decode(mla, c, c.codes, c.entries, 1, err)
    torch.cuda.synchronize()
    for planned in (False, True):
        ws = None
        if planned:
            ws, g = mla.decode_plan(c.seq_lens, n_q=1, H=24, max_pages=c.max_pages, num_pages=c.num_pages,
                                    page_size=128)
            torch.cuda.synchronize()
        ws, g = mla.decode_paged_fp8(want["q_abs"], c.codes, c.entries, c.table, c.seq_lens, planned=planned,
                                     workspace=ws, err_word=err, n_q=1, softmax_scale=ref.SCALE)
        u, lse = mla.combine(ws, B=2, n_q=1, H=24, num_splits=g)
        torch.cuda.synchronize()
        assert torch.equal(bits(u), bits(want["u"])) and torch.equal(bits(lse), bits(want["lse"]))
    # a bf16 query is taken as it is: its values are fp16 numbers too
    q = mla.absorb_q(c.q_nope, c.q_rope, c.w_uk)
    assert (q.to(torch.float16).float() == q.float()).all()
    res = []
    for query in (q, q.to(torch.float16)):
        ws, g = mla.decode_paged_fp8(query, c.codes, c.entries, c.table, c.seq_lens, n_q=1, err_word=err)
        res.append(mla.combine(ws, B=2, n_q=1, H=24, num_splits=g))
        torch.cuda.synchronize()
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(*res)) and int(err.item()) == 0


def test_queries_in_bf16_outside_fp16_are_reported(mla, err):
    import torch
    c = Blocks([1, 1], [70, 70], H=16, seed=8)
    for d, value, want in ((3, 65536.0, RANGE), (560, -65536.0, RANGE), (3, 65280.0, 0)):
        q = mla.absorb_q(c.q_nope, c.q_rope, c.w_uk)
        q[1, 5, d] = value
        err.zero_()
        mla.decode_paged_fp8(q, c.codes, c.entries, c.table, c.seq_lens, n_q=1, err_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == want


def test_decode_reports_bad_pages(mla, err):
    import torch
    c = Blocks([1, 1], [200, 70], H=16, seed=8)
    c.table[0, 1] = -1
    got = decode(mla, c, c.codes, c.entries, 1, err)
    torch.cuda.synchronize()
    assert int(err.item()) == BOUNDS
    check_decode(c, got, 1, skip=(0,))


def test_captured_step(mla, err):
    """CapturedStep on a block-scaled cache, the cache and the lengths changing between replays."""
    import torch
    c = Blocks([1, 1], [70, 300], H=16, block=16, seed=8)
    step = mla.CapturedStep(c.w_uk, c.w_uv, c.codes, c.table, c.seq_lens, n_q=1, fp8_scales=c.entries, err_word=err)
    for k in range(3):
        got = {key: v.clone() for key, v in step(c.q_nope, c.q_rope).items()}
        want = decode(mla, c, c.codes, c.entries, 1)
        torch.cuda.synchronize()
        assert all(torch.equal(bits(got[key]), bits(want[key])) for key in ("u", "lse", "out"))
        check_decode(c, want, 1)
        c.lens = [c.lens[0] - 7, c.lens[1] - 90]
        c.seq_lens.copy_(torch.tensor(c.lens, dtype=torch.int32))
        c.codes.bitwise_xor_(0x80)  # every value's sign
        c.cache.neg_()
    assert int(err.item()) == 0


def test_captured_step_with_host_buffers(mla, err):
    """replay_host reads queries, table and lengths from pinned memory and writes out and lse there."""
    import torch
    c = Blocks([2, 2, 2], [70, 300, 2], H=24, block=32, seed=9)
    step = mla.CapturedStep(c.w_uk, c.w_uv, c.codes, c.table, c.seq_lens, n_q=2, fp8_scales=c.entries, err_word=err,
                            host_io=True)
    for k in range(2):
        step.host["q_nope"].copy_(c.q_nope)
        step.host["q_rope"].copy_(c.q_rope)
        step.host["seq_lens"].copy_(c.seq_lens)
        torch.cuda.synchronize()
        step.replay_host()
        want = decode(mla, c, c.codes, c.entries, 2)
        torch.cuda.synchronize()
        assert all(torch.equal(bits(step.host[key].cuda()), bits(want[key])) for key in ("lse", "out"))
        c.seq_lens.sub_(torch.tensor([5, 200, 0], dtype=torch.int32, device="cuda"))
    assert int(err.item()) == 0


def test_test_build_finds_no_bad_address(mla):
    """The same decode in the test build, whose kernel checks every shared and tensor memory address."""
    import ctypes

    import torch
    lib, dbg = mla.lib(), mla.debug_lib()
    c = Blocks([2] * 5, [2, 64, 65, 700, 129], H=40, page=128, block=16, seed=8)
    q = mla.absorb_q(c.q_nope, c.q_rope, c.w_uk)
    assert dbg.mla_debug_reset() == 0
    out = []
    for L in (lib, dbg):
        g = mla.default_splits(2)
        ws = torch.empty(mla.workspace_bytes(5, 2, 40, g), dtype=torch.uint8, device="cuda")
        e = torch.zeros(1, dtype=torch.int32, device="cuda")
        s = torch.cuda.current_stream().cuda_stream
        st = L.mla_decode_paged_blocks(q.data_ptr(), 0, c.codes.data_ptr(), c.entries.data_ptr(), 16,
                                       c.table.data_ptr(),
                                       c.seq_lens.data_ptr(), 5, 2, 40, c.num_pages, 128, c.max_pages, ref.SCALE, g,
                                       ws.data_ptr(), ws.numel(), e.data_ptr(), s)
        assert st == 0
        torch.cuda.synchronize()
        out.append(mla.combine(ws, B=5, n_q=2, H=40, num_splits=g))
        torch.cuda.synchronize()
        assert int(e.item()) == 0
    n = (ctypes.c_ulonglong * 4)()
    assert dbg.mla_debug_read_counters(n, 4) == 0 and n[1] == 0
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(*out))


@pytest.mark.parametrize("lens", [[70], [4096] * 8])
def test_waits_that_run_out_are_reported(mla, lens):
    """The test build's decode with a producer that loads nothing: every wait gives up, the kernel reports it
    and ends, and the library works as before."""
    import torch
    dbg = mla.debug_lib()
    c = Blocks([1] * len(lens), lens, H=16, block=16, seed=8)
    q = mla.absorb_q(c.q_nope, c.q_rope, c.w_uk)
    g = mla.default_splits(1)
    ws = torch.empty(mla.workspace_bytes(len(lens), 1, 16, g), dtype=torch.uint8, device="cuda")
    e = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    try:
        assert dbg.mla_debug_set_wait_limit(2_000_000) == 0 and dbg.mla_debug_set_skip_producer(1) == 0
        st = dbg.mla_decode_paged_blocks(q.data_ptr(), 0, c.codes.data_ptr(), c.entries.data_ptr(), 16,
                                         c.table.data_ptr(),
                                         c.seq_lens.data_ptr(), len(lens), 1, 16, c.num_pages, 64, c.max_pages,
                                         ref.SCALE, g, ws.data_ptr(), ws.numel(), e.data_ptr(),
                                         torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert st == 0 and int(e.item()) == 5  # MLA_ERR_TIMEOUT
    finally:
        assert dbg.mla_debug_reset() == 0
    e.zero_()
    check_decode(c, decode(mla, c, c.codes, c.entries, 1, e), 1)
    assert int(e.item()) == 0


# ------------------------------------------------------------------ attend_chunk
CHUNKS = [
    (16, 64, 64, [1], [1], 0),
    (4, 64, 16, [5, 0, 70], [5, 9, 200], 4),
    (128, 128, 32, [4] * 3, [300, 4, 129], 0),
    (7, 128, 16, [130, 1, 257], [1000, 64, 257], 3),
    (40, 64, 32, [37, 300], [1500, 300], 0),
]


def attend(mla, c, cache, scales, form, err=None):
    import torch
    out = torch.full((c.T, c.H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.T, c.H), 7.0, dtype=torch.float32, device="cuda")
    mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, cache, c.table, c.seq_lens, c.cu, max_tokens=sum(c.lens),
                     fp8_scales=scales, form=form, out=out, lse=lse, err_word=err)
    return out, lse


def absorbed_bound(c):
    """(out, lse, bounds): chunk_reference's for an FP8 cache whose scales are 1 (absorbed query, weights and u in
    fp16). A score, and so lse, is off by the query's rounding times the absolute products, 1.25 as there, and by
    the exchanged half's, an offset of at most half its spread, which those products bound too."""
    import torch
    c.fp8, c.scales = True, torch.ones(576, device=c.dev)
    values, c.values = c.values, lambda b, lo=0, hi=None: c.cache.view(-1, 576)[c.rows(b, lo, hi)].double()
    want, lse, bounds = ref.attend(c)
    dz = []
    for b, n in enumerate(c.new):
        if n:
            at, x = sum(c.new[:b]), c.values(b).abs()
            qa = torch.einsum("thd,hdc->thc", c.q_nope[at:at + n].double(), c.w_uk.double())
            q = torch.cat([qa, c.q_rope[at:at + n].double()], 2).abs()
            dz.append(ref.SCALE * (2.25 * ref.U_F16 * (q @ x.t()).amax(-1) + ref.TINY_F16 * x.sum(-1).max()))
    c.fp8, c.scales, c.values = False, None, values
    return want, lse, bounds["absorbed"], torch.cat(dz) + 2.0 ** -15 + 2.0 ** -20 * lse.abs()


@pytest.mark.parametrize("H,page,block,new,lens,pad", CHUNKS)
def test_expanded_attention_is_the_bf16_one_on_the_same_values(mla, err, H, page, block, new, lens, pad):
    import torch
    c = Blocks(new, lens, H=H, page=page, block=block, seed=11, pad_rows=pad)
    got, want = (attend(mla, c, k, e, "expanded", err) for k, e in ((c.codes, c.entries), (c.cache, None)))
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert torch.equal(bits(got[0]), bits(want[0])) and torch.equal(bits(got[1]), bits(want[1]))
    assert (got[0][c.total:] == 7.0).all() and (got[1][c.total:] == 7.0).all()


@pytest.mark.parametrize("H,page,block,new,lens,pad", CHUNKS)
def test_absorbed_attention(mla, err, H, page, block, new, lens, pad):
    import torch
    c = Blocks(new, lens, H=H, page=page, block=block, seed=11, pad_rows=pad, spread=0.5)
    out, lse = attend(mla, c, c.codes, c.entries, "absorbed", err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and (out[c.total:] == 7.0).all() and (lse[c.total:] == 7.0).all()
    want, want_lse, bound, lse_bound = absorbed_bound(c)
    assert ((out[:c.total].double() - want).abs() <= bound).all()
    assert ((lse[:c.total].double() - want_lse).abs() <= lse_bound).all()


@pytest.mark.parametrize("H,page,block,new,lens,pad", CHUNKS[3:])
def test_calls_repeat_their_bits(mla, err, H, page, block, new, lens, pad):
    """Slots of codes and operands pass between the roles of a CTA hundreds of times in a call: one handed on too
    early shows as bits that change from call to call."""
    import torch
    c = Blocks(new, lens, H=H, page=page, block=block, seed=11, pad_rows=pad, spread=0.5)
    want = [bits(x) for x in attend(mla, c, c.codes, c.entries, "absorbed", err)]
    for _ in range(60):
        got = [bits(x) for x in attend(mla, c, c.codes, c.entries, "absorbed", err)]
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert int(err.item()) == 0


def test_expanded_and_auto_against_64_bits(mla, err):
    """A ragged chunk within the bounds that chunk_reference derives for a bf16 cache (the values are the
    cache's own, so its quantisation is no part of the error)."""
    import torch
    c = Blocks([9, 1, 60], [700, 1, 60], H=8, block=16, seed=12, spread=0.5)
    want, lse, bounds = ref.attend(c)
    for form in ("expanded", "auto"):
        got, _ = attend(mla, c, c.codes, c.entries, form, err)
        torch.cuda.synchronize()
        bound = torch.maximum(*bounds.values()) if form == "auto" else bounds[form]
        assert int(err.item()) == 0 and ((got.double() - want).abs() <= bound).all()


def test_a_nan_code_reaches_the_queries_that_see_it(mla):
    """A NaN in token 40 of 70 new ones: rows 40 and on are NaN, those before are as without it, in both forms."""
    import torch
    for form in ("expanded", "absorbed"):
        c = Blocks([70], [70], H=4, block=64, seed=3)
        want, _ = attend(mla, c, c.codes, c.entries, form)
        c.codes.view(-1, 576)[c.rows(0)[40], 100] = 0x7F
        got, _ = attend(mla, c, c.codes, c.entries, form)
        torch.cuda.synchronize()
        assert torch.equal(bits(got[:40]), bits(want[:40])) and torch.isnan(got[40:].float()).all(), form


# ------------------------------------------------------------------ append_chunk, and all of it together
@pytest.mark.parametrize("new,lens,d_model,page,block,pad", [
    ([1], [1], 64, 64, 64, 0),
    ([3, 0, 70], [3, 9, 200], 128, 64, 16, 4),          # one split: the GEMM's own epilogue
    ([1] * 33, list(range(1, 331, 10)), 512, 64, 32, 0),  # split over d_model
    ([200, 0, 57], [7000, 3, 57], 1024, 128, 16, 130),
])
def test_append_is_the_bf16_append_written(mla, err, new, lens, d_model, page, block, pad):
    """append_chunk's rows as a bf16 cache gets them, then write_kv."""
    import torch
    c = Blocks(new, lens, H=1, page=page, block=block, seed=5, pad_rows=pad)
    g = torch.Generator(device="cuda").manual_seed(6)
    h = torch.randn(c.T, d_model, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(576, d_model, generator=g, device="cuda") * d_model ** -0.5).to(torch.bfloat16)
    mla.append_chunk(h, w, *c.paged(), err_word=err)
    first = torch.tensor([L - n for L, n in zip(lens, new)], dtype=torch.int32, device="cuda")
    rows = mla.read_kv(*c.paged(), n_rows=c.T, first=first)
    rows[c.total:] = 0
    want = c.codes.clone(), c.entries.clone()
    mla.write_kv(rows, want[0], c.table, c.seq_lens, c.cu, fp8_scales=want[1])
    ws = mla.append_chunk(h, w, *c.paged8(), fp8_scales=c.entries, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and ws.numel() == mla.append_chunk_blocks_workspace_bytes(c.T, d_model)
    assert torch.equal(c.codes, want[0]) and torch.equal(c.entries, want[1])


@pytest.mark.parametrize("page,block", [(64, 64), (128, 16)])
def test_serving_loop(mla, err, page, block):
    """Prompts arrive, their pages are assigned on the GPU, written and attended (chunk_step), decode steps
    append a token each, one sequence finishes and another takes its pages: after each step the attention
    is that of a bf16 cache read back from the 8-bit one."""
    import torch
    B, H, d, max_pages, num_pages = 3, 8, 256, 6, 10
    bf, i32 = torch.bfloat16, torch.int32
    g = torch.Generator(device="cuda").manual_seed(0)
    normal = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(bf)  # noqa: E731
    i = lambda v: torch.tensor(v, dtype=i32, device="cuda")  # noqa: E731
    w_dkr = normal(576, d, std=d ** -0.5)
    w_uk, w_uv = normal(H, 128, 512, std=512 ** -0.5), normal(H, 128, 512, std=512 ** -0.5)
    codes = torch.full((num_pages, page, 576), 0x7F, dtype=torch.uint8, device="cuda")
    entries = torch.zeros(num_pages, page // block, 8, dtype=torch.uint8, device="cuda")
    table = torch.full((B, max_pages), -1, dtype=i32, device="cuda")
    held, free, count = i([0] * B), i(list(range(num_pages))), i([num_pages])
    book = blk.Pages(table.tolist(), [0] * B, list(range(num_pages)), page)
    lens = [0] * B
    for step, new in enumerate(([150, 0, 70], [1, 0, 1], [1, 129, 1], [1, 1, 1], [0, 1, 1], [100, 1, 1], [1, 1, 1])):
        if step == 4:
            lens[0] = 0  # finished
        lens = [L + n for L, n in zip(lens, new)]
        T = sum(new) + 2
        cu, sl = i([sum(new[:b]) for b in range(B + 1)]), i(lens)
        slots = torch.empty(T, dtype=torch.int64, device="cuda")
        mla.update_pages(table, held, sl, free, count, page_size=page, cu=cu, slots=slots, err_word=err)
        assert slots.tolist() == book.update(lens, new, T) and table.tolist() == book.table
        h, qn, qr = normal(T, d), normal(T, H, 128), normal(T, H, 64)
        got = mla.chunk_step(h, qn, qr, w_dkr, w_uk, w_uv, codes, table, sl, cu, max_tokens=sum(lens),
                             fp8_scales=entries, form="expanded", err_word=err)
        # the rows at the slots, as the 8-bit cache holds them
        first = i([L - n for L, n in zip(lens, new)])
        rows = mla.read_kv(codes, table, sl, cu, n_rows=T, first=first, fp8_scales=entries, err_word=err)[:T - 2]
        values = blk.values(codes.cpu().numpy(), entries.cpu().numpy())
        flat = torch.from_numpy(values).cuda().to(bf)
        assert torch.equal(rows, flat.view(-1, 576)[slots[:T - 2]])
        want = mla.attend_chunk(qn, qr, w_uk, w_uv, flat, table, sl, cu, max_tokens=sum(lens), form="expanded")
        assert torch.equal(bits(got[:T - 2]), bits(want[:T - 2]))
        if min(new) == 1 == max(new):  # a decode step's own call on the same cache, at the library's parity tolerance
            a = mla.decode_step(qn[:B], qr[:B], w_uk, w_uv, codes, table, sl, n_q=1, fp8_scales=entries, err_word=err)
            off = (a["out"].double() - want[:B].double()).abs()
            assert off.max() <= 2e-2 and off.sum() <= 5e-3 * want[:B].double().abs().sum()
        torch.cuda.synchronize()
        assert int(err.item()) == 0, step


def test_a_captured_serving_step(mla, err):
    """update_pages, write_kv and the decode in one graph, replayed while lengths, rows and queries change."""
    import torch
    torch.manual_seed(3)
    B, H, page, block = 4, 16, 64, 32
    c = Blocks([1] * B, [1] * B, H=H, page=page, block=block, seed=1)
    i32 = torch.int32
    num_pages, max_pages = 12, 4
    codes = torch.full((num_pages, page, 576), 0x7F, dtype=torch.uint8, device="cuda")
    entries = torch.zeros(num_pages, page // block, 8, dtype=torch.uint8, device="cuda")
    table = torch.full((B, max_pages), -1, dtype=i32, device="cuda")
    held, free = torch.zeros(B, dtype=i32, device="cuda"), torch.arange(num_pages, dtype=i32, device="cuda")
    count = torch.full((1,), num_pages, dtype=i32, device="cuda")
    lens, cu = torch.full((B,), 60, dtype=i32, device="cuda"), torch.arange(B + 1, dtype=i32, device="cuda")
    rows = torch.zeros(B, 576, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(B, dtype=torch.int64, device="cuda")
    g = mla.default_splits(1)
    bufs = dict(workspace=torch.empty(mla.workspace_bytes(B, 1, H, g), dtype=torch.uint8, device="cuda"))

    def step():
        mla.update_pages(table, held, lens, free, count, page_size=page, cu=cu, slots=slots, err_word=err)
        mla.write_kv(rows, codes, table, lens, cu, fp8_scales=entries, err_word=err)
        return mla.decode_step(c.q_nope, c.q_rope, c.w_uk, c.w_uv, codes, table, lens, n_q=1, num_splits=g, bufs=bufs,
                               fp8_scales=entries, err_word=err)

    # a first write fills the contexts (and loads the modules)
    prompt = (torch.randn(60 * B, 576, device="cuda")).to(torch.bfloat16)
    long = torch.arange(0, 60 * B + 1, 60, dtype=i32, device="cuda")
    mla.update_pages(table, held, lens, free, count, page_size=page, err_word=err)
    mla.write_kv(prompt, codes, table, lens, long, fp8_scales=entries, err_word=err)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = step()
    for k in range(9):
        lens += 1
        rows.copy_(torch.randn(B, 576, device="cuda") * 2.0 ** (k % 5))
        c.q_nope.normal_()
        graph.replay()
        got = r["out"].clone()
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and held.tolist() == [1 + (lens[0].item() > 64)] * B
        flat = torch.from_numpy(blk.values(codes.cpu().numpy(), entries.cpu().numpy())).cuda().to(torch.bfloat16)
        want = mla.decode_step(c.q_nope, c.q_rope, c.w_uk, c.w_uv, codes, table, lens, n_q=1, num_splits=g,
                               fp8_scales=entries)
        assert torch.equal(bits(got), bits(want["out"]))
        d = (flat.view(-1, 576)[slots].float() - rows.float()).abs()
        assert (d <= 2.0 ** -4 * rows.float().abs() + 2.0 ** -10 * 2.0 ** -6 * 16).all()  # powers <= 2^-2 here


def test_far_pages(mla, err):
    """Rows past 2^32 bytes of codes: written, read, decoded and attended there."""
    import torch
    page, block, num_pages = 128, 64, 62000  # 4.57 GB of codes
    codes = torch.zeros(num_pages, page, 576, dtype=torch.uint8, device="cuda")
    entries = torch.zeros(num_pages, page // block, 8, dtype=torch.uint8, device="cuda")
    c = Blocks([200], [200], H=16, page=page, block=block, seed=1, spare=2)
    c.table[0, :2] = torch.tensor([61999, 58255], dtype=torch.int32)
    near = c.host_table[0][:2]
    rows = draw_rows(c, 4, 0.5)
    mla.write_kv(rows, codes, c.table, c.seq_lens, c.cu, fp8_scales=entries, err_word=err)
    c.table[0, :2] = torch.tensor(near, dtype=torch.int32)
    mla.write_kv(rows, *c.paged8(), fp8_scales=c.entries, err_word=err)
    far = torch.tensor([61999, 58255], device="cuda")
    assert torch.equal(codes[far][0], c.codes[near[0]]) and torch.equal(codes[far][1, :72], c.codes[near[1], :72])
    assert torch.equal(entries[far], c.entries[torch.tensor(near, device="cuda")])
    for form in ("expanded", "absorbed"):
        res = []
        for k, e, t in ((codes, entries, far), (c.codes, c.entries, torch.tensor(near, device="cuda"))):
            c.table[0, :2] = t.to(torch.int32)
            res.append(mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, k, c.table, c.seq_lens, c.cu,
                                        max_tokens=200, fp8_scales=e, form=form, err_word=err))
            res.append(mla.read_kv(k, c.table, c.seq_lens, c.cu, n_rows=200, fp8_scales=e, err_word=err))
        torch.cuda.synchronize()
        assert torch.equal(bits(res[0]), bits(res[2])) and torch.equal(bits(res[1]), bits(res[3]))
    assert int(err.item()) == 0


def test_on_another_stream(mla, err):
    import torch
    c = Blocks([9, 60], [100, 60], H=8, seed=2)
    rows = draw_rows(c, 3)
    want = c.codes.clone(), c.entries.clone()
    mla.write_kv(rows, want[0], c.table, c.seq_lens, c.cu, fp8_scales=want[1])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    mla.write_kv(rows, *c.paged8(), fp8_scales=c.entries, err_word=err, stream=s)
    a = mla.read_kv(*c.paged8(), n_rows=69, fp8_scales=c.entries, stream=s)
    args = (c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged8())
    b = mla.attend_chunk(*args, max_tokens=160, fp8_scales=c.entries, stream=s)
    s.synchronize()
    assert torch.equal(c.codes, want[0]) and torch.equal(c.entries, want[1]) and int(err.item()) == 0
    assert torch.equal(bits(a), bits(mla.read_kv(*c.paged8(), n_rows=69, fp8_scales=c.entries)))
    assert torch.equal(bits(b), bits(mla.attend_chunk(*args, max_tokens=160, fp8_scales=c.entries)))


def test_python_checks(mla):
    import torch
    c = Blocks([9], [100], H=2, seed=2)
    rows = draw_rows(c, 3)
    with pytest.raises(ValueError, match="block scales"):
        mla.write_kv(rows, *c.paged8(), fp8_scales=torch.ones(576, device="cuda"))
    with pytest.raises(ValueError, match="scales"):
        mla.write_kv(rows, *c.paged(), fp8_scales=c.entries)  # a bf16 cache
    with pytest.raises(ValueError, match="rows"):
        mla.write_kv(rows[:, :512], *c.paged8(), fp8_scales=c.entries)
    with pytest.raises(ValueError, match="fp8_scales"):
        mla.read_kv(*c.paged8(), n_rows=9, fp8_scales=c.entries[:1])
    with pytest.raises(ValueError, match="on cpu"):
        mla.read_kv(*c.paged8(), n_rows=9, fp8_scales=c.entries.cpu())
    step = (c.q_nope[:1], c.q_rope[:1], c.w_uk, c.w_uv, c.codes, c.table, c.seq_lens)
    for k, bad in ((0, c.q_nope[:2]), (1, c.q_rope[:1].float()), (2, c.w_uk[:1]), (3, c.w_uv.transpose(0, 1)),
                   (5, c.table[:, ::2]), (6, c.seq_lens.long())):
        with pytest.raises(ValueError):
            mla.decode_step(*step[:k], bad, *step[k + 1:], n_q=1, fp8_scales=c.entries)
    with pytest.raises(ValueError, match="q_abs"):
        mla.decode_step(*step, n_q=1, fp8_scales=c.entries, bufs=dict(q_abs=mla.absorb_q(*step[:3])))
    with pytest.raises(mla.MlaError, match="WORKSPACE"):
        mla.decode_step(*step, n_q=1, fp8_scales=c.entries, bufs=dict(workspace=c.codes[0]))
    with pytest.raises(ValueError, match="rows of 2 heads"):  # nine tokens' queries for one sequence
        mla.decode_paged_fp8(mla.absorb_q(c.q_nope, c.q_rope, c.w_uk), c.codes, c.entries, c.table, c.seq_lens, n_q=1)
    with pytest.raises(ValueError, match="q_abs"):
        mla.decode_paged_fp8(mla.absorb_q(*step[:3]).float(), c.codes, c.entries, c.table, c.seq_lens, n_q=1)
    with pytest.raises(ValueError, match="seq_lens"):
        mla.decode_paged_fp8(mla.absorb_q(*step[:3]), c.codes, c.entries, c.table, c.seq_lens.long(), n_q=1)
    with pytest.raises(ValueError, match="shape"):
        q = mla.absorb_q(c.q_nope[:1], c.q_rope[:1], c.w_uk)
        mla.decode_paged_fp8(q, c.codes, c.entries[1:], c.table, c.seq_lens, n_q=1)
