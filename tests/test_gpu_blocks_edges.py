"""The decode and the absorbed attention on a block-scaled cache where their fp16 operands end: weights far below
the largest, values below fp16's normal range and above it, contexts that hold a NaN."""
import numpy as np
import pytest

from tests import chunk_reference as ref
from tests.test_gpu_blocks import Blocks, attend, bits, check_decode, decode

pytestmark = pytest.mark.gpu

RANGE = 7


@pytest.fixture(scope="module")
def mla():
    import mla_latent_kv_paged_gb300 as m
    m.build()
    return m


@pytest.fixture()
def err():
    import torch
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def e4m3(codes):
    import torch
    return codes.view(torch.float8_e4m3fn).double()


@pytest.mark.parametrize("splits", [1, 3])
def test_many_light_tokens_beside_a_heavy_one(mla, err, splits):
    """One token of score 0 and 131072 behind it of 2^-d each: together they hold up to an eighth of the sum, and a
    sink keeps neither more nor less than its share. All values are of one sign.

    A weight is held in fp16, 2^7 times its size, so off by 2^-11 of itself or by 2^-25 / 2^7 at most; ex2 and the
    scores (whose sums here are single products) by 2^-15. The L products of a value are added in fp32, each addend
    cut below 2^-24 of the sum: L 2^-24 of the absolute sum, which is a tight bound where the heavy token's value
    is zero (columns 128 to 191) and a loose one elsewhere. The partial is rounded to fp16, the merged u to bf16. The
    sum of the weights grows by one tile's in every second of the L / 64 tiles, each time rounded by 2^-24."""
    import torch
    d = [20.0, 24.5, 25.5, 27.25, 30.0, 31.5, 33.0, 60.0]
    H, L, dev = len(d), 131073, "cuda"
    # page 0: light tokens, page 1: the heavy one and light ones behind it, page 2: a light one
    g = torch.Generator(device=dev).manual_seed(1)
    codes = torch.randint(0x30, 0x40, (3, 64, 576), dtype=torch.uint8, generator=g, device=dev)  # 0.5 .. 1.875
    codes[..., :64] = 0x38          # 1 in every token
    codes[..., 64:128] = 0x40       # 2 in the light tokens, 1 in the heavy one
    codes[1, 0, 64:128] = 0x38
    codes[..., 128:192] = 0x38      # 1 in the light tokens, 0 in the heavy one
    codes[1, 0, 128:192] = 0
    codes[..., 512:] = 0
    codes[..., 575] = 0xB8          # the key: -1 in the light tokens
    codes[1, 0, 575] = 0
    entries = torch.full((3, 2, 8), 127, dtype=torch.uint8, device=dev)
    table = torch.zeros(1, -(-L // 64), dtype=torch.int32, device=dev)
    table[0, 0], table[0, -1] = 1, 2
    q = torch.zeros(1, H, 576, dtype=torch.float16, device=dev)
    q[0, :, 575] = torch.tensor(d, device=dev)
    lens = torch.tensor([L], dtype=torch.int32, device=dev)
    scale = float(np.log(2.0))
    ws, g = mla.decode_paged_fp8(q, codes, entries, table, lens, n_q=1, num_splits=splits, softmax_scale=scale,
                                 err_word=err)
    u, lse = mla.combine(ws, B=1, n_q=1, H=H, num_splits=g)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    rows = e4m3(codes).view(-1, 576)
    at = (table[0].long()[:, None] * 64 + torch.arange(64, device=dev)).view(-1)[:L]
    lat = rows[at, :512]
    w = torch.exp2(q[0, :, 575].double()[:, None] * rows[at, 575][None])
    total = w.sum(-1, keepdim=True)
    want = w @ lat / total
    # splits: a range without the heavy token has a reference of its own, 2^-d
    held = torch.full_like(w, 2.0 ** -32)
    bound = (w @ lat * (ref.U_F16 + 2.0 ** -15 + L * ref.U_F32) + held @ lat) / total
    bound += 1.01 * (ref.U_F16 + ref.U_BF16) * want
    assert ((u[0].double() - want).abs() <= bound).all()
    assert ((lse[0].double() - total[:, 0].log()).abs()
            <= 2.0 ** -15 + L / 128 * ref.U_F32 + 2.0 ** -20 * total[:, 0].log().abs()).all()


@pytest.mark.parametrize("block", [16, 64])
def test_values_below_fp16_are_rounded_once(mla, err, block):
    """One attended token a sequence, of powers from 2^-16 down: u is the value rounded once to fp16 (2^-24's
    multiples there, ties to even), and that to bf16."""
    import torch
    powers = list(range(-36, -15))
    B, dev = len(powers), "cuda"
    g = torch.Generator(device=dev).manual_seed(block)
    codes = torch.randint(0, 255, (B, 64, 576), dtype=torch.uint8, generator=g, device=dev)
    codes[(codes & 0x7F) == 0x7F] = 0x09
    codes[:, 0, :508] = torch.arange(254, dtype=torch.uint8, device=dev).repeat(2)  # all but 0x7F, 0xFE and 0xFF
    codes[:, 0, 127] = codes[:, 0, 381] = 0x7E
    entries = torch.zeros(B, 64 // block, 8, dtype=torch.uint8, device=dev)
    entries[:, :, :5] = torch.tensor([127 + p for p in powers], dtype=torch.uint8, device=dev)[:, None, None]
    q = torch.randn(B, 3, 576, generator=g, device=dev).to(torch.float16)
    ws, splits = mla.decode_paged_fp8(q, codes, entries, torch.arange(B, dtype=torch.int32, device=dev)[:, None],
                                      torch.ones(B, dtype=torch.int32, device=dev), n_q=1, err_word=err)
    u, _ = mla.combine(ws, B=B, n_q=1, H=3, num_splits=splits)
    torch.cuda.synchronize()
    v = e4m3(codes[:, 0, :512]) * torch.exp2(torch.tensor(powers, dtype=torch.float64, device=dev))[:, None]
    want = (v * 2.0 ** 24).round() * 2.0 ** -24  # (half to even)
    want = torch.where(v.abs() < 2.0 ** -14, want, v.to(torch.float16).double()).to(torch.bfloat16)
    assert int(err.item()) == 0 and (u.float() == want.float()[:, None]).all()
    # (at 2^-25 the codes above 1, 0x39 .. 0x7E and 0xB9 .. 0xFD, are not zero: 139 of them, twice)
    assert (want[0] == 0).all() and (want[powers.index(-25), :508] != 0).sum() >= 2 * 139


@pytest.mark.parametrize("col", [77, 570])
@pytest.mark.parametrize("kind", ["blocks", "bf16"])
def test_a_nan_in_contexts_of_every_length(mla, err, kind, col):
    """A latent or a positional NaN gives NaN to all of its sequence's results, whether one CTA pair has the whole
    context or several share it, and to no other sequence's."""
    import torch
    c = Blocks([1] * 6, [1, 40, 64, 100, 1000, 70], H=16, block=32, seed=8)
    for b in range(5):
        row = c.rows(b)[c.lens[b] // 2]
        c.codes.view(-1, 576)[row, col] = 0xFF
        c.cache.view(-1, 576)[row, col] = float("nan")
    got = decode(mla, c, *((c.codes, c.entries) if kind == "blocks" else (c.cache, None)), 1, err)
    torch.cuda.synchronize()
    for k in ("u", "lse", "out"):
        assert torch.isnan(got[k][:5].float()).all() and torch.isfinite(got[k][5].float()).all(), k
    if kind == "blocks":
        check_decode(c, got, 1, skip=range(5))


def test_absorbed_attention_reports_values_outside_fp16(mla, err):
    """A value of the context of 65520 or more is reported, one behind it is not; the expanded form, which takes
    rows in bf16, has its own limits (the keys and values that it makes of them)."""
    import torch
    for at, entry, want in ((60, 127 + 8, RANGE), (60, 127 + 7, 0), (75, 127 + 20, 0)):
        c = Blocks([5], [70], H=16, block=16, seed=8)
        pool = c.rows(0)[at].item() if at < 70 else c.host_table[0][1] * 64 + at - 64
        rows = slice(pool // 16 * 16, pool // 16 * 16 + 16)
        c.codes.view(-1, 576)[rows, 256:384] = 0
        c.codes.view(-1, 576)[pool, 300] = 0x7E
        c.entries.view(-1, 8)[pool // 16, 2] = entry
        c.q_nope.zero_()  # (scores of ordinary size)
        c.w_uv.mul_(2.0 ** -6)
        err.zero_()
        attend(mla, c, c.codes, c.entries, "absorbed", err)
        torch.cuda.synchronize()
        assert int(err.item()) == want, (at, entry)


def test_small_values_in_every_reader(mla, err):
    """Latents of about 2^-20. Read back and the expanded attention take them as they are; the decode and the
    absorbed attention hold values, partials and (the attention) u to 2^-25, whatever their size, and so does the
    decode of a bf16 cache with its partials."""
    import torch
    c = Blocks([40, 3], [200, 130], H=8, block=16, seed=8, powers=(-20, -20), spread=0.0)
    c.codes, c.entries = c.codes.clone(), c.entries.clone()
    assert c.cache.nan_to_num().abs().max() < 2.0 ** -17
    back = mla.read_kv(c.codes, c.table, c.seq_lens, c.cu, n_rows=43, fp8_scales=c.entries, err_word=err)
    for b, n in enumerate(c.new):
        rows = back[sum(c.new[:b]):sum(c.new[:b]) + n]
        assert torch.equal(rows, c.cache.view(-1, 576)[c.rows(b, 0, n)])
    got = {form: attend(mla, c, c.codes, c.entries, form, err)[0].double() for form in ("expanded", "absorbed")}
    torch.cuda.synchronize()
    want, _, bounds = ref.attend(c)
    held = c.w_uv.double().abs().sum(-1)  # each latent of u off by 2^-25: [H, 128]
    keys = torch.expm1(torch.tensor(2 * ref.SCALE * 576 * 6 * ref.TINY_F16)).item() * want.abs().max()
    assert ((got["expanded"] - want).abs() <= bounds["expanded"] + keys).all()
    assert ((got["absorbed"] - want).abs() <= bounds["absorbed"] + 4 * ref.TINY_F16 * held + keys).all()
    # a step on either cache
    last = [sum(c.new[:b + 1]) - 1 for b in range(2)]
    c.q_nope, c.q_rope = c.q_nope[last].contiguous(), c.q_rope[last].contiguous()
    blocks = decode(mla, c, c.codes, c.entries, 1, err)
    plain = mla.decode_step(c.q_nope, c.q_rope, c.w_uk, c.w_uv, c.cache, c.table, c.seq_lens, n_q=1, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check_decode(c, blocks, 1)
    for b in range(2):
        x = c.values(b)
        z = (torch.einsum("hd,hdc->hc", c.q_nope[b].double(), c.w_uk.double()) @ x[:, :512].t()
             + c.q_rope[b].double() @ x[:, 512:].t()) * ref.SCALE
        u = torch.softmax(z, -1) @ x[:, :512]
        # (weights of nearly equal tokens; the query in bf16 or fp16 moves scores of 2^-17 by nothing)
        near = 2.0 ** -7 * x[:, :512].abs().amax(0)
        for r, parts in ((blocks, 2), (plain, 1)):
            assert ((r["u"][b].double() - u).abs() <= near + parts * ref.TINY_F16).all()
    assert bits(blocks["u"]).shape == bits(plain["u"]).shape


def test_decode_paged_refusals(mla, err):
    """decode_paged_fp8 with block scales checks what it passes on, as the calls beside it do."""
    import torch
    c = Blocks([1, 1], [70, 100], H=16, seed=8)
    q = mla.absorb_q(c.q_nope, c.q_rope, c.w_uk)
    good = dict(q_abs=q, cache8=c.codes, scales=c.entries, block_table=c.table, seq_lens=c.seq_lens, n_q=1,
                err_word=err)
    ws = torch.zeros(2 * mla.workspace_bytes(2, 1, 16, mla.default_splits(1)), dtype=torch.uint8, device="cuda")
    for name, bad in (("cache8", c.codes[..., :512].contiguous()), ("q_abs", q[..., :512].contiguous()),
                      ("q_abs", q.float()), ("q_abs", q[0, 0]), ("q_abs", q[:1].contiguous()),
                      ("block_table", c.table.long()), ("block_table", c.table[0]), ("seq_lens", c.seq_lens[:1]),
                      ("seq_lens", c.seq_lens.cpu()), ("err_word", err.long()), ("err_word", err.cpu()),
                      ("workspace", ws[::2]), ("workspace", ws.cpu()), ("scales", c.entries[:, :, :7].contiguous())):
        with pytest.raises(ValueError):
            mla.decode_paged_fp8(**{**good, name: bad})
    with pytest.raises(mla.MlaError, match="WORKSPACE_TOO_SMALL"):
        mla.decode_paged_fp8(**good, workspace=ws[:1024])
    side = torch.cuda.Stream()
    want = mla.combine(mla.decode_paged_fp8(**good)[0], B=2, n_q=1, H=16, num_splits=mla.default_splits(1))
    torch.cuda.synchronize()
    ws, g = mla.decode_paged_fp8(**good, stream=side)
    got = mla.combine(ws, B=2, n_q=1, H=16, num_splits=g, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(bits(x), bits(y)) for x, y in zip(got, want)) and int(err.item()) == 0


@pytest.mark.parametrize("kind", ["blocks", "bf16", "columns"])
def test_a_nan_in_the_last_draft_reaches_only_the_query_that_sees_it(mla, err, kind):
    """Two new tokens, the second with a NaN: the first one's results are, bit for bit, those without it, wherever
    the second lies in its tile."""
    import torch
    lens = [65, 64, 129, 200, 2, 1000, 128]
    c = Blocks([2] * len(lens), lens, H=16, block=16, seed=8)
    scales = torch.ones(576, device="cuda")
    cache = {"blocks": c.codes, "bf16": c.cache, "columns": c.codes}[kind]
    kw = {"blocks": c.entries, "bf16": None, "columns": scales}[kind]
    want = {k: v.clone() for k, v in decode(mla, c, cache, kw, 2, err).items() if k in ("u", "lse", "out")}
    rows = torch.stack([c.rows(b)[-1] for b in range(len(lens))])
    for col in (70, 300, 570):
        cache.view(-1, 576)[rows, col] = float("nan") if kind == "bf16" else 0x7F
    got = decode(mla, c, cache, kw, 2, err)
    torch.cuda.synchronize()
    for k in ("u", "lse", "out"):
        assert torch.equal(bits(got[k][::2]), bits(want[k][::2])), k
        assert torch.isfinite(want[k].float()).all() and torch.isnan(got[k][1::2].float()).all(), k
    assert int(err.item()) == 0
