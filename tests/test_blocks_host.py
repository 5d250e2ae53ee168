"""Host-side checks of the block-scaled cache's and the page tables' entry points: every refusal
returns a status (or raises) before any launch. And the reference itself against torch's conversion.
No GPU is needed."""
import numpy as np
import pytest

import mla_latent_kv_paged_gb300 as mla
from tests import blocks_reference as ref


@pytest.fixture(scope="module")
def lib():
    mla.build()
    return mla.lib()


P = 1 << 20  # a 16-byte aligned address that is never dereferenced


def refusals(call, pointers):
    for name in pointers:
        assert call(**{name: None}) == 1 and call(**{name: P + 4}) == 1, name


def test_write_kv_refusals(lib):
    def call(**kw):
        a = dict(rows=P, cache=P, entries=P, block=32, bt=P, sl=P, cu=P, B=2, T=9, pages=8, page=64, maxp=4)
        a.update(kw)
        return lib.mla_write_kv(*a.values(), None, None)

    refusals(call, ("rows", "cache", "entries", "bt", "sl", "cu"))
    for block in (0, 1, 8, 24, 128, -16):
        assert call(block=block) == 2
    assert call(B=0) == 1 and call(T=0) == 1 and call(pages=0) == 1 and call(maxp=0) == 1
    assert call(B=4097) == 2 and call(T=(1 << 20) + 1) == 2 and call(page=32) == 2
    assert call(page=128, maxp=(1 << 23) + 1) == 2 and call(pages=1 << 25) == 2


def test_append_chunk_blocks_refusals(lib):
    ws = lib.mla_append_chunk_blocks_workspace_bytes(9, 512)
    assert ws == lib.mla_append_chunk_workspace_bytes(9, 512) + 9 * 1152
    assert lib.mla_append_chunk_blocks_workspace_bytes(0, 512) == 0
    assert lib.mla_append_chunk_blocks_workspace_bytes(9, 100) == 0

    def call(**kw):
        a = dict(h=P, w=P, cache=P, entries=P, block=64, bt=P, sl=P, cu=P, B=2, T=9, d=512, pages=8, page=64, maxp=4,
                 theta=1e4, ws=P, wsb=ws)
        a.update(kw)
        return lib.mla_append_chunk_blocks(*a.values(), None, None)

    refusals(call, ("h", "w", "cache", "entries", "bt", "sl", "cu", "ws"))
    assert call(block=48) == 2 and call(B=0) == 1 and call(T=0) == 1 and call(theta=1.0) == 1
    assert call(d=96) == 2 and call(page=32) == 2 and call(wsb=ws - 1) == 3


def test_read_kv_blocks_refusals(lib):
    def call(**kw):
        a = dict(cache=P, entries=P, block=16, bt=P, sl=P, first=None, cu=P, rows=P, B=2, n=9, pages=8, page=64, maxp=4)
        a.update(kw)
        return lib.mla_read_kv_blocks(*a.values(), None, None)

    refusals(call, ("cache", "entries", "bt", "sl", "cu", "rows"))
    assert call(first=P + 4) == 1 and call(block=17) == 2 and call(B=0) == 1 and call(n=0) == 1
    assert call(B=4097) == 2 and call(page=16) == 2


@pytest.mark.parametrize("planned", [False, True])
def test_decode_blocks_refusals(lib, planned):
    ws = lib.mla_decode_workspace_bytes(2, 1, 16, 4)

    def call(**kw):
        a = dict(q=P, f16=0, cache=P, entries=P, block=16, bt=P, sl=P, B=2, n_q=1, H=16, pages=8, page=64, maxp=4,
                 scale=0.07, splits=4, ws=P, wsb=ws)
        a.update(kw)
        if planned:
            a.pop("sl")
        fn = lib.mla_decode_paged_planned_blocks if planned else lib.mla_decode_paged_blocks
        return fn(*a.values(), None, None)

    refusals(call, ("q", "cache", "entries", "bt", "ws") + (() if planned else ("sl",)))
    assert call(block=0) == 2 and call(scale=0.0) == 1 and call(scale=float("nan")) == 1 and call(B=0) == 1
    assert call(n_q=3) == 2 and call(H=129) == 2 and call(page=32) == 2 and call(wsb=ws - 1) == 3


def test_decode_step_blocks_refusals(lib):
    """(out and lse come last among the checks: their kind of memory is asked of the runtime.)"""
    ws = lib.mla_decode_workspace_bytes(2, 1, 16, 4)

    def call(**kw):
        a = dict(qn=P, qr=P, uk=P, uv=P, cache=P, entries=P, block=16, bt=P, sl=P, B=2, n_q=1, H=16, pages=8, page=64,
                 maxp=4, scale=0.07, splits=4, qa=P, u=P, lse=None, out=P, ws=P, wsb=ws)
        a.update(kw)
        return lib.mla_decode_step_blocks(*a.values(), None, None)

    refusals(call, ("qn", "qr", "uk", "uv", "cache", "entries", "bt", "sl", "qa", "u", "out", "ws"))
    assert call(lse=P + 2) == 1 and call(block=8) == 2 and call(scale=0.0) == 1 and call(B=0) == 1
    assert call(n_q=3) == 2 and call(H=0) == 2 and call(page=96) == 2 and call(wsb=ws - 1) == 3 and call(splits=0) == 1


def test_attend_chunk_blocks_refusals(lib):
    ws = lib.mla_attend_chunk_workspace_bytes(2, 300, 16, 1000, 1)

    def call(**kw):
        a = dict(qn=P, qr=P, uk=P, uv=P, cache=P, entries=P, block=32, bt=P, sl=P, cu=P, B=2, T=300, H=16, pages=8,
                 page=64, maxp=8, maxt=1000, scale=0.07, form=1, out=P, lse=None, ws=P, wsb=ws)
        a.update(kw)
        return lib.mla_attend_chunk_blocks(*a.values(), None, None)

    refusals(call, ("qn", "qr", "uk", "uv", "cache", "entries", "bt", "sl", "cu", "out", "ws"))
    assert call(lse=P + 2) == 1 and call(block=128) == 2 and call(form=3) == 1 and call(scale=-1.0) == 1
    assert call(B=5000) == 2 and call(H=0) == 2 and call(T=5000, form=2) == 2 and call(wsb=ws - 1) == 3


def test_update_pages_refusals(lib):
    def call(**kw):
        a = dict(bt=P, held=P, sl=P, free=P, count=P, cu=P, slots=P, B=3, n=9, pages=8, page=64, maxp=4)
        a.update(kw)
        return lib.mla_update_pages(*a.values(), None, None)

    refusals(call, ("bt", "held", "sl", "free", "count", "cu", "slots"))
    assert call(B=0) == 1 and call(n=0) == 1 and call(n=-1) == 1 and call(pages=0) == 1 and call(maxp=0) == 1
    assert call(cu=None, slots=None, n=-1) == 1
    assert call(B=4097) == 2 and call(n=(1 << 20) + 1) == 2 and call(page=32) == 2
    assert call(maxp=(1 << 24) + 1) == 2 and call(pages=1 << 26) == 2


def test_python_refusals():
    import torch
    t = lambda *s, dtype=torch.uint8: torch.zeros(*s, dtype=dtype)  # noqa: E731
    i = lambda *s: t(*s, dtype=torch.int32)  # noqa: E731
    cache = t(8, 128, 576)
    for shape in ((8, 2), (8, 3, 8), (8, 0, 8), (8, 1, 8), (8, 16, 8), (576,)):
        with pytest.raises(ValueError, match="blocks of 16, 32 or 64"):
            mla._block_tokens(cache, t(*shape))
    with pytest.raises(ValueError, match="shape"):
        mla._block_tokens(cache, t(7, 2, 8))
    with pytest.raises(ValueError, match="shape"):
        mla._block_tokens(cache, t(8, 2, 5))
    with pytest.raises(ValueError, match="contiguous"):
        mla._block_tokens(cache, t(8, 8, 2).transpose(1, 2))
    assert [mla._block_tokens(cache, t(8, k, 8)) for k in (2, 4, 8)] == [64, 32, 16]
    assert mla._block_tokens(cache, t(576, dtype=torch.float32)) == 0 and mla._block_tokens(cache, None) == 0
    with pytest.raises(ValueError, match="CUDA device"):
        mla.write_kv(t(4, 576, dtype=torch.bfloat16), cache, i(2, 4), i(2), i(3), fp8_scales=t(8, 2, 8))
    with pytest.raises(ValueError, match="CUDA device"):
        mla.update_pages(i(2, 4), i(2), i(2), i(8), i(1))


def test_reference_codes_are_torchs():
    import torch
    g = torch.Generator().manual_seed(1)
    x = torch.cat([torch.randn(20000, generator=g) * torch.exp2(torch.randint(-12, 9, (20000,), generator=g).float()),
                   torch.tensor(ref._MID, dtype=torch.float32), -torch.tensor(ref._UP, dtype=torch.float32)])
    x = x[x.abs() <= 448]
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (ref.codes(x.numpy()) == want).all()
    assert np.array_equal(ref.VALUE, torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy(),
                          equal_nan=True)


@pytest.mark.parametrize("top,e", [(448.0, 0), (448.0001, 1), (447.9, 0), (224.0, -1), (1.0, -8), (1.76, -7),
                                   (1.75, -8), (0.0, -110), (2.0 ** -120, -110), (2.0 ** 126, 118)])
def test_reference_powers(top, e):
    assert ref.power(top) == e and (top <= 448 * 2.0 ** e) and (e == -110 or top > 448 * 2.0 ** (e - 1))


def test_reference_write_twice_is_write_once():
    """Writing the same rows again changes nothing; writing a run in two parts differs from writing it at
    once by at most the second rounding of the first part."""
    r = np.random.default_rng(2)
    rows = r.standard_normal((40, 576)) * np.exp2(r.integers(-2, 3, (40, 1)))
    one = [np.zeros((1, 64, 576), np.uint8), np.zeros((1, 2, 8), np.uint8)]
    ref.write(*one, rows, [[0]], [40], [40], 64, 32)
    again = [a.copy() for a in one]
    ref.write(*again, rows[30:], [[0]], [40], [10], 64, 32)
    assert all((a == b).all() for a, b in zip(one, again))
    two = [np.zeros((1, 64, 576), np.uint8), np.zeros((1, 2, 8), np.uint8)]
    ref.write(*two, rows[:20], [[0]], [20], [20], 64, 32)
    ref.write(*two, rows[20:], [[0]], [40], [20], 64, 32)
    assert (two[1] == one[1]).all()
    d = np.abs(ref.values(*two)[0, :40] - rows)
    step = np.exp2(one[1][0, :, :5].astype(float) - 127).max()
    assert (d <= 2 * (2.0 ** -4 * np.abs(rows) + 2.0 ** -10 * step)).all()
    assert np.abs(ref.values(*one)[0, 40:]).max() == 0


def test_reference_pages_go_back_and_forth():
    p = ref.Pages([[5, 1, -1, -1], [2, -1, -1, -1], [-1] * 4], [2, 1, 0], [7, 0, 3, 6, 4], 64)
    start = ([list(r) for r in p.table], list(p.held), list(p.free))
    slots = p.update([10, 130, 64], [0, 70, 64], 140)
    assert p.refused == [] and p.held == [1, 3, 1] and p.table[1] == [2, 1, 4, -1] and p.table[2][0] == 6
    assert slots[:5] == [2 * 64 + 60, 2 * 64 + 61, 2 * 64 + 62, 2 * 64 + 63, 64] and slots[134:] == [-1] * 6
    p.update([128, 64, 0])
    assert (p.table, p.held, p.free) == start
    # page 1 comes back and is the first to be taken, then 4 and 6: place 3 is page 6
    assert p.update([64, 64 * 4, 64 * 4], [0, 1, 1], 2) == [6 * 64 + 63, -1] and p.refused == [2]


@pytest.mark.parametrize("what,match", [
    (dict(cache8=(4, 64, 512)), "cache8: shape"), (dict(cache8=(4, 64, 640)), "cache8: shape"),
    (dict(cache8=(4, 64, 576)), "a CUDA device is needed"),
])
def test_decode_refuses_caches_of_another_width(what, match):
    """A row of another width would be read past the cache's end."""
    import torch
    z = lambda shape, dtype: torch.zeros(shape, dtype=dtype)  # noqa: E731
    with pytest.raises(ValueError, match=match):
        mla.decode_paged_fp8(z((2, 16, 576), torch.float16), z(what["cache8"], torch.uint8), z((4, 2, 8), torch.uint8),
                             z((2, 2), torch.int32), z((2,), torch.int32), n_q=1, num_splits=4)
