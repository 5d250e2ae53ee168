"""Host-side checks of the chunk entry points: every refusal returns a status (or raises)
before any launch. No GPU is needed."""
import pytest

import mla_latent_kv_paged_gb300 as mla


@pytest.fixture(scope="module")
def lib():
    mla.build()
    return mla.lib()


P = 1 << 20  # a 16-byte aligned address that is never dereferenced


def test_append_chunk_refusals(lib):
    ws = lib.mla_append_chunk_workspace_bytes(9, 512)
    assert ws > 0
    for T, d in ((0, 512), (9, 0), (9, 100), (9, 65600), ((1 << 20) + 1, 512)):
        assert lib.mla_append_chunk_workspace_bytes(T, d) == 0

    def call(**kw):
        a = dict(h=P, w=P, cache=P, s=None, bt=P, sl=P, cu=P, B=2, T=9, d=512, pages=8, page=64, maxp=4, theta=1e4, ws=P,
                 wsb=ws)
        a.update(kw)
        return lib.mla_append_chunk(a["h"], a["w"], a["cache"], a["s"], a["bt"], a["sl"], a["cu"], a["B"], a["T"],
                                    a["d"], a["pages"], a["page"], a["maxp"], a["theta"], a["ws"], a["wsb"], None, None)

    for name in ("h", "w", "cache", "bt", "sl", "cu", "ws"):
        assert call(**{name: None}) == 1 and call(**{name: P + 4}) == 1, name
    assert call(s=P + 8) == 1
    assert call(B=0) == 1 and call(T=0) == 1 and call(pages=0) == 1 and call(maxp=0) == 1
    assert call(theta=1.0) == 1 and call(theta=float("nan")) == 1 and call(theta=float("inf")) == 1
    assert call(B=5000) == 2 and call(T=(1 << 20) + 1) == 2 and call(page=32) == 2 and call(d=96) == 2
    assert call(page=128, maxp=(1 << 23) + 1) == 2
    assert call(wsb=ws - 1) == 3


def test_read_kv_refusals(lib):
    def call(**kw):
        a = dict(cache=P, s=None, bt=P, sl=P, first=None, cu=P, rows=P, B=2, n=9, pages=8, page=64, maxp=4)
        a.update(kw)
        return lib.mla_read_kv(a["cache"], a["s"], a["bt"], a["sl"], a["first"], a["cu"], a["rows"], a["B"], a["n"],
                               a["pages"], a["page"], a["maxp"], None, None)

    for name in ("cache", "bt", "sl", "cu", "rows"):
        assert call(**{name: None}) == 1 and call(**{name: P + 4}) == 1, name
    assert call(first=P + 4) == 1 and call(s=P + 4) == 1
    assert call(B=0) == 1 and call(n=0) == 1 and call(pages=0) == 1 and call(maxp=0) == 1
    assert call(B=4097) == 2 and call(page=16) == 2 and call(page=64, maxp=(1 << 24) + 1) == 2


def test_attend_chunk_refusals(lib):
    ws = lib.mla_attend_chunk_workspace_bytes(2, 300, 16, 1000, 1)
    assert ws > 0
    for a in ((0, 300, 16, 1000, 1), (2, 0, 16, 1000, 1), (2, 300, 129, 1000, 1), (2, 300, 16, 0, 1),
              (2, 300, 16, 1 << 31, 1), (2, 300, 16, 1000, 3), (2, 300, 16, 1000, -1), (2, 5000, 16, 1000, 2)):
        assert lib.mla_attend_chunk_workspace_bytes(*a) == 0, a

    def call(**kw):
        a = dict(qn=P, qr=P, uk=P, uv=P, cache=P, s=None, bt=P, sl=P, cu=P, B=2, T=300, H=16, pages=8, page=64, maxp=8,
                 maxt=1000, scale=0.07, form=1, out=P, lse=None, ws=P, wsb=ws)
        a.update(kw)
        return lib.mla_attend_chunk(a["qn"], a["qr"], a["uk"], a["uv"], a["cache"], a["s"], a["bt"], a["sl"], a["cu"],
                                    a["B"], a["T"], a["H"], a["pages"], a["page"], a["maxp"], a["maxt"], a["scale"],
                                    a["form"], a["out"], a["lse"], a["ws"], a["wsb"], None, None)

    for name in ("qn", "qr", "uk", "uv", "cache", "bt", "sl", "cu", "out", "ws"):
        assert call(**{name: None}) == 1 and call(**{name: P + 4}) == 1, name
    assert call(s=P + 8) == 1 and call(lse=P + 2) == 1
    assert call(B=0) == 1 and call(T=0) == 1 and call(pages=0) == 1 and call(maxp=0) == 1 and call(maxt=0) == 1
    assert call(scale=0.0) == 1 and call(scale=-1.0) == 1 and call(scale=float("nan")) == 1
    assert call(scale=float("inf")) == 1
    assert call(form=3) == 1 and call(form=-1) == 1
    assert call(B=5000) == 2 and call(T=(1 << 20) + 1) == 2 and call(H=129) == 2 and call(H=0) == 2
    assert call(page=256) == 2 and call(maxt=(1 << 30) + 1) == 2
    assert call(T=5000, form=2) == 2
    assert call(wsb=ws - 1) == 3


def test_the_expanded_workspace_is_bounded_by_head_groups(lib):
    """All heads' keys and values while those fit 2 GiB, fewer at a time beyond."""
    size = lambda tokens: lib.mla_attend_chunk_workspace_bytes(1, 2048, 128, tokens, 1)  # noqa: E731
    assert size(16384) >= 128 * 16384 * 512
    assert size(1 << 20) < (2 << 30) + (1 << 20) * 1152 + (64 << 20)


def test_python_refusals():
    import torch
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA device"):
        mla.append_chunk(t(4, 512), t(576, 512), t(8, 64, 576), i(2, 4), i(2), i(3))
    with pytest.raises(ValueError, match="CUDA device"):
        mla.read_kv(t(8, 64, 576), i(2, 4), i(2), i(3), n_rows=4)
    with pytest.raises(ValueError, match="CUDA device"):
        mla.attend_chunk(t(4, 2, 128), t(4, 2, 64), t(2, 128, 512), t(2, 128, 512), t(8, 64, 576), i(2, 4), i(2), i(3),
                         max_tokens=9)
    with pytest.raises(ValueError, match="dtype"):
        mla._tensor("x", t(2, 3), torch.int32, (2, 3), -1)
    with pytest.raises(ValueError, match="shape"):
        mla._tensor("x", t(2, 3), torch.bfloat16, (2, 4), -1)
    with pytest.raises(ValueError, match="shape"):
        mla._tensor("x", t(2, 3), torch.bfloat16, (2, 3, 1), -1)
    with pytest.raises(ValueError, match="contiguous"):
        mla._tensor("x", t(3, 2).t(), torch.bfloat16, (2, 3), -1)
    with pytest.raises(ValueError, match="on cpu"):
        mla._tensor("x", t(2, 3), torch.bfloat16, (2, 3), 0)
    mla._tensor("x", t(2, 3), torch.bfloat16, (2, 3), -1)
