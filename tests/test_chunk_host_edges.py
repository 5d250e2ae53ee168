"""The limits of the chunk entry points, both sides of each, on the host: a call within them
goes on to the next check (a workspace one byte short, a device), one beyond is refused.
Nothing is launched."""
import pytest

import mla_latent_kv_paged_gb300 as mla

P = 1 << 20  # a 16-byte aligned address that is never dereferenced
SHAPE, SMALL = 2, 3


@pytest.fixture(scope="module")
def lib():
    mla.build()
    return mla.lib()


def append(lib, wsb, T=9, d=512, page=64, maxp=4):
    return lib.mla_append_chunk(P, P, P, None, P, P, P, 2, T, d, 8, page, maxp, 1e4, P, wsb, None, None)


def attend(lib, wsb, B=2, T=300, H=16, page=64, maxp=8, max_tokens=1000, form=1):
    return lib.mla_attend_chunk(P, P, P, P, P, None, P, P, P, B, T, H, 8, page, maxp, max_tokens, 0.07, form, P, None, P,
                                wsb, None, None)


def test_contexts_and_rows_of_up_to_2_to_the_30(lib):
    ws = lib.mla_append_chunk_workspace_bytes(9, 512)
    for page in (64, 128):
        most = (1 << 30) // page
        assert append(lib, ws - 1, page=page, maxp=most) == SMALL
        assert append(lib, ws - 1, page=page, maxp=most + 1) == SHAPE
        need = lib.mla_attend_chunk_workspace_bytes(2, 300, 16, 1000, 1)
        assert attend(lib, need - 1, page=page, maxp=most) == SMALL
        assert attend(lib, need - 1, page=page, maxp=most + 1) == SHAPE
    assert lib.mla_read_kv(P, None, P, P, None, P, P, 2, (1 << 30) + 1, 8, 64, 4, None, None) == SHAPE
    assert lib.mla_attend_chunk_workspace_bytes(2, 300, 16, (1 << 30) + 1, 1) == 0
    need = lib.mla_attend_chunk_workspace_bytes(2, 300, 16, 1 << 30, 1)
    assert need > (1 << 30) * 1152
    assert attend(lib, need - 1, max_tokens=1 << 30) == SMALL
    assert attend(lib, need - 1, max_tokens=(1 << 30) + 1) == SHAPE


def test_absorbed_rows_whose_tiles_pass_32_bits_are_refused(lib):
    """4096 rows that may each see 2^25 tokens are 2^31 tiles of 64 for the decode plan."""
    for page, most in ((64, (1 << 19) - 1), (128, (1 << 18) - 1)):
        assert attend(lib, 1, T=4096, page=page, maxp=most, form=2) != SHAPE
        assert attend(lib, 1, T=4096, page=page, maxp=most + 1, form=2) == SHAPE
        assert attend(lib, 1, T=4095, page=page, maxp=most + 1, form=2) != SHAPE
