"""The bounded waits of the chunk calls' MMA kernels give up, report it and leave the context
usable (GPU only).

As for the decode kernel (tests/test_gpu_wait_timeout.py): the test build leaves out some of
a kernel's loads and shortens the limit to about a millisecond. The waits on them run out,
also in the CTA of a pair that does not issue and in warps that meet at named barriers; the
call returns with the error recorded, and the next one, in the same context, is right."""
import pytest

from tests import chunk_reference as ref

pytestmark = pytest.mark.gpu

TIMEOUT = 5
APPEND, EXPAND, ATTEND = 0, 1, 2


@pytest.fixture()
def dbg(monkeypatch):
    """The module, its calls made to the test build."""
    import mla_latent_kv_paged_gb300 as mla
    lib = mla.debug_lib()
    monkeypatch.setattr(mla, "lib", lambda: lib)
    assert lib.mla_debug_reset() == 0
    yield mla, lib
    assert lib.mla_debug_reset() == 0


def gives_up(lib, kernel, what, call, err):
    import torch
    assert lib.mla_debug_set_wait_limit(2_000_000) == 0  # about 1 ms of SM cycles
    assert lib.mla_debug_set_skip_loads(kernel, what) == 0
    call()
    torch.cuda.synchronize()  # returns: every wait ended by its limit
    assert int(err.item()) == TIMEOUT
    assert lib.mla_debug_reset() == 0
    err.zero_()


@pytest.mark.parametrize("what", [1, 2])
@pytest.mark.parametrize("d_model,fp8", [(64, False), (512, True), (2048, False)])
def test_append_gives_up_then_recovers(dbg, what, d_model, fp8):
    import torch
    mla, lib = dbg
    c = ref.Chunk([300, 5], [400, 90], H=1, fp8=fp8, seed=110)
    g = torch.Generator(device="cuda").manual_seed(111)
    h = torch.randn(c.T, d_model, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(576, d_model, generator=g, device="cuda") * d_model ** -0.5).to(torch.bfloat16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = c.cache.clone()
    rows, want, slack = ref.append(c, h, w)
    other = torch.ones(c.num_pages * c.page, dtype=torch.bool, device="cuda")
    other[rows] = False

    def call():
        mla.append_chunk(h, w, *c.paged(), fp8_scales=c.scales, err_word=err)

    gives_up(lib, APPEND, what, call, err)
    raw = (lambda t: t) if fp8 else (lambda t: t.view(torch.int16))
    assert torch.equal(raw(c.cache).view(-1, 576)[other], raw(before).view(-1, 576)[other])
    call()
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    got = c.cache.view(-1, 576)[rows]
    if fp8:
        s = c.scales.double()
        got, want, slack = got.view(torch.float8_e4m3fn).double(), (want / s).clamp(-448, 448), slack / s
        assert ((got - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -10 + 1.1 * slack).all()
    else:
        assert ((got.double() - want).abs() <= ref.U_BF16 * want.abs() + 1.1 * slack).all()


@pytest.mark.parametrize("kernel,what", [(EXPAND, 1), (EXPAND, 2), (EXPAND, 3), (ATTEND, 1), (ATTEND, 2), (ATTEND, 3)])
@pytest.mark.parametrize("new,lens,H", [([5], [4000], 1), ([600, 3, 130], [900, 2500, 130], 40)])
def test_attend_gives_up_then_recovers(dbg, kernel, what, new, lens, H):
    import torch
    mla, lib = dbg
    c = ref.Chunk(new, lens, H=H, seed=112, pad_rows=2)
    want, _, bound = ref.attend(c)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    room = torch.full((c.T + 4, H, 128), 3.0, dtype=torch.bfloat16, device="cuda")

    def call():
        mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=sum(lens), form="expanded",
                         out=room[:c.T], err_word=err)

    gives_up(lib, kernel, what, call, err)
    assert (room[c.total:] == 3.0).all()
    call()
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert ((room[:c.total].double() - want).abs() <= bound["expanded"]).all()
    assert (room[c.total:] == 3.0).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_absorbed_gives_up_then_recovers(dbg, fp8):
    import torch
    mla, lib = dbg
    c = ref.Chunk([4, 30], [400, 200], H=5, fp8=fp8, seed=113, pad_rows=2)
    want, _, bound = ref.attend(c)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        return mla.attend_chunk(c.q_nope, c.q_rope, c.w_uk, c.w_uv, *c.paged(), max_tokens=600, fp8_scales=c.scales,
                                form="absorbed", err_word=err)

    assert lib.mla_debug_set_skip_producer(1) == 0
    gives_up(lib, APPEND, 0, call, err)
    got = call()
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert ((got[:c.total].double() - want).abs() <= bound["absorbed"]).all()
