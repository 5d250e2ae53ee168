"""CapturedStep keeps the tensors that its graphs read."""
import pytest

from tests.test_gpu_blocks import Blocks, bits, decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    import mla_latent_kv_paged_gb300 as m
    m.build()
    return m


@pytest.mark.parametrize("kind", ["bf16", "blocks"])
@pytest.mark.parametrize("host_io", [False, True])
def test_captured_step_outlives_its_callers_references(mla, kind, host_io):
    """The caller's tensors go out of scope and others of their sizes are allocated: replays read what they did."""
    import weakref

    import torch
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = Blocks([1, 1], [700, 300], H=16, block=32, seed=8)
    cache = c.cache if kind == "bf16" else c.codes
    given = [t.clone() for t in (c.w_uk, c.w_uv, cache, c.table, c.seq_lens, c.entries)]
    sizes = [(t.shape, t.dtype) for t in given]
    step = mla.CapturedStep(*given[:5], n_q=1, fp8_scales=None if kind == "bf16" else given[5], err_word=err,
                            host_io=host_io)
    torch.cuda.synchronize()
    alive = [weakref.ref(t) for t in given[:5 if kind == "bf16" else 6]]
    del given
    assert all(r() is not None for r in alive)
    other = [torch.full(shape, 1, dtype=dtype, device="cuda") for shape, dtype in sizes for _ in range(3)]
    want = decode(mla, c, *((c.cache, None) if kind == "bf16" else (c.codes, c.entries)), 1)
    got = step(c.q_nope, c.q_rope)
    torch.cuda.synchronize()
    assert all(torch.equal(bits(got[k]), bits(want[k])) for k in ("u", "lse", "out"))
    if host_io:
        step.host["q_nope"].copy_(c.q_nope)
        step.host["q_rope"].copy_(c.q_rope)
        torch.cuda.synchronize()
        step.replay_host()
        torch.cuda.synchronize()
        assert all(torch.equal(bits(step.host[k].cuda()), bits(want[k])) for k in ("lse", "out"))
    assert int(err.item()) == 0 and len(other) == 18
