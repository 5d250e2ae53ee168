"""A decode's split plan is computed while the kernels before it still run, and written to the workspace only
after they have finished: the workspace may be one that an earlier decode or merge still uses, or memory that
a call still reads its rows, its cache or its own workspace from (an allocator hands such memory on as soon as its
owner has given it back, in the order of the stream). Each call is compared bit for bit with the same run alone."""
import numpy as np
import pytest

from tests.helpers import plan_mirror
from tests.test_gpu_blocks import Blocks, bits
from tests.test_gpu_parity import plan_arrays

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    import mla_latent_kv_paged_gb300 as m
    m.build()
    return m


LENGTHS = {"warp": ([4096] * 8, [64, 5000, 1, 700, 3000, 130, 2000, 900]),
           "block": ([700] * 50, [1 + (977 * b) % 1900 for b in range(50)])}


@pytest.mark.parametrize("kind", ["bf16", "blocks"])
@pytest.mark.parametrize("lens", LENGTHS.values(), ids=LENGTHS.keys())
def test_decode_and_merge_in_turn_on_one_workspace(mla, lens, kind):
    """decode_paged, combine, decode_paged on other lengths: the merge lets the next plan start while the decode
    before it still runs."""
    import torch
    H, B, G = 128, len(lens[0]), 60
    cs = [Blocks([1] * B, v, H=H, seed=3 + k) for k, v in enumerate(lens)]
    qs = [mla.absorb_q(c.q_nope, c.q_rope, c.w_uk) for c in cs]
    need = mla.workspace_bytes(B, 1, H, G)

    def step(k, ws):
        c = cs[k]
        if kind == "bf16":
            mla.decode_paged(qs[k], c.cache, c.table, c.seq_lens, n_q=1, num_splits=G, workspace=ws)
        else:
            mla.decode_paged_fp8(qs[k], c.codes, c.entries, c.table, c.seq_lens, n_q=1, num_splits=G, workspace=ws)
        return mla.combine(ws, B=B, n_q=1, H=H, num_splits=G)

    want = []
    for k in range(2):
        want.append(step(k, torch.zeros(need, dtype=torch.uint8, device="cuda")))
        torch.cuda.synchronize()
    one = torch.zeros(need, dtype=torch.uint8, device="cuda")
    got = [(i % 2, step(i % 2, one)) for i in range(8)]
    torch.cuda.synchronize()
    for k, pair in got:
        assert all(torch.equal(bits(x), bits(y)) for x, y in zip(pair, want[k]))


def plan_into(mla, memory, B=32):
    """A plan of B sequences whose workspace starts at byte ``memory``'s."""
    import torch
    lens = torch.full((B,), 4096, dtype=torch.int32, device="cuda")
    need = mla.workspace_bytes(B, 1, 1, 76)
    assert memory.numel() >= need and memory.dtype == torch.uint8
    return lambda: mla.decode_plan(lens, n_q=1, H=1, max_pages=64, num_pages=2048, num_splits=76, workspace=memory)


@pytest.mark.parametrize("where", [0.0, 0.5, 0.9])
def test_plan_over_rows_being_written_and_read(mla, where):
    """write_kv's rows, append_chunk's own workspace and the cache that read_kv reads become the next plan's
    workspace: what the calls give is as without it."""
    import torch
    new = [9000, 7000, 4000]
    need = [-(-n // 64) for n in new]
    table = torch.full((3, max(need)), -1, dtype=torch.int32, device="cuda")
    order, at = torch.randperm(sum(need), device="cuda").int(), 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, cu, T = i(new), i([0] + np.cumsum(new).tolist()), sum(new)
    g = torch.Generator(device="cuda").manual_seed(2)
    rows = torch.randn(T, 576, generator=g, device="cuda").to(torch.bfloat16)
    codes = lambda: (torch.zeros(sum(need), 64, 576, dtype=torch.uint8, device="cuda"),  # noqa: E731
                     torch.zeros(sum(need), 2, 8, dtype=torch.uint8, device="cuda"))

    def spot(t):  # a place of t's memory for a workspace
        flat = t.view(torch.uint8).view(-1)
        return flat[int(flat.numel() * where) // 256 * 256:]

    want, want_e = codes()
    mla.write_kv(rows, want, table, lens, cu, fp8_scales=want_e)
    back = mla.read_kv(want, table, lens, cu, n_rows=T, fp8_scales=want_e)
    h = torch.randn(T, 64, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(576, 64, generator=g, device="cuda").to(torch.bfloat16)
    appended, appended_e = codes()
    ws = mla.append_chunk(h, w, appended, table, lens, cu, fp8_scales=appended_e)
    torch.cuda.synchronize()
    for _ in range(5):
        used = rows.clone()
        plan = plan_into(mla, spot(used))
        got, got_e = codes()
        torch.cuda.synchronize()
        mla.write_kv(used, got, table, lens, cu, fp8_scales=got_e)
        plan()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(got_e, want_e)

        plan = plan_into(mla, spot(ws))
        got, got_e = codes()
        torch.cuda.synchronize()
        mla.append_chunk(h, w, got, table, lens, cu, fp8_scales=got_e, workspace=ws)
        plan()
        torch.cuda.synchronize()
        assert torch.equal(got, appended) and torch.equal(got_e, appended_e)

        used = want.clone()
        plan = plan_into(mla, spot(used))
        torch.cuda.synchronize()
        got = mla.read_kv(used, table, lens, cu, n_rows=T, fp8_scales=want_e)
        plan()
        torch.cuda.synchronize()
        assert torch.equal(bits(got), bits(back))


def test_steps_that_allocate_for_themselves(mla):
    """append_chunk and write_kv whose rows and workspaces nobody keeps, each followed by a decode step without
    buffers of its own."""
    import torch
    c = Blocks([5000, 3000], [5000, 3000], H=16, seed=5)
    g = torch.Generator(device="cuda").manual_seed(7)
    rows = torch.randn(8000, 576, generator=g, device="cuda").to(torch.bfloat16)
    h = torch.randn(8000, 128, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(576, 128, generator=g, device="cuda") / 11).to(torch.bfloat16)
    q = [t[:2].contiguous() for t in (c.q_nope, c.q_rope)]

    def fresh():
        return torch.zeros_like(c.codes), torch.zeros_like(c.entries)

    def step(codes, entries):
        return mla.decode_step(*q, c.w_uk, c.w_uv, codes, c.table, c.seq_lens, n_q=1, fp8_scales=entries)

    def run(sync):
        res = []
        for write in (lambda k: mla.write_kv(torch.cat([rows[:, :512], rows[:, 512:]], 1), k[0], c.table, c.seq_lens,
                                             c.cu, fp8_scales=k[1]),
                      lambda k: mla.append_chunk(h * 1, w, k[0], c.table, c.seq_lens, c.cu, fp8_scales=k[1])):
            k = fresh()
            write(k)
            if sync:
                torch.cuda.synchronize()
            r = step(*k)
            res += [*k, bits(r["u"]), bits(r["lse"]), bits(r["out"])]
        torch.cuda.synchronize()
        return res

    want = run(True)
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(run(False), want))


@pytest.mark.parametrize("lens,G", [([6400, 1, 700000], 11000), ([300 + 97 * b for b in range(60)], 11000),
                                    ([65 * b + 1 for b in range(4096)], 76)])
def test_large_plans(mla, lens, G):
    """Plans that do not fit into shared memory are written in place after the wait; the largest batch fits."""
    import torch
    B, max_pages = len(lens), -(-max(lens) // 64)
    ws, _ = mla.decode_plan(torch.tensor(lens, dtype=torch.int32, device="cuda"), n_q=1, H=1, max_pages=max_pages,
                            num_pages=1 << 20, num_splits=G)
    torch.cuda.synchronize()
    pl, host = plan_mirror(lens, 1, max_pages, G), ws.cpu().numpy()
    offs, _ = plan_arrays(host, B, G)
    i32 = lambda k, n: host[offs[k]:offs[k] + 4 * n].view(np.int32)  # noqa: E731
    n = len(pl["items"])
    assert i32(0, 3).tolist() == [n, pl["Ge"], pl["total"]] and np.array_equal(i32(1, G + 1), pl["range_item"])
    assert np.array_equal(i32(2, B + 1), pl["seq_item"]) and i32(3, B).tolist() == lens
    assert all(np.array_equal(i32(4 + k, n), pl["items"][:, k]) for k in range(3))
