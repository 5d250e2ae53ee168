"""Cases of the operators around a latent cache held in 8 bits with block scales, for timing and
for comparison.

  pages   block tables and slot maps kept by the GPU: every sequence's pages brought to what its
          length needs, from and to a stack of free pages, and the pool row of each new token
  write   rows of new tokens quantised into their pages: e4m3 codes, and for each block of 16, 32 or
          64 tokens and group of 128 columns (the 64 positional columns are a group of their own) a
          power of two; a block that holds older tokens is requantised where its power grows
  read    rows of the sequences read back from those pages into one array, as bf16
  decode  a decode step over the cache for one or two new tokens of each sequence
  attend  attention of a ragged chunk of new tokens over the cache

``run`` computes each in its plain form (elementary torch operations in 32 bits) or, with ``own``
set, through the package's entry points. ``exact`` gives the same outputs in 64 bits.
"""
import math
import random

import torch

own = False

D_NOPE, D_R, D_C, D_V, D_ROW = 128, 64, 512, 128, 576
SCALE = 1.0 / math.sqrt(D_NOPE + D_R)
GROUPS = 5          # four of 128 latent columns, one of 64 positional ones; an 8-byte entry for each block
LEAST = 17          # the smallest power: 2^(17 - 127)
SPARE_ROWS = 3      # rows of a padded batch behind its last sequence


# ------------------------------------------------------------------ cases
def listed():
    return [
        # 32 running sequences between two decode steps: a token more each, a few finish, a few start
        dict(name="pages_serving_32", op="pages", B=32, ctx_hi=4096, prompt_hi=700, page=64, shape=1),
        # a full server: 2048 places, long prompts started where others finish
        dict(name="pages_prompts_2048", op="pages", B=2048, ctx_hi=16384, prompt_hi=4096, page=128, shape=2),
        # one new token for each of 128 running sequences
        dict(name="write_decode_128", op="write", B=128, new_lo=1, new_hi=1, old_lo=0, old_hi=4096, page=64, block=64,
             shape=3),
        # prompts and prompt pieces of odd lengths
        dict(name="write_prompts", op="write", B=24, new_lo=1, new_hi=4096, old_lo=0, old_hi=900, page=128, block=16,
             shape=4),
        # a small batch's rows read back, odd starts
        dict(name="read_small", op="read", B=7, rows_lo=1, rows_hi=600, first_lo=0, first_hi=900, page=128, block=32,
             shape=5),
        # four contexts of 65536 tokens read back whole
        dict(name="read_long", op="read", B=4, rows_lo=65536, rows_hi=65536, first_lo=0, first_hi=0, page=64, block=64,
             shape=6),
        # 16 heads on short contexts, a drafted token beside the new one: latency
        dict(name="decode_tiny", op="decode", B=2, H=16, n_q=2, ctx_lo=250, ctx_hi=256, page=64, block=64, shape=7),
        # the step of 32 sequences of 4096 tokens
        dict(name="decode_32x4096", op="decode", B=32, H=128, n_q=1, ctx_lo=4096, ctx_hi=4096, page=64, block=64,
             shape=8),
        # ragged contexts, from one token on
        dict(name="decode_ragged", op="decode", B=61, H=128, n_q=1, ctx_lo=1, ctx_hi=16384, page=128, block=16,
             shape=9),
        # four drafted tokens for each of 32 sequences of about 4096 tokens
        dict(name="attend_drafts", op="attend", B=32, H=128, new_lo=4, new_hi=4, old_lo=4092, old_hi=4092, page=64,
             block=64, shape=10),
        # ragged prompt pieces, odd lengths
        dict(name="attend_ragged", op="attend", B=6, H=40, new_lo=37, new_hi=1500, old_lo=0, old_hi=6000, page=128,
             block=32, shape=11),
        # a 2048-token piece of a prompt of 16384 tokens
        dict(name="attend_chunk_16k", op="attend", B=1, H=128, new_lo=2048, new_hi=2048, old_lo=14336, old_hi=14336,
             page=64, block=64, shape=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One more case: the operator, then its sizes over their logarithms, within the largest listed cost."""
    op = rng.choice(["pages", "write", "read", "decode", "decode", "attend", "attend"])
    c = dict(op=op, page=rng.choice([64, 128]), shape=rng.randrange(100, 1 << 20))
    if op == "pages":
        c.update(B=_log_int(rng, 1, 2048), ctx_hi=_log_int(rng, 1, 16384), prompt_hi=_log_int(rng, 1, 4096))
        return c
    c["block"] = rng.choice([16, 32, 64])
    if op == "write":
        c.update(B=_log_int(rng, 1, 1024))
        c["new_hi"] = _log_int(rng, 1, max(1, 65536 // c["B"]))
        c["new_lo"] = rng.randint(0, 1) if c["new_hi"] > 1 else 1
        c["old_lo"], c["old_hi"] = 0, _log_int(rng, 1, max(1, min(4096, 400000 // c["B"])))
    elif op == "read":
        c.update(B=_log_int(rng, 1, 64))
        c["rows_lo"], c["rows_hi"] = 1, _log_int(rng, 1, max(1, 262144 // c["B"]))
        c["first_lo"], c["first_hi"] = 0, _log_int(rng, 1, 2048)
    elif op == "decode":
        c.update(H=rng.choice([128, 128, _log_int(rng, 1, 128)]), n_q=rng.choice([1, 1, 2]))
        c["ctx_hi"] = _log_int(rng, c["n_q"], 131072)
        c["B"] = _log_int(rng, 1, max(1, min(256, 600000 // c["ctx_hi"])))
        c["ctx_lo"] = rng.choice([c["n_q"], c["ctx_hi"]])
    else:
        c["H"] = rng.choice([128, 128, _log_int(rng, 4, 128)])
        c["new_hi"] = _log_int(rng, 1, 2048)
        room = (1 << 32) // (c["H"] * c["new_hi"])  # heads x new tokens x context of one sequence
        c["old_hi"] = _log_int(rng, 1, max(1, min(16384, room)))
        c["B"] = _log_int(rng, 1, max(1, min(32, 20000 // (c["new_hi"] + c["old_hi"]))))
        c["new_lo"], c["old_lo"] = max(1, c["new_hi"] // 3), 0
    return c


def _lengths(case):
    """(new, old) or (rows, first) of each sequence, from the case alone."""
    r = random.Random(case["shape"])
    if case["op"] == "decode":
        ctx = [r.randint(max(case["ctx_lo"], case["n_q"]), case["ctx_hi"]) for _ in range(case["B"])]
        return [case["n_q"]] * case["B"], [L - case["n_q"] for L in ctx]
    a, b = ("rows", "first") if case["op"] == "read" else ("new", "old")
    n = [r.randint(case[a + "_lo"], case[a + "_hi"]) for _ in range(case["B"])]
    if sum(n) == 0:
        n[0] = 1
    return n, [r.randint(case[b + "_lo"], case[b + "_hi"]) for _ in range(case["B"])]


def _serving(case):
    """Two moments of a server: the sequences' lengths at each, and the new tokens of the step to it.
    One in eight places is empty before and holds a prompt after, one in eight the other way round."""
    r = random.Random(case["shape"])
    before, after, new_after, new_before = [], [], [], []
    for b in range(case["B"]):
        kind = (b + case["shape"]) % 8
        ctx, prompt = r.randint(1, case["ctx_hi"]), r.randint(1, case["prompt_hi"])
        pair = (0, prompt) if kind == 0 else (prompt, 0) if kind == 1 else (ctx, ctx + 1)
        before.append(pair[0])
        after.append(pair[1])
        new_after.append(prompt if kind == 0 else 0 if kind == 1 else 1)
        new_before.append(prompt if kind == 1 else 0)
    return before, after, new_before, new_after


# ------------------------------------------------------------------ inputs
def _cum(v):
    at, out = 0, [0]
    for n in v:
        at += n
        out.append(at)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def _prepare_pages(case, g):
    B, page, i32 = case["B"], case["page"], torch.int32
    before, after, new_before, new_after = _serving(case)
    pages = lambda v: [-(-L // page) for L in v]  # noqa: E731
    pb, pa = pages(before), pages(after)
    num_pages, max_pages = max(sum(pb), sum(pa)) + 5, max(max(pb), max(pa)) + 1
    order = torch.randperm(num_pages, generator=g, device="cuda").to(i32)
    held = torch.tensor(pb, dtype=i32, device="cuda")
    j = torch.arange(max_pages, device="cuda")
    mine = j[None, :] < held[:, None]
    table = torch.full((B, max_pages), -1, dtype=i32, device="cuda")
    table[mine] = order[:sum(pb)]
    free = torch.full((num_pages,), -1, dtype=i32, device="cuda")
    free[:num_pages - sum(pb)] = order[sum(pb):]
    s = dict(case=case, table=table, held=held, free=free, num_pages=num_pages,
             count=torch.tensor([num_pages - sum(pb)], dtype=i32, device="cuda"))
    for name, lens, new in (("after", after, new_after), ("before", before, new_before)):
        s[name] = torch.tensor(lens, dtype=i32, device="cuda")
        s["cu_" + name] = _cum(new)
        s["slots_" + name] = torch.empty(sum(new) + SPARE_ROWS, dtype=torch.int64, device="cuda")
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "pages":
        return _prepare_pages(case, g)
    new, old = _lengths(case)
    lens = [a + b for a, b in zip(new, old)]
    B, page, block = case["B"], case["page"], case["block"]
    bf, i32 = torch.bfloat16, torch.int32

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(bf)

    # a shuffled pool with a few pages to spare; unused block-table entries are -1
    need = [-(-L // page) for L in lens]
    num_pages, max_pages = sum(need) + 4, max(max(need), 1)
    order = torch.randperm(num_pages, generator=g, device="cuda").to(i32)
    table = torch.full((B, max_pages), -1, dtype=i32, device="cuda")
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    s = dict(case=case, new=new, lens=lens, total=sum(new), table=table, cu=_cum(new), max_tokens=sum(lens),
             seq_lens=torch.tensor(lens, dtype=i32, device="cuda"))
    # channels of unequal size, and blocks of tokens of unequal size
    rows = normal(num_pages * page, D_ROW)
    rows *= 0.5 + torch.rand(D_ROW, generator=g, device="cuda").to(bf)
    size = torch.randn(num_pages * page // 16, 1, generator=g, device="cuda").mul_(0.5).exp2_().to(bf)
    rows.view(-1, 16 * D_ROW).mul_(size)
    power = _power(_largest(rows).view(-1, block, GROUPS).amax(1))
    s["cache"] = _codes(rows, power.repeat_interleave(block, 0)).view(num_pages, page, D_ROW)
    s["scales"] = torch.zeros(num_pages, page // block, 8, dtype=torch.uint8, device="cuda")
    s["scales"].view(-1, 8)[:, :GROUPS] = power.to(torch.uint8)
    if case["op"] == "write":
        s["rows"] = normal(s["total"], D_ROW)
        s["rows"] *= torch.randn(s["total"], 1, generator=g, device="cuda").exp2_().to(bf)
    elif case["op"] == "read":
        s["first"] = torch.tensor(old, dtype=i32, device="cuda")
    else:
        H = case["H"]
        s["q_nope"], s["q_rope"] = normal(s["total"], H, D_NOPE), normal(s["total"], H, D_R)
        s["w_uk"], s["w_uv"] = normal(H, D_NOPE, D_C, std=D_C ** -0.5), normal(H, D_V, D_C, std=D_C ** -0.5)
    return s


# ------------------------------------------------------------------ plain forms
def _largest(rows):
    """The largest finite magnitude of each row's five groups, fp32."""
    x = rows.float().abs_()
    x.masked_fill_(~torch.isfinite(x), 0)
    return torch.cat([x[:, :D_C].view(-1, 4, 128).amax(2), x[:, D_C:].amax(1, keepdim=True)], 1)


def _power(top):
    """127 + the smallest power e with top <= 448 * 2^e, at least LEAST (int32)."""
    bits = top.contiguous().view(torch.int32)
    return ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp_(min=LEAST)


def _columns(power):
    """2^e of each of the 576 columns, from the powers of the five groups."""
    step = (power.int() << 23).view(torch.float32)
    return torch.cat([step[:, :4].repeat_interleave(128, 1), step[:, 4:5].expand(-1, D_R)], 1)


def _codes(rows, power):
    """e4m3 codes of rows by their powers (nearest, ties to even); what is not finite becomes NaN."""
    x = rows.float() / _columns(power)
    return x.masked_fill_(~torch.isfinite(x), float("nan")).to(torch.float8_e4m3fn).view(torch.uint8)


def _values(s, row):
    """fp32 values of rows of the pool."""
    power = s["scales"].view(-1, 8)[row // s["case"]["block"], :GROUPS]
    return s["cache"].view(-1, D_ROW)[row].view(torch.float8_e4m3fn).float() * _columns(power)


def _places(s, first):
    """Position of each new (or read) row in its sequence, and its row in the pool."""
    t = torch.arange(s["total"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu"], t, right=True).long() - 1
    pos = first[b].long() + (t - s["cu"][b]).long()
    page = s["case"]["page"]
    return pos, s["table"][b, pos // page].long() * page + pos % page


def _update_pages(s, lens, cu, slots):
    page, (B, width) = s["case"]["page"], s["table"].shape
    table, held, free, N = s["table"], s["held"], s["free"], s["num_pages"]
    count = s["count"].long()
    j = torch.arange(width, device="cuda")[None, :]
    need = (lens + page - 1) // page
    back = (j >= need[:, None]) & (j < held[:, None])
    take = (j >= held[:, None]) & (j < need[:, None])
    nth_back = (back.flatten().cumsum(0) - 1).view(B, width)
    nth_take = (take.flatten().cumsum(0) - 1).view(B, width)
    given = back.sum()
    last = nth_take[:, -1]  # a sequence is served whole or not at all, in order
    served = (need <= held) | (last < count + given)
    take &= served[:, None]
    taken = take.sum()
    # the pages given back, the first of them on top of the stack, then the stack downwards
    returned = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
    returned[torch.where(back, nth_back, N)] = table
    down = (count - 1 - (nth_take - given)).clamp(0, N - 1)
    page_id = torch.where(nth_take < given, returned[nth_take.clamp(0, N)], free[down])
    table.copy_(torch.where(take, page_id, torch.where(back, -1, table)))
    put = torch.where(back & (nth_back >= taken), count + given - 1 - nth_back, N)
    longer = torch.cat([free, free[:1]])
    longer[put] = torch.where(put < N, returned[nth_back.clamp(0, N)], longer[put])
    free.copy_(longer[:N])
    s["count"].copy_(count + given - taken)
    held.copy_(torch.where(served, need, held))
    t = torch.arange(slots.shape[0], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(cu, t, right=True).long() - 1
    mine = b < B
    b = b.clamp(max=B - 1)
    pos = (lens[b] - cu[b + 1] + t).long().clamp(min=0)
    row = table[b, (pos // page).clamp(max=width - 1)].long() * page + pos % page
    slots.copy_(torch.where(mine & served[b], row, -1))


def _write(s):
    block, page = s["case"]["block"], s["case"]["page"]
    n = s["cu"][1:] - s["cu"][:-1]
    first = s["seq_lens"] - n
    _, row = _places(s, first)
    codes, entry = s["cache"].view(-1, D_ROW), s["scales"].view(-1, 8)
    top = torch.zeros(entry.shape[0], GROUPS, device="cuda")
    touched = torch.zeros(entry.shape[0], dtype=torch.bool, device="cuda")
    at = row // block
    top.scatter_reduce_(0, at[:, None].expand(-1, GROUPS), _largest(s["rows"]), "amax")
    touched[at] = True
    before = entry[:, :GROUPS].int()
    power = torch.where(touched[:, None], _power(top), before)
    # blocks that hold older tokens: one at most for each sequence
    mixed = (n > 0) & (first % block != 0)
    b, p0 = torch.arange(len(n), device="cuda")[mixed], first[mixed].long()
    start = (s["table"][b, p0 // page].long() * page + p0 % page) // block
    power[start] = torch.maximum(power[start], before[start])
    inside = torch.arange(block, device="cuda")[None, :]
    older = (start[:, None] * block + inside)[inside < (p0 % block)[:, None]]
    codes[older] = _codes(_values(s, older), power[older // block])
    codes[row] = _codes(s["rows"], power[at])
    entry[touched] = torch.nn.functional.pad(power, (0, 3))[touched].to(torch.uint8)
    return s["cache"].view(torch.float8_e4m3fn), s["scales"]


def _read(s):
    _, row = _places(s, s["first"])
    return _values(s, row).to(torch.bfloat16)


def _decode(s):
    B, H, n, page = (s["case"][k] for k in ("B", "H", "n_q", "page"))
    tok = torch.arange(max(s["lens"]), device="cuda")
    row = s["table"][:, tok // page].long().clamp(min=0) * page + tok % page
    x = _values(s, row.flatten()).view(B, -1, D_ROW)
    c = x[..., :D_C]
    q = torch.cat([torch.einsum("thd,hdc->thc", s["q_nope"].float(), s["w_uk"].float()), s["q_rope"].float()], 2)
    z = (q.view(B, n * H, D_ROW) @ x.transpose(1, 2)).view(B, n, H, -1)
    seen = s["seq_lens"][:, None] - n + 1 + torch.arange(n, device="cuda")
    z.mul_(SCALE).masked_fill_(tok >= seen[..., None, None], float("-inf"))
    z.sub_(z.amax(-1, keepdim=True)).exp_()
    z.div_(z.sum(-1, keepdim=True))
    u = (z.view(B, n * H, -1) @ c).view(B * n, H, D_C)
    return [torch.einsum("thc,hvc->thv", u, s["w_uv"].float()).to(torch.bfloat16), u.to(torch.bfloat16)]


def _attend(s):
    outs, at, page = [], 0, s["case"]["page"]
    w_uk, w_uv = s["w_uk"].float(), s["w_uv"].float()
    for b, (n, L) in enumerate(zip(s["new"], s["lens"])):  # the scores of all of them at once would not fit
        if n == 0:
            continue
        tok = torch.arange(L, device="cuda")
        x = _values(s, s["table"][b, tok // page].long() * page + tok % page)
        c, kr = x[:, :D_C], x[:, D_C:]
        qn = s["q_nope"][at:at + n].float().transpose(0, 1)  # [H, n, 128]
        qr = s["q_rope"][at:at + n].float().transpose(0, 1)
        few = n < 128  # fewer products on the latents themselves than on expanded keys and values
        z = (qn @ w_uk) @ c.t() if few else qn @ (w_uk @ c.t())
        z += qr @ kr.t()
        hidden = tok[None, :] > (torch.arange(n, device="cuda") + (L - n))[:, None]
        z.mul_(SCALE).masked_fill_(hidden, float("-inf"))
        z.sub_(z.amax(-1, keepdim=True)).exp_()
        total = z.sum(-1, keepdim=True)
        o = (z @ c) @ w_uv.transpose(1, 2) if few else z @ (w_uv @ c.t()).transpose(1, 2)
        outs.append((o / total).transpose(0, 1).to(torch.bfloat16))
        at += n
    return torch.cat(outs)


def _pages(s, when):
    """The step of a server to `when`: the pages of finished sequences go to those that start or grow."""
    if own:
        import mla_latent_kv_paged_gb300 as mla
        mla.update_pages(s["table"], s["held"], s[when], s["free"], s["count"], page_size=s["case"]["page"],
                         cu=s["cu_" + when], slots=s["slots_" + when])
    else:
        _update_pages(s, s[when], s["cu_" + when], s["slots_" + when])


def run(s):
    op = s["case"]["op"]
    if op == "pages":
        _pages(s, "after")  # and back: the stack of free pages then is as it was
        _pages(s, "before")
        return [s[k] for k in ("slots_after", "slots_before", "table", "held", "free", "count")]
    if own:
        import mla_latent_kv_paged_gb300 as mla
        paged = (s["cache"], s["table"], s["seq_lens"], s["cu"])
        if op == "write":
            mla.write_kv(s["rows"], *paged, fp8_scales=s["scales"])
            return s["cache"].view(torch.float8_e4m3fn), s["scales"]
        if op == "read":
            return mla.read_kv(*paged, n_rows=s["total"], first=s["first"], fp8_scales=s["scales"])
        if op == "decode":
            r = mla.decode_step(s["q_nope"], s["q_rope"], s["w_uk"], s["w_uv"], s["cache"], s["table"], s["seq_lens"],
                                n_q=s["case"]["n_q"], softmax_scale=SCALE, fp8_scales=s["scales"])
            return [r["out"], r["u"]]
        return mla.attend_chunk(s["q_nope"], s["q_rope"], s["w_uk"], s["w_uv"], *paged, max_tokens=s["max_tokens"],
                                fp8_scales=s["scales"], softmax_scale=SCALE)
    return _write(s) if op == "write" else _read(s) if op == "read" else _decode(s) if op == "decode" else _attend(s)


# ------------------------------------------------------------------ cost
def work(case):
    B = case["B"]
    if case["op"] == "pages":
        total, page = 0, case["page"]
        before, after, new_before, new_after = _serving(case)
        for a, b in zip(before, after):
            pa, pb = -(-a // page), -(-b // page)
            total += 2 * abs(pa - pb) * (2 * 4 + 4)  # a page's id read, written, its old place cleared
        rows = sum(new_before) + sum(new_after) + 2 * SPARE_ROWS
        return {"bytes": total + 8 * rows + 2 * B * 4 * 4, "flops": 0}
    new, old = _lengths(case)
    T = sum(new)
    entry = 8.0 / case["block"]
    if case["op"] == "write":
        blocks = sum(-(-(o + n) // case["block"]) - o // case["block"] for n, o in zip(new, old) if n)
        return {"bytes": T * 3 * D_ROW + 2 * 8 * blocks, "flops": 2 * T * D_ROW}
    if case["op"] == "read":
        return {"bytes": T * (3 * D_ROW + entry), "flops": T * D_ROW}
    H, flops = case["H"], 0
    for n, p in zip(new, old):
        pairs = n * p + n * (n + 1) // 2
        expanded = (n + p) * D_C * (D_NOPE + D_V) + pairs * (D_NOPE + D_R + D_V)
        absorbed = n * D_C * (D_NOPE + D_V) + pairs * (D_ROW + D_C)
        flops += 2 * H * (absorbed if case["op"] == "decode" else min(expanded, absorbed))
    data = sum(n + p for n, p in zip(new, old) if n) * (D_ROW + entry) + 2 * T * H * (D_NOPE + D_R + D_V)
    if case["op"] == "decode":
        data += T * H * 2 * D_C
    return {"bytes": data + 2 * H * D_C * (D_NOPE + D_V) + 8 * B, "flops": flops}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The outputs from the definitions, in 64 bits; codes before their rounding, none for whole numbers."""
    if case["op"] == "pages":
        return None
    s = prepare(case, seed)
    new, old = _lengths(case)
    page, block = case["page"], case["block"]
    groups = [slice(128 * i, 128 * i + 128) for i in range(4)] + [slice(D_C, D_ROW)]
    codes = s["cache"].view(torch.float8_e4m3fn).double().reshape(-1, D_ROW)
    power = s["scales"].reshape(-1, 8).double() - 127
    table = s["table"].cpu().tolist()

    def rows_of(b, lo, hi):
        return torch.tensor([table[b][p // page] * page + p % page for p in range(lo, hi)], dtype=torch.long,
                            device="cuda")

    def values(row):
        x = codes[row]
        for i, cols in enumerate(groups):
            x[:, cols] *= torch.exp2(power[row // block, i])[:, None]
        return x

    if case["op"] == "write":
        at = 0
        for b, (n, p) in enumerate(zip(new, old)):
            for lo in range(p // block * block, p + n, block) if n else ():
                hi = min(lo + block, p + n)
                cut = max(lo, p)
                row, mine = rows_of(b, lo, hi), s["rows"][at + cut - p:at + hi - p].double()
                held = values(row[:cut - lo])
                for i, cols in enumerate(groups):
                    e = torch.ceil(torch.log2(mine[:, cols].abs().max() / 448)).clamp(min=LEAST - 127)
                    if cut > lo:
                        e = torch.maximum(e, power[row[0] // block, i])
                    codes[row, cols] = torch.cat([held, mine])[:, cols] / torch.exp2(e)
            at += n
        return codes.reshape(s["cache"].shape), None
    if case["op"] == "read":
        return torch.cat([values(rows_of(b, p, p + n)) for b, (n, p) in enumerate(zip(new, old))])
    T, H = sum(new), case["H"]
    out = torch.empty(T, H, D_V, dtype=torch.float64, device="cuda")
    us = torch.empty(T, H, D_C, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, p) in enumerate(zip(new, old)):
        x = values(rows_of(b, 0, n + p))
        keep = torch.ones(n, n + p, dtype=torch.bool, device="cuda").tril_(p)
        for h in range(H):
            key = torch.cat([x[:, :D_C] @ s["w_uk"][h].double().t(), x[:, D_C:]], 1)
            q = torch.cat([s["q_nope"][at:at + n, h], s["q_rope"][at:at + n, h]], 1).double()
            a = torch.softmax((q @ key.t() * SCALE).masked_fill(~keep, float("-inf")), -1)
            w_uv = s["w_uv"][h].double()
            out[at:at + n, h] = a @ (x[:, :D_C] @ w_uv.t())
            if case["op"] == "decode":
                us[at:at + n, h] = a @ x[:, :D_C]
        at += n
    return [out, us] if case["op"] == "decode" else out
