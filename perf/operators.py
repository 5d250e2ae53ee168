"""Cases of the prompt-side operators of the paged latent cache, for timing and for comparison.

  append  the cache rows of a ragged chunk of new tokens, [h W^DKV ; RoPE(h W^KR)], written into their
          pages as bf16 or quantised to e4m3 codes with one scale per column
  read    rows of the sequences read back from their pages into one array, as bf16
  attend  attention of a ragged chunk of new tokens over the paged cache: query j of a sequence with
          n new tokens and context L sees tokens 0 .. L - n + j

``run`` computes each in its plain form (elementary torch operations in 32 bits) or, with ``own``
set, through the package's entry points. ``exact`` gives the same outputs in 64 bits.
"""
import math
import random

import torch

own = False

D_NOPE, D_R, D_C, D_V, D_ROW = 128, 64, 512, 128, 576
THETA = 10000.0
SCALE = 1.0 / math.sqrt(D_NOPE + D_R)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token for each of 32 running sequences, the cache append beside a decode step
        dict(name="append_decode_32", op="append", B=32, new_lo=1, new_hi=1, old_lo=64, old_hi=4096, d_model=7168,
             page=64, fp8=False, shape=1),
        # a mixed batch of prompt pieces into an FP8 cache, odd lengths
        dict(name="append_fp8_mixed", op="append", B=5, new_lo=37, new_hi=700, old_lo=0, old_hi=3000, d_model=5120,
             page=128, fp8=True, shape=2),
        # whole prompts into an FP8 cache: 16 sequences of up to 1024 tokens
        dict(name="append_fp8_prompts", op="append", B=16, new_lo=200, new_hi=1024, old_lo=0, old_hi=0, d_model=7168,
             page=64, fp8=True, shape=3),
        # a small batch's rows read back, odd starts
        dict(name="read_fp8_small", op="read", B=7, rows_lo=1, rows_hi=600, first_lo=0, first_hi=900, page=128,
             fp8=True, shape=4),
        # four contexts of 131072 tokens read back whole
        dict(name="read_long", op="read", B=4, rows_lo=131072, rows_hi=131072, first_lo=0, first_hi=0, page=64,
             fp8=False, shape=5),
        # 16 heads, a few tokens on a short context: latency
        dict(name="attend_tiny", op="attend", B=2, H=16, new_lo=3, new_hi=6, old_lo=100, old_hi=250, page=64,
             fp8=False, shape=6),
        # four drafted tokens per sequence for 32 sequences of about 4096 tokens
        dict(name="attend_drafts", op="attend", B=32, H=128, new_lo=4, new_hi=4, old_lo=4092, old_hi=4092, page=64,
             fp8=False, shape=7),
        # a prompt without context
        dict(name="attend_prompt", op="attend", B=1, H=128, new_lo=2048, new_hi=2048, old_lo=0, old_hi=0, page=64,
             fp8=False, shape=8),
        # ragged prompt pieces on an FP8 cache, odd lengths, pages of 128
        dict(name="attend_ragged_fp8", op="attend", B=6, H=40, new_lo=37, new_hi=1500, old_lo=0, old_hi=6000,
             page=128, fp8=True, shape=9),
        # a prompt's last 1024 tokens on a long context, few heads
        dict(name="attend_long_few_heads", op="attend", B=1, H=16, new_lo=1024, new_hi=1024, old_lo=64512,
             old_hi=64512, page=64, fp8=False, shape=10),
        # a 2048-token piece of a prompt of 16384 tokens
        dict(name="attend_chunk_16k", op="attend", B=1, H=128, new_lo=2048, new_hi=2048, old_lo=14336, old_hi=14336,
             page=64, fp8=False, shape=11),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One more case: the operator, then its sizes over their logarithms, within the largest listed cost."""
    op = rng.choice(["append", "read", "attend", "attend"])
    c = dict(op=op, page=rng.choice([64, 128]), fp8=rng.random() < 0.5, shape=rng.randrange(100, 1 << 20))
    if op == "append":
        c.update(B=_log_int(rng, 1, 64), d_model=64 * _log_int(rng, 8, 112))
        c["new_hi"] = _log_int(rng, 1, max(1, 8192 // c["B"]))
        c["new_lo"] = rng.randint(0, 1) if c["new_hi"] > 1 else 1
        c["old_hi"] = _log_int(rng, 1, 4096)
        c["old_lo"] = 0
    elif op == "read":
        c.update(B=_log_int(rng, 1, 64))
        c["rows_hi"] = _log_int(rng, 1, max(1, 262144 // c["B"]))
        c["rows_lo"] = 1
        c["first_lo"], c["first_hi"] = 0, _log_int(rng, 1, 2048)
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
    a, b = ("rows", "first") if case["op"] == "read" else ("new", "old")
    n = [r.randint(case[a + "_lo"], case[a + "_hi"]) for _ in range(case["B"])]
    if sum(n) == 0:
        n[0] = 1
    return n, [r.randint(case[b + "_lo"], case[b + "_hi"]) for _ in range(case["B"])]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new, old = _lengths(case)
    lens = [a + b for a, b in zip(new, old)]
    B, page = case["B"], case["page"]
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

    def cum(v):
        return torch.tensor([sum(v[:i]) for i in range(B + 1)], dtype=i32, device="cuda")

    s = dict(case=case, new=new, lens=lens, total=sum(new), table=table, cu=cum(new), max_tokens=sum(lens),
             seq_lens=torch.tensor(lens, dtype=i32, device="cuda"))
    rows = normal(num_pages, page, D_ROW)
    s["scales"] = None
    if case["fp8"]:
        col = (0.5 + torch.rand(D_ROW, generator=g, device="cuda"))  # channels of unequal size
        amax = (rows.view(-1, D_ROW).float() * col).abs().amax(0)
        s["scales"] = (amax / 448.0).contiguous()
        codes = (rows.float() * col / s["scales"]).clamp_(-448, 448).to(torch.float8_e4m3fn)
        s["cache"] = codes.view(torch.uint8)
    else:
        s["cache"] = rows
    if case["op"] == "append":
        s["h"] = normal(s["total"], case["d_model"])
        s["w_dkr"] = normal(D_ROW, case["d_model"], std=case["d_model"] ** -0.5)
    elif case["op"] == "read":
        s["first"] = torch.tensor(old, dtype=i32, device="cuda")
    else:
        H = case["H"]
        s["q_nope"], s["q_rope"] = normal(s["total"], H, D_NOPE), normal(s["total"], H, D_R)
        s["w_uk"], s["w_uv"] = normal(H, D_NOPE, D_C, std=D_C ** -0.5), normal(H, D_V, D_C, std=D_C ** -0.5)
    return s


# ------------------------------------------------------------------ plain forms
def _places(s, first):
    """Position of each new (or read) row in its sequence, and its row in the pool."""
    t = torch.arange(s["total"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu"], t, right=True).long() - 1
    pos = first[b].long() + (t - s["cu"][b]).long()
    page = s["case"]["page"]
    return pos, s["table"][b, pos // page].long() * page + pos % page


def _values(s, rows):
    """fp32 values of rows of the pool."""
    if s["scales"] is None:
        return rows.float()
    return rows.view(torch.float8_e4m3fn).float() * s["scales"]


def _append(s):
    first = s["seq_lens"] - (s["cu"][1:] - s["cu"][:-1])
    pos, row = _places(s, first)
    x = s["h"].float() @ s["w_dkr"].float().t()
    freq = THETA ** (-torch.arange(0, D_R, 2, device="cuda", dtype=torch.float64) / D_R)
    angle = pos.double()[:, None] * freq  # far positions need 64 bits
    cos, sin = angle.cos().float(), angle.sin().float()
    a, b = x[:, D_C::2].clone(), x[:, D_C + 1::2].clone()
    x[:, D_C::2], x[:, D_C + 1::2] = a * cos - b * sin, a * sin + b * cos
    pool = s["cache"].view(-1, D_ROW)
    if s["scales"] is None:
        pool[row] = x.to(torch.bfloat16)
        return s["cache"]
    pool[row] = (x / s["scales"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return s["cache"].view(torch.float8_e4m3fn)


def _read(s):
    _, row = _places(s, s["first"])
    return _values(s, s["cache"].view(-1, D_ROW)[row]).to(torch.bfloat16)


def _attend(s):
    outs, at, page = [], 0, s["case"]["page"]
    w_uk, w_uv = s["w_uk"].float(), s["w_uv"].float()
    for b, (n, L) in enumerate(zip(s["new"], s["lens"])):
        tok = torch.arange(L, device="cuda")
        row = s["table"][b, tok // page].long() * page + tok % page
        x = _values(s, s["cache"].view(-1, D_ROW)[row])
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


def run(s):
    op = s["case"]["op"]
    if own:
        import mla_latent_kv_paged_gb300 as mla
        if op == "append":
            mla.append_chunk(s["h"], s["w_dkr"], s["cache"], s["table"], s["seq_lens"], s["cu"],
                             fp8_scales=s["scales"], rope_theta=THETA)
            return s["cache"] if s["scales"] is None else s["cache"].view(torch.float8_e4m3fn)
        if op == "read":
            return mla.read_kv(s["cache"], s["table"], s["seq_lens"], s["cu"], n_rows=s["total"], first=s["first"],
                               fp8_scales=s["scales"])
        return mla.attend_chunk(s["q_nope"], s["q_rope"], s["w_uk"], s["w_uv"], s["cache"], s["table"],
                                s["seq_lens"], s["cu"], max_tokens=s["max_tokens"], fp8_scales=s["scales"],
                                softmax_scale=SCALE)
    return _append(s) if op == "append" else _read(s) if op == "read" else _attend(s)


# ------------------------------------------------------------------ cost
def work(case):
    new, old = _lengths(case)
    T, B = sum(new), case["B"]
    row = D_ROW * (1 if case["fp8"] else 2)
    if case["op"] == "append":
        d = case["d_model"]
        return {"bytes": 2 * T * d + 2 * D_ROW * d + T * row, "flops": 2 * T * d * D_ROW}
    if case["op"] == "read":
        return {"bytes": T * (row + 2 * D_ROW), "flops": T * D_ROW if case["fp8"] else 0}
    H, flops = case["H"], 0
    for n, p in zip(new, old):
        pairs = n * p + n * (n + 1) // 2
        expanded = (n + p) * D_C * (D_NOPE + D_V) + pairs * (D_NOPE + D_R + D_V)
        absorbed = n * D_C * (D_NOPE + D_V) + pairs * (D_ROW + D_C)
        flops += 2 * H * min(expanded, absorbed)
    data = sum(n + p for n, p in zip(new, old)) * row + 2 * T * H * (D_NOPE + D_R + D_V)
    return {"bytes": data + 2 * H * D_C * (D_NOPE + D_V) + 8 * B, "flops": flops}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The outputs from the definitions, in 64 bits; an 8-bit output before its rounding."""
    s = prepare(case, seed)
    new, old = _lengths(case)
    page, f8 = case["page"], torch.float8_e4m3fn
    pool = (s["cache"].view(f8) if case["fp8"] else s["cache"]).double().reshape(-1, D_ROW)
    table = s["table"].cpu().tolist()

    def rows_of(b, lo, hi):
        return torch.tensor([table[b][p // page] * page + p % page for p in range(lo, hi)], device="cuda")

    if case["op"] == "append":
        y = s["h"].double() @ s["w_dkr"].double().t()
        at = 0
        for b, (n, p) in enumerate(zip(new, old)):
            if n == 0:
                continue
            x = y[at:at + n]
            pos = torch.arange(p, p + n, dtype=torch.float64, device="cuda")
            freq = torch.tensor([THETA ** (-2.0 * i / D_R) for i in range(D_R // 2)], dtype=torch.float64,
                                device="cuda")
            turn = torch.polar(torch.ones(n, D_R // 2, dtype=torch.float64, device="cuda"), torch.outer(pos, freq))
            key = torch.view_as_real(torch.view_as_complex(x[:, D_C:].reshape(n, D_R // 2, 2).contiguous()) * turn)
            x = torch.cat([x[:, :D_C], key.reshape(n, D_R)], 1)
            if case["fp8"]:
                x = (x / s["scales"].double()).clamp(-448, 448)
            pool[rows_of(b, p, p + n)] = x
            at += n
        return pool.reshape(s["cache"].shape)
    if case["fp8"]:
        pool = pool * s["scales"].double()
    if case["op"] == "read":
        return torch.cat([pool[rows_of(b, p, p + n)] for b, (n, p) in enumerate(zip(new, old))])
    out = torch.empty(sum(new), case["H"], D_V, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, p) in enumerate(zip(new, old)):
        x = pool[rows_of(b, 0, n + p)]
        keep = torch.ones(n, n + p, dtype=torch.bool, device="cuda").tril_(p)
        for h in range(case["H"]):
            key = torch.cat([x[:, :D_C] @ s["w_uk"][h].double().t(), x[:, D_C:]], 1)
            q = torch.cat([s["q_nope"][at:at + n, h], s["q_rope"][at:at + n, h]], 1).double()
            a = torch.softmax((q @ key.t() * SCALE).masked_fill_(~keep, float("-inf")), -1)
            out[at:at + n, h] = a @ (x[:, :D_C] @ s["w_uv"][h].double().t())
        at += n
    return out
