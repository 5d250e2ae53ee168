"""Plain 64-bit reference of the chunk operators (append_chunk, read_kv, attend_chunk)
and the error bounds their tests use. Torch tensors on one device, elementary
operations only; shares no code with the library."""
import math

import torch

D_C, D_R, D_ROW = 512, 64, 576
SCALE = 1.0 / math.sqrt(192.0)
U_BF16, U_F16, U_F32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24  # half a step, relative
TINY_F16 = 2.0 ** -25  # half a step of fp16 below its normal range (2^-14)
NAN_CODE = 0x7F  # e4m3 NaN


class Chunk:
    """A ragged chunk on a shuffled paged cache. Spare pages and the slack behind each
    context hold NaN, unused block-table entries -1."""

    def __init__(self, new, lens, *, H=4, page=64, fp8=False, seed=0, pad_rows=0, spare=3, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.new, self.lens, self.H, self.page, self.fp8, self.dev = list(new), list(lens), H, page, fp8, device
        B, i32, bf = len(self.new), torch.int32, torch.bfloat16
        self.T = sum(self.new) + pad_rows
        self.total = sum(self.new)
        need = [-(-L // page) for L in self.lens]
        self.num_pages, self.max_pages = sum(need) + spare, max(max(need), 1) + 1
        order = torch.randperm(self.num_pages, generator=g, device=device)
        table = torch.full((B, self.max_pages), -1, dtype=i32, device=device)
        at = 0
        for b, k in enumerate(need):
            table[b, :k] = order[at:at + k].to(i32)
            at += k
        self.table = table
        self.host_table = table.cpu().tolist()
        self.seq_lens = torch.tensor(self.lens, dtype=i32, device=device)
        self.cu = torch.tensor([sum(self.new[:i]) for i in range(B + 1)], dtype=i32, device=device)

        def normal(*shape, std=1.0):
            return (torch.randn(*shape, generator=g, device=device) * std).to(bf)

        pool = torch.full((self.num_pages * page, D_ROW), float("nan"), dtype=bf, device=device)
        for b in range(B):
            if self.lens[b]:
                pool[self.rows(b)] = normal(self.lens[b], D_ROW)
        self.scales = None
        if fp8:
            self.scales = (0.5 + torch.rand(D_ROW, generator=g, device=device)) * (5.0 / 448.0)
            codes = (pool.float() / self.scales).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            codes[torch.isnan(pool)] = NAN_CODE
            self.cache = codes.view(self.num_pages, page, D_ROW)
        else:
            self.cache = pool.view(self.num_pages, page, D_ROW)
        rows = max(self.T, 1)
        self.q_nope, self.q_rope = normal(rows, H, 128), normal(rows, H, 64)
        self.w_uk, self.w_uv = normal(H, 128, D_C, std=D_C ** -0.5), normal(H, 128, D_C, std=D_C ** -0.5)

    def rows(self, b, lo=0, hi=None):
        """Rows of the pool that hold tokens [lo, hi) of sequence b."""
        hi = self.lens[b] if hi is None else hi
        t = self.host_table[b]
        return torch.tensor([t[p // self.page] * self.page + p % self.page for p in range(lo, hi)], dtype=torch.long,
                            device=self.dev)

    def values(self, b, lo=0, hi=None):
        """Cached values of those tokens, 64 bits."""
        x = self.cache.view(-1, D_ROW)[self.rows(b, lo, hi)]
        return x.view(torch.float8_e4m3fn).double() * self.scales.double() if self.fp8 else x.double()

    def paged(self):
        return self.cache, self.table, self.seq_lens, self.cu


def attend(c: Chunk, scale=SCALE):
    """(out, lse, bounds): 64-bit results for the chunk's rows and, per form, a bound of
    |got - out| from the roundings of that form.

    A score is off by at most dz (the rounding of the keys, or of the absorbed query,
    times the absolute products), which moves a weight by a factor exp(+-2 dz); a weight
    is rounded once more before the value product, a value once:
      expanded  keys, values and weights in fp16 (u = 2^-11); rows of an FP8 cache are
                first rounded to fp16 as well
      absorbed  absorbed query and weights in bf16 (2^-8; on an FP8 cache in fp16, the
                query times the scales), partials, u and W^UV in fp16
    plus the output's own rounding to bf16 and the fp32 sums. Those are off by 2^-24 of
    the absolute products per term, whatever the products cancel to: 512 terms for a key
    or a value (2^-15 of |c| |W|), 192 for a score, 128 for an absorbed query. The sums
    over the keys have at most a few thousand terms: below 2^-11 of sum p |v|, counted as
    one more fp16 unit. Below 2^-14 fp16 rounds by 2^-25 whatever the value is."""
    outs, lses, be, ba = [], [], [], []
    for b, (n, L) in enumerate(zip(c.new, c.lens)):
        if n == 0:
            continue
        at = sum(c.new[:b])
        x = c.values(b)
        lat, kr = x[:, :D_C], x[:, D_C:]
        hidden = torch.ones(n, L, dtype=torch.bool, device=c.dev).triu_(L - n + 1)
        o = torch.empty(n, c.H, 128, dtype=torch.float64, device=c.dev)
        z_all = torch.empty(n, c.H, dtype=torch.float64, device=c.dev)
        e1, e2 = torch.empty_like(o), torch.empty_like(o)
        for h in range(c.H):
            uk, uv = c.w_uk[h].double(), c.w_uv[h].double()
            k, v = lat @ uk.t(), lat @ uv.t()
            qn, qr = c.q_nope[at:at + n, h].double(), c.q_rope[at:at + n, h].double()
            z = ((qn @ k.t() + qr @ kr.t()) * scale).masked_fill(hidden, float("-inf"))
            p = torch.softmax(z, -1)
            o[:, h] = p @ v
            z_all[:, h] = torch.logsumexp(z, -1)
            rows_u = U_F16 if c.fp8 else 0.0
            kabs, vabs = lat.abs() @ uk.abs().t(), lat.abs() @ uv.abs().t()
            # expanded
            rope_abs = qr.abs() @ kr.abs().t()
            tiny = TINY_F16 * (qn.abs().sum(-1, keepdim=True) + k.abs().sum(-1)[None])
            dz = scale * ((qn.abs() @ k.abs().t()) * 2 * U_F16 + tiny + (rows_u + 512 * U_F32) * (qn.abs() @ kabs.t())
                          + (rows_u + 192 * U_F32) * rope_abs)
            dz = dz.masked_fill(hidden, 0).amax(-1, keepdim=True)
            e1[:, h] = U_BF16 * o[:, h].abs() + (p @ v.abs()) * (3 * U_F16 + torch.expm1(2 * dz))
            e1[:, h] += TINY_F16 + (rows_u + 512 * U_F32) * (p @ vabs)
            # absorbed
            qa = qn @ uk
            unit = U_F16 if c.fp8 else U_BF16
            dz = scale * unit * 1.25 * (qa.abs() @ lat.abs().t() + rope_abs)
            dz += scale * 128 * U_F32 * ((qn.abs() @ uk.abs()) @ lat.abs().t())
            if c.fp8:
                dz += scale * TINY_F16 * (x / c.scales.double()).abs().sum(-1)
            dz = dz.masked_fill(hidden, 0).amax(-1, keepdim=True)
            u = p @ lat
            du = U_F16 * u.abs() + (p @ lat.abs()) * (unit + 3 * U_F16 + torch.expm1(2 * dz))
            e2[:, h] = 1.01 * U_BF16 * o[:, h].abs() + du @ uv.abs().t() + U_F16 * (u.abs() @ uv.abs().t())
        outs.append(o), lses.append(z_all), be.append(e1), ba.append(e2)
    return torch.cat(outs), torch.cat(lses), {"expanded": torch.cat(be), "absorbed": torch.cat(ba)}


def append(c: Chunk, h, w_dkr, theta=10000.0):
    """(pool rows, rows in 64 bits, error bound before rounding) of the chunk's new rows."""
    y = h[:c.total].double() @ w_dkr.double().t()
    # fp32 sums of d products in any order: at most d half steps of the absolute sum
    slack = h.shape[1] * U_F32 * (h[:c.total].double().abs() @ w_dkr.double().abs().t())
    pos = torch.cat([torch.arange(L - n, L, dtype=torch.float64, device=c.dev) for n, L in zip(c.new, c.lens)])
    ang = pos[:, None] * torch.tensor([theta ** (-2.0 * i / D_R) for i in range(D_R // 2)], dtype=torch.float64,
                                      device=c.dev)
    cs, sn = ang.cos(), ang.sin()
    a, b = y[:, D_C::2].clone(), y[:, D_C + 1::2].clone()
    y[:, D_C::2], y[:, D_C + 1::2] = a * cs - b * sn, a * sn + b * cs
    # both members of a pair mix; the angle, its sine and cosine and the rotation are in fp32
    both = slack[:, D_C::2] + slack[:, D_C + 1::2] + 8 * U_F32 * (a.abs() + b.abs())
    slack[:, D_C::2], slack[:, D_C + 1::2] = both, both
    rows = torch.cat([c.rows(b, L - n, L) for b, (n, L) in enumerate(zip(c.new, c.lens))])
    return rows, y, slack
