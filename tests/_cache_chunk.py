"""Paged caches filled with ragged requests, and the plain definitions (64 bits, on the tensors'
device) of the cache and chunk operators, for their tests.  Shares no code with the kernels.

Tolerances, derived from the operators' arithmetic (u16 = 2^-8 is half a bf16 step relative to the
value, u32 = 2^-24 half an f32 step):
  * a logit is a sum of 576 exact products accumulated in f32 in some order and then scaled, so it is
    off by at most E = tau * sum|q||k| * 600 * 2^-23 + |logit| * 2^-22 (2^-23: the accumulation may
    truncate), and its exponential by a factor 1 +- 2 E for E < 1/2; ex2 and the running base add
    2^-20;
  * tensor cores multiply weights rounded to bf16: relative u16 each.  Numerator and normaliser use
    the same rounded weights, so out is off by at most (2 u16 + 2 * (2 E + 2^-20)) * A with
    A = sum p |v| of the exact softmax, plus the accumulation 2^-23 * n / 16 * A over n rows, plus
    the output's own rounding u16 * |out|;
  * lse moves with the normaliser: u16 + 2 E + 2^-20, plus 2^-22 * |lse|;
  * f32 caches (no rounded weights): the same without the u16 terms, n * 2^-23 for n rows summed.
"""
import math

import torch

import sparse_attention_06_b200 as dsa

PAGE = 64
FP8 = torch.float8_e4m3fn


class Requests:
    """Chunks of `news[r]` tokens behind `ctxs[r]` cached ones, over shuffled pages of one pool."""

    def __init__(self, ctxs, news, seed=0, pad=0, extra_blocks=2, min_block=0, device="cuda"):
        self.ctxs, self.news = list(ctxs), list(news)
        self.gen = torch.Generator().manual_seed(seed)
        lens = [c + n for c, n in zip(ctxs, news)]
        blocks = [-(-n // PAGE) for n in lens]
        self.num_blocks = sum(blocks) + extra_blocks + min_block
        ids = torch.randperm(sum(blocks) + extra_blocks, generator=self.gen) + min_block
        width = max(max(blocks), 1)
        table = torch.full((len(news), width), -1, dtype=torch.int32)
        at = 0
        for r, n in enumerate(blocks):
            table[r, :n] = ids[at:at + n]
            at += n
        cu = [0]
        for n in news:
            cu.append(cu[-1] + n)
        self.total, self.tokens = cu[-1], cu[-1] + pad
        self.lens = lens
        self.table = table.to(device)
        self.cu = torch.tensor(cu, dtype=torch.int32, device=device)
        self.seq = torch.tensor(lens, dtype=torch.int32, device=device)
        self.max_context = max(max(lens), 1)
        self.req = [r for r, n in enumerate(news) for _ in range(n)]
        self.pos = [c + i for c, n in zip(ctxs, news) for i in range(n)]

    def chunks(self):
        return dsa.Chunks(self.cu, self.seq, self.table, self.max_context)

    def rows(self, r, lo=0, hi=None):
        """Pool rows (page * 64 + slot) of positions lo .. hi-1 of request r."""
        p = torch.arange(lo, self.lens[r] if hi is None else hi, device=self.table.device)
        return self.table[r].long()[p // PAGE] * PAGE + p % PAGE

    def token_rows(self):
        return torch.cat([self.rows(r, c) for r, c in enumerate(self.ctxs)])


def randn(reqs, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=reqs.gen).cuda().to(dtype)


def pow2(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float64), e)


def quantise(x, group):
    """(e4m3 values, scales) in 64 bits of x [..., n] in groups: the smallest power of two with
    |x| <= 448 * scale over the group's finite elements, within 2^-100 .. 2^119, 1 for zeros; values
    nearest to x / scale, ties to even, saturating; NaN where x is not finite."""
    g = x.double().unflatten(-1, (-1, group))
    fin = torch.isfinite(g)
    amax = torch.where(fin, g, 0.0).abs().amax(-1)
    m, e = torch.frexp(amax)                       # amax = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-100, 119)
    scale = torch.where(amax > 0, pow2(e), 1.0)
    y = (g / scale.unsqueeze(-1)).clamp(-448.0, 448.0)
    _, ye = torch.frexp(y)
    step = pow2((ye - 1).clamp(min=-6) - 3)
    v = torch.where(fin, torch.round(y / step) * step, math.nan)
    return v.flatten(-2), scale


def make_latent(kind, reqs, rows=None):
    """A pool of latent rows; (PagedCache, its values in 64 bits [num_blocks * 64, 576])."""
    n = reqs.num_blocks * PAGE
    x = randn(reqs, n, 576) if rows is None else rows
    if kind == "f32":
        return dsa.PagedCache(x.float().view(-1, PAGE, 576)), x.double()
    x = x.bfloat16()
    if kind == "bf16":
        return dsa.PagedCache(x.view(-1, PAGE, 576)), x.double()
    v, s = quantise(x[:, :512], 128)
    data = torch.cat([v.float().to(FP8).view(torch.uint8), x[:, 512:].contiguous().view(torch.uint8)], 1)
    values = torch.cat([v * s.repeat_interleave(128, 1), x[:, 512:].double()], 1)
    return dsa.PagedCache(data.view(-1, PAGE, 640).contiguous(), s.float().view(-1, PAGE, 4).contiguous()), values


def attend(q, values, d_v, tau, limits, kind):
    """Softmax attention of query rows q [m, H, d] over value rows [n, d], row i over the first
    limits[i] of them (0 and -inf where that is none); out, lse and their tolerances."""
    q64 = q.double()
    n = values.shape[0]
    z = torch.einsum("thd,sd->ths", q64, values) * tau
    zabs = torch.einsum("thd,sd->ths", q64.abs(), values.abs()) * tau
    hidden = torch.arange(n, device=q.device)[None, None, :] >= limits[:, None, None]
    z = z.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(z, -1)
    p = torch.where(hidden, 0.0, torch.exp(z - lse[..., None]))
    out = p @ values[:, :d_v]
    A = p @ values[:, :d_v].abs()
    lse_size = torch.where(lse == -math.inf, 0.0, lse.abs())
    E = (zabs * 600 * 2.0 ** -23 + z.masked_fill(hidden, 0.0).abs() * 2.0 ** -22).masked_fill(hidden, 0.0).amax(-1)
    w = 2 * E + 2.0 ** -20
    if kind == "f32":
        return out, lse, (2 * w + 2 * n * 2.0 ** -23)[..., None] * A + 2.0 ** -24 * out.abs(), w + n * 2.0 ** -23 + 2.0 ** -22 * lse_size
    tol = (2 * 2.0 ** -8 + 2 * w + n / 16 * 2.0 ** -23)[..., None] * A + 2.0 ** -8 * out.abs()
    return out, lse, tol, 2.0 ** -8 + w + 2.0 ** -22 * lse_size


def close(got, want, tol, what=""):
    g = got.double()
    bad = ~((g == want) | ((g - want).abs() <= tol))
    if bool(bad.any()):
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError("%s: %d of %d off, first at %s: got %r, want %r, tolerance %.3g" %
                             (what, int(bad.sum()), bad.numel(), i, got[i].item(), want[i].item(), tol[i].item()))


def check_chunk(reqs, q, cache, values, tau, out, lse, kind, d_v=512, tokens=None):
    """The chunk attention's outputs of every request against the definition."""
    start = 0
    for r, n in enumerate(reqs.news):
        if n:
            v = values[reqs.rows(r)]
            for i in range(0, n, 256):
                m = min(256, n - i)
                lim = reqs.ctxs[r] + i + 1 + torch.arange(m, device=q.device)
                s = slice(start + i, start + i + m)
                o, l, to, tl = attend(q[s], v[:reqs.ctxs[r] + i + m], d_v, tau, lim, kind)
                close(out[s], o, to, "out of request %d" % r)
                if lse is not None:
                    close(lse[s], l, tl, "lse of request %d" % r)
        start += n


def run_chunk(reqs, q, cache, tau, d_v=512, with_lse=True, stream=None, fill=7.0):
    T, H = q.shape[:2]
    out = torch.full((T, H, d_v), fill, dtype=q.dtype, device="cuda")
    lse = torch.full((T, H), fill, device="cuda") if with_lse else None
    size = dsa.dsa_chunk_mla_workspace_size(T, len(reqs.news), H, d_v, reqs.max_context)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    dsa.dsa_chunk_mla(q, cache, reqs.chunks(), tau, out, lse, ws, stream)
    return out, lse
