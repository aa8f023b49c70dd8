"""What is measured of the paged-cache operators: quantised append, read-back, chunk attention and
sparse attention over the quantised latent cache.

Geometry: 64-token blocks, shuffled block tables; an indexer key has 128 elements, a latent row 512
latent + 64 RoPE elements.  A quantised latent row holds 512 e4m3 codes and the 64 RoPE elements in
bf16 (640 bytes); each group of 128 codes has a power-of-two f32 scale, the smallest 2^e with
|x| <= 448 * 2^e for the group.  A quantised key row holds 128 codes and one such scale.
"""
import math

import torch

own = False

BLOCK, KEY, LAT, ROPE, GROUP, TOPK = 64, 128, 512, 64, 128, 2048
ROW = LAT + ROPE
FP8 = torch.float8_e4m3fn


def listed():
    return [
        # one decode step of a batch: every request's new token enters both caches
        {"name": "append_decode", "op": "append", "reqs": 64, "new": 1, "spread": 0, "ctx": 4096, "x": "bf16"},
        # the prompts of three requests enter the caches, of odd and unequal lengths
        {"name": "append_prompts", "op": "append", "reqs": 3, "new": 5461, "spread": 1, "ctx": 0, "x": "bf16"},
        # one request's prefix is read back
        {"name": "read_prefix", "op": "read", "reqs": 1, "new": 1000, "spread": 0, "ctx": 0, "cache": "latent_e4m3"},
        # the caches of a whole batch are read back (hand-over to a worker that holds bf16 rows)
        {"name": "read_batch", "op": "read", "reqs": 24, "new": 12000, "spread": 1, "ctx": 0, "cache": "latent_e4m3"},
        # one new token attends densely to a short context: the smallest call
        {"name": "chunk_token", "op": "chunk", "reqs": 1, "new": 1, "spread": 0, "ctx": 2047, "heads": 128, "cache": "latent_e4m3"},
        # four drafted tokens of each request of a batch are checked in one pass
        {"name": "chunk_drafts", "op": "chunk", "reqs": 16, "new": 4, "spread": 0, "ctx": 8000, "heads": 128, "cache": "latent_e4m3"},
        # a prompt's first 2048 tokens: all of them below the top-K, hence dense
        {"name": "chunk_prompt", "op": "chunk", "reqs": 1, "new": 2048, "spread": 0, "ctx": 0, "heads": 128, "cache": "bf16"},
        # odd chunks of several requests, the heads of one GPU of eight
        {"name": "chunk_ragged", "op": "chunk", "reqs": 7, "new": 190, "spread": 1, "ctx": 3777, "heads": 16, "cache": "latent_e4m3"},
        # a chunk late in a long prompt, 64 heads
        {"name": "chunk_late", "op": "chunk", "reqs": 1, "new": 512, "spread": 0, "ctx": 16384, "heads": 64, "cache": "bf16"},
        # decode of one request over its selected rows
        {"name": "sparse_token", "op": "sparse", "reqs": 1, "new": 1, "ctx": 32768, "heads": 128},
        # decode of a batch
        {"name": "sparse_batch", "op": "sparse", "reqs": 64, "new": 1, "ctx": 16384, "heads": 128},
        # a prefill chunk, each query with a selection of its own
        {"name": "sparse_prefill", "op": "sparse", "reqs": 1, "new": 1024, "ctx": 16384, "heads": 64},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "chunk", "sparse"])
    if op == "append":
        reqs = _log(rng, 1, 96)
        return {"op": op, "reqs": reqs, "new": _log(rng, 1, 16384 // reqs), "spread": rng.randint(0, 1),
                "ctx": rng.randint(0, 4096), "x": rng.choice(["bf16", "f32"])}
    if op == "read":
        reqs = _log(rng, 1, 32)
        return {"op": op, "reqs": reqs, "new": _log(rng, 20, 262144 // reqs), "spread": rng.randint(0, 1),
                "ctx": rng.randint(0, 500), "cache": rng.choice(["latent_e4m3", "key_e4m3", "bf16"])}
    if op == "chunk":
        heads = rng.choice([8, 16, 32, 64, 128])
        reqs = _log(rng, 1, 16)
        ctx = _log(rng, 1, 16384)
        return {"op": op, "reqs": reqs, "new": _log(rng, 1, max(1, min(2048, (3 << 26) // (heads * reqs * max(ctx, 2048))))),
                "spread": rng.randint(0, 1), "ctx": ctx, "heads": heads, "cache": rng.choice(["latent_e4m3", "bf16"])}
    if rng.random() < 0.5:
        return {"op": op, "reqs": _log(rng, 1, 96), "new": 1, "ctx": _log(rng, 100, 16384), "heads": rng.choice([64, 128])}
    return {"op": op, "reqs": rng.randint(1, 3), "new": _log(rng, 2, 256), "ctx": _log(rng, 500, 16384),
            "heads": rng.choice([64, 128])}


def _lengths(case):
    """(context before the chunk, new tokens) of each request: plain numbers that follow from the case alone."""
    reqs, new, ctx = case["reqs"], case["new"], case["ctx"]
    ctxs = [ctx if reqs == 1 else ctx * (8 + 9 * r % 25) // 32 for r in range(reqs)]
    news = [new if reqs == 1 or not case.get("spread") else max(1, new * (3 + 7 * r % 11) // 8) for r in range(reqs)]
    return ctxs, news


def _pow2_quantise(x, group):
    """e4m3 codes and power-of-two scales of x [..., n] in groups of `group` elements."""
    g = x.float().unflatten(-1, (-1, group))
    m, e = torch.frexp(g.abs().amax(-1))          # amax = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(-100, 119)
    scale = torch.where(m > 0, ((e + 127) << 23).view(torch.float32), 1.0)  # exactly 2^e
    codes = (g / scale.unsqueeze(-1)).clamp(-448.0, 448.0).to(FP8)
    return codes.flatten(-2), scale


def _latents(n, gen):
    """Latent rows as a normalised projection gives them: unit variance, a few strong channels; RoPE keys are larger."""
    x = torch.randn(n, ROW, generator=gen, device="cuda")
    gain = torch.exp(0.4 * torch.randn(ROW, generator=gen, device="cuda"))
    gain[LAT:] *= 2.0
    return x.mul_(gain)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)
    ctxs, news = _lengths(case)
    reqs, total = len(news), sum(news)
    lens = [c + n for c, n in zip(ctxs, news)]
    blocks = [-(-n // BLOCK) for n in lens]
    nblk = sum(blocks) + 3
    perm = torch.randperm(nblk, generator=gen, device="cuda").to(torch.int32)
    width = max(blocks)
    nb = torch.tensor(blocks, device="cuda")
    first = nb.cumsum(0) - nb
    col = torch.arange(width, device="cuda")
    table = torch.where(col < nb[:, None], perm[(first[:, None] + col).clamp(max=nblk - 1)], -1).to(torch.int32)
    new_t = torch.tensor(news, device="cuda")
    cu = torch.zeros(reqs + 1, dtype=torch.int32, device="cuda")
    cu[1:] = new_t.cumsum(0)
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    req = torch.repeat_interleave(torch.arange(reqs, device="cuda"), new_t)
    pos = torch.arange(total, device="cuda") - cu[req].long() + (seq[req].long() - new_t[req])
    s = {"case": dict(case), "cu": cu, "seq": seq, "table": table, "req": req, "pos": pos, "max_new": max(news),
         "max_len": max(lens), "total": total}
    op = case["op"]
    if op == "append":
        dt = torch.bfloat16 if case["x"] == "bf16" else torch.float32
        s["k"] = torch.randn(total, KEY, generator=gen, device="cuda").to(dt)
        s["kv"] = _latents(total, gen).to(dt)
        # the pools hold other tokens' rows already
        s["key_data"] = torch.randint(0, 120, (nblk, BLOCK, KEY), generator=gen, device="cuda", dtype=torch.uint8)
        s["key_scale"] = torch.full((nblk, BLOCK), 2.0 ** -7, device="cuda")
        s["lat_data"] = torch.randint(0, 63, (nblk, BLOCK, LAT + 2 * ROPE), generator=gen, device="cuda", dtype=torch.uint8)
        s["lat_scale"] = torch.full((nblk, BLOCK, LAT // GROUP), 2.0 ** -7, device="cuda")
        return s
    if op == "read" and case["cache"] == "key_e4m3":
        codes, scale = _pow2_quantise(torch.randn(nblk * BLOCK, KEY, generator=gen, device="cuda").bfloat16(), KEY)
        s["data"] = codes.view(torch.uint8).view(nblk, BLOCK, KEY)
        s["scale"] = scale.view(nblk, BLOCK)
        s["out"] = torch.empty(total, KEY, dtype=torch.bfloat16, device="cuda")
        return s
    rows = _latents(nblk * BLOCK, gen).bfloat16()
    if case.get("cache", "latent_e4m3") == "bf16":
        s["data"], s["scale"] = rows.view(nblk, BLOCK, ROW), None
    else:
        codes, scale = _pow2_quantise(rows[:, :LAT], GROUP)
        s["data"] = torch.cat([codes.view(torch.uint8), rows[:, LAT:].contiguous().view(torch.uint8)], 1).view(nblk, BLOCK, -1)
        s["scale"] = scale.view(nblk, BLOCK, -1)
        del codes, scale
    del rows
    if op == "read":
        s["out"] = torch.empty(total, ROW, dtype=torch.bfloat16, device="cuda")
        return s
    heads = case["heads"]
    s["tau"] = 1.0 / math.sqrt(192.0 if heads != 64 else 256.0)
    # queries whose logits spread over a few units
    s["q"] = torch.randn(total, heads, ROW, generator=gen, device="cuda").bfloat16()
    s["out"] = torch.empty(total, heads, LAT, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty(total, heads, device="cuda")
    s["workspace"] = None
    if op == "sparse":
        # a selection: distinct visible positions, ascending, -1 behind them
        r = torch.rand(total, s["max_len"], generator=gen, device="cuda")
        r.masked_fill_(torch.arange(s["max_len"], device="cuda") > pos[:, None], -1.0)
        got = r.topk(min(TOPK, s["max_len"]), dim=1)
        idx = torch.where(got.values >= 0, got.indices, 1 << 30).sort(1).values
        idx = torch.where(idx == 1 << 30, -1, idx).to(torch.int32)
        s["idx"] = torch.full((total, TOPK), -1, dtype=torch.int32, device="cuda")
        s["idx"][:, :idx.shape[1]] = idx
        s["q_req"], s["q_pos"] = req.to(torch.int32), pos.to(torch.int32)
    return s


def _rows_f32(s, req, pos):
    """Dequantised rows of (request, position) pairs, f32; pairs outside a request's table read row 0."""
    blk = s["table"].long()[req, (pos // BLOCK).clamp(0, s["table"].shape[1] - 1)].clamp(min=0)
    d = s["data"][blk, pos % BLOCK]
    if s["scale"] is None:
        return d.float()
    sc = s["scale"][blk, pos % BLOCK]
    if sc.dim() < d.dim():
        return d.view(FP8).float() * sc.unsqueeze(-1)
    lat = d[..., :LAT].contiguous().view(FP8).float().unflatten(-1, (-1, GROUP)) * sc.unsqueeze(-1)
    return torch.cat([lat.flatten(-2), d[..., LAT:].contiguous().view(torch.bfloat16).float()], -1)


def _softmax_mix(logits, keep, values):
    """softmax over the kept columns, times values; a row that keeps nothing gives 0 and -inf."""
    logits = logits.masked_fill_(~keep, -math.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = logits.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, values) / torch.where(total > 0, total, 1.0)
    return o, (top + total.log()).squeeze(-1)


def _plain(s):
    op = s["case"]["op"]
    if op == "append":
        blk = s["table"].long()[s["req"], s["pos"] // BLOCK]
        off = s["pos"] % BLOCK
        codes, scale = _pow2_quantise(s["k"], KEY)
        s["key_data"][blk, off] = codes.view(torch.uint8)
        s["key_scale"][blk, off] = scale.squeeze(-1)
        codes, scale = _pow2_quantise(s["kv"][:, :LAT], GROUP)
        s["lat_data"][blk, off] = torch.cat([codes.view(torch.uint8), s["kv"][:, LAT:].bfloat16().contiguous().view(torch.uint8)], 1)
        s["lat_scale"][blk, off] = scale
        return
    if op == "read":
        s["out"].copy_(_rows_f32(s, s["req"], s["pos"]))
        return
    q, heads = s["q"].float(), s["q"].shape[1]
    if op == "sparse":
        idx = s["idx"].long()
        rows = _rows_f32(s, s["req"][:, None].expand_as(idx), idx.clamp(min=0))
        o, lse = _softmax_mix(torch.matmul(q, rows.transpose(1, 2)) * s["tau"], (idx >= 0)[:, None, :], rows[..., :LAT])
        s["out"].copy_(o)
        s["lse"].copy_(lse)
        return
    # chunk attention: every request's new tokens side by side, padded to the longest chunk
    reqs, width = s["seq"].numel(), s["max_new"]
    slot = torch.arange(s["total"], device="cuda") - s["cu"].long()[s["req"]]
    padded = q.new_zeros(reqs, width, heads, ROW)
    padded[s["req"], slot] = q
    limit = torch.full((reqs, width), -1, dtype=torch.long, device="cuda")
    limit[s["req"], slot] = s["pos"]
    at = torch.arange(s["max_len"], device="cuda")
    rows = _rows_f32(s, torch.arange(reqs, device="cuda")[:, None].expand(-1, s["max_len"]), at.expand(reqs, -1))
    rows.masked_fill_((at >= s["seq"][:, None])[..., None], 0.0)   # nothing behind a request's last token
    keep = (at <= limit[..., None]).repeat_interleave(heads, 1)
    o, lse = _softmax_mix(torch.matmul(padded.flatten(1, 2), rows.transpose(1, 2)) * s["tau"], keep, rows[..., :LAT])
    s["out"].copy_(o.unflatten(1, (width, heads))[s["req"], slot])
    s["lse"].copy_(lse.unflatten(1, (width, heads))[s["req"], slot])


def _framework(s):
    import sparse_attention_06_b200 as dsa
    op = s["case"]["op"]
    if op == "append":
        chunks = dsa.Chunks(s["cu"], s["seq"], s["table"], s["max_len"])
        dsa.dsa_cache_append(s["k"], s["kv"], dsa.PagedCache(s["key_data"], s["key_scale"]),
                             dsa.PagedCache(s["lat_data"], s["lat_scale"]), chunks)
        return
    cache = dsa.PagedCache(s["data"], s["scale"])
    chunks = dsa.Chunks(s["cu"], s["seq"], s["table"], s["max_len"])
    if op == "read":
        dsa.dsa_cache_read(cache, chunks, s["out"])
        return
    if s["workspace"] is None:  # a program allocates its scratch once
        size = (dsa.dsa_mla_workspace_size(s["total"], s["q"].shape[1], LAT, TOPK) if op == "sparse" else
                dsa.dsa_chunk_mla_workspace_size(s["total"], s["seq"].numel(), s["q"].shape[1], LAT, s["max_len"]))
        s["workspace"] = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    if op == "chunk":
        dsa.dsa_chunk_mla(s["q"], cache, chunks, s["tau"], s["out"], s["lse"], s["workspace"])
        return
    batch = dsa.Batch(s["q_req"], s["q_pos"], s["table"], s["max_len"])
    call = dsa.dsa_sparse_mla_decode if s["case"]["new"] == 1 else dsa.dsa_sparse_mla_prefill
    call(s["q"], cache, batch, s["idx"], s["tau"], s["out"], s["lse"], s["workspace"])


def run(state):
    if own:
        _framework(state)
    else:
        _plain(state)
    if state["case"]["op"] == "append":
        return {"k": state["key_data"].view(FP8), "k_scale": state["key_scale"],
                "latent": state["lat_data"][..., :LAT].view(FP8), "rope": state["lat_data"][..., LAT:].view(torch.bfloat16),
                "latent_scale": state["lat_scale"]}
    if state["case"]["op"] == "read":
        return state["out"]
    return {"out": state["out"], "lse": state["lse"]}


def work(case):
    ctxs, news = _lengths(case)
    total = sum(news)
    q8 = LAT + 2 * ROPE + 4 * (LAT // GROUP)
    if case["op"] == "append":
        size = 2 if case["x"] == "bf16" else 4
        return {"bytes": total * ((KEY + ROW) * size + KEY + 4 + q8), "flops": total * 4 * (KEY + LAT)}
    if case["op"] == "read":
        row, n = {"latent_e4m3": (q8, ROW), "key_e4m3": (KEY + 4, KEY), "bf16": (2 * ROW, ROW)}[case["cache"]]
        return {"bytes": total * (row + 2 * n), "flops": total * n}
    heads = case["heads"]
    ends = total * heads * (2 * ROW + 2 * LAT + 4)
    if case["op"] == "chunk":
        row = q8 if case["cache"] == "latent_e4m3" else 2 * ROW
        pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctxs, news))
        return {"bytes": ends + row * sum(c + n for c, n in zip(ctxs, news)), "flops": 2 * pairs * heads * (ROW + LAT)}
    pairs = sum(min(TOPK, c + i + 1) for c, n in zip(ctxs, news) for i in range(n))
    rows = sum(min(c + n, n * TOPK) for c, n in zip(ctxs, news))
    return {"bytes": ends + 4 * total * TOPK + q8 * rows, "flops": 2 * pairs * heads * (ROW + LAT)}


# the definitions in 64 bits, request by request -----------------------------------------------------------------


def _e4m3_64(x, group):
    """Nearest e4m3 values (ties to even) of x / 2^e, and 2^e, by the format's definition."""
    g = x.double().reshape(*x.shape[:-1], -1, group)
    amax = g.abs().max(-1).values
    e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448.0)).long()
    e = torch.where(448.0 * _two_to(e - 1) >= amax, e - 1, e)
    e = torch.where(448.0 * _two_to(e) < amax, e + 1, e).clamp(-100, 119)
    scale = torch.where(amax > 0, _two_to(e), 1.0)
    y = g / scale[..., None]
    step = _two_to(((y.abs().view(torch.int64) >> 52) - 1023).clamp(min=-6) - 3)
    return (torch.round(y / step) * step).reshape(x.shape), scale


def _two_to(e):
    return ((e + 1023) << 52).view(torch.float64)


def _slots(s, r, lo, hi):
    at = torch.arange(lo, hi, device="cuda")
    return s["table"][r].long()[at // BLOCK], at % BLOCK


def _values64(s, blk, off):
    d = s["data"][blk, off]
    if s["scale"] is None:
        return d.double()
    sc = s["scale"][blk, off].double()
    if sc.dim() == 1:
        return d.view(FP8).double() * sc[:, None]
    lat = d[:, :LAT].contiguous().view(FP8).double() * sc.repeat_interleave(GROUP, 1)
    return torch.hstack([lat, d[:, LAT:].contiguous().view(torch.bfloat16).double()])


def exact(case, seed):
    s = prepare(case, seed)
    ctxs, news = _lengths(case)
    op, reqs = case["op"], len(news)
    starts = [sum(news[:r]) for r in range(reqs + 1)]
    if op == "append":
        k, ks = s["key_data"].view(FP8).double(), s["key_scale"].double()
        lat, rope = s["lat_data"][..., :LAT].view(FP8).double(), s["lat_data"][..., LAT:].view(torch.bfloat16).double()
        ls = s["lat_scale"].double()
        for r in range(reqs):
            blk, off = _slots(s, r, ctxs[r], ctxs[r] + news[r])
            mine = slice(starts[r], starts[r + 1])
            v, sc = _e4m3_64(s["k"][mine], KEY)
            k[blk, off], ks[blk, off] = v, sc[:, 0]
            v, sc = _e4m3_64(s["kv"][mine][:, :LAT], GROUP)
            lat[blk, off], ls[blk, off] = v, sc
            rope[blk, off] = s["kv"][mine][:, LAT:].double()
        return {"k": k, "k_scale": ks, "latent": lat, "rope": rope, "latent_scale": ls}
    if op == "read":
        return torch.vstack([_values64(s, *_slots(s, r, ctxs[r], ctxs[r] + news[r])) for r in range(reqs)])
    heads = case["heads"]
    out = torch.zeros(s["total"], heads, LAT, dtype=torch.float64, device="cuda")
    lse = torch.full((s["total"], heads), -math.inf, dtype=torch.float64, device="cuda")
    if op == "sparse":
        for t in range(s["total"]):
            r = int(torch.searchsorted(s["cu"], t, right=True)) - 1 if reqs > 1 else 0
            at = s["idx"][t][s["idx"][t] >= 0].long()
            if at.numel():
                v = _values64(s, s["table"][r].long()[at // BLOCK], at % BLOCK)
                z = s["q"][t].double() @ v.T * s["tau"]
                lse[t] = torch.logsumexp(z, 1)
                out[t] = torch.exp(z - lse[t][:, None]) @ v[:, :LAT]
        return {"out": out, "lse": lse}
    for r in range(reqs):
        v = _values64(s, *_slots(s, r, 0, ctxs[r] + news[r]))
        for i in range(0, news[r], 64):
            n = min(64, news[r] - i)
            seen = ctxs[r] + i + n
            mine = slice(starts[r] + i, starts[r] + i + n)
            z = torch.einsum("thd,sd->ths", s["q"][mine].double(), v[:seen]) * s["tau"]
            hidden = torch.arange(seen, device="cuda")[None] > (ctxs[r] + i + torch.arange(n, device="cuda"))[:, None]
            z = torch.where(hidden[:, None], -math.inf, z)
            lse[mine] = torch.logsumexp(z, 2)
            out[mine] = torch.einsum("ths,sd->thd", torch.exp(z - lse[mine][..., None]), v[:seen, :LAT])
    return {"out": out, "lse": lse}
