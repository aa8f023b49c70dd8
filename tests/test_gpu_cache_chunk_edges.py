"""Cache and chunk operators where one row, unit or call could reach into another: units that follow each other on a CTA
pair, rows that are skipped, first calls."""
import math

import pytest
import torch

import sparse_attention_06_b200 as dsa
from _cache_chunk import Requests, attend, check_chunk, close, make_latent, quantise, randn, run_chunk

pytestmark = pytest.mark.gpu

TAU = 1.0 / math.sqrt(192.0)


@pytest.fixture(autouse=True)
def _clean_error_word():
    torch.cuda.init()
    dsa.dsa_clear_device_error()
    yield
    dsa.dsa_clear_device_error()


def no_error():
    assert dsa.dsa_get_device_error() == 0


def sparse(reqs, q, cache, idx, rows=slice(None), entry="prefill"):
    """Sparse attention of the chosen queries, each alone on the pool."""
    T, H = q[rows].shape[:2]
    out, lse = torch.empty(T, H, 512, dtype=q.dtype, device="cuda"), torch.empty(T, H, device="cuda")
    batch = dsa.Batch(torch.tensor(reqs.req, dtype=torch.int32, device="cuda")[rows].contiguous(),
                      torch.tensor(reqs.pos, dtype=torch.int32, device="cuda")[rows].contiguous(), reqs.table, reqs.max_context)
    size = dsa.dsa_mla_workspace_size(T, H, 512, idx.shape[1])
    ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    fn = dsa.dsa_sparse_mla_prefill if entry == "prefill" else dsa.dsa_sparse_mla_decode
    fn(q[rows].contiguous(), cache, batch, idx[rows].contiguous(), TAU, out, lse, ws)
    return out, lse


def chosen(reqs, k, seed):
    g = torch.Generator().manual_seed(seed)
    idx = torch.full((reqs.total, k), -1, dtype=torch.int32)
    for t, p in enumerate(reqs.pos):
        n = min(k, p + 1)
        idx[t, :n] = torch.randperm(p + 1, generator=g)[:n].sort().values
    return idx.cuda()


# ------------------------------------------------------------------------------------------ units behind each other


@pytest.mark.parametrize("heads", [128, 64, 20])
@pytest.mark.parametrize("k", [128, 640])
def test_units_behind_each_other_equal_units_alone(heads, k):
    # ten units a CTA pair, short ones among them, bit for bit what one unit a pair gives: no unit's outputs reach
    # into the next one's weights, nor the other way round
    reqs = Requests([700, 0], [700, 40], seed=71 + heads)
    cache, _ = make_latent("q", reqs)
    q = randn(reqs, reqs.total, heads, 576, dtype=torch.bfloat16)
    idx = chosen(reqs, k, 1)
    out, lse = sparse(reqs, q, cache, idx)
    for at in range(0, reqs.total, 60):
        rows = slice(at, min(at + 60, reqs.total))
        o, l = sparse(reqs, q, cache, idx, rows)
        assert torch.equal(out[rows], o) and torch.equal(lse[rows], l), at
    no_error()


@pytest.mark.parametrize("kind", ["q", "bf16"])
def test_prompt_of_many_units_repeats_itself(kind):
    # some seven units a pair, twice each: equal bits, and the definition's values
    reqs = Requests([0, 129, 64], [300, 150, 77], seed=75)
    cache, values = make_latent(kind, reqs)
    q = randn(reqs, reqs.total, 128, 576, dtype=torch.bfloat16)
    a, b = run_chunk(reqs, q, cache, TAU), run_chunk(reqs, q, cache, TAU)
    no_error()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check_chunk(reqs, q, cache, values, TAU, a[0], a[1], kind)


# ------------------------------------------------------------------------------------------ rows that are skipped


def spoil(cache, row, group):
    """A bad scale for one group of a quantised row, and NaN codes under the good scales of the others."""
    cache.scale.view(-1, 4)[row, group] = 0.3
    codes = cache.data.view(-1, 640)[row, :512].view(4, 128)
    codes[[g for g in range(4) if g != group], 5] = 0x7F
    cache.data.view(-1, 640)[row, :512] = codes.flatten()


@pytest.mark.parametrize("group", [0, 1, 2, 3])
@pytest.mark.parametrize("heads", [32, 128])
def test_chunk_skips_the_whole_of_a_bad_row(group, heads):
    # rows of pages of either CTA of a pair, seen by every token and by some, expanded first (128 heads) and not
    reqs = Requests([400], [6], seed=81)
    cache, values = make_latent("q", reqs)
    q = randn(reqs, 6, heads, 576, dtype=torch.bfloat16)
    rows = reqs.rows(0)
    skipped = [10, 70, 200, 300, 403]
    for p in skipped:
        spoil(cache, int(rows[p]), group)
    out, lse = run_chunk(reqs, q, cache, TAU)
    assert dsa.dsa_get_device_error() == dsa.DEVERR_SCALE
    keep = torch.ones(406, dtype=torch.bool, device="cuda")
    keep[skipped] = False
    o, l, to, tl = attend(q, values[rows[keep]], 512, TAU, keep.cumsum(0)[400:], "q")
    close(out, o, to, "out")
    close(lse, l, tl, "lse")


@pytest.mark.parametrize("group", [0, 1, 2, 3])
@pytest.mark.parametrize("heads", [8, 64, 128])
@pytest.mark.parametrize("entry", ["prefill", "decode"])
def test_sparse_skips_the_whole_of_a_bad_row(group, heads, entry):
    # the spoiled rows come in the first, second and last 64 selected rows
    reqs = Requests([500], [2], seed=82)
    cache, values = make_latent("q", reqs)
    q = randn(reqs, 2, heads, 576, dtype=torch.bfloat16)
    idx = chosen(reqs, 200, 3)
    bad = idx[0, [3, 90, 199]].tolist()
    for p in bad:
        spoil(cache, int(reqs.rows(0)[p]), group)
    out, lse = sparse(reqs, q, cache, idx, entry=entry)
    assert dsa.dsa_get_device_error() == dsa.DEVERR_SCALE
    for t in range(2):
        at = torch.tensor([p for p in idx[t].tolist() if p not in bad], device="cuda")
        o, l, to, tl = attend(q[t:t + 1], values[reqs.rows(0)[at]], 512, TAU, torch.tensor([at.numel()], device="cuda"), "q")
        close(out[t:t + 1], o, to, "out")
        close(lse[t:t + 1], l, tl, "lse")


# ------------------------------------------------------------------------------------------ forms of a cache


@pytest.mark.parametrize("tail", [(), (1,)])
def test_key_scales_in_either_shape(tail):
    # [num_blocks, 64] and [num_blocks, 64, 1] are the same array
    reqs = Requests([0, 60], [70, 9], seed=84)
    k = randn(reqs, reqs.total, 128)
    data = torch.zeros(reqs.num_blocks, 64, 128, dtype=torch.uint8, device="cuda")
    scale = torch.ones(reqs.num_blocks, 64, *tail, device="cuda")
    keys = dsa.PagedCache(data, scale)
    dsa.dsa_cache_append(k, None, keys, None, reqs.chunks())
    back = torch.empty(reqs.total, 128, device="cuda")
    dsa.dsa_cache_read(keys, reqs.chunks(), back)
    no_error()
    v, s = quantise(k, 128)
    assert torch.equal(back.double(), v * s)
    q, w = randn(reqs, 1, 64, 128, dtype=torch.bfloat16), torch.ones(1, 64, device="cuda")
    pos = torch.tensor([69], dtype=torch.int32, device="cuda")
    scores = torch.zeros(1, 72, device="cuda")
    dsa.dsa_indexer_scores(q, w, keys, dsa.Batch(torch.zeros_like(pos), pos, reqs.table, 70), scores)
    no_error()
    want = torch.relu(q[0].double() @ (v * s)[:70].T).sum(0)
    # 128 exact products and 64 heads summed in f32; two e4m3 terms carry bf16 queries to 2^-8 relative
    size = (q[0].double().abs() @ (v * s)[:70].T.abs()).sum(0)
    close(scores[0, :70], want, 2.0 ** -8 * size, "scores")


# ------------------------------------------------------------------------------------------ infinite logits


@pytest.mark.parametrize("kind,q_dtype", [("f32", torch.float32), ("q", torch.float32), ("bf16", torch.bfloat16), ("q", torch.bfloat16)])
@pytest.mark.parametrize("at", [0, 2])
def test_a_logit_of_minus_infinity_has_no_weight(kind, q_dtype, at):
    # exp(-inf) = 0 wherever the row comes, the first of all among them; a token that sees nothing else has the sum 0
    reqs = Requests([0], [70], seed=85)
    cache, values = make_latent(kind, reqs)
    q = randn(reqs, 70, 6, 576, dtype=q_dtype)
    q[:, :, 530] = 1.0
    rows = reqs.rows(0)
    if kind == "q":
        cache.data.view(-1, 640)[rows[at]].view(torch.bfloat16)[256 + 530 - 512] = -math.inf
    else:
        cache.data.view(-1, 576)[rows[at], 530] = -math.inf
    out, lse = run_chunk(reqs, q, cache, TAU)
    no_error()
    keep = torch.ones(70, dtype=torch.bool, device="cuda")
    keep[at] = False
    first = 1 if at == 0 else 0
    o, l, to, tl = attend(q[first:], values[rows[keep]], 512, TAU, keep.cumsum(0)[first:], "f32" if q_dtype is torch.float32 else kind)
    close(out[first:], o, to, "out")
    close(lse[first:], l, tl, "lse")
    if at == 0:
        assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())


# ------------------------------------------------------------------------------------------ the normaliser


def fine_tolerances(q, values, limits, tau, out, lse):
    """Bounds for bf16 queries with the normaliser summed from the weights before their rounding to bf16.
    lse: no rounded weights in it, so what moves it is the logits' error, 2 E + 2^-20 as in _cache_chunk.py, the sum
    of n weights in f32 (n partial sums at most, each to 2^-24 of the whole: n * 2^-24) and the final logarithm and its
    sum, 2^-22 * (|lse| + 1).
    out: weights rounded to bf16 once (2^-8 * A, A = sum p |v|), logits (numerator and normaliser: 2 * (2 E + 2^-20) * A),
    accumulation n / 16 * 2^-23 * A and n * 2^-24 * A, and the output's rounding 2^-8 * |out|."""
    n = values.shape[0]
    hidden = torch.arange(n, device=q.device)[None, None, :] >= limits[:, None, None]
    z = torch.einsum("thd,sd->ths", q.double(), values) * tau
    zabs = torch.einsum("thd,sd->ths", q.double().abs(), values.abs()) * tau
    E = (zabs * 600 * 2.0 ** -23 + z.abs() * 2.0 ** -22).masked_fill(hidden, 0.0).amax(-1)
    w = 2 * E + 2.0 ** -20
    p = torch.where(hidden, 0.0, torch.exp(z - lse[..., None]))
    A = p @ values[:, :512].abs()
    return ((2.0 ** -8 + 2 * w + n / 16 * 2.0 ** -23 + n * 2.0 ** -24)[..., None] * A + 2.0 ** -8 * out.abs(),
            w + n * 2.0 ** -24 + 2.0 ** -22 * (lse.abs() + 1))


@pytest.mark.parametrize("kind", ["q", "bf16"])
@pytest.mark.parametrize("ctx,new,heads", [(0, 90, 16), (2047, 1, 128), (3000, 5, 64), (700, 200, 24), (9000, 2, 128)])
def test_chunk_normaliser_sums_unrounded_weights(kind, ctx, new, heads):
    reqs = Requests([ctx, 130], [new, 3], seed=86 + ctx)
    cache, values = make_latent(kind, reqs)
    # logits of a few tenths: every key counts, so that a lost or rounded weight shows
    q = (randn(reqs, reqs.total, heads, 576) * 0.2).bfloat16()
    out, lse = run_chunk(reqs, q, cache, TAU)
    no_error()
    start = 0
    for r, n in enumerate(reqs.news):
        v, s = values[reqs.rows(r)], slice(start, start + n)
        limits = reqs.ctxs[r] + 1 + torch.arange(n, device="cuda")
        o, l, _, _ = attend(q[s], v, 512, TAU, limits, kind)
        to, tl = fine_tolerances(q[s], v, limits, TAU, o, l)
        close(out[s], o, to, "out of request %d" % r)
        close(lse[s], l, tl, "lse of request %d" % r)
        start += n


@pytest.mark.parametrize("heads", [128, 64, 12])
@pytest.mark.parametrize("entry", ["prefill", "decode"])
def test_sparse_normaliser_sums_unrounded_weights(heads, entry):
    reqs = Requests([3000], [3], seed=87)
    cache, values = make_latent("q", reqs)
    q = (randn(reqs, 3, heads, 576) * 0.2).bfloat16()
    idx = chosen(reqs, 2048, 4)
    out, lse = sparse(reqs, q, cache, idx, entry=entry)
    no_error()
    for t in range(3):
        v = values[reqs.rows(0)[idx[t].long()]]
        limits = torch.tensor([2048], device="cuda")
        o, l, _, _ = attend(q[t:t + 1], v, 512, TAU, limits, "q")
        to, tl = fine_tolerances(q[t:t + 1], v, limits, TAU, o, l)
        close(out[t:t + 1], o, to, "out")
        close(lse[t:t + 1], l, tl, "lse")


# ------------------------------------------------------------------------------------------ calls behind each other


@pytest.mark.parametrize("heads", [128, 16])
def test_calls_behind_each_other_see_what_the_last_one_wrote(heads):
    # one graph of 48 decode steps with nothing between the calls: the token's row is written, attended to densely and by
    # selection, and read back, next to rows (and scales, in the same sectors) that the step before has read
    steps, ctx = 48, 150
    reqs = Requests([ctx + steps - 1], [1], seed=88)
    cache, _ = make_latent("q", reqs)
    fresh = (cache.data.clone(), cache.scale.clone())
    kv = randn(reqs, steps, 576, dtype=torch.bfloat16)
    q = randn(reqs, steps, heads, 576, dtype=torch.bfloat16)
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    lens = [torch.tensor([ctx + i + 1], dtype=torch.int32, device="cuda") for i in range(steps)]
    chunks = [dsa.Chunks(one, n, reqs.table, reqs.max_context) for n in lens]
    batches = [dsa.Batch(one[:1], n - 1, reqs.table, reqs.max_context) for n in lens]
    idx = torch.full((steps, 256), -1, dtype=torch.int32)
    for i in range(steps):
        idx[i, :100] = torch.arange(ctx + i + 1 - 100, ctx + i + 1)
    idx = idx.cuda()
    dense, some = (torch.zeros(steps, heads, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lse, lse2 = (torch.zeros(steps, heads, device="cuda") for _ in range(2))
    back = torch.zeros(steps, 576, dtype=torch.bfloat16, device="cuda")
    size = max(dsa.dsa_chunk_mla_workspace_size(1, 1, heads, 512, reqs.max_context), dsa.dsa_mla_workspace_size(1, heads, 512, 256), 1)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def step(i):
        s = slice(i, i + 1)
        dsa.dsa_cache_append(None, kv[s], None, cache, chunks[i])
        dsa.dsa_chunk_mla(q[s], cache, chunks[i], TAU, dense[s], lse[s], ws)
        dsa.dsa_sparse_mla_decode(q[s], cache, batches[i], idx[s], TAU, some[s], lse2[s], ws)
        dsa.dsa_cache_read(cache, chunks[i], back[s])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(0)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(steps):
            step(i)
    v, s = quantise(kv[:, :512], 128)
    new = torch.cat([v * s.repeat_interleave(128, 1), kv[:, 512:].double()], 1)
    for _ in range(5):
        # the rows to come hold other values until their step writes them
        cache.data.copy_(fresh[0])
        cache.scale.copy_(fresh[1])
        before = torch.empty(ctx, 576, dtype=torch.float32, device="cuda")
        dsa.dsa_cache_read(cache, dsa.Chunks(torch.tensor([0, ctx], dtype=torch.int32, device="cuda"),
                                             torch.tensor([ctx], dtype=torch.int32, device="cuda"), reqs.table, reqs.max_context), before)
        values = torch.cat([before.double(), new])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(back.double(), new)
        o, l, to, tl = attend(q, values, 512, TAU, ctx + 1 + torch.arange(steps, device="cuda"), "q")
        close(dense, o, to, "dense")
        close(lse, l, tl, "lse, dense")
        for i in range(steps):
            o, l, to, tl = attend(q[i:i + 1], values[ctx + i + 1 - 100:ctx + i + 1], 512, TAU, torch.tensor([100], device="cuda"), "q")
            close(some[i:i + 1], o, to, "selected")
            close(lse2[i:i + 1], l, tl, "lse, selected")
    no_error()


# ------------------------------------------------------------------------------------------ calls the documentation allows


@pytest.mark.parametrize("dim", [1, 7, 64, 100, 200, 256])
@pytest.mark.parametrize("kind", ["e4m3", "bf16", "f32"])
@pytest.mark.parametrize("x_dtype", [torch.bfloat16, torch.float32])
def test_keys_of_other_widths(dim, kind, x_dtype):
    reqs = Requests([0, 63, 100], [5, 70, 1], seed=90 + dim, pad=2)
    k = (randn(reqs, reqs.tokens, dim) * torch.exp(4 * randn(reqs, reqs.tokens, 1))).to(x_dtype)
    dt = {"e4m3": torch.uint8, "bf16": torch.bfloat16, "f32": torch.float32}[kind]
    keys = dsa.PagedCache(torch.zeros(reqs.num_blocks, 64, dim, dtype=dt, device="cuda"),
                          torch.ones(reqs.num_blocks, 64, device="cuda") if kind == "e4m3" else None)
    dsa.dsa_cache_append(k, None, keys, None, reqs.chunks())
    back = torch.full((reqs.tokens, dim), 7.0, device="cuda")
    dsa.dsa_cache_read(keys, reqs.chunks(), back)
    no_error()
    n = reqs.total
    if kind == "e4m3":
        v, s = quantise(k[:n], dim)
        want = v * s
    else:
        want = k[:n].to(dt).double()
    assert torch.equal(back[:n].double(), want) and bool((back[n:] == 7.0).all())


@pytest.mark.parametrize("kind", ["q", "bf16"])
@pytest.mark.parametrize("heads", [3, 200, 1024])
def test_chunk_rows_in_front_empty_requests_and_a_loose_bound(kind, heads):
    # rows before the first request belong to none; requests without tokens anywhere; max_context above every length
    reqs = Requests([70, 5, 0, 200], [0, 3, 9, 0], seed=91, pad=1)
    cache, values = make_latent(kind, reqs)
    table = torch.full((4, 20), -1, dtype=torch.int32, device="cuda")
    table[:, :reqs.table.shape[1]] = reqs.table
    lead, T = 2, reqs.tokens + 2
    q = randn(reqs, T, heads, 576, dtype=torch.bfloat16)
    out, lse = torch.full((T, heads, 512), 7.0, dtype=q.dtype, device="cuda"), torch.full((T, heads), 7.0, device="cuda")
    size = dsa.dsa_chunk_mla_workspace_size(T, 4, heads, 512, 1280)
    ws = torch.full((max(size, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    dsa.dsa_chunk_mla(q, cache, dsa.Chunks(reqs.cu + lead, reqs.seq, table, 1280), TAU, out, lse, ws)
    no_error()
    check_chunk(reqs, q[lead:], cache, values, TAU, out[lead:], lse[lead:], kind)
    for x in (out, lse):
        assert bool((x[:lead] == 7.0).all()) and bool((x[lead + reqs.total:] == 7.0).all())


@pytest.mark.parametrize("heads", [7, 64, 128])
@pytest.mark.parametrize("k", [1, 37, 300])
@pytest.mark.parametrize("entry", ["prefill", "decode"])
def test_sparse_selections_in_any_order_with_repeats(heads, k, entry):
    # a position selected twice counts twice; -1 may stand anywhere
    reqs = Requests([0, 400], [3, 4], seed=92)
    cache, values = make_latent("q", reqs)
    q = randn(reqs, reqs.total, heads, 576, dtype=torch.bfloat16)
    g = torch.Generator().manual_seed(k)
    idx = torch.stack([torch.randint(0, p + 1, (k,), generator=g) for p in reqs.pos]).to(torch.int32)
    idx[torch.rand(idx.shape, generator=g) < 0.3] = -1
    idx = idx.cuda()
    out, lse = sparse(reqs, q, cache, idx, entry=entry)
    no_error()
    for t in range(reqs.total):
        at = idx[t][idx[t] >= 0].long()
        if not at.numel():
            assert bool((out[t] == 0).all()) and bool((lse[t] == -math.inf).all())
            continue
        v = values[reqs.rows(reqs.req[t])[at]]
        o, l, to, tl = attend(q[t:t + 1], v, 512, TAU, torch.tensor([at.numel()], device="cuda"), "q")
        close(out[t:t + 1], o, to, "out")
        close(lse[t:t + 1], l, tl, "lse")
