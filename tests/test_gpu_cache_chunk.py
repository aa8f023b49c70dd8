"""The cache operators (append with quantisation, read-back), chunk attention and sparse attention over
the quantised latent cache, against their definitions in 64 bits."""
import math

import pytest
import torch

import sparse_attention_06_b200 as dsa
from _cache_chunk import FP8, PAGE, Requests, attend, check_chunk, close, make_latent, pow2, quantise, randn, run_chunk

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


# ------------------------------------------------------------------------------------------ append and read


def empty_caches(key_kind, lat_kind, nb):
    """Caches full of a marker byte, so that a row that was not to be written shows."""
    def raw(*shape):
        return torch.full(shape, 0x55, dtype=torch.uint8, device="cuda")
    kd = {"e4m3": (torch.uint8, 1), "bf16": (torch.bfloat16, 2), "f32": (torch.float32, 4)}
    dt, size = kd[key_kind]
    keys = dsa.PagedCache(raw(nb, PAGE, 128 * size).view(dt),
                          raw(nb, PAGE, 4).view(torch.float32).squeeze(-1) if key_kind == "e4m3" else None)
    if lat_kind == "q":
        lat = dsa.PagedCache(raw(nb, PAGE, 640), raw(nb, PAGE, 16).view(torch.float32))
    else:
        dt, size = kd[lat_kind]
        lat = dsa.PagedCache(raw(nb, PAGE, 576 * size).view(dt))
    return keys, lat


def raw_rows(t):
    return t.contiguous().view(torch.uint8).view(t.shape[0] * t.shape[1], -1)


def bits_equal(got, want, what):
    """Equal values, NaN equal to NaN, and zeros of the same sign."""
    g, w = got.double(), want.double()
    same = (g == w) & (torch.signbit(g) == torch.signbit(w)) | (g.isnan() & w.isnan())
    assert bool(same.all()), what


def check_appended(reqs, k, kv, keys, lat, key_kind, lat_kind):
    rows = reqs.token_rows()
    others = torch.ones(reqs.num_blocks * PAGE, dtype=torch.bool, device="cuda")
    others[rows] = False
    for c, quant in ((keys, key_kind == "e4m3"), (lat, lat_kind == "q")):
        assert bool((raw_rows(c.data)[others] == 0x55).all())
        if quant:
            s = c.scale if c.scale.dim() == 3 else c.scale.unsqueeze(-1)
            assert bool((raw_rows(s)[others] == 0x55).all())
    n = reqs.total
    if key_kind == "e4m3":
        v, s = quantise(k[:n], 128)
        bits_equal(keys.data.view(-1, 128).view(FP8)[rows], v, "key codes")
        bits_equal(keys.scale.view(-1)[rows], s.squeeze(-1), "key scales")
    else:
        bits_equal(keys.data.view(-1, 128)[rows], k[:n].to(keys.data.dtype), "keys")
    if lat_kind == "q":
        v, s = quantise(kv[:n, :512], 128)
        row = lat.data.view(-1, 640)[rows]
        bits_equal(row[:, :512].contiguous().view(FP8), v, "latent codes")
        bits_equal(lat.scale.view(-1, 4)[rows], s, "latent scales")
        bits_equal(row[:, 512:].contiguous().view(torch.bfloat16), kv[:n, 512:].bfloat16(), "RoPE part")
    else:
        bits_equal(lat.data.view(-1, 576)[rows], kv[:n].to(lat.data.dtype), "latents")


@pytest.mark.parametrize("x_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("key_kind,lat_kind", [("e4m3", "q"), ("bf16", "bf16"), ("f32", "f32"), ("e4m3", "bf16"), ("bf16", "q")])
@pytest.mark.parametrize("layout", ["dense", "slice", "odd"])
def test_append(x_dtype, key_kind, lat_kind, layout):
    # requests that start, cross and end at page borders; one without new tokens; rows behind the last
    reqs = Requests([0, 63, 64, 130, 200, 1], [1, 1, 64, 0, 57, 129], seed=3, pad=5)
    wide = {"dense": 0, "slice": 64, "odd": 3}[layout]
    k = randn(reqs, reqs.tokens, 128 + wide, dtype=x_dtype)[:, wide:]
    kv = (randn(reqs, reqs.tokens, 576 + wide) * torch.exp(3 * randn(reqs, 1, 576 + wide))).to(x_dtype)[:, wide:]
    keys, lat = empty_caches(key_kind, lat_kind, reqs.num_blocks)
    dsa.dsa_cache_append(k, kv, keys, lat, reqs.chunks())
    no_error()
    check_appended(reqs, k, kv, keys, lat, key_kind, lat_kind)


def test_append_one_cache_at_a_time():
    reqs = Requests([5], [70], seed=4)
    k, kv = randn(reqs, 70, 128), randn(reqs, 70, 576)
    keys, lat = empty_caches("e4m3", "q", reqs.num_blocks)
    dsa.dsa_cache_append(k, None, keys, None, reqs.chunks())
    assert bool((raw_rows(lat.data) == 0x55).all())
    dsa.dsa_cache_append(None, kv, None, lat, reqs.chunks())
    no_error()
    check_appended(reqs, k, kv, keys, lat, "e4m3", "q")


@pytest.mark.parametrize("x_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("aligned", [True, False])
def test_append_magnitudes(x_dtype, aligned):
    # groups of zeros, of the smallest and largest numbers, at both sides of every border of a scale,
    # and ties between codes
    reqs = Requests([0], [40], seed=5)
    off = 0 if aligned else 1
    kv = torch.zeros(40, 577, device="cuda")
    base = randn(reqs, 40, 576)
    mags = [0.0, 2.0 ** -149, 2.0 ** -133, 2.0 ** -126, 2.0 ** -110, 2.0 ** -100, 2.0 ** -92, 2.0 ** -91, 1e-20, 448.0,
            448.0 * (1 + 2.0 ** -7), 449.0, 1.0, 3e38, 1e30, 2.0 ** 120]
    kv[:16, :576] = base[:16].clamp(-1, 1) * torch.tensor(mags, device="cuda")[:, None]
    kv[9, :] = 448.0
    kv[10, :] = 448.0 * (1 + 2.0 ** -7)
    kv[16:, :576] = torch.arange(24 * 576, device="cuda").view(24, 576).float() / 64.0 - 100.0   # many exact ties
    kv = kv.to(x_dtype)
    src = torch.zeros(40, 577, device="cuda", dtype=x_dtype)
    src[:, off:off + 576] = kv[:, :576]
    x = src[:, off:off + 576] if not aligned else kv[:, :576].contiguous()
    keys, lat = empty_caches("e4m3", "q", reqs.num_blocks)
    dsa.dsa_cache_append(x[:, :128], x, keys, lat, reqs.chunks())
    no_error()
    check_appended(reqs, x[:, :128], x, keys, lat, "e4m3", "q")


@pytest.mark.parametrize("aligned", [True, False])
def test_append_nonfinite(aligned):
    reqs = Requests([0], [6], seed=6)
    off = 0 if aligned else 1
    kv = torch.zeros(6, 580, device="cuda")[:, off:off + 576]
    kv.copy_(randn(reqs, 6, 576))
    kv[1, 3], kv[2, 200], kv[3, 511], kv[4, 128:256] = math.nan, math.inf, -math.inf, math.nan
    keys, lat = empty_caches("e4m3", "q", reqs.num_blocks)
    dsa.dsa_cache_append(None, kv, None, lat, reqs.chunks())
    assert dsa.dsa_get_device_error() == dsa.DEVERR_NONFINITE
    rows = reqs.token_rows()
    v, s = quantise(kv[:, :512], 128)
    bits_equal(lat.data.view(-1, 640)[rows][:, :512].contiguous().view(FP8), v, "codes")
    bits_equal(lat.scale.view(-1, 4)[rows], s, "scales")
    # unquantised caches and RoPE elements keep what they are given
    dsa.dsa_clear_device_error()
    kv[0, 540] = math.inf
    _, plain = empty_caches("bf16", "f32", reqs.num_blocks)
    dsa.dsa_cache_append(None, kv, None, plain, reqs.chunks())
    no_error()
    bits_equal(plain.data.view(-1, 576)[rows], kv, "f32 latents")


def test_append_bad_pages_and_requests():
    reqs = Requests([0, 0, 0], [100, 30, 30], seed=7)
    k, kv = randn(reqs, 160, 128), randn(reqs, 160, 576)
    keys, lat = empty_caches("e4m3", "q", reqs.num_blocks)
    good = reqs.table.clone()
    reqs.table[0, 1] = reqs.num_blocks          # tokens 64..99 of request 0 have no page
    reqs.table[1, 0] = -1
    dsa.dsa_cache_append(k, kv, keys, lat, reqs.chunks())
    assert dsa.dsa_get_device_error() == dsa.DEVERR_BLOCK_ID
    reqs.table.copy_(good)
    written = torch.cat([reqs.rows(0, 0, 64), reqs.rows(2)])
    mask = torch.zeros(reqs.num_blocks * PAGE, dtype=torch.bool, device="cuda")
    mask[written] = True
    assert bool((raw_rows(lat.data)[~mask] == 0x55).all()) and bool((raw_rows(keys.data)[~mask] == 0x55).all())
    src = torch.cat([torch.arange(64), torch.arange(130, 160)]).cuda()
    bits_equal(lat.data.view(-1, 640)[written][:, :512].contiguous().view(FP8), quantise(kv[src, :512], 128)[0], "codes")
    # lengths outside the call's bounds
    for lens in ([reqs.max_context + 1, 30, 30], [99, 30, 30], [-5, 30, 30]):
        dsa.dsa_clear_device_error()
        keys, lat = empty_caches("e4m3", "q", reqs.num_blocks)
        reqs.seq.copy_(torch.tensor(lens, dtype=torch.int32))
        dsa.dsa_cache_append(k, kv, keys, lat, reqs.chunks())
        assert dsa.dsa_get_device_error() == dsa.DEVERR_REQUEST
        mask = torch.zeros(reqs.num_blocks * PAGE, dtype=torch.bool, device="cuda")
        mask[torch.cat([reqs.rows(1), reqs.rows(2)])] = True
        assert bool((raw_rows(lat.data)[~mask] == 0x55).all())
        bits_equal(lat.data.view(-1, 640)[reqs.rows(2)][:, :512].contiguous().view(FP8), quantise(kv[130:, :512], 128)[0], "codes")


@pytest.mark.parametrize("kind", ["q", "e4m3", "bf16", "f32"])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_read(kind, out_dtype):
    reqs = Requests([0, 63, 64, 130, 3], [1, 1, 64, 0, 129], seed=8, pad=4)
    if kind == "e4m3":
        n = reqs.num_blocks * PAGE
        codes = torch.randint(0, 256, (n, 128), generator=reqs.gen, dtype=torch.uint8).cuda()
        codes[(codes & 0x7F) == 0x7F] = 0
        scale = torch.rand(n, generator=reqs.gen).cuda() + 0.01     # any positive scale
        cache = dsa.PagedCache(codes.view(-1, PAGE, 128), scale.view(-1, PAGE))
        values = codes.view(FP8).double() * scale.double()[:, None]
    else:
        cache, values = make_latent(kind, reqs)
    dim = values.shape[1]
    out = torch.full((reqs.tokens, dim), 7.0, dtype=out_dtype, device="cuda")
    dsa.dsa_cache_read(cache, reqs.chunks(), out)
    no_error()
    want = values[reqs.token_rows()]
    # f32: code * scale is rounded once (e4m3); bf16: that and one more rounding
    rel = {("e4m3", torch.float32): 2.0 ** -24, ("e4m3", torch.bfloat16): 2.0 ** -8 + 2.0 ** -23,
           ("f32", torch.bfloat16): 2.0 ** -8}.get((kind, out_dtype), 0.0)
    close(out[:reqs.total], want, rel * want.abs(), "read")
    assert bool((out[reqs.total:] == 7.0).all())


def test_read_every_code_at_the_ends_of_the_scale_range():
    # a quantised row's 256 codes (NaN among them), and scales 2^-100, 2^7, 2^8 and 2^119
    reqs = Requests([0], [4], seed=9)
    cache, _ = make_latent("q", reqs)
    rows = reqs.token_rows()
    codes = torch.arange(512, device="cuda").remainder(256).to(torch.uint8)
    codes = codes.view(4, 128).repeat(1, 1).flatten()
    cache.data.view(-1, 640)[rows, :512] = codes
    e = torch.tensor([[-100, 119, 7, 8], [119, -100, 0, -7], [8, 7, 119, -100], [0, 1, -100, 119]], device="cuda")
    cache.scale.view(-1, 4)[rows] = pow2(e).float()
    want = codes.view(FP8).double()[None] * pow2(e).repeat_interleave(128, 1)
    for dt in (torch.bfloat16, torch.float32):
        out = torch.empty(4, 576, dtype=dt, device="cuda")
        dsa.dsa_cache_read(cache, reqs.chunks(), out)
        bits_equal(out[:, :512], want, str(dt))
    no_error()


def test_read_bad_page_leaves_the_row():
    reqs = Requests([0], [70], seed=10)
    cache, values = make_latent("q", reqs)
    rows = reqs.token_rows()
    reqs.table[0, 1] = 1 << 20
    out = torch.full((70, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_cache_read(cache, reqs.chunks(), out)
    assert dsa.dsa_get_device_error() == dsa.DEVERR_BLOCK_ID
    assert bool((out[64:] == 7.0).all())
    bits_equal(out[:64], values[rows[:64]], "rows with a page")


# ------------------------------------------------------------------------------------------ chunk attention


@pytest.mark.parametrize("kind", ["q", "bf16"])
@pytest.mark.parametrize("heads", [1, 5, 16, 64, 96, 128, 160])
def test_chunk_ragged(kind, heads):
    # one-token chunks, chunks that start and end at page borders, a request without new tokens,
    # prompts from position 0, rows behind the last request
    reqs = Requests([0, 63, 64, 130, 700, 1, 0], [1, 1, 64, 0, 37, 3, 150], seed=heads, pad=3)
    cache, values = make_latent(kind, reqs)
    q = randn(reqs, reqs.tokens, heads, 576, dtype=torch.bfloat16)
    out, lse = run_chunk(reqs, q, cache, TAU)
    no_error()
    check_chunk(reqs, q, cache, values, TAU, out, lse, kind)
    assert bool((out[reqs.total:] == 7.0).all()) and bool((lse[reqs.total:] == 7.0).all())


@pytest.mark.parametrize("kind", ["q", "bf16"])
@pytest.mark.parametrize("ctx,new,heads", [(0, 1, 128), (1, 1, 128), (2047, 1, 128), (62, 1, 16), (63, 1, 16), (64, 1, 8), (127, 2, 64),
                                           (5000, 4, 128), (9001, 3, 8), (0, 300, 128), (300, 5, 24)])
def test_chunk_one_request(kind, ctx, new, heads):
    reqs = Requests([ctx], [new], seed=ctx + heads)
    cache, values = make_latent(kind, reqs)
    q = randn(reqs, new, heads, 576, dtype=torch.bfloat16)
    out, lse = run_chunk(reqs, q, cache, TAU)
    no_error()
    check_chunk(reqs, q, cache, values, TAU, out, lse, kind)
    out2, _ = run_chunk(reqs, q, cache, TAU, with_lse=False)
    assert torch.equal(out, out2)


@pytest.mark.parametrize("kind", ["q", "bf16"])
def test_chunk_many_requests(kind):
    # more requests than a warp has lanes, lengths from nothing to several pages
    news = [(7 * r) % 5 for r in range(83)]
    ctxs = [(37 * r) % 400 for r in range(83)]
    reqs = Requests(ctxs, news, seed=21, pad=1)
    cache, values = make_latent(kind, reqs)
    q = randn(reqs, reqs.tokens, 16, 576, dtype=torch.bfloat16)
    out, lse = run_chunk(reqs, q, cache, TAU)
    no_error()
    check_chunk(reqs, q, cache, values, TAU, out, lse, kind)


@pytest.mark.parametrize("kind,q_dtype", [("f32", torch.float32), ("q", torch.float32)])
def test_chunk_f32_queries(kind, q_dtype):
    reqs = Requests([0, 70], [20, 3], seed=22, pad=1)
    cache, values = make_latent(kind, reqs)
    q = randn(reqs, reqs.tokens, 6, 576, dtype=q_dtype)
    out, lse = run_chunk(reqs, q, cache, TAU)
    no_error()
    check_chunk(reqs, q, cache, values, TAU, out, lse, "f32")
    assert bool((out[reqs.total:] == 7.0).all())


@pytest.mark.parametrize("d_v,d_rope", [(32, 16), (48, 0), (640, 8)])
def test_chunk_other_widths(d_v, d_rope):
    reqs = Requests([10, 100], [9, 4], seed=23)
    n = reqs.num_blocks * PAGE
    rows = randn(reqs, n, d_v + d_rope)
    cache = dsa.PagedCache(rows.view(-1, PAGE, d_v + d_rope))
    q = randn(reqs, reqs.total, 3, d_v + d_rope)
    out, lse = run_chunk(reqs, q, cache, 0.2, d_v=d_v)
    no_error()
    check_chunk(reqs, q, cache, rows.double(), 0.2, out, lse, "f32", d_v=d_v)


@pytest.mark.parametrize("kind", ["q", "bf16"])
@pytest.mark.parametrize("gain", [40.0, 0.001])
def test_chunk_logit_ranges(kind, gain):
    # softmaxes of one row (the maximum moves all the time) and nearly uniform ones
    reqs = Requests([900], [40], seed=24)
    cache, values = make_latent(kind, reqs)
    q = (randn(reqs, 40, 16, 576) * gain).bfloat16()
    out, lse = run_chunk(reqs, q, cache, TAU)
    no_error()
    check_chunk(reqs, q, cache, values, TAU, out, lse, kind)


def poison(cache, row, kind, part):
    """NaN, or an infinity where the cache can hold one, in pool row `row`."""
    if kind == "q":
        if part == "latent":
            cache.data.view(-1, 640)[row, 77] = 0x7F
        else:
            cache.data.view(-1, 640)[row].view(torch.bfloat16)[256 + 10] = math.nan
    else:
        cache.data.view(-1, 576)[row, 77 if part == "latent" else 530] = math.nan


@pytest.mark.parametrize("kind", ["q", "bf16"])
@pytest.mark.parametrize("heads", [128, 16, 1])
@pytest.mark.parametrize("part", ["latent", "rope"])
def test_chunk_nan_reaches_only_who_sees_it(kind, heads, part):
    # NaN behind the last token of a page, in every unused page, and in the row of the chunk's 20th token
    reqs = Requests([100], [30], seed=25)
    cache, values = make_latent(kind, reqs)
    q = randn(reqs, 30, heads, 576, dtype=torch.bfloat16)
    used = torch.zeros(reqs.num_blocks * PAGE, dtype=torch.bool, device="cuda")
    used[reqs.rows(0)] = True
    for row in (~used).nonzero().flatten().tolist():
        poison(cache, row, kind, "latent")
        poison(cache, row, kind, "rope")
    if kind == "q":
        cache.scale.view(-1, 4)[~used] = math.nan
    out, lse = run_chunk(reqs, q, cache, TAU)
    no_error()
    check_chunk(reqs, q, cache, values, TAU, out, lse, kind)
    poison(cache, int(reqs.rows(0, 119, 120)), kind, part)
    out2, lse2 = run_chunk(reqs, q, cache, TAU)
    no_error()
    assert torch.equal(out[:19], out2[:19]) and torch.equal(lse[:19], lse2[:19])
    assert bool(out2[19:].isnan().all()) and bool(lse2[19:].isnan().all())


@pytest.mark.parametrize("heads", [128, 16])
def test_chunk_infinity_hidden_from_earlier_tokens(heads):
    reqs = Requests([64], [40], seed=26)
    cache, values = make_latent("bf16", reqs)
    q = randn(reqs, 40, heads, 576, dtype=torch.bfloat16)
    out, lse = run_chunk(reqs, q, cache, TAU)
    cache.data.view(-1, 576)[reqs.rows(0, 64 + 25, 64 + 26), 5] = math.inf
    out2, lse2 = run_chunk(reqs, q, cache, TAU)
    no_error()
    assert torch.equal(out[:25], out2[:25]) and torch.equal(lse[:25], lse2[:25])


@pytest.mark.parametrize("kind", ["q", "bf16"])
@pytest.mark.parametrize("heads", [16, 128])
def test_chunk_bad_page_is_skipped(kind, heads):
    reqs = Requests([200, 0], [10, 5], seed=27)
    cache, values = make_latent(kind, reqs)
    q = randn(reqs, 15, heads, 576, dtype=torch.bfloat16)
    keep = torch.cat([torch.arange(0, 64), torch.arange(128, 210)]).cuda()
    rows = reqs.rows(0)
    reqs.table[0, 1] = reqs.num_blocks + 5
    reqs.table[1, 0] = -7                       # the second request has no page at all
    out, lse = run_chunk(reqs, q, cache, TAU)
    assert dsa.dsa_get_device_error() == dsa.DEVERR_BLOCK_ID
    lim = 64 + 73 + torch.arange(10, device="cuda")
    o, l, to, tl = attend(q[:10], values[rows[keep]], 512, TAU, lim, kind)
    close(out[:10], o, to, "out")
    close(lse[:10], l, tl, "lse")
    assert bool((out[10:] == 0).all()) and bool((lse[10:] == -math.inf).all())


@pytest.mark.parametrize("bad", [0.3, -0.125, 2.0 ** -101, 2.0 ** 120, math.inf, math.nan, 0.0])
def test_chunk_bad_scale_is_skipped(bad):
    reqs = Requests([70], [6], seed=28)
    cache, values = make_latent("q", reqs)
    q = randn(reqs, 6, 32, 576, dtype=torch.bfloat16)
    rows = reqs.rows(0)
    cache.scale.view(-1, 4)[rows[30], 2] = bad
    cache.scale.view(-1, 4)[rows[72], 0] = bad  # a row that some of the tokens do not see
    out, lse = run_chunk(reqs, q, cache, TAU)
    assert dsa.dsa_get_device_error() == dsa.DEVERR_SCALE
    keep = torch.ones(76, dtype=torch.bool, device="cuda")
    keep[30] = keep[72] = False
    lim = torch.tensor([70, 71, 71, 72, 73, 74], device="cuda")
    o, l, to, tl = attend(q, values[rows[keep]], 512, TAU, lim, "q")
    close(out, o, to, "out")
    close(lse, l, tl, "lse")


def test_chunk_scale_range():
    # values from 2^-109 to 448 * 2^100 (beyond 2^109 the f32 accumulators, which hold sums of
    # weights of up to 2^8 times values, may overflow)
    reqs = Requests([100], [4], seed=29)
    cache, values = make_latent("q", reqs)
    n = reqs.num_blocks * PAGE
    e = torch.randint(-100, 101, (n, 4), generator=reqs.gen).cuda()
    scale = pow2(e)
    old = cache.scale.view(-1, 4).double()
    values[:, :512] = values[:, :512] / old.repeat_interleave(128, 1) * scale.repeat_interleave(128, 1)
    cache.scale.view(-1, 4).copy_(scale)
    # queries that see the RoPE part only, so that the logits stay ordinary
    q = randn(reqs, 4, 16, 576, dtype=torch.bfloat16)
    q[:, :, :512] = 0
    out, lse = run_chunk(reqs, q, cache, TAU)
    no_error()
    check_chunk(reqs, q, cache, values, TAU, out, lse, "q")


def test_chunk_bad_requests_are_left_alone():
    reqs = Requests([10, 20, 30], [8, 8, 8], seed=30)
    cache, values = make_latent("bf16", reqs)
    q = randn(reqs, 24, 16, 576, dtype=torch.bfloat16)
    for lens in ([18, 7, 38], [18, reqs.max_context + 1, 38], [18, -1, 38]):
        dsa.dsa_clear_device_error()
        reqs.seq.copy_(torch.tensor(lens, dtype=torch.int32))
        out, lse = run_chunk(reqs, q, cache, TAU)
        assert dsa.dsa_get_device_error() == dsa.DEVERR_REQUEST
        assert bool((out[8:16] == 7.0).all()) and bool((lse[8:16] == 7.0).all())
        for r, s in ((0, slice(0, 8)), (2, slice(16, 24))):
            lim = reqs.ctxs[r] + 1 + torch.arange(8, device="cuda")
            o, l, to, tl = attend(q[s], values[reqs.rows(r)], 512, TAU, lim, "bf16")
            close(out[s], o, to, "out")


def test_chunk_offsets_past_32_bits():
    # the request's pages lie behind 2^32 bytes of the pool
    first = (1 << 32) // (PAGE * 640) + 10
    reqs = Requests([90], [5], seed=31)
    small, values = make_latent("q", reqs)
    big = torch.empty(first + reqs.num_blocks, PAGE, 640, dtype=torch.uint8, device="cuda")
    scale = torch.empty(first + reqs.num_blocks, PAGE, 4, device="cuda")
    big[first:], scale[first:] = small.data, small.scale
    q = randn(reqs, 5, 16, 576, dtype=torch.bfloat16)
    want, _ = run_chunk(reqs, q, small, TAU)
    reqs.table += first
    far = dsa.PagedCache(big, scale)
    out, lse = run_chunk(reqs, q, far, TAU)
    back = torch.empty(5, 576, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_cache_read(far, reqs.chunks(), back)
    kv = randn(reqs, 5, 576)
    dsa.dsa_cache_append(None, kv, None, far, reqs.chunks())
    no_error()
    assert torch.equal(out, want)
    rows = reqs.token_rows() - first * PAGE
    bits_equal(back, values[rows], "read")
    v, _ = quantise(kv[:, :512], 128)
    bits_equal(big[first:].view(-1, 640)[rows][:, :512].contiguous().view(FP8), v, "append")


def test_chunk_equal_runs():
    reqs = Requests([3000, 100, 7], [6, 200, 1], seed=32)
    cache, _ = make_latent("q", reqs)
    q = randn(reqs, reqs.total, 64, 576, dtype=torch.bfloat16)
    first = run_chunk(reqs, q, cache, TAU)
    for _ in range(3):
        again = run_chunk(reqs, q, cache, TAU)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_chunk_unaligned_queries():
    # queries and outputs that do not start on 16 bytes
    reqs = Requests([90], [5], seed=33)
    cache, values = make_latent("q", reqs)
    q = torch.empty(5 * 16 * 576 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(5, 16, 576)
    q.copy_(randn(reqs, 5, 16, 576))
    out = torch.empty(5 * 16 * 512 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(5, 16, 512)
    size = dsa.dsa_chunk_mla_workspace_size(5, 1, 16, 512, reqs.max_context)
    dsa.dsa_chunk_mla(q, cache, reqs.chunks(), TAU, out, workspace=torch.empty(size, dtype=torch.uint8, device="cuda") if size else None)
    no_error()
    check_chunk(reqs, q, cache, values, TAU, out, None, "q")


# ------------------------------------------------------------------------------------------ sparse attention, quantised


def selection(reqs, k, seed, fill):
    """int32 [T, k]: for each token a choice of its visible positions, ascending, -1 behind them."""
    g = torch.Generator().manual_seed(seed)
    idx = torch.full((reqs.total, k), -1, dtype=torch.int32)
    for t, p in enumerate(reqs.pos):
        n = min(k, p + 1, max(1, int(k * fill)))
        idx[t, :n] = torch.randperm(p + 1, generator=g)[:n].sort().values
    return idx.cuda()


def run_sparse(reqs, q, cache, idx, entry="decode", k=None):
    T, H = q.shape[:2]
    out = torch.empty(T, H, 512, dtype=q.dtype, device="cuda")
    lse = torch.empty(T, H, device="cuda")
    batch = dsa.Batch(torch.tensor(reqs.req, dtype=torch.int32, device="cuda"),
                      torch.tensor(reqs.pos, dtype=torch.int32, device="cuda"), reqs.table, reqs.max_context)
    if entry == "noalloc":
        dsa.dsa_sparse_mla_decode_noalloc(q, cache, batch, idx, TAU, out, lse)
        return out, lse
    size = dsa.dsa_mla_workspace_size(T, H, 512, k if idx is None else idx.shape[1])
    ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    fn = dsa.dsa_sparse_mla_decode if entry == "decode" else dsa.dsa_sparse_mla_prefill
    fn(q, cache, batch, idx, TAU, out, lse, ws, **({"k": k} if idx is None else {}))
    return out, lse


def check_sparse(reqs, q, values, idx, out, lse, kind="q"):
    for t in range(q.shape[0]):
        at = idx[t][idx[t] >= 0].long()
        rows = reqs.table[reqs.req[t]].long()[at // PAGE] * PAGE + at % PAGE
        o, l, to, tl = attend(q[t:t + 1], values[rows], 512, TAU, torch.tensor([at.numel()], device="cuda"), kind)
        close(out[t:t + 1], o, to, "out of query %d" % t)
        close(lse[t:t + 1], l, tl, "lse of query %d" % t)


@pytest.mark.parametrize("heads", [128, 64, 16, 100])
@pytest.mark.parametrize("entry", ["decode", "prefill", "noalloc"])
@pytest.mark.parametrize("k,fill", [(2048, 1.0), (100, 1.0), (640, 0.4)])
def test_sparse_quantised(heads, entry, k, fill):
    reqs = Requests([2999, 400, 30], [1, 2, 1] if entry == "decode" else [3, 1, 2], seed=heads + k)
    cache, values = make_latent("q", reqs)
    q = randn(reqs, reqs.total, heads, 576, dtype=torch.bfloat16)
    idx = selection(reqs, k, 5, fill)
    out, lse = run_sparse(reqs, q, cache, idx, entry)
    no_error()
    check_sparse(reqs, q, values, idx, out, lse)


def test_sparse_quantised_many_queries():
    # more (query, split) units than SMs, so that several share a CTA
    reqs = Requests([1500], [170], seed=41)
    cache, values = make_latent("q", reqs)
    q = randn(reqs, 170, 128, 576, dtype=torch.bfloat16)
    idx = selection(reqs, 512, 6, 1.0)
    for entry in ("decode", "prefill"):
        out, lse = run_sparse(reqs, q, cache, idx, entry)
        no_error()
        check_sparse(reqs, q, values, idx, out, lse)


@pytest.mark.parametrize("heads", [128, 64, 24])
def test_sparse_quantised_dense_case(heads):
    # no selection: every visible position
    reqs = Requests([130, 20], [2, 3], seed=42)
    cache, values = make_latent("q", reqs)
    q = randn(reqs, 5, heads, 576, dtype=torch.bfloat16)
    idx = torch.full((5, 192), -1, dtype=torch.int32)
    for t, p in enumerate(reqs.pos):
        idx[t, :p + 1] = torch.arange(p + 1)
    for entry in ("decode", "prefill"):
        out, lse = run_sparse(reqs, q, cache, None, entry, k=192)
        no_error()
        check_sparse(reqs, q, values, idx.cuda(), out, lse)


def test_sparse_quantised_f32_queries():
    reqs = Requests([130], [3], seed=43)
    cache, values = make_latent("q", reqs)
    q = randn(reqs, 3, 8, 576)
    idx = selection(reqs, 64, 7, 1.0)
    out, lse = run_sparse(reqs, q, cache, idx)
    no_error()
    check_sparse(reqs, q, values, idx, out, lse, "f32")


def test_sparse_quantised_flags():
    reqs = Requests([300], [3], seed=44)
    cache, values = make_latent("q", reqs)
    q = randn(reqs, 3, 128, 576, dtype=torch.bfloat16)
    idx = selection(reqs, 128, 8, 1.0)
    idx[0, 5] = 1000                            # a position the query does not see
    idx[1, :] = -1                              # nothing selected
    bad = int(idx[2, 9])                        # a row with a bad scale, skipped by every query that selects it
    cache.scale.view(-1, 4)[reqs.rows(0)[bad], 3] = 0.7
    out, lse = run_sparse(reqs, q, cache, idx)
    assert dsa.dsa_get_device_error() == dsa.DEVERR_INDEX | dsa.DEVERR_SCALE
    assert bool((out[1] == 0).all()) and bool((lse[1] == -math.inf).all())
    idx[0, 5] = -1
    idx[idx == bad] = -1
    for t in (0, 2):
        at = idx[t][idx[t] >= 0].long()
        rows = reqs.table[0].long()[at // PAGE] * PAGE + at % PAGE
        o, l, to, tl = attend(q[t:t + 1], values[rows], 512, TAU, torch.tensor([at.numel()], device="cuda"), "q")
        close(out[t:t + 1], o, to, "out")
        close(lse[t:t + 1], l, tl, "lse")


def test_sparse_quantised_unselected_nan():
    reqs = Requests([300], [2], seed=45)
    cache, values = make_latent("q", reqs)
    q = randn(reqs, 2, 64, 576, dtype=torch.bfloat16)
    idx = selection(reqs, 128, 9, 0.7)
    chosen = torch.zeros(reqs.num_blocks * PAGE, dtype=torch.bool, device="cuda")
    for t in range(2):
        at = idx[t][idx[t] >= 0].long()
        chosen[reqs.table[0].long()[at // PAGE] * PAGE + at % PAGE] = True
    cache.data.view(-1, 640)[~chosen] = 0x7F
    cache.scale.view(-1, 4)[~chosen] = math.nan
    out, lse = run_sparse(reqs, q, cache, idx)
    no_error()
    check_sparse(reqs, q, values, idx, out, lse)


# ------------------------------------------------------------------------------------------ together


def test_serving_steps_from_prompt_to_decode():
    # two prompts enter the caches in chunks, attend densely below the top-K; then decode steps append
    # a token, score, select and attend sparsely; the caches are read back at the end
    H, K, Hi = 64, 64, 64
    reqs = Requests([0, 0], [200, 131], seed=50)
    g = reqs.gen
    keys_x, lat_x = torch.randn(2, 220, 128, generator=g).cuda(), torch.randn(2, 220, 576, generator=g).cuda()
    nb, width = 12, 6
    table = torch.randperm(nb, generator=g).to(torch.int32).view(2, width).cuda()
    keys = dsa.PagedCache(torch.zeros(nb, PAGE, 128, dtype=torch.uint8, device="cuda"), torch.zeros(nb, PAGE, device="cuda"))
    lat = dsa.PagedCache(torch.zeros(nb, PAGE, 640, dtype=torch.uint8, device="cuda"), torch.zeros(nb, PAGE, 4, device="cuda"))
    v, s = quantise(lat_x.bfloat16()[..., :512], 128)
    values = torch.cat([v * s.repeat_interleave(128, -1), lat_x.bfloat16()[..., 512:].double()], -1)
    done = [0, 0]

    def step(news, sparse):
        ends = [d + n for d, n in zip(done, news)]
        cu = torch.tensor([0, news[0], sum(news)], dtype=torch.int32, device="cuda")
        ch = dsa.Chunks(cu, torch.tensor(ends, dtype=torch.int32, device="cuda"), table, max(ends))
        cut = lambda x: torch.cat([x[r, done[r]:ends[r]] for r in range(2)]).bfloat16()
        T = sum(news)
        dsa.dsa_cache_append(cut(keys_x), cut(lat_x), keys, lat, ch)
        q = torch.randn(T, H, 576, generator=g).cuda().bfloat16()
        out, lse = torch.empty(T, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, device="cuda")
        req = [r for r in range(2) for _ in range(news[r])]
        pos = [done[r] + i for r in range(2) for i in range(news[r])]
        if sparse:
            b = dsa.Batch(torch.tensor(req, dtype=torch.int32, device="cuda"), torch.tensor(pos, dtype=torch.int32, device="cuda"),
                          table, max(ends))
            qi, w = torch.randn(T, Hi, 128, generator=g).cuda().bfloat16(), torch.rand(T, Hi, generator=g).cuda()
            scores = torch.empty(T, (max(ends) + 3) // 4 * 4, device="cuda")
            idx = torch.empty(T, K, dtype=torch.int32, device="cuda")
            dsa.dsa_indexer_topk(qi, w, keys, b, K, scores, idx)
            size = dsa.dsa_mla_workspace_size(T, H, 512, K)
            dsa.dsa_sparse_mla_decode(q, lat, b, idx, TAU, out, lse, torch.empty(max(size, 1), dtype=torch.uint8, device="cuda"))
        else:
            size = dsa.dsa_chunk_mla_workspace_size(T, 2, H, 512, max(ends))
            dsa.dsa_chunk_mla(q, lat, ch, TAU, out, lse, torch.empty(max(size, 1), dtype=torch.uint8, device="cuda"))
        for t in range(T):
            at = idx[t][idx[t] >= 0].long() if sparse else torch.arange(pos[t] + 1, device="cuda")
            assert not sparse or at.numel() == K
            o, l, to, tl = attend(q[t:t + 1], values[req[t]][at], 512, TAU, torch.tensor([at.numel()], device="cuda"), "q")
            close(out[t:t + 1], o, to, "out")
            close(lse[t:t + 1], l, tl, "lse")
        done[:] = ends

    for news in ([64, 1], [0, 100], [136, 30]):
        step(news, False)
    for _ in range(3):
        step([1, 1], True)
    step([4, 2], True)
    no_error()
    ch = dsa.Chunks(torch.tensor([0, done[0], sum(done)], dtype=torch.int32, device="cuda"),
                    torch.tensor(done, dtype=torch.int32, device="cuda"), table, max(done))
    back = torch.empty(sum(done), 576, device="cuda")
    dsa.dsa_cache_read(lat, ch, back)
    bits_equal(back, torch.cat([values[0, :done[0]], values[1, :done[1]]]), "read back")


def test_captured_step_follows_the_lengths():
    # append and chunk attention captured once for a padded batch, replayed as the requests grow
    H, T, B, nb, width = 16, 8, 3, 14, 4
    g = torch.Generator().manual_seed(51)
    table = torch.randperm(nb, generator=g)[:B * width].to(torch.int32).view(B, width).cuda()
    lat = dsa.PagedCache(torch.zeros(nb, PAGE, 640, dtype=torch.uint8, device="cuda"), torch.zeros(nb, PAGE, 4, device="cuda"))
    cu, seq = torch.zeros(B + 1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    kv = torch.zeros(T, 576, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(T, H, 576, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros(T, H, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, H, device="cuda")
    ch = dsa.Chunks(cu, seq, table, width * PAGE)
    size = dsa.dsa_chunk_mla_workspace_size(T, B, H, 512, width * PAGE)
    ws = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")

    def step():
        dsa.dsa_cache_append(None, kv, None, lat, ch)
        dsa.dsa_chunk_mla(q, lat, ch, TAU, out, lse, ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    held = [torch.zeros(0, 576, dtype=torch.float64, device="cuda") for _ in range(B)]
    for news in ([4, 1, 0], [1, 1, 1], [0, 0, 8], [3, 2, 2], [0, 0, 0], [1, 6, 1]):
        n = sum(news)
        x = torch.randn(T, 576, generator=g).bfloat16().cuda()
        kv.copy_(x)
        q.copy_(torch.randn(T, H, 576, generator=g))
        out.fill_(7.0)
        v, s = quantise(x[:, :512], 128)
        vals = torch.cat([v * s.repeat_interleave(128, -1), x[:, 512:].double()], -1)
        cu.copy_(torch.tensor([0, news[0], news[0] + news[1], n], dtype=torch.int32))
        at = 0
        for r in range(B):
            held[r] = torch.cat([held[r], vals[at:at + news[r]]])
            at += news[r]
        seq.copy_(torch.tensor([h.shape[0] for h in held], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        at = 0
        for r in range(B):
            if news[r]:
                lim = held[r].shape[0] - news[r] + 1 + torch.arange(news[r], device="cuda")
                o, l, to, tl = attend(q[at:at + news[r]], held[r], 512, TAU, lim, "q")
                close(out[at:at + news[r]], o, to, "out")
                close(lse[at:at + news[r]], l, tl, "lse")
            at += news[r]
        assert bool((out[n:] == 7.0).all())
    no_error()


def test_two_streams_with_their_own_workspaces():
    reqs = [Requests([1500 + 100 * i], [4], seed=52 + i) for i in range(2)]
    caches = [make_latent("q", r) for r in reqs]
    qs = [randn(r, 4, 128, 576, dtype=torch.bfloat16) for r in reqs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [None, None]
    for _ in range(4):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                outs[i] = run_chunk(reqs[i], qs[i], caches[i][0], TAU)
    torch.cuda.synchronize()
    no_error()
    for i in range(2):
        check_chunk(reqs[i], qs[i], caches[i][0], caches[i][1], TAU, outs[i][0], outs[i][1], "q")


# ------------------------------------------------------------------------------------------ both ways of reading quantised chunks


def chunk_with(reqs, q, cache, full):
    """Chunk attention with the whole workspace (quantised rows of several row tiles are expanded once)
    or with none where a call needs none (each row tile turns them into bf16 itself)."""
    T, H = q.shape[:2]
    out = torch.full((T, H, 512), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    size = dsa.dsa_chunk_mla_workspace_size(T, len(reqs.news), H, 512, reqs.max_context)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") if full else None   # NaN wherever it is read unwritten
    dsa.dsa_chunk_mla(q, cache, reqs.chunks(), TAU, out, lse, ws)
    return out, lse


@pytest.mark.parametrize("full", [True, False])
def test_chunk_quantised_bad_rows_many_tiles(full):
    # row tiles enough for one unit per SM and more, so that nothing is split: bad scales, a page outside the
    # pool, a request without tokens, NaN codes, and garbage in every row that no request has
    reqs = Requests([100, 5, 0, 300], [150, 0, 90, 40], seed=61, pad=2)
    cache, values = make_latent("q", reqs)
    q = randn(reqs, reqs.tokens, 128, 576, dtype=torch.bfloat16)
    used = torch.zeros(reqs.num_blocks * PAGE, dtype=torch.bool, device="cuda")
    for r in range(4):
        used[reqs.rows(r)] = True
    cache.data.view(-1, 640)[~used] = 0x7F
    cache.scale.view(-1, 4)[~used] = math.nan
    skipped = {0: [7, 110, 249], 2: [0, 33], 3: []}
    for r, ps in skipped.items():
        for i, p in enumerate(ps):
            cache.scale.view(-1, 4)[reqs.rows(r, p, p + 1), i % 4] = 0.3
    skipped[3] = list(range(64, 128))
    rows3 = reqs.rows(3)
    reqs.table[3, 1] = 1 << 28
    nan_at = 120                                    # of request 0: its tokens from position 120 on get NaN
    cache.data.view(-1, 640)[reqs.rows(0, nan_at, nan_at + 1), 300] = 0xFF
    out, lse = chunk_with(reqs, q, cache, full)
    assert dsa.dsa_get_device_error() == dsa.DEVERR_SCALE | dsa.DEVERR_BLOCK_ID
    assert bool((out[reqs.total:] == 7.0).all()) and bool((lse[reqs.total:] == 7.0).all())
    start = 0
    for r, n in enumerate(reqs.news):
        if n:
            keep = torch.ones(reqs.lens[r], dtype=torch.bool, device="cuda")
            keep[skipped[r]] = False
            s = slice(start, start + (n if r else nan_at - reqs.ctxs[0]))
            lim = keep.cumsum(0)[reqs.ctxs[r]:reqs.ctxs[r] + s.stop - s.start]
            o, l, to, tl = attend(q[s], values[(rows3 if r == 3 else reqs.rows(r))[keep]], 512, TAU, lim, "q")
            close(out[s], o, to, "out of request %d" % r)
            close(lse[s], l, tl, "lse of request %d" % r)
        start += n
    tail = slice(nan_at - reqs.ctxs[0], reqs.news[0])
    assert bool(out[tail].isnan().all()) and bool(lse[tail].isnan().all())


def test_chunk_expanded_equals_unexpanded():
    reqs = Requests([0, 700, 64], [200, 33, 150], seed=62)
    cache, values = make_latent("q", reqs)
    q = randn(reqs, reqs.total, 128, 576, dtype=torch.bfloat16)
    a, b = chunk_with(reqs, q, cache, True), chunk_with(reqs, q, cache, False)
    no_error()
    # the same rows, products and order of sums
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check_chunk(reqs, q, cache, values, TAU, a[0], a[1], "q")


@pytest.mark.parametrize("kind", ["q", "bf16"])
def test_chunk_ragged_splits(kind):
    # requests of very different lengths whose row tiles are split: units handed out as CTAs become free; used twice,
    # with a workspace that the first call has left dirty
    reqs = Requests([6000, 40, 2500, 0, 900], [3, 4, 1, 2, 2], seed=63)
    cache, values = make_latent(kind, reqs)
    q = randn(reqs, reqs.total, 128, 576, dtype=torch.bfloat16)
    size = dsa.dsa_chunk_mla_workspace_size(reqs.total, 5, 128, 512, reqs.max_context)
    assert size > 0
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    got = []
    for _ in range(2):
        out, lse = torch.empty(reqs.total, 128, 512, dtype=q.dtype, device="cuda"), torch.empty(reqs.total, 128, device="cuda")
        dsa.dsa_chunk_mla(q, cache, reqs.chunks(), TAU, out, lse, ws)
        got.append((out, lse))
    no_error()
    check_chunk(reqs, q, cache, values, TAU, got[0][0], got[0][1], kind)
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_chunk_workspace_is_checked():
    reqs = Requests([4000], [2], seed=64)
    cache, _ = make_latent("bf16", reqs)
    q = randn(reqs, 2, 128, 576, dtype=torch.bfloat16)
    out = torch.empty(2, 128, 512, dtype=torch.bfloat16, device="cuda")
    size = dsa.dsa_chunk_mla_workspace_size(2, 1, 128, 512, reqs.max_context)
    ws = torch.empty(size + 256, dtype=torch.uint8, device="cuda")
    for bad in (None, ws[:size - 1], ws[1:1 + size]):
        with pytest.raises(dsa.DsaError):
            dsa.dsa_chunk_mla(q, cache, reqs.chunks(), TAU, out, workspace=bad)
    dsa.dsa_chunk_mla(q, cache, reqs.chunks(), TAU, out, workspace=ws[:size])
    no_error()


def test_two_captured_graphs_with_their_own_workspaces():
    # the same call captured twice, replayed on two streams at once
    reqs = Requests([2500, 300, 0], [4, 7, 3], seed=65)
    cache, values = make_latent("q", reqs)
    qs = [randn(reqs, reqs.total, 128, 576, dtype=torch.bfloat16) for _ in range(2)]
    size = dsa.dsa_chunk_mla_workspace_size(reqs.total, 3, 128, 512, reqs.max_context)
    runs = []
    for q in qs:
        ws = torch.full((max(size, 1),), 0xFF, dtype=torch.uint8, device="cuda")
        out, lse = torch.empty(reqs.total, 128, 512, dtype=q.dtype, device="cuda"), torch.empty(reqs.total, 128, device="cuda")
        call = lambda: dsa.dsa_chunk_mla(q, cache, reqs.chunks(), TAU, out, lse, ws)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        runs.append((g, side, q, out, lse, ws))
    for g, side, *_ in runs:
        with torch.cuda.stream(side):
            for _ in range(3):
                g.replay()
    torch.cuda.synchronize()
    no_error()
    for _, _, q, out, lse, _ in runs:
        check_chunk(reqs, q, cache, values, TAU, out, lse, "q")


@pytest.mark.parametrize("heads", [1, 16, 128])
def test_sparse_quantised_equals_bf16_values(heads):
    # a quantised cache and a bf16 one with the same values give the same up to the order of sums
    reqs = Requests([1200], [3], seed=66)
    cache, values = make_latent("q", reqs)
    plain = dsa.PagedCache(values.bfloat16().view(-1, PAGE, 576))
    assert torch.equal(plain.data.double().view(-1, 576), values)
    q = randn(reqs, 3, heads, 576, dtype=torch.bfloat16)
    idx = selection(reqs, 256, 10, 1.0)
    for c in (cache, plain):
        out, lse = run_sparse(reqs, q, c, idx)
        check_sparse(reqs, q, values, idx, out, lse)
    no_error()


def test_tensors_of_another_device_are_refused():
    if torch.cuda.device_count() < 2:
        pytest.skip("one device")
    reqs = Requests([10], [2], seed=67, device="cuda:0")
    cache, _ = make_latent("q", reqs)
    with torch.cuda.device(1), pytest.raises(ValueError):
        dsa.dsa_cache_read(cache, reqs.chunks(), torch.empty(2, 576, device="cuda:0"))


def test_empty_chunks_do_nothing():
    reqs = Requests([10, 20], [0, 0], seed=68)
    cache, _ = make_latent("q", reqs)
    q = torch.empty(0, 16, 576, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_chunk_mla(q, cache, reqs.chunks(), TAU, torch.empty(0, 16, 512, dtype=torch.bfloat16, device="cuda"))
    dsa.dsa_cache_read(cache, reqs.chunks(), torch.empty(0, 576, device="cuda"))
    dsa.dsa_cache_append(None, torch.empty(0, 576, device="cuda"), None, cache, reqs.chunks())
    # rows that belong to no request
    out = torch.full((3, 576), 7.0, device="cuda")
    dsa.dsa_cache_read(cache, reqs.chunks(), out)
    q = torch.zeros(3, 16, 576, dtype=torch.bfloat16, device="cuda")
    o = torch.full((3, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    size = dsa.dsa_chunk_mla_workspace_size(3, 2, 16, 512, reqs.max_context)
    dsa.dsa_chunk_mla(q, cache, reqs.chunks(), TAU, o, workspace=torch.empty(max(size, 1), dtype=torch.uint8, device="cuda"))
    no_error()
    assert bool((out == 7.0).all()) and bool((o == 7.0).all())
