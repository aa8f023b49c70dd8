"""Refusals of the cache and chunk entry points on the host (no GPU), and the definitions their GPU
tests compare with, checked against brute force."""
import ctypes
import math

import pytest
import torch

import sparse_attention_06_b200 as dsa
from _cache_chunk import FP8, quantise
from sparse_attention_06_b200 import build as dsa_build


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return dsa.load_library()


FAKE = 4096   # a device address that is never dereferenced on the host


def chunks(**kw):
    d = dict(num_tokens=4, num_reqs=2, cu_tokens=FAKE, seq_len=FAKE, block_table=FAKE, max_blocks=4, max_context=256)
    d.update(kw)
    return dsa._Chunks(*d.values())


def cache(dtype, dim, scale=None, data=FAKE, blocks=4, block_size=64):
    return dsa._PagedCache(data, scale, blocks, block_size, dim, dtype, 0)


BAD_CHUNKS = [
    (dict(num_tokens=-1), b"negative"),
    (dict(num_reqs=-2), b"negative"),
    (dict(cu_tokens=None), b"NULL"),
    (dict(seq_len=None), b"NULL"),
    (dict(block_table=None), b"NULL"),
    (dict(max_blocks=0), b"max_blocks"),
    (dict(max_context=0), b"max_context"),
    (dict(max_context=257), b"max_blocks"),
]


def append(lib, ch, keys=None, lat=None, k=FAKE, ks=128, kv=FAKE, kvs=576, x=dsa.DSA_BF16):
    keys = cache(dsa.DSA_E4M3, 128, FAKE) if keys is None else keys
    lat = cache(dsa.DSA_LATENT_E4M3, 576, FAKE) if lat is None else lat
    return lib.dsa_cache_append(k, ks, kv, kvs, x, ctypes.byref(keys) if keys else None, ctypes.byref(lat) if lat else None,
                                ctypes.byref(ch) if ch else None, None)


def read(lib, ch, c, out=FAKE, dt=dsa.DSA_BF16):
    return lib.dsa_cache_read(ctypes.byref(c) if c else None, ctypes.byref(ch) if ch else None, out, dt, None)


def chunk(lib, ch, c, q=FAKE, qd=dsa.DSA_BF16, H=16, dv=512, dr=64, scale=0.1, out=FAKE, ws=None, ws_bytes=0):
    return lib.dsa_chunk_mla(q, qd, H, dv, dr, ctypes.byref(c) if c else None, ctypes.byref(ch) if ch else None, scale,
                             out, None, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,word", BAD_CHUNKS)
def test_bad_chunks_are_refused(lib, kw, word):
    lat = cache(dsa.DSA_LATENT_E4M3, 576, FAKE)
    for call in (lambda: append(lib, chunks(**kw)), lambda: read(lib, chunks(**kw), lat), lambda: chunk(lib, chunks(**kw), lat)):
        assert call() == dsa.DSA_ERR_INVALID_ARG
        assert word in lib.dsa_last_error_message()


def test_missing_structures_are_refused(lib):
    assert append(lib, None) == dsa.DSA_ERR_INVALID_ARG
    assert read(lib, None, cache(dsa.DSA_BF16, 576)) == dsa.DSA_ERR_INVALID_ARG
    assert read(lib, chunks(), None) == dsa.DSA_ERR_INVALID_ARG
    assert chunk(lib, None, cache(dsa.DSA_BF16, 576)) == dsa.DSA_ERR_INVALID_ARG
    assert chunk(lib, chunks(), None) == dsa.DSA_ERR_INVALID_ARG


BAD_LATENTS = [
    cache(dsa.DSA_LATENT_E4M3, 576),                         # no scales
    cache(dsa.DSA_LATENT_E4M3, 576, FAKE + 4),               # scales not on 16 bytes
    cache(dsa.DSA_LATENT_E4M3, 512, FAKE),                   # rows of another width
    cache(dsa.DSA_LATENT_E4M3, 576, FAKE, block_size=32),
    cache(dsa.DSA_LATENT_E4M3, 576, FAKE, blocks=0),
    cache(dsa.DSA_LATENT_E4M3, 576, FAKE, data=FAKE + 8),    # data not on 16 bytes
    cache(dsa.DSA_LATENT_E4M3, 576, FAKE, data=None),
    cache(7, 576, FAKE),                                     # no such dtype
]


@pytest.mark.parametrize("c", BAD_LATENTS)
def test_bad_latent_caches_are_refused(lib, c):
    assert append(lib, chunks(), lat=c) == dsa.DSA_ERR_INVALID_ARG
    assert read(lib, chunks(), c) == dsa.DSA_ERR_INVALID_ARG
    assert chunk(lib, chunks(), c) == dsa.DSA_ERR_INVALID_ARG
    b = dsa._Batch(1, 1, FAKE, FAKE, FAKE, 4, 256, 1, 0)
    for fn in (lib.dsa_sparse_mla_decode, lib.dsa_sparse_mla_prefill):
        assert fn(FAKE, dsa.DSA_BF16, 16, 512, 64, ctypes.byref(c), ctypes.byref(b), FAKE, 64, 0.1, FAKE, None, None, 0,
                  None) == dsa.DSA_ERR_INVALID_ARG


def test_append_refusals(lib):
    keys, lat = cache(dsa.DSA_E4M3, 128, FAKE), cache(dsa.DSA_LATENT_E4M3, 576, FAKE)
    bad = [
        dict(k=None),                                        # a cache without its input, and the other way round
        dict(kv=None),
        dict(keys=False),
        dict(lat=False),
        dict(x=dsa.DSA_E4M3),
        dict(ks=127),                                        # rows shorter than the cache's
        dict(kvs=575),
        dict(kvs=-576),
        dict(keys=cache(dsa.DSA_E4M3, 128)),                 # no scales
        dict(keys=cache(dsa.DSA_LATENT_E4M3, 576, FAKE)),    # a latent cache in the keys' place
        dict(lat=cache(dsa.DSA_E4M3, 576, FAKE)),
    ]
    for kw in bad:
        assert append(lib, chunks(), **kw) == dsa.DSA_ERR_INVALID_ARG, kw
    assert append(lib, chunks(num_tokens=0)) == dsa.DSA_OK
    assert append(lib, chunks(num_reqs=0)) == dsa.DSA_OK
    assert lib.dsa_cache_append(None, 0, None, 0, dsa.DSA_BF16, None, None, ctypes.byref(chunks()), None) == dsa.DSA_OK
    del keys, lat


def test_read_refusals(lib):
    lat = cache(dsa.DSA_LATENT_E4M3, 576, FAKE)
    assert read(lib, chunks(), lat, out=None) == dsa.DSA_ERR_INVALID_ARG
    assert read(lib, chunks(), lat, dt=dsa.DSA_E4M3) == dsa.DSA_ERR_INVALID_ARG
    assert read(lib, chunks(), cache(dsa.DSA_E4M3, 128)) == dsa.DSA_ERR_INVALID_ARG
    assert read(lib, chunks(num_tokens=0), lat) == dsa.DSA_OK


def test_chunk_refusals(lib):
    lat = cache(dsa.DSA_LATENT_E4M3, 576, FAKE)
    bad = [dict(q=None), dict(out=None), dict(H=0), dict(dv=0), dict(dv=448, dr=128), dict(dv=2048), dict(scale=0.0),
           dict(scale=-1.0), dict(scale=math.nan), dict(qd=dsa.DSA_E4M3)]
    for kw in bad:
        assert chunk(lib, chunks(), lat, **kw) == dsa.DSA_ERR_INVALID_ARG, kw
    # an unquantised cache has the queries' type
    assert chunk(lib, chunks(), cache(dsa.DSA_BF16, 576), qd=dsa.DSA_F32) == dsa.DSA_ERR_INVALID_ARG
    assert chunk(lib, chunks(), cache(dsa.DSA_F32, 576)) == dsa.DSA_ERR_INVALID_ARG
    assert chunk(lib, chunks(), cache(dsa.DSA_E4M3, 576, FAKE)) == dsa.DSA_ERR_INVALID_ARG
    assert chunk(lib, chunks(num_tokens=0), lat) == dsa.DSA_OK


def test_indexer_refuses_latent_rows(lib):
    kc = cache(dsa.DSA_LATENT_E4M3, 576, FAKE)
    b = dsa._Batch(1, 1, FAKE, FAKE, FAKE, 4, 256, 1, 0)
    st = lib.dsa_indexer_scores(FAKE, 1, None, 16, 576, FAKE, ctypes.byref(kc), ctypes.byref(b), FAKE, 256, None, None)
    assert st == dsa.DSA_ERR_INVALID_ARG


def test_workspace_sizes_are_host_only_and_bounded(lib):
    for args in ((0, 1, 128, 512, 4096), (1, 0, 128, 512, 4096), (1, 1, 0, 512, 4096), (1, 1, 128, 512, 0), (4, 1, 128, 64, 4096)):
        assert dsa.dsa_chunk_mla_workspace_size(*args) == 0
    assert dsa.dsa_chunk_mla_workspace_size(1, 1, 128, 512, 64) == 0    # one tile of keys: nothing to split


def test_quantise_definition_against_all_codes():
    # the tests' quantiser: every e4m3 value is its own code at scale 1, every midpoint goes to the even
    # code, and the scale is the smallest one
    v = torch.arange(256, dtype=torch.uint8).view(FP8).double()
    v = v[torch.isfinite(v)].sort().values.unique()
    mids = (v[1:] + v[:-1]) / 2
    for x in list(v.tolist()) + mids.tolist() + (mids * (1 + 1e-9)).tolist():
        row = torch.zeros(128, dtype=torch.float64)
        row[0], row[1] = x, 300.0
        got, s = quantise(row, 128)
        assert s.item() == 1.0
        d = (v - x).abs()
        best = v[d == d.min()]
        assert got[0].item() in best.tolist()
        if best.numel() == 2:
            code = torch.tensor([got[0].item()]).to(FP8).view(torch.uint8).item()
            assert code % 2 == 0
    for amax, want in ((448.0, 1.0), (449.0, 2.0), (224.0, 0.5), (224.1, 1.0), (2.0 ** -140, 2.0 ** -100), (0.0, 1.0),
                       (1.7e38, 2.0 ** 119)):
        row = torch.zeros(128, dtype=torch.float64)
        row[5] = -amax
        got, s = quantise(row, 128)
        assert s.item() == want and abs(got[5].item() * s.item() + amax) <= max(amax * 2.0 ** -4, 2.0 ** -110)


def test_python_checks():
    cpu = torch.zeros(2, 64, 640, dtype=torch.uint8)
    with pytest.raises(ValueError):
        dsa.PagedCache(cpu, torch.zeros(2, 64, 4, dtype=torch.float64))._c()
    with pytest.raises(ValueError):
        dsa.PagedCache(cpu[:, :, :576].contiguous(), torch.zeros(2, 64, 4))._c()
    with pytest.raises(ValueError):
        dsa.PagedCache(cpu, torch.zeros(2, 64, 2))._c()
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        dsa.Chunks(i.long(), i[:1], i[:1, None], 64)._c(1)
    with pytest.raises(ValueError):
        dsa.Chunks(i, i, i[:1, None], 64)._c(1)
    assert dsa.PagedCache(cpu, torch.zeros(2, 64, 4)).dim == 576
