"""Which tensors a PagedCache takes (no GPU): what the kernels read and write through its pointers has to be there."""
import pytest
import torch

import sparse_attention_06_b200 as dsa

# CPU tensors pass the checks of type and shape and then meet this refusal
TAKEN = "must be a CUDA tensor"


def keys(nb=3, dim=128, dtype=torch.uint8):
    return torch.zeros(nb, 64, dim, dtype=dtype)


@pytest.mark.parametrize("data", [keys(), keys(dtype=torch.float8_e4m3fn)])
@pytest.mark.parametrize("scale", [
    torch.zeros(3, 64, dtype=torch.bfloat16),   # two bytes a row
    torch.zeros(3, 64, dtype=torch.float64),
    torch.zeros(3, 64, dtype=torch.int32),
    torch.zeros(3),                             # one per block
    torch.zeros(2, 64),                         # a block short
    torch.zeros(3, 63),
    torch.zeros(0),
], ids=lambda t: "%s%s" % (t.dtype, list(t.shape)))
def test_key_scales_that_are_too_small_are_refused(data, scale):
    with pytest.raises(ValueError, match="float32"):
        dsa.PagedCache(data, scale)._c()


@pytest.mark.parametrize("scale", [torch.zeros(3, 64), torch.zeros(192), torch.zeros(5, 64)])
def test_key_scales_of_a_row_each_are_taken(scale):
    with pytest.raises(ValueError, match=TAKEN):
        dsa.PagedCache(keys(), scale)._c()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unquantised_caches_do_not_look_at_a_scale(dtype):
    with pytest.raises(ValueError, match=TAKEN):
        dsa.PagedCache(keys(dtype=dtype), torch.zeros(1))._c()


def test_key_scales_with_a_last_dimension_of_one_are_a_key_caches():
    for dim in (128, 576, 640):
        c = dsa.PagedCache(keys(dim=dim), torch.zeros(3, 64, 1))
        assert c.dim == dim
        with pytest.raises(ValueError, match=TAKEN):
            c._c()
    with pytest.raises(ValueError, match="float32"):
        dsa.PagedCache(keys(), torch.zeros(3, 64, 1, dtype=torch.bfloat16))._c()


def test_scales_of_groups_are_a_quantised_latent_caches():
    c = dsa.PagedCache(keys(dim=640), torch.zeros(3, 64, 4))
    assert c.dim == 576
    with pytest.raises(ValueError, match=TAKEN):
        c._c()
    for data, scale in ((keys(), torch.zeros(3, 64, 4)), (keys(dim=640), torch.zeros(3, 64, 5)), (keys(dim=640), torch.zeros(2, 64, 4))):
        with pytest.raises(ValueError, match="quantised latent"):
            dsa.PagedCache(data, scale)._c()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unquantised_caches_do_not_look_at_group_scales(dtype):
    c = dsa.PagedCache(keys(dtype=dtype), torch.zeros(3, 64, 4))
    assert c.dim == 128
    with pytest.raises(ValueError, match=TAKEN):
        c._c()
