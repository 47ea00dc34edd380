"""Cache views as the entry points of the 4-bit latent cache take them: built field by field, and with a tensor on a
device of its own."""
import pytest
import torch

import long_context_sparse_11_b200 as dsa
from long_context_sparse_11_b200 import binding as B


@pytest.fixture(scope="module")
def lib():
    from long_context_sparse_11_b200.build import build
    build()
    return dsa.load()


def calls(view):
    """The three entry points on CPU tensors: they get as far as the check of the device, and no further."""
    x, pos = torch.zeros(2, 576), torch.zeros(2, dtype=torch.int32)
    q, idx = torch.zeros(2, 64, 576, dtype=torch.bfloat16), torch.zeros(2, 8, dtype=torch.int32)
    yield lambda: dsa.latent_append(x, pos, view)
    yield lambda: dsa.latent_read(view, pos)
    if view.dtype == B.DSA_MXFP4:
        yield lambda: dsa.sparse_mla_attn(q, view, idx, 8, 0.04)


def views():
    bt, lens = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    yield dsa.paged_view(dsa.latent_pool4(4, "cpu"), None, bt, lens)
    yield dsa.paged_view(torch.zeros(4, 64, 576, dtype=torch.uint8), torch.zeros(4, 64), bt, lens)


def refused(call):
    with pytest.raises(dsa.DsaError) as e:
        call()
    assert e.value.status == B.DSA_ERR_INVALID_ARG
    return str(e.value)


@pytest.mark.parametrize("which", [0, 1])
def test_views_without_tensors_of_their_own(lib, which):
    """A view filled in field by field, or copied out of a group's arguments, holds no tensors."""
    view = B.CacheView.from_buffer_copy(list(views())[which])
    for call in calls(view):
        assert "CUDA device" in refused(call)


class Elsewhere(torch.Tensor):
    """A tensor that says it lies on another GPU."""

    device = torch.device("cuda:1")

    def get_device(self):
        return 1


@pytest.mark.parametrize("part", [1, 2, 3])
def test_every_tensor_of_an_e4m3_view_lies_on_the_calls_device(lib, part):
    made = [torch.zeros(4, 64, 576, dtype=torch.uint8), torch.zeros(4, 64), torch.zeros(2, 2, dtype=torch.int32),
            torch.ones(2, dtype=torch.int32)]
    made[part] = made[part].as_subclass(Elsewhere)
    for call in calls(dsa.paged_view(*made)):
        assert "tensors on cpu and cuda:1" in refused(call)


@pytest.mark.parametrize("part", [2, 3])
def test_every_tensor_of_a_4bit_view_lies_on_one_device(lib, part):
    made = [dsa.latent_pool4(4, "cpu"), None, torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)]
    made[part] = made[part].as_subclass(Elsewhere)
    assert "cuda:1" in refused(lambda: dsa.paged_view(*made))
