"""moe_route on logits that are zeros of both signs: equal, so the lowest number comes first, for few and for many tokens."""
import pytest
import torch

from tests.test_gpu_route import TYPES, bias_of
from tests.test_gpu_route_many import check

pytestmark = pytest.mark.gpu


def zeros_of(T, E, dtype, seed=0, share=0.5, below=0.3):
    """Rows of +0 and -0, a part of them below zero."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.where(torch.rand((T, E), generator=g, device="cuda") < share, 0.0, -0.0)
    z = torch.where(torch.rand((T, E), generator=g, device="cuda") < below, -torch.rand((T, E), generator=g, device="cuda") - 0.5, z)
    return z.to(TYPES[dtype])


@pytest.mark.parametrize("T", [20, 8195])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("E,k,n_group,topk_group", [(64, 1, 1, 1), (64, 6, 8, 3), (128, 8, 1, 1), (128, 8, 8, 5), (256, 8, 8, 4), (256, 7, 1, 1),
                                                    (512, 8, 16, 5), (512, 3, 1, 1)])
def test_signs_of_zero_do_not_rank(lib, T, dtype, E, k, n_group, topk_group):
    few_open = zeros_of(30, E, dtype, seed=E, below=1.0 - 2.0 / k if k > 2 else 0.9)     # the threshold lies among the zeros, or below
    for flags in (0, lib.MOE_ROUTE_SOFTMAX, lib.MOE_ROUTE_RENORM, lib.MOE_ROUTE_GROUP_PAIR):
        for z in (zeros_of(30, E, dtype, seed=k), few_open):
            check(lib, z, k, None, n_group, topk_group, flags=flags, T=T)
            check(lib, z, k, 0.0 * bias_of(E), n_group, topk_group, flags=flags, T=T)


@pytest.mark.parametrize("T", [1, 8191, 8192])
def test_a_negative_zero_in_front(lib, T):
    z = torch.full((1, 64), -1.0, device="cuda")
    z[0, 0], z[0, 5] = -0.0, 0.0
    check(lib, z, 1, T=T)
    check(lib, z, 2, T=T)
    check(lib, z.relu_().neg_(), 8, T=T)              # rectified and turned: -0 throughout
    check(lib, torch.where(torch.arange(64, device="cuda") % 3 == 0, 0.0, z), 8, T=T)
