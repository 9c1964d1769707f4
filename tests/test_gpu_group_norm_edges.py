"""GPU tests of the grouped norm: group sizes between the listed ones of each vector form, and the widest
rows. Tolerances as in test_gpu_group_norm.py."""
import pytest
import torch

from oracle import linattn as ol
from state_space_sequence_mamba_b200 import binding as m3
from test_gpu_group_norm import BF, F32, bound, check, err

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("T,C,G", [(1, 512, 1), (7, 1536, 4), (40, 528, 2), (300, 3120, 6), (5, 264, 1), (90, 1024, 2),
                                   (200, 520, 1), (33, 1032, 1), (21, 2064, 2)])
def test_groups_of_several_vectors_a_lane(cuda_dev, T, C, G, gate, dtype):
    check(cuda_dev, T, C, G, dtype, gate=gate)
    check(cuda_dev, T, C, G, dtype, gate=gate, center=False, silu=False)


def test_widest_rows_of_the_smallest_groups(cuda_dev):
    """2^24 channels in groups of four, fp32: the most groups that a call may have, 64 of them to a CTA."""
    C, G, T = 1 << 24, 1 << 22, 2
    g = torch.Generator(device=cuda_dev).manual_seed(3)
    x, d = (torch.randn(T, C, generator=g, device=cuda_dev) for _ in range(2))
    w = torch.rand(C, generator=g, device=cuda_dev) + 0.5
    out = m3.group_norm_fwd(x, G, weight=w, bias=w)
    r = m3.group_norm_bwd(d, x, G, weight=w, bias=w)
    torch.cuda.synchronize()
    for lo in (0, C // 2 - 512, C - 4096):      # (a group stands for itself)
        part = slice(lo, lo + 4096)
        args = x[:, part].cpu(), 1024, w[part].cpu(), w[part].cpu()
        assert err(out[:, part], ol.group_norm_forward(*args)) <= bound(F32, 4)
        dx, _, dw, db = ol.group_norm_gradients(d[:, part].cpu(), *args)
        assert err(r["dweight"][part], dw) <= bound(F32, T) and err(r["dbias"][part], db) <= bound(F32, T)
        assert err(r["dx"][:, part], dx) <= 4 * bound(F32, 4)
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 6, 9])
def test_few_rows(cuda_dev, rows):
    for C, G in ((4096, 64), (96, 3)):
        check(cuda_dev, rows, C, G, BF)
        check(cuda_dev, rows, C, G, F32, affine=False, gate=False)


