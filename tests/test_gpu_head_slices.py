"""One token in every slice of a larger tensor: [S, 1, d], whose middle stride
says nothing. The same bits as from a copy."""
import pytest

import token_perturbation_estimator_gb300 as dust
from helpers import cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S", [2, 9, 40])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_token_of_every_slice(S, dtype):
    import torch
    dev = cuda()
    T, d, V = 7, 72, 300
    g = torch.Generator().manual_seed(S)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    Y = torch.randn((S, T, d), generator=g).to(dt).to(dev)
    E = (torch.randn((V, d), generator=g) * (2.0 / d ** 0.5)).to(dt).to(dev)
    for t in (0, 3, T - 1):
        H = Y[:, t:t + 1]
        y = torch.tensor([17 * t + 5], dtype=torch.int32, device=dev)
        copy = H.clone(memory_format=torch.contiguous_format)
        a = dust.dust_head_loss(H, E, y, changes=True)
        b = dust.dust_head_loss(copy, E, y, changes=True)
        gl = torch.ones((S, 1), device=dev)
        a += dust.dust_head_loss_grad(H, E, y, a[1], gl)
        b += dust.dust_head_loss_grad(copy, E, y, b[1], gl)
        ids = torch.tensor([[3, -1, 250]], dtype=torch.int32, device=dev)
        z = torch.tensor([[0.5, 0.0, 1.5]], device=dev)
        c, e = dust.dust_distill_loss(H, E, ids, z), dust.dust_distill_loss(copy, E, ids, z)
        a += c + dust.dust_distill_loss_grad(H, E, ids, z, c[1], c[2], gl)
        b += e + dust.dust_distill_loss_grad(copy, E, ids, z, e[1], e[2], gl)
        assert len(a) == len(b)
        for p, q in zip(a, b):
            assert torch.equal(p, q)


def test_slices_over_one_another_are_refused():
    import torch
    dev = cuda()
    Y = torch.zeros((20, 64), device=dev)
    E, y = torch.zeros((50, 64), device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    with pytest.raises(ValueError):
        dust.dust_head_loss(Y[:1].expand(3, 1, 64), E, y)
    with pytest.raises(ValueError):
        dust.dust_head_loss(Y.as_strided((3, 1, 64), (32, 32, 1)), E, y)
