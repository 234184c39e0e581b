"""Zeros and the smallest numbers through the norm and its codes, bit for bit, on the GPU."""
import numpy as np
import pytest

import oracle.smla_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def smla():
    import sparse_mla_decode_smla_gb300 as m
    m.lib()
    return m


def _torch():
    import torch
    return torch


@pytest.mark.parametrize("dim", [96, 1024, 7168])
@pytest.mark.parametrize("group", [128, 0])
@pytest.mark.parametrize("mode", [0, 1])
def test_code_bytes_are_those_of_the_rounded_quotient(smla, dim, group, mode):
    """Rows of +-1 have the norm 1, so y is the weight exactly; a third of the weights are zero, so that zeros of both signs occur."""
    torch = _torch()
    g = torch.Generator().manual_seed(dim + group)
    x = torch.where(torch.rand((6, dim), generator=g) < 0.5, -1.0, 1.0).to(torch.bfloat16)
    w = torch.randn((dim,), generator=g) * torch.exp2(torch.randint(-30, 12, (dim,), generator=g).float())
    w[::3] = 0.0
    w = w.to(torch.bfloat16)
    codes = torch.empty((6, dim), dtype=torch.uint8, device="cuda")
    scales = torch.empty((6, -(-dim // 128) if group else 1), device="cuda")
    smla.add_rmsnorm(x.cuda(), None, w.cuda(), 0.0, codes=codes, scales=scales, group=group, scale_mode=mode)
    y = (x.float() * w.float()).numpy()
    width = group or dim
    for b in range(0, dim, width):
        part = y[:, b:b + width]
        ratio = np.abs(part).max(1) / np.float32(448)
        scale = ratio if mode == smla.SMLA_SCALE_FP32 else O.pow2_ceil_f32(ratio).astype(np.float32)
        want = O.e4m3_encode_rne_satfinite((part / scale[:, None].astype(np.float32)).astype(np.float32))
        assert np.array_equal(codes[:, b:b + width].cpu().numpy(), want)


@pytest.mark.parametrize("dim", [64, 1024, 7168])
def test_zeros_keep_their_sign_without_a_residual(smla, dim):
    torch = _torch()
    x = torch.randn((5, dim), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    x[:, ::3], x[:, 1::7] = -0.0, 0.0
    x, w = x.cuda(), torch.ones(dim, device="cuda").to(torch.bfloat16)
    total, y = torch.empty_like(x), torch.empty_like(x)
    smla.add_rmsnorm(x, None, w, 1e-6, residual_out=total, y=y)
    assert torch.equal(total.view(torch.int16), x.view(torch.int16))
    assert torch.equal(torch.signbit(y), torch.signbit(x))
