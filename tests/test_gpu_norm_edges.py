"""Zeros and the smallest numbers through the norm and its codes, bit for bit, on the GPU."""
import numpy as np
import pytest

import oracle.prompt_oracle as PO
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


@pytest.mark.parametrize("group", [128, 0])
@pytest.mark.parametrize("mode", [0, 1])
def test_values_whose_scale_would_round_to_zero(smla, group, mode):
    """y of some 2^-142.5 where it is not 0: a 448th of that is below fp32's smallest number, 2^-149, which is the scale then."""
    torch = _torch()
    x = torch.cat([torch.ones(3, 128), torch.full((3, 128), 2.0 ** -10)], 1).to(torch.bfloat16)
    w = torch.zeros(256)
    w[128::2] = 2.0 ** -133  # bf16's smallest number
    w = w.to(torch.bfloat16)
    codes = torch.empty((3, 256), dtype=torch.uint8, device="cuda")
    scales = torch.empty((3, 2 if group else 1), device="cuda")
    smla.add_rmsnorm(x.cuda(), None, w.cuda(), 0.0, codes=codes, scales=scales, group=group, scale_mode=mode)
    s = scales.double().cpu().numpy()
    assert (s[:, -1] == 2.0 ** -149).all()
    if group:
        assert (s[:, 0] == 1).all()
    _, ref, _ = PO.add_rmsnorm(x.double().numpy(), None, w.double().numpy(), 0.0, group)
    value = O.e4m3_decode(codes.cpu().numpy()) * np.repeat(s, group or 256, 1)
    # y itself is a whole number of 2^-149, off by a few roundings to such; a code is off by 2^-4 of it at most
    assert (np.abs(value - ref) <= np.abs(ref) * 2.0 ** -4 + 2 * 2.0 ** -149).all()
