"""A token's attention is its own: other rows, other requests and far positions leave it as it is, on the GPU."""
import numpy as np
import pytest

import oracle.prompt_oracle as PO
from test_gpu_prompt_attention import Prompt, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def smla():
    import sparse_mla_decode_smla_gb300 as m
    m.lib()
    return m


def _torch():
    import torch
    return torch


def _same(a, b):
    """Bit for bit."""
    return _torch().equal(a.contiguous().view(_torch().uint8), b.contiguous().view(_torch().uint8))


@pytest.mark.parametrize("rope,bias", [(64, False), (0, False), (0, True)])
@pytest.mark.parametrize("value", [200.0, float("nan"), float("inf")])
def test_a_capped_token_does_not_depend_on_other_queries(smla, rope, bias, value):
    """The first 40 tokens, whose scores are small beside the cap, in front of large queries: later ones of their own request
    and another request's, over key tiles that all of them see."""
    p = Prompt(smla, [70, 90], [600, 300], 2, 2, rope=rope, cap=20.0, bias=bias, seed=31, sink=True, spread=0.3).run()
    out, lse = p.out.clone(), p.lse.clone()
    first = int(p.cu_q[0]) + 40
    p.q[first:].copy_(p.q[first:] * value if np.isfinite(value) else _torch().full_like(p.q[first:], value))
    p.run()
    assert _same(p.out[:first], out[:first]) and _same(p.lse[:first], lse[:first])


@pytest.mark.parametrize("value", [200.0, float("nan")])
def test_a_capped_token_does_not_depend_on_other_heads(smla, value):
    """Grouped heads of one token stand beside one another in a row tile."""
    p = Prompt(smla, [30], [700], 8, 2, cap=20.0, seed=32, spread=0.3).run()
    out, lse = p.out.clone(), p.lse.clone()
    p.q[:, 1].copy_(p.q[:, 1] * value if np.isfinite(value) else _torch().full_like(p.q[:, 1], value))
    p.run()
    others = [h for h in range(8) if h != 1]
    assert _same(p.out[:, others], out[:, others]) and _same(p.lse[:, others], lse[:, others])


@pytest.mark.parametrize("bias", [False, True])
def test_small_and_large_scores_beside_one_another(smla, bias):
    p = Prompt(smla, [150, 33], [400, 150], 4, 2, cap=20.0, bias=bias, seed=33, sink=True)
    p.q.copy_(p.q * _torch().where(_torch().arange(p.T, device="cuda") % 3 == 0, 15.0, 0.2)[:, None, None])
    p.run().check()


def test_scores_up_to_a_cap_that_is_large_beside_the_scale(smla):
    """Powers of scale / cap that leave fp32: scores from next to nothing up to 0.63 of the cap."""
    torch = _torch()
    for cap in (2e3, 5e4, 1e6, 1e9):
        p = Prompt(smla, [130], [130], 2, 2, cap=cap, seed=34)
        # s = scale * 192 a b, up to 0.63 cap: a in whole numbers up to 85, b a power of two or 27 / 16 of one, exact in bf16
        b = 2.0 ** np.floor(np.log2(0.63 * cap / (p.scale * 192 * 85)))
        p.q.copy_((1 + torch.arange(p.T, device="cuda") * 84 // p.T)[:, None, None].to(p.q.dtype).expand_as(p.q))
        p.k.fill_(b)
        p.rope.fill_(b)
        p.run().check()
        p.k.fill_(b * 1.6875)
        p.rope.fill_(b * 1.6875)
        p.run().check()


def test_a_bias_by_distance_past_two_to_the_24_keys(smla):
    """Positions that fp32 does not hold: all but the nearest keys weigh nothing, so the last 300 are the reference."""
    torch = _torch()
    n, near, slope = (1 << 24) + 130, 300, 1.0
    g = torch.Generator(device="cuda").manual_seed(35)
    q = torch.randn((3, 1, 128), generator=g, device="cuda").to(torch.bfloat16)
    k, v = (torch.zeros((n, 1, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for t in (k, v):
        t[-near:] = torch.randn((near, 1, 128), generator=g, device="cuda").to(torch.bfloat16)
    out, lse = torch.zeros((3, 1, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((3, 1), device="cuda")
    d = smla.make_prompt_desc(3, n, 1, 1, 1, 0, 128 ** -0.5)
    ws = torch.zeros(smla.prompt_workspace_size(d), dtype=torch.uint8, device="cuda")
    smla.prompt_attention(d, q, k, v, None, _i32([0, 3]), _i32([0, n]), None, torch.full((1,), slope, device="cuda"), None, out, lse, ws)
    assert smla.read_error(None, ws) == 0
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    ref, rl, size, big = PO.prompt_attention(f(q), f(k[-near:]), f(v[-near:]), None, [0, 3], [0, near], 128 ** -0.5, slopes=[slope])
    # keys 40 steps away weigh e^-40: the others' scores are of size 40 + 8 at most, in fp32 as elsewhere
    e = 48 * 200 * 2.0 ** -24
    assert (np.abs(f(lse) - rl) <= e).all(), np.abs(f(lse) - rl).max()
    assert (np.abs(f(out) - ref) <= size * (2.0 ** -8 + 2 * e) + np.abs(ref) * 2.0 ** -8).all()
