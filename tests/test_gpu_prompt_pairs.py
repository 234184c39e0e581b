"""Values that are not finite in items of one row tile, whose key tiles alternate between two halves of a CTA, on the GPU."""
import pytest

from test_gpu_prompt_attention import Prompt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def smla():
    import sparse_mla_decode_smla_gb300 as m
    m.lib()
    return m


def _spoil(smla, nq, nk, heads, kv_heads, rope, keys, **kw):
    """One value that is not finite, at each of `keys` in turn. A value that every token sees takes part in the sums: its dim is
    not finite then, and no other one changes. One that some tokens do not see makes those that do NaN in every dim. The others
    and all lse stay as they are, bit for bit, call after call."""
    import torch
    p = Prompt(smla, [nq], [nk], heads, kv_heads, rope=rope, seed=51, **kw).run()
    p.check()
    out, lse, v = p.out.clone(), p.lse.clone(), p.v.clone()
    g, h = heads // kv_heads, kv_heads - 1
    for j in keys:
        for dim in (9, 100):
            for value in (float("nan"), float("inf")):
                p.v.copy_(v)
                p.v[int(p.cu_k[0]) + j, h, dim] = value
                first = int(p.cu_q[0]) + max(0, j - (nk - nq))  # the token that stands at it
                sees = torch.zeros((p.T, heads), dtype=torch.bool, device="cuda")
                sees[first:int(p.cu_q[1]), h * g:h * g + g] = True
                for _ in range(3):
                    p.out.fill_(7.0)
                    p.run()
                    if j > nk - nq:
                        assert torch.isnan(p.out[sees].float()).all(), (j, dim, value)
                    else:
                        assert not torch.isfinite(p.out[sees][:, dim].float()).any(), (j, dim, value)
                        rest = [d for d in range(128) if d != dim]
                        assert torch.equal(p.out[sees][:, rest], out[sees][:, rest])
                    assert torch.equal(p.out[~sees], out[~sees]) and torch.equal(p.lse, lse)


@pytest.mark.parametrize("rope", [64, 0])
@pytest.mark.parametrize("nq,heads,kv_heads", [(1, 1, 1), (2, 1, 1), (40, 1, 1), (128, 2, 2), (1, 8, 1), (5, 16, 2)])
@pytest.mark.parametrize("tiles", [2, 3, 4, 5])
def test_every_dim_of_the_tokens_that_see_it(smla, rope, nq, heads, kv_heads, tiles):
    nk = 128 * tiles - 7
    # among the new keys: in the last key tile, and where there are as many in the one before
    _spoil(smla, nq, nk, heads, kv_heads, rope, sorted({nk - 1, nk - nq, nk - 1 - nq // 2}))


@pytest.mark.parametrize("rope", [64, 0])
@pytest.mark.parametrize("nq,nk,heads,kv_heads", [(1, 9001, 1, 1), (40, 9100, 1, 1), (100, 9000, 2, 2), (3, 20011, 8, 2)])
def test_in_items_that_several_sms_share(smla, rope, nq, nk, heads, kv_heads):
    _spoil(smla, nq, nk, heads, kv_heads, rope, sorted({nk - 1, nk - nq, nk - 1 - nq // 2}))


def test_with_a_prefix_that_reaches_past_a_token(smla):
    """Tokens that see a value behind them."""
    import torch
    p = Prompt(smla, [60], [390], 1, 1, seed=52, prefix=[385], cap=20.0).run()
    lse = p.lse.clone()
    p.v[int(p.cu_k[0]) + 384, 0, 70] = float("nan")
    for _ in range(5):
        p.out.fill_(7.0)
        p.run()
        assert torch.isnan(p.out[int(p.cu_q[0]):int(p.cu_q[1]), 0, 70].float()).all() and torch.equal(p.lse, lse)


@pytest.mark.parametrize("nk", [400, 9000])
@pytest.mark.parametrize("cap", [0.0, 60.0])
def test_one_key_that_has_nearly_all_the_weight(smla, nk, cap):
    """A late key some 2^15 above the ones before: its weight's rounding would be all of the result's, in one direction."""
    import numpy as np
    import torch
    H = 64
    p = Prompt(smla, [1], [nk], H, H, rope=0, seed=53, cap=cap)
    g = torch.Generator(device="cuda").manual_seed(54)
    sign = torch.where(torch.rand((H, 128), generator=g, device="cuda") < 0.5, -1.0, 1.0)
    top = 7
    p.q[int(p.cu_q[0])] = sign.to(torch.bfloat16)
    p.k.mul_(0.01)
    # s = 128^0.5 c: 14.4 to 16 in log2 of the ones before, which are about 0 (10.2 to 11 of a cap of 60 stays as it is but for 1 %)
    p.k[int(p.cu_k[1]) - top] = (sign * torch.linspace(0.885, 0.97, H, device="cuda")[:, None]).to(torch.bfloat16)
    p.run()
    out, lse = p.check()
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    q, k, v = f(p.q[int(p.cu_q[0])]), f(p.k[int(p.cu_k[0]):int(p.cu_k[1])]), f(p.v[int(p.cu_k[0]):int(p.cu_k[1])])
    s = np.einsum("hd,nhd->hn", q, k) * p.scale
    s = cap * np.tanh(s / cap) if cap else s
    w = np.exp(s - s.max(1, keepdims=True))
    rest = np.einsum("hn,nhd->hd", np.delete(w, nk - top, 1), np.abs(np.delete(v, nk - top, 0))) / w.sum(1)[:, None]
    want, got = out[int(p.cu_q[0])], f(p.out)[int(p.cu_q[0])]
    # the result's rounding, the other weights', and scores of 11 in fp32 as elsewhere
    e = 11 * 200 * 2.0 ** -24 + cap * 2.0 ** -20 + nk * 2.0 ** -24
    assert (np.abs(got - want) <= np.abs(want) * 2.0 ** -8 + rest * 2.0 ** -8 + e * (np.abs(want) + rest)).all()
