"""The operators around a prompt where byte and element offsets pass 32 bits: the last rows against float64, on the GPU."""
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


def _i32(v):
    return _torch().tensor(v, dtype=_torch().int32, device="cuda")


def _f64(t):
    return t.double().cpu().numpy()


def _near(out, lse, q, k, v):
    """One causal prompt of its own keys."""
    n = q.shape[0]
    ref, rl, size, _ = PO.prompt_attention(_f64(q), _f64(k), _f64(v), None, [0, n], [0, n], 128 ** -0.5)
    assert np.abs(_f64(lse) - rl).max() <= 1e-4
    # weights and the result are rounded to bf16: 2^-8 of each at most; scores in fp32 as above
    assert (np.abs(_f64(out) - ref) <= size * (2.0 ** -8 + 2e-4) + np.abs(ref) * 2.0 ** -8).all()


def test_attention_of_far_rows(smla):
    torch = _torch()
    n, gap = 300, 1 << 23  # 5 GB from the first token to the last
    q, k, v = (torch.empty(n * gap, dtype=torch.bfloat16, device="cuda").as_strided((n, h, 128), (gap, 136, 1)) for h in (4, 2, 2))
    for t in (q, k, v):
        t.copy_(torch.randn(t.shape, device="cuda"))
    out, lse = torch.zeros((n, 4, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((n, 4), device="cuda")
    d = smla.make_prompt_desc(n, n, 4, 2, 1, 0, 128 ** -0.5, q_strides=q.stride()[:2], k_strides=k.stride()[:2], v_strides=v.stride()[:2])
    ws = torch.zeros(smla.prompt_workspace_size(d), dtype=torch.uint8, device="cuda")
    smla.prompt_attention(d, q, k, v, None, _i32([0, n]), _i32([0, n]), None, None, None, out, lse, ws)
    assert smla.read_error(None, ws) == 0
    _near(out, lse, q, k, v)


def test_attention_of_many_rows(smla):
    torch = _torch()
    B, n, H = 1000, 140, 128  # 2.3e9 elements of q and of the output
    T = B * n
    q = torch.zeros((T, H, 128), dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros((T, 1, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for a in (0, T - n):
        for t in (q, k, v):
            t[a:a + n] = torch.randn(t[a:a + n].shape, device="cuda").to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty((T, H), device="cuda")
    d = smla.make_prompt_desc(T, T, H, 1, B, 0, 128 ** -0.5)
    ws = torch.zeros(smla.prompt_workspace_size(d), dtype=torch.uint8, device="cuda")
    cu = _i32([n * i for i in range(B + 1)])
    smla.prompt_attention(d, q, k, v, None, cu, cu, None, None, None, out, lse, ws)
    assert smla.read_error(None, ws) == 0
    for a in (0, T - n):
        _near(out[a:a + n], lse[a:a + n], q[a:a + n], k[a:a + n], v[a:a + n])
    assert not out[n:T - n].any()


def test_read_of_a_large_pool(smla):
    torch = _torch()
    P, pages, B, n = 64, 110000, 70, 62000  # 4.6 GB of pages, 4.4 GB of latents
    kv = torch.empty((pages, P, 656), dtype=torch.uint8, device="cuda")
    table = torch.empty((B, -(-n // P)), dtype=torch.int32, device="cuda")
    last = torch.arange(pages - 100, pages, dtype=torch.int32, device="cuda")
    table[:] = last[torch.arange(table.shape[1], device="cuda") % 100]
    g = torch.Generator().manual_seed(3)
    raw = torch.cat([(torch.randn((100 * P, 512), generator=g) * 50).to(torch.float8_e4m3fn).view(torch.uint8),
                     torch.exp2(torch.randint(-3, 3, (100 * P, 4), generator=g).float()).view(torch.uint8),
                     torch.randn((100 * P, 64), generator=g).to(torch.bfloat16).view(torch.uint8)], 1)
    kv[pages - 100:] = raw.reshape(100, P, 656).cuda()
    lat = torch.empty((B * n, 512), dtype=torch.bfloat16, device="cuda")
    rope, err = torch.empty((B * n, 64), dtype=torch.bfloat16, device="cuda"), _i32([0])
    d = smla.make_read_desc(smla.SMLA_KV_FP8_DS, P, pages, B, table.shape[1], B * n)
    smla.cache_read(d, kv, table, _i32([0] * B), _i32([n * i for i in range(B + 1)]), lat, rope, err)
    want = O.dequant_rows(raw.numpy(), "fp8_ds")  # E4M3 times a power of two: exact in bf16
    for r in (0, B - 1):
        for a in (0, n - 400):
            at = np.arange(a, a + 400) % (100 * P)
            assert np.array_equal(_f64(lat[r * n + a:r * n + a + 400]), want[at, :512])
            assert np.array_equal(_f64(rope[r * n + a:r * n + a + 400]), want[at, 512:])
    assert err.item() == 0


def test_norm_of_many_rows(smla):
    torch = _torch()
    n, dim = 300000, 8192  # 2.5e9 elements
    x, res = (torch.zeros((n, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for t in (x, res):
        t[-5:] = torch.randn((5, dim), device="cuda").to(torch.bfloat16)
    w = torch.randn(dim, device="cuda").to(torch.bfloat16)
    added, y = torch.empty_like(x), torch.empty_like(x)
    codes, scales = torch.empty((n, dim), dtype=torch.uint8, device="cuda"), torch.empty((n, dim // 128), device="cuda")
    smla.add_rmsnorm(x, res, w, 1e-6, residual_out=added, y=y, codes=codes, scales=scales)
    h, ref, amax = PO.add_rmsnorm(_f64(x[-5:]), _f64(res[-5:]), _f64(w), 1e-6, 128)
    assert (np.abs(_f64(added[-5:]) - h) <= np.abs(h) * 2.0 ** -8).all()
    assert (np.abs(_f64(y[-5:]) - ref) <= np.abs(ref) * 1.01 * 2.0 ** -8).all()
    s = np.repeat(_f64(scales[-5:]), 128, 1)
    back = _f64(codes[-5:].view(torch.float8_e4m3fn)) * s
    assert (np.abs(back - ref) <= np.abs(ref) * 1.01 * 2.0 ** -4 + s * 2.0 ** -10).all()  # half a step, of subnormals too
    assert not (codes[:-5] & 127).any() and not y[:-5].any() and not added[:-5].any() and (scales[:-5] == 1).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_logprobs_of_far_rows(smla, dtype):
    torch = _torch()
    n, v, gap = 4, 5001, (1 << 30) + 3
    x = torch.empty(3 * gap + v, dtype=getattr(torch, dtype), device="cuda").as_strided((n, v), (gap, 1))
    x.copy_(torch.randn((n, v), device="cuda") * 3)
    lp, ids = torch.empty((n, 1), device="cuda"), torch.empty((n, 7), dtype=torch.int32, device="cuda")
    smla.token_logprobs(x, _i32([[5000 - i] for i in range(n)]), lp, top_ids=ids)
    want = PO.token_logprobs(_f64(x), np.array([[5000 - i] for i in range(n)]), 7)
    assert np.array_equal(ids.cpu().numpy(), want[2]) and np.abs(_f64(lp) - want[0]).max() <= 1e-4
