"""Offsets that go back and on again: requests that would write one another's rows, on the GPU."""
import numpy as np
import pytest

from test_gpu_prompt_attention import Prompt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def smla():
    import sparse_mla_decode_smla_gb300 as m
    m.lib()
    return m


def _with(p, smla, cu_q, cu_k):
    import torch
    p.cu_q, p.cu_k = np.asarray(cu_q), np.asarray(cu_k)
    p.desc.num_requests = len(cu_q) - 1
    p.ws = torch.zeros(smla.prompt_workspace_size(p.desc), dtype=torch.uint8, device="cuda")
    p.out.fill_(7.0)
    p.lse.fill_(7.0)
    p.run()
    return p.out.clone(), p.lse.clone(), smla.read_error(None, p.ws)


@pytest.mark.parametrize("heads,kv_heads", [(2, 2), (8, 2)])
@pytest.mark.parametrize("lead", [0, 40, 300])  # requests without tokens in front: the others in one warp, and in several
def test_requests_that_overlap_are_left_out(smla, heads, kv_heads, lead):
    import torch
    p = Prompt(smla, [60, 50], [100, 300], heads, kv_heads, seed=61, lead=0)
    a = _with(p, smla, [0, 60], [0, 100])
    b = _with(p, smla, [90, 110], [100, 300])
    assert a[2] == b[2] == 0
    # 60 -> 40 goes back, 40 -> 90 starts before 60, 90 -> 110 fits
    cu_q, cu_k = [0, 60, 40, 90, 110], [0, 100, 100, 100, 300]
    for gap in (0, 40, 300) if lead else (0,):  # and requests without tokens between them
        q = [0] * lead + cu_q[:2] + [60] * gap + [40] + [40] * gap + cu_q[3:]
        k = [0] * lead + cu_k[:2] + [100] * gap + [100] + [100] * gap + cu_k[3:]
        out, lse, err = _with(p, smla, q, k)
        assert err == smla.SMLA_DEVERR_INDEX
        assert torch.equal(out[:60], a[0][:60]) and torch.equal(lse[:60], a[1][:60])
        assert torch.equal(out[90:110], b[0][90:110]) and torch.equal(lse[90:110], b[1][90:110])
        assert (out[60:90] == 7).all() and (lse[60:90] == 7).all() and (out[110:] == 7).all()


@pytest.mark.parametrize("requests", [32, 2000])
def test_offsets_to_and_fro(smla, requests):
    """Every second request would have all rows: the first one has."""
    import torch
    p = Prompt(smla, [113], [300], 4, 2, rope=0, seed=62, lead=0)
    want = _with(p, smla, [0, 113], [0, 300])
    out, lse, err = _with(p, smla, [0, 113] * (requests // 2) + [0], [0, 300] + [300] * (requests - 1))
    assert err == smla.SMLA_DEVERR_INDEX
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_a_long_request_behind_one_that_is_left_out(smla):
    """Items that several SMs share, and the way from one request to the next past those without items."""
    import torch
    p = Prompt(smla, [3, 200, 1], [9000, 5000, 700], 4, 4, seed=63, lead=0)
    p.run().check()
    out, lse, cq, ck = p.out.clone(), p.lse.clone(), p.cu_q, p.cu_k
    got = _with(p, smla, [0, 3, 2, 2, 3, 203, 204], [0, 9000, 9000, 9000, 9000, 14000, 14700])
    assert got[2] == smla.SMLA_DEVERR_INDEX
    p.cu_q, p.cu_k, p.desc.num_requests = cq, ck, 3
    assert torch.equal(got[0][:204], out[:204]) and torch.equal(got[1][:204], lse[:204])
