"""One attention workspace under calls of different descriptions, on the GPU."""
import numpy as np
import pytest

from test_gpu_prompt_attention import Prompt, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def smla():
    import sparse_mla_decode_smla_gb300 as m
    m.lib()
    return m


def _batch(smla, requests, seed):
    """`requests` short ones, the first and one in the middle so long that several SMs share their items."""
    r = np.random.default_rng(seed)
    nq = r.integers(0, 4, requests)
    nk = nq + r.integers(0, 200, requests)
    nq[0], nk[0] = 2, 9000
    nq[requests // 2], nk[requests // 2] = 140, 5000
    return Prompt(smla, nq.tolist(), nk.tolist(), 4, 2, rope=64 if requests % 2 else 0, seed=seed)


def test_one_workspace_for_batches_of_any_size(smla):
    import torch
    order = [64, 40, 1, 700, 33, 2, 48, 20, 31, 64, 16, 1, 700, 1]
    batches = {n: _batch(smla, n, 40 + n) for n in set(order)}
    size = smla.prompt_workspace_size(batches[700].desc)
    assert all(smla.prompt_workspace_size(b.desc) <= size for b in batches.values())
    shared = torch.zeros(size, dtype=torch.uint8, device="cuda")
    want = {}
    for n, b in batches.items():  # on a workspace of their own
        b.run()
        assert smla.read_error(None, b.ws) == 0
        want[n] = b.out.clone(), b.lse.clone()
    for captured in (False, True):
        if captured:  # all of them behind one another, nothing between them
            graph = torch.cuda.CUDAGraph()
            keep = []
            for n in order:
                b = batches[n]
                keep.append((b, _i32(b.cu_q), _i32(b.cu_k), torch.full_like(b.out, 7.0), torch.full_like(b.lse, 7.0)))
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                for b, cq, ck, out, lse in keep:
                    smla.prompt_attention(b.desc, b.q, b.k, b.v, b.rope, cq, ck, None, None, None, out, lse, shared)
            for _ in range(2):
                graph.replay()
            torch.cuda.synchronize()
            got = [(out, lse) for _, _, _, out, lse in keep]
        else:
            got = []
            for n in order:
                b = batches[n]
                b.ws = shared
                b.out.fill_(7.0)
                b.lse.fill_(7.0)
                b.run()
                got.append((b.out.clone(), b.lse.clone()))
        assert smla.read_error(None, shared) == 0
        for i, (n, (out, lse)) in enumerate(zip(order, got)):
            assert torch.equal(out, want[n][0]) and torch.equal(lse, want[n][1]), (captured, i, n)
