"""Calls behind one another on a stream, none of which waits on the host: each sees what the ones before it wrote, and
writes nothing that they still read."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def smla():
    import sparse_mla_decode_smla_gb300 as m
    m.lib()
    return m


def _chain(smla, rows, vocab, seed):
    """A step's calls over shared buffers, as a list of functions, and the tensors that they write."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    bf = lambda *n: torch.randn(n, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    P, H, pages = 64, 4, -(-rows // 64)
    x, w = bf(rows, 640), torch.ones(640, device="cuda").to(torch.bfloat16)
    kv = torch.zeros((pages, P, 1152), dtype=torch.uint8, device="cuda")
    slots = torch.arange(rows, dtype=torch.int64, device="cuda")
    latent, rope = torch.zeros((rows, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((rows, 64), dtype=torch.bfloat16, device="cuda")
    table, cu, zero, err = i32([list(range(pages))]), i32([0, rows]), i32([0]), i32([0])
    rd = smla.make_read_desc(smla.SMLA_KV_BF16, P, pages, 1, pages, rows)
    q = bf(rows, H, 192)
    k = latent.view(rows, 2, 256)[..., :128]
    v = latent.view(rows, 2, 256)[..., 128:]
    pd = smla.make_prompt_desc(rows, rows, H, 2, 1, 64, 192 ** -0.5, k_strides=k.stride()[:2], v_strides=v.stride()[:2])
    ws = torch.zeros(smla.prompt_workspace_size(pd), dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros((rows, H, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((rows, H), device="cuda")
    logits = out.view(-1)[:(rows * H * 128) // vocab * vocab].view(-1, vocab)
    n = logits.shape[0]
    tok = torch.randint(0, vocab, (n, 1), generator=g, device="cuda", dtype=torch.int32)
    lp, ent = torch.zeros((n, 1), device="cuda"), torch.zeros(n, device="cuda")
    ids, alt = torch.zeros((n, 5), dtype=torch.int32, device="cuda"), torch.zeros((n, 5), device="cuda")
    codes, scales = torch.zeros((rows, 512), dtype=torch.uint8, device="cuda"), torch.zeros((rows, 4), device="cuda")
    w512 = torch.ones(512, device="cuda").to(torch.bfloat16)
    steps = [
        lambda: smla.add_rmsnorm(x, None, w, 1e-6, y=x),                                                # in place
        lambda: smla.pack_kv(smla.SMLA_KV_BF16, smla.SMLA_SCALE_POW2, x[:, :512].contiguous(), x[:, 512:576].contiguous(), slots, kv, rows),
        lambda: smla.cache_read(rd, kv, table, zero, cu, latent, rope, err),
        lambda: smla.prompt_attention(pd, q, k, v, rope, cu, cu, None, None, None, out, lse, ws),
        lambda: smla.token_logprobs(logits, tok, lp, entropy=ent, top_ids=ids, top_logprobs=alt, error_word=err),
        lambda: smla.add_rmsnorm(latent, out.view(rows, H * 128), w512, 1e-6, residual_out=out.view(rows, H * 128), codes=codes, scales=scales),
        lambda: smla.token_logprobs(logits, tok, lp, entropy=ent, top_ids=ids, top_logprobs=alt, error_word=err),
        lambda: smla.add_rmsnorm(x[:, :512], out.view(rows, H * 128), w512, 1e-6, y=out.view(rows, H * 128)),  # overwrites the logits
        lambda: smla.add_rmsnorm(x, x, w, 1e-6, residual_out=x),
    ]
    return steps, [x, kv, latent, rope, out, lse, lp, ent, ids, alt, codes, scales, err]


@pytest.mark.parametrize("rows,vocab", [(5, 512), (300, 1001), (6000, 2000), (9000, 40000)])
def test_calls_on_one_stream_take_effect_in_order(smla, rows, vocab):
    import torch
    steps, want = _chain(smla, rows, vocab, 3)
    for _ in range(4):
        for f in steps:
            f()
            torch.cuda.synchronize()
    for captured in (False, True):
        steps, got = _chain(smla, rows, vocab, 3)
        torch.cuda.synchronize()
        if captured:
            first = [t.clone() for t in got]
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for f in steps:
                    f()
            s.synchronize()
            for t, f in zip(got, first):
                t.copy_(f)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                for f in steps:
                    f()
            for _ in range(4):
                graph.replay()
        else:
            for _ in range(4):
                for f in steps:
                    f()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(want, got)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (captured, i)
