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


@pytest.mark.parametrize("requests", [33, 700])
def test_many_requests_behind_the_kernels_that_write_their_inputs(smla, requests):
    """More requests than a warp lays out: lengths, keys and queries are written right in front of each call, and the output is
    overwritten right behind it."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    n, H = 7 * requests, 4
    xs = [torch.randn((n, 1024), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3)]
    w = torch.ones(1024, device="cuda").to(torch.bfloat16)
    w128 = torch.ones(H * 128, device="cuda").to(torch.bfloat16)
    cus = [torch.arange(0, n + 1, 7, dtype=torch.int32, device="cuda"),
           torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((requests,), n, dtype=torch.int32, device="cuda")])]
    y, cu = torch.zeros_like(xs[0]), torch.zeros(requests + 1, dtype=torch.int32, device="cuda")
    q, k, v = y[:, :512].view(n, H, 128), y[:, 512:768].view(n, 2, 128), y[:, 768:].view(n, 2, 128)
    d = smla.make_prompt_desc(n, n, H, 2, requests, 0, 128 ** -0.5, q_strides=q.stride()[:2], k_strides=k.stride()[:2], v_strides=v.stride()[:2])
    ws = torch.zeros(smla.prompt_workspace_size(d), dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros((n, H, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((n, H), device="cuda")

    def once(i, wait):
        keep = torch.zeros_like(out)
        for f in (lambda: cu.copy_(cus[i % 2]), lambda: smla.add_rmsnorm(xs[i % 3], None, w, 1e-6, y=y),
                  lambda: smla.prompt_attention(d, q, k, v, None, cu, cu, None, None, None, out, lse, ws),
                  lambda: smla.add_rmsnorm(out.view(n, H * 128), None, w128, 1e-6, y=keep.view(n, H * 128)),
                  lambda: smla.add_rmsnorm(y[:, :512], None, w128, 1e-6, y=out.view(n, H * 128))):
            f()
            if wait:
                torch.cuda.synchronize()
        return keep

    want = [once(i, True) for i in range(6)]
    got = [once(i, False) for i in range(6)]
    torch.cuda.synchronize()
    assert smla.read_error(None, ws) == 0
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
