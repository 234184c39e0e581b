"""Attention of packed prompts against float64, on the GPU."""
import numpy as np
import pytest

import oracle.prompt_oracle as PO

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
    return _torch().tensor([int(x) for x in v], dtype=_torch().int32, device="cuda")


class Prompt:
    """Random prompts: nq and nk tokens and keys a request; rows before the first and behind the last request."""

    def __init__(self, smla, nq, nk, heads, kv_heads, rope=64, causal=True, prefix=None, cap=0.0, bias=False, sink=False, seed=0,
                 lead=2, layout="kv", spread=2.0):
        torch = _torch()
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.smla, self.causal, self.cap = smla, causal, cap
        self.cu_q = lead + np.concatenate([[0], np.cumsum(nq)]).astype(np.int64)
        self.cu_k = lead + np.concatenate([[0], np.cumsum(nk)]).astype(np.int64)
        T, N = int(self.cu_q[-1]) + 3, int(self.cu_k[-1]) + 1
        self.T, self.N, self.H, self.HK, self.rope_dim = T, N, heads, kv_heads, rope
        D = 128 + rope
        rnd = lambda *n: torch.randn(n, generator=g, device="cuda")  # noqa: E731
        if layout == "heads":  # heads before tokens, rows with a gap
            self.q = (rnd(heads, T, D + 8) * spread).to(torch.bfloat16)[..., :D].permute(1, 0, 2)
            kv = rnd(2, kv_heads, N, 136).to(torch.bfloat16)[..., :128].permute(0, 2, 1, 3)
            self.k, self.v = kv[0], kv[1]
        else:
            self.q = (rnd(T, heads, D) * spread).to(torch.bfloat16)
            kv = rnd(N, kv_heads, 256).to(torch.bfloat16)
            self.k, self.v = kv[..., :128], kv[..., 128:]
        self.rope = rnd(N, 64).to(torch.bfloat16) if rope else None
        self.prefix = prefix
        self.slopes = torch.exp2(-torch.arange(heads, device="cuda") * 8.0 / heads) if bias else None
        self.sink = rnd(heads) if sink else None
        self.out = torch.full((T, heads, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((T, heads), 7.0, device="cuda")
        self.scale = float(np.float32(D ** -0.5))
        self.desc = smla.make_prompt_desc(T, N, heads, kv_heads, len(nq), rope, self.scale, causal=causal, softcap=cap,
                                          q_strides=self.q.stride()[:2], k_strides=self.k.stride()[:2], v_strides=self.v.stride()[:2])
        self.ws = torch.zeros(smla.prompt_workspace_size(self.desc), dtype=torch.uint8, device="cuda")

    def run(self):
        self.smla.prompt_attention(self.desc, self.q, self.k, self.v, self.rope, _i32(self.cu_q), _i32(self.cu_k),
                                   None if self.prefix is None else _i32(self.prefix), self.slopes, self.sink, self.out, self.lse,
                                   self.ws)
        return self

    def oracle(self):
        f = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
        return PO.prompt_attention(f(self.q), f(self.k), f(self.v), f(self.rope), self.cu_q, self.cu_k, self.scale, self.causal,
                                   self.prefix, self.cap, f(self.slopes), f(self.sink))

    def check(self, flags=0):
        out, lse, A, big = self.oracle()
        got, gl = self.out.double().cpu().numpy(), self.lse.double().cpu().numpy()
        assert self.smla.read_error(None, self.ws) == flags
        real = ~np.isnan(lse)
        none = np.ones(self.T, bool)
        none[int(self.cu_q[0]):int(self.cu_q[-1])] = False
        assert (got[none] == 7).all() and (gl[none] == 7).all()
        # scores: 192 products and sums of 2^-24 each of the terms' size, the cap 2^-20 of itself; the sum of weights
        # n 2^-24, exponentials 2^-22. Each weight enters PV off by 2^-8 of itself at most, and the result is rounded to bf16.
        keys = max([int(b - a) for a, b in zip(self.cu_k[:-1], self.cu_k[1:])] + [1])
        e = big * 200 * 2.0 ** -24 + self.cap * 2.0 ** -20 + keys * 2.0 ** -24 + 2.0 ** -20
        assert np.array_equal(np.isneginf(gl[real]), np.isneginf(lse[real]))
        f = real & np.isfinite(lse)
        assert (np.abs(gl - np.where(f, lse, 0))[f] <= (e + np.abs(np.where(f, lse, 0)) * 2.0 ** -22)[f]).all(), \
            np.nanmax(np.abs(gl - lse)[f])
        ok = np.isfinite(out)
        tol = A * (2.0 ** -8 + 2 * e[..., None]) + np.abs(np.where(ok, out, 0)) * 2.0 ** -8 + 1e-30
        bad = ok & ~(np.abs(got - np.where(ok, out, 0)) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], out[bad][:4], bad.sum())
        return out, lse


CASES = [
    dict(nq=[24], nk=[24], heads=4, kv_heads=4),
    dict(nq=[1], nk=[1], heads=1, kv_heads=1),
    dict(nq=[128], nk=[128], heads=2, kv_heads=2),
    dict(nq=[256], nk=[256], heads=2, kv_heads=1, rope=0),
    dict(nq=[257], nk=[300], heads=2, kv_heads=2, sink=True),
    dict(nq=[300, 1, 0, 129, 64], nk=[300, 1, 0, 700, 65], heads=3, kv_heads=3),
    dict(nq=[300, 40], nk=[500, 40], heads=4, kv_heads=2, causal=False),
    dict(nq=[200, 131], nk=[200, 260], heads=4, kv_heads=4, prefix=[77, 200]),
    dict(nq=[200, 131, 5], nk=[200, 260, 9], heads=8, kv_heads=2, rope=0, prefix=[500, -3, 1], bias=True),
    dict(nq=[150, 33], nk=[400, 33], heads=4, kv_heads=4, cap=20.0),
    dict(nq=[150, 33], nk=[400, 33], heads=4, kv_heads=4, cap=5.0, bias=True, sink=True, rope=0),
    dict(nq=[150, 33], nk=[400, 150], heads=4, kv_heads=2, bias=True),
    dict(nq=[700], nk=[1500], heads=2, kv_heads=2),
    dict(nq=[5, 3], nk=[0, 2], heads=2, kv_heads=2),               # no keys, and tokens that stand before the first key
    dict(nq=[300], nk=[100], heads=2, kv_heads=1, sink=True),
    dict(nq=[300, 2], nk=[100, 1], heads=3, kv_heads=1, prefix=[10, 0], rope=0),
    dict(nq=[1, 1, 1], nk=[5000, 1, 130], heads=8, kv_heads=2, rope=0),  # single tokens
    dict(nq=[1, 1], nk=[3000, 777], heads=4, kv_heads=4),
    dict(nq=[1], nk=[20000], heads=2, kv_heads=1, cap=30.0),       # one token over many SMs
    dict(nq=[3], nk=[9001], heads=12, kv_heads=4, rope=0, bias=True, sink=True),
    dict(nq=[40], nk=[40], heads=256, kv_heads=2, rope=0),         # a group of 128 heads
    dict(nq=[40], nk=[41], heads=96, kv_heads=2),                  # of 48: sixteen beside one another
    dict(nq=[600], nk=[5000], heads=2, kv_heads=2, causal=False),
    dict(nq=[260], nk=[900], heads=2, kv_heads=2, cap=300.0),      # small beside the cap: by the polynomial
    dict(nq=[260], nk=[900], heads=2, kv_heads=2, cap=0.5, rope=0),  # and all but cut off
    dict(nq=[1, 130], nk=[2600, 131], heads=2, kv_heads=2, prefix=[5, 131], bias=True),
    dict(nq=[130], nk=[300], heads=2, kv_heads=2, cap=1e-7),       # whose polynomial's powers would leave fp32
    dict(nq=[130], nk=[300], heads=2, kv_heads=2, cap=1e30),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()).replace(" ", ""))
@pytest.mark.parametrize("layout", ["kv", "heads"])
def test_against_float64(smla, case, layout):
    Prompt(smla, **case, seed=3, layout=layout).run().check()


def test_many_small_requests(smla):
    r = np.random.default_rng(5)
    nq = r.integers(0, 4, 700)
    nk = nq + r.integers(0, 200, 700)
    Prompt(smla, nq.tolist(), nk.tolist(), 2, 1, rope=64, seed=4).run().check()


def test_a_long_request_among_many(smla):
    """More requests than a warp lays out, one of them over many SMs."""
    r = np.random.default_rng(6)
    nq = r.integers(0, 3, 60)
    nk = nq + r.integers(0, 90, 60)
    nq[[17, 41]], nk[[17, 41]] = [1, 150], [9000, 2000]
    Prompt(smla, nq.tolist(), nk.tolist(), 4, 2, rope=0, seed=18).run().check()


@pytest.mark.parametrize("heads,kv_heads,rope", [(7, 7, 64), (8, 8, 0), (10, 5, 64), (9, 3, 0)])
@pytest.mark.parametrize("requests", [30, 90])
def test_requests_of_one_row_tile(smla, heads, kv_heads, rope, requests):
    """More of them than SMs, each of a few tokens over a few key tiles, and a value that spoils one head of one of them."""
    r = np.random.default_rng(heads)
    nq = r.integers(0, 65 if heads == kv_heads else 30, requests)
    nk = nq + r.integers(0, 400, requests)
    nq[3], nk[3], nq[4], nk[4] = 1, 1, 3, 2
    p = Prompt(smla, nq.tolist(), nk.tolist(), heads, kv_heads, rope=rope, seed=23, sink=heads == 8, cap=20.0 if heads == 10 else 0.0,
               bias=heads == 9).run()
    p.check()
    # a value that one head's later tokens alone see
    torch = _torch()
    out, lse = p.out.clone(), p.lse.clone()
    big = int(np.argmax(nq))
    j, h = int(nk[big]) - 1 - int(nq[big]) // 2, kv_heads // 2
    p.v[int(p.cu_k[big]) + j, h, 9] = float("nan")
    p.run()
    first, g = int(p.cu_q[big]) + j - int(nk[big] - nq[big]), heads // kv_heads
    same = torch.ones((p.T, heads), dtype=torch.bool, device="cuda")
    same[first:int(p.cu_q[big + 1]), h * g:h * g + g] = False
    assert torch.equal(p.out[same], out[same]) and torch.equal(p.lse, lse)
    assert torch.isnan(p.out[first:int(p.cu_q[big + 1]), h * g].float()).any(-1).all()


def test_single_tokens_of_many_heads_over_long_contexts(smla):
    """More heads than SMs, and items that several SMs share."""
    Prompt(smla, [1, 2, 1], [9000, 5000, 700], 60, 60, seed=24).run().check()


def test_single_head_group_of_many_blocks(smla):
    """128 query heads on one kv head: two tokens a row tile pair, more blocks than a warp has lanes."""
    Prompt(smla, [300, 7], [310, 500], 128, 1, rope=64, seed=19).run().check()


@pytest.mark.parametrize("heads,requests", [(256, 1), (128, 35)])
def test_items_off_the_counter(smla, heads, requests):
    """More short items than SMs: a few heads of the result against float64."""
    torch = _torch()
    nq = [1500] if requests == 1 else [300] * requests
    p = Prompt(smla, nq, nq, heads, heads, seed=20, sink=True).run()
    sel = [0, 1, heads // 2, heads - 1]
    p.q, p.k, p.v, p.sink = p.q[:, sel], p.k[:, sel], p.v[:, sel], p.sink[sel]
    p.out, p.lse, p.H, p.HK = p.out[:, sel], p.lse[:, sel], 4, 4
    p.check()
    assert torch.isfinite(p.out.float()).all()


@pytest.mark.parametrize("case", [dict(nq=[1, 1], nk=[3000, 777], heads=4, kv_heads=4), dict(nq=[700], nk=[1500], heads=2, kv_heads=2),
                                  dict(nq=[1], nk=[20000], heads=2, kv_heads=1, cap=30.0)])
def test_the_first_call_on_a_workspace_is_as_good_as_any(smla, case):
    """Parts of cut items that are read before they are written would be zeros here, and right ones in later calls."""
    torch = _torch()
    first = Prompt(smla, **case, seed=22).run()
    again = first.out.clone()
    first.run()
    real = slice(int(first.cu_q[0]), int(first.cu_q[-1]))
    assert torch.equal(first.out[real], again[real])
    for _ in range(8):
        p = Prompt(smla, **case, seed=22).run()
        assert torch.equal(p.out[real], again[real]) and torch.equal(p.lse, first.lse)


def test_output_on_a_border_of_sixteen_bytes_and_no_lse(smla):
    torch = _torch()
    p = Prompt(smla, [70, 300], [400, 300], 3, 3, seed=25, sink=True).run()
    want = p.out.clone()
    room = torch.full((p.out.numel() + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    p.out, lse, p.lse = room[8:].view(want.shape), p.lse, None
    assert p.out.data_ptr() % 32 == 16
    p.run()
    assert torch.equal(p.out, want)
    p.lse = lse
    p.check()


def test_large_scores_and_equal_ones(smla):
    Prompt(smla, [90], [400], 2, 2, seed=8, spread=40.0).run().check()
    for cap in (0.0, 1e-7, 30.0):
        p = Prompt(smla, [90], [400], 2, 2, seed=9, cap=cap)
        p.q.zero_()
        p.run().check()
    # the maximum grows from key tile to key tile: the sums are rescaled every time
    p = Prompt(smla, [130], [1300], 2, 2, seed=10)
    p.q.fill_(1.0)
    p.k.copy_((_torch().arange(p.N, device="cuda")[:, None, None] / 90.0).to(p.k.dtype).expand_as(p.k))
    p.run().check()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_hidden_values_that_are_not_finite(smla, value):
    nq, nk = [200, 70, 1], [333, 70, 140]
    p = Prompt(smla, nq, nk, 2, 2, seed=11).run()
    out, lse = p.out.clone(), p.lse.clone()
    # rows of no request, and a whole request
    p.k[:int(p.cu_k[0])] = value
    p.v[:int(p.cu_k[0])] = value
    p.rope[int(p.cu_k[3]):] = value
    p.v[int(p.cu_k[3]):] = value
    p.k[int(p.cu_k[1]):int(p.cu_k[2])] = value
    p.v[int(p.cu_k[1]):int(p.cu_k[2])] = value
    p.run()
    keep = np.ones(p.T, bool)
    keep[int(p.cu_q[1]):int(p.cu_q[2])] = False
    torch = _torch()
    keep = torch.from_numpy(keep).cuda()
    assert torch.equal(p.out[keep], out[keep]) and torch.equal(p.lse[keep], lse[keep])
    # one value of the first request: the tokens before it do not see it
    p = Prompt(smla, nq, nk, 2, 2, seed=11)
    j, h = 250, 1
    p.v[int(p.cu_k[0]) + j, h, 5] = value
    p.run()
    first = int(p.cu_q[0]) + j - (nk[0] - nq[0])  # the token that stands at it
    same = torch.ones((p.T, 2), dtype=torch.bool, device="cuda")
    same[first:int(p.cu_q[1]), h] = False
    assert torch.equal(p.out[same], out[same]) and torch.equal(p.lse, lse)
    assert not torch.isfinite(p.out[first:int(p.cu_q[1]), h].float()).all(-1).any()
    # and a key
    p = Prompt(smla, nq, nk, 2, 2, seed=11)
    p.k[int(p.cu_k[0]) + j, h] = value
    p.run()
    assert torch.equal(p.out[same], out[same]) and torch.equal(p.lse[same], lse[same])


def test_values_that_are_not_finite_in_cut_items(smla):
    torch = _torch()
    p = Prompt(smla, [130], [9000], 1, 1, seed=12).run()
    out, lse = p.out.clone(), p.lse.clone()
    p.v[int(p.cu_k[0]) + 8950, 0, 3] = float("nan")
    p.run()
    first = int(p.cu_q[0]) + 8950 - (9000 - 130)
    assert torch.equal(p.out[:first], out[:first]) and torch.equal(p.lse, lse)
    assert torch.isnan(p.out[first:int(p.cu_q[1])].float()).all()


def test_offsets_that_do_not_fit(smla):
    torch = _torch()
    for cq, ck in (([0, 50, 40], [0, 100, 150]), ([0, 50, 90], [0, 100, 90]), ([-1, 50, 90], [0, 100, 150]),
                   ([0, 50, 1000], [0, 100, 150]), ([0, 50, 90], [0, 100, 1000])):
        p = Prompt(smla, [50, 40], [100, 50], 2, 2, seed=13, lead=0)
        p.cu_q, p.cu_k = np.asarray(cq), np.asarray(ck)
        p.run()
        assert smla.read_error(None, p.ws) == smla.SMLA_DEVERR_INDEX
        bad = 0 if cq[0] < 0 else 1
        other = slice(50, 90) if bad == 0 else slice(0, 50)
        assert (p.out[slice(0, 50) if bad == 0 else slice(50, 93)] == 7).all()
        assert torch.isfinite(p.out[other].float()).all() and not (p.out[other] == 7).all()


def test_results_do_not_change_from_call_to_call(smla):
    torch = _torch()
    p = Prompt(smla, [1, 200, 3], [12000, 4000, 700], 4, 4, seed=14).run()
    out, lse = p.out.clone(), p.lse.clone()
    for _ in range(10):
        p.out.fill_(0)
        p.run()
        real = slice(int(p.cu_q[0]), int(p.cu_q[-1]))
        assert torch.equal(p.out[real], out[real]) and torch.equal(p.lse, lse)


def test_captured_call_serves_other_lengths(smla):
    torch = _torch()
    p = Prompt(smla, [100, 200], [400, 200], 4, 2, seed=15, lead=0)
    cu_q, cu_k = _i32(p.cu_q), _i32(p.cu_k)

    def call():
        smla.prompt_attention(p.desc, p.q, p.k, p.v, p.rope, cu_q, cu_k, None, None, None, p.out, p.lse, p.ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        call()
    for nq, nk in (([100, 200], [400, 200]), ([3, 290], [5, 595]), ([1, 0], [600, 0])):
        p.cu_q, p.cu_k = np.asarray([0, nq[0], sum(nq)]), np.asarray([0, nk[0], sum(nk)])
        p.out.fill_(7.0)
        p.lse.fill_(7.0)
        cu_q.copy_(_i32(p.cu_q))
        cu_k.copy_(_i32(p.cu_k))
        g.replay()
        p.check()


def test_two_streams_with_their_own_workspaces(smla):
    torch = _torch()
    a = Prompt(smla, [300, 1], [2000, 9000], 4, 4, seed=16)
    b = Prompt(smla, [150], [8000], 4, 2, seed=17, rope=0, cap=10.0)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(sa):
            a.run()
        with torch.cuda.stream(sb):
            b.run()
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_a_prompt_from_hidden_states_to_log_probabilities(smla):
    """Norm, the cache write, the context read back, the expansion to heads, attention, log probabilities: a second chunk
    of two prompts over what the first left in the cache."""
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(21)
    H, P, dim, vocab = 4, 16, 256, 1003
    past, new = [70, 3], [40, 19]
    nk = [a + b for a, b in zip(past, new)]
    T, N, pages = sum(new), sum(nk), 12
    rnd = lambda *n: (torch.randn(n, generator=g, device="cuda") / n[-1] ** 0.5).to(torch.bfloat16)  # noqa: E731
    hidden, res = (torch.randn((T, dim), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    wn, wq, wkv, wup, wo = torch.ones(dim, device="cuda").to(torch.bfloat16), rnd(H * 192, dim), rnd(576, dim), rnd(H * 256, 512), rnd(vocab, H * 128)
    y = torch.empty_like(hidden)
    smla.add_rmsnorm(hidden, res, wn, 1e-6, residual_out=res, y=y)
    q = (y @ wq.T).view(T, H, 192)
    lat = y @ wkv.T
    kv = torch.zeros((pages, P, 656), dtype=torch.uint8, device="cuda")
    table = torch.full((2, 8), -1, dtype=torch.int32)
    table[0, :7], table[1, :2] = torch.tensor([9, 2, 5, 0, 11, 4, 7]), torch.tensor([3, 8])
    old = torch.randn((pages * P, 576), generator=g, device="cuda").to(torch.bfloat16)
    smla.pack_kv(1, 0, old[:, :512].contiguous(), old[:, 512:].contiguous(), torch.arange(pages * P, device="cuda"), kv, pages * P)
    slots = torch.cat([table[r, torch.arange(past[r], nk[r]) // P].long() * P + torch.arange(past[r], nk[r]) % P for r in range(2)]).cuda()
    smla.pack_kv(1, 0, lat[:, :512].contiguous(), lat[:, 512:].contiguous(), slots, kv, pages * P)
    cu_q, cu_k = _i32([0, new[0], T]), _i32([0, nk[0], N])
    back, rope = torch.empty((N, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((N, 64), dtype=torch.bfloat16, device="cuda")
    err = _i32([0])
    smla.cache_read(smla.make_read_desc(1, P, pages, 2, 8, N), kv, table.cuda(), _i32([0, 0]), cu_k, back, rope, err)
    up = (back @ wup.T).view(N, H, 256)
    out, lse = torch.empty((T, H, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((T, H), device="cuda")
    d = smla.make_prompt_desc(T, N, H, H, 2, 64, 192 ** -0.5, k_strides=up.stride()[:2], v_strides=up.stride()[:2])
    ws = torch.zeros(smla.prompt_workspace_size(d), dtype=torch.uint8, device="cuda")
    smla.prompt_attention(d, q, up[..., :128], up[..., 128:], rope, cu_q, cu_k, None, None, None, out, lse, ws)
    logits = (out.view(T, H * 128) @ wo.T).float()
    tokens = torch.randint(0, vocab, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    lp, ent = torch.empty((T, 1), device="cuda"), torch.empty(T, device="cuda")
    smla.token_logprobs(logits, tokens, lp, entropy=ent, error_word=err)
    assert err.item() == 0 and smla.read_error(None, ws) == 0
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    want, wl, A, big = PO.prompt_attention(f(q), f(up[..., :128]), f(up[..., 128:]), f(rope), [0, new[0], T], [0, nk[0], N], 192 ** -0.5)
    e = big * 200 * 2.0 ** -24 + 2.0 ** -19
    assert (np.abs(f(out) - want) <= A * (2.0 ** -8 + 2 * e[..., None]) + np.abs(want) * 2.0 ** -8).all()
    assert (np.abs(f(lse) - wl) <= e + np.abs(wl) * 2.0 ** -22).all()
    glp, gent, _, _ = PO.token_logprobs(f(logits), tokens.cpu().numpy(), 0)
    assert np.abs(f(lp) - glp).max() <= 1e-5 and np.abs(f(ent) - gent).max() <= 1e-5
