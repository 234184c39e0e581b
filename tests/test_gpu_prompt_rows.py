"""Cache rows read back, the norm and the log probabilities against float64, on the GPU."""
import numpy as np
import pytest

import oracle.prompt_oracle as PO
import oracle.smla_oracle as O

pytestmark = pytest.mark.gpu
FMT = {"bf16": 0, "fp8_ds": 1, "fp8_tensor": 2}


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


# ---------------------------------------------------------------- cache rows


def _cache(fmt, rows, seed):
    torch = _torch()
    g = torch.Generator().manual_seed(seed)
    if fmt == "bf16":
        raw = torch.randn((rows, 576), generator=g).to(torch.bfloat16).view(torch.uint8)
    elif fmt == "fp8_tensor":
        raw = torch.randn((rows, 576), generator=g).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        codes = (torch.randn((rows, 512), generator=g) * 50).to(torch.float8_e4m3fn).view(torch.uint8)
        scales = torch.exp2(torch.randn((rows, 4), generator=g)).view(torch.uint8)
        rope = torch.randn((rows, 64), generator=g).to(torch.bfloat16).view(torch.uint8)
        raw = torch.cat([codes, scales, rope], 1)
    return raw.contiguous()


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("page,lens,starts", [
    (64, [200, 0, 1, 63], [0, 5, 64, 1]), (1, [3, 17], [2, 0]), (16, [0, 0], [0, 0]), (256, [1000], [24]),
    (4, [1 + (i * 7) % 90 for i in range(150)], [(i * 5) % 11 for i in range(150)])])
def test_read(smla, fmt, page, lens, starts):
    torch = _torch()
    need = [-(-(a + n) // page) for a, n in zip(starts, lens)]
    stride, pool = max(max(need), 1), sum(need) + 3
    perm = np.random.default_rng(1).permutation(pool)
    table = np.full((len(lens), stride), -1, dtype=np.int64)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n
    raw = _cache(fmt, pool * page, 2)
    cu = 2 + np.concatenate([[0], np.cumsum(lens)])  # two rows before the first request, three behind the last
    N = int(cu[-1]) + 3
    latent = torch.full((N, 520), 7.0, dtype=torch.bfloat16, device="cuda")
    rope = torch.full((N, 72), 7.0, dtype=torch.bfloat16, device="cuda")
    err = _i32([0])
    d = smla.make_read_desc(FMT[fmt], page, pool, len(lens), stride, N, kv_scale=0.7, latent_stride=520, rope_stride=72)
    smla.cache_read(d, raw.cuda(), _i32(table.tolist()), _i32(starts), _i32(cu.tolist()), latent, rope, err)
    want = torch.full((N, 576), 7.0, dtype=torch.bfloat16)
    for r, n in enumerate(lens):
        if n:
            s = starts[r] + np.arange(n)
            keys = O.dequant_rows(raw.numpy()[table[r, s // page] * page + s % page], fmt, float(np.float32(0.7)))
            want[cu[r]:cu[r + 1]] = torch.from_numpy(np.asarray(keys).astype(np.float32)).to(torch.bfloat16)
    assert err.item() == 0
    assert torch.equal(latent[:, :512].cpu(), want[:, :512]) and torch.equal(rope[:, :64].cpu(), want[:, 512:])
    assert (latent[:, 512:] == 7).all() and (rope[:, 64:] == 7).all()


def test_read_entries_that_are_no_pages(smla):
    torch = _torch()
    raw = _cache("bf16", 4 * 16, 3)
    table = _i32([[0, 9, 1], [-1, 2, 3]])
    latent = torch.full((70, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    rope = torch.full((70, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    err = _i32([0])
    d = smla.make_read_desc(0, 16, 4, 2, 3, 70)
    smla.cache_read(d, raw.cuda(), table, _i32([0, 0]), _i32([0, 40, 70]), latent, rope, err)
    assert err.item() == smla.SMLA_DEVERR_PAGE
    assert (latent[16:32] == 0).all() and (latent[40:56] == 0).all() and (rope[16:32] == 0).all()
    assert torch.equal(latent[32:40].cpu(), raw.view(torch.bfloat16)[16:24, :512])
    for starts in ([-3, 0], [40, 0]):  # slots before the first and past the last page of the table
        err.zero_()
        smla.cache_read(d, raw.cuda(), _i32([[0, 1, 2], [3, 2, 1]]), _i32(starts), _i32([0, 40, 70]), latent, rope, err)
        assert err.item() == smla.SMLA_DEVERR_INDEX
        none = slice(0, 3) if starts[0] < 0 else slice(8, 40)
        assert (latent[none] == 0).all()
    for cu in ([0, -5, 3], [60, 20, 10], [-9, -5, -1], [500, 600, 700]):  # offsets that do not ascend, or lie outside
        latent.fill_(7.0)
        smla.cache_read(d, raw.cuda(), _i32([[0, 1, 2], [3, 2, 1]]), _i32([0, 0]), _i32(cu), latent, rope, err)
    torch.cuda.synchronize()
    assert (latent == 7).all()


# ---------------------------------------------------------------- the norm


def _check_norm(smla, n, dim, residual, group, mode, eps=1e-6, x_stride=None, zero_row=False, alias=False, seed=0):
    torch = _torch()
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, x_stride or dim), generator=g) * torch.exp2(torch.randint(-3, 8, (n, 1), generator=g).float())
    x[:, ::37] *= 20
    if zero_row:
        x[0] = 0
        x[-1, : min(dim, 128)] = 0
    x = x.to(torch.bfloat16).cuda()[:, :dim]
    res = torch.randn((n, dim), generator=g).to(torch.bfloat16).cuda() if residual else None
    if residual and zero_row:
        res[0] = 0
    w = (1 + 0.3 * torch.randn((dim,), generator=g)).to(torch.bfloat16).cuda()
    x64, r64 = x.double().cpu().numpy(), None if res is None else res.double().cpu().numpy()
    blocks = -(-dim // 128) if group else 1
    codes = torch.full((n, dim), 255, dtype=torch.uint8, device="cuda")
    scales = torch.full((n, blocks), -1.0, device="cuda")
    total = res if alias else torch.empty((n, dim), dtype=torch.bfloat16, device="cuda")
    y = x if alias and x.is_contiguous() else torch.empty((n, dim), dtype=torch.bfloat16, device="cuda")
    smla.add_rmsnorm(x, res, w, eps, residual_out=total, y=y, codes=codes, scales=scales, group=group, scale_mode=mode)
    h, ref, amax = PO.add_rmsnorm(x64, r64, w.double().cpu().numpy(), eps, group)
    # the sum is rounded twice: fp32, then bf16
    assert (np.abs(total.double().cpu().numpy() - h) <= np.abs(h) * (2.0 ** -8 + 2.0 ** -23)).all()
    # y: the fp32 sum of squares, in at most 4 * 8 + 10 steps of 2^-24, the root halves its error; five roundings more
    rel = 32 * 2.0 ** -24
    assert (np.abs(y.double().cpu().numpy() - ref) <= np.abs(ref) * (2.0 ** -8 + rel)).all()
    s = scales.double().cpu().numpy()
    ratio = amax / 448
    if mode == smla.SMLA_SCALE_FP32:
        assert (np.abs(s - np.where(amax == 0, 1.0, ratio)) <= np.where(amax == 0, 0, ratio * (rel + 2.0 ** -24))).all()
    else:
        assert (np.exp2(np.round(np.log2(s))) == s).all()
        live = amax > 0
        assert (s[live] >= ratio[live] * (1 - 2 * rel)).all() and (s[live] / 2 < ratio[live] * (1 + 2 * rel)).all()
        assert (s[~live] == 1).all()
    width = group or dim
    value = O.e4m3_decode(codes.cpu().numpy()) * np.repeat(s, width, 1)[:, :dim]
    step = np.repeat(s, width, 1)[:, :dim] * 2.0 ** -10  # half a step of the subnormal codes
    assert (np.abs(value - ref) <= np.maximum(np.abs(ref) * 2.0 ** -4, step) + np.abs(ref) * 2 * rel).all()


@pytest.mark.parametrize("n,dim", [(1, 8), (5, 64), (9, 136), (17, 512), (3, 1024), (2, 1032), (33, 1536), (4, 7168), (2, 16384),
                                   (1, 32768), (2, 10008), (300, 128), (1001, 248)])
@pytest.mark.parametrize("residual,group,mode", [(True, 128, 0), (False, 0, 1), (True, 0, 0), (False, 128, 1)])
def test_norm(smla, n, dim, residual, group, mode):
    _check_norm(smla, n, dim, residual, group, mode, seed=n + dim)


def test_norm_of_a_slice_zero_rows_and_in_place(smla):
    _check_norm(smla, 6, 1536, False, 128, 0, x_stride=2112)  # q's part of one projection's output
    _check_norm(smla, 6, 512, True, 0, 1, x_stride=576)
    _check_norm(smla, 6, 2048, True, 128, 0, zero_row=True)
    _check_norm(smla, 6, 256, True, 0, 0, zero_row=True, eps=1e-3)
    _check_norm(smla, 40, 7168, True, 128, 0, alias=True)


@pytest.mark.parametrize("dim", [96, 1024, 7168])
@pytest.mark.parametrize("group", [128, 0])
@pytest.mark.parametrize("mode", [0, 1])
def test_codes_are_those_of_the_rounded_quotient(smla, dim, group, mode):
    """Rows of +-1 have the norm 1, so y is the weight exactly: scales and codes bit for bit."""
    torch = _torch()
    g = torch.Generator().manual_seed(dim + group)
    x = torch.where(torch.rand((6, dim), generator=g) < 0.5, -1.0, 1.0).to(torch.bfloat16)
    w = torch.randn((dim,), generator=g) * torch.exp2(torch.randint(-30, 12, (dim,), generator=g).float())
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
        assert np.array_equal(scales[:, b // width].cpu().numpy(), scale.astype(np.float32))
        want = O.e4m3_encode_rne_satfinite((part / scale[:, None].astype(np.float32)).astype(np.float32))
        got = codes[:, b:b + width].cpu().numpy()
        assert np.array_equal(O.e4m3_decode(got), O.e4m3_decode(want))


def test_norm_single_outputs(smla):
    torch = _torch()
    x = torch.randn((5, 640), device="cuda").to(torch.bfloat16)
    w = torch.ones(640, device="cuda").to(torch.bfloat16)
    y, y2, total = (torch.empty_like(x) for _ in range(3))
    codes = torch.empty((5, 640), dtype=torch.uint8, device="cuda")
    codes2, scales, scales2 = torch.empty_like(codes), torch.empty((5, 5), device="cuda"), torch.empty((5, 5), device="cuda")
    smla.add_rmsnorm(x, x, w, 1e-6, residual_out=total, y=y, codes=codes, scales=scales)
    smla.add_rmsnorm(x, x, w, 1e-6, y=y2)
    smla.add_rmsnorm(x, x, w, 1e-6, codes=codes2, scales=scales2)
    assert torch.equal(y, y2) and torch.equal(codes, codes2) and torch.equal(scales, scales2)
    assert torch.equal(total, x + x)


# ---------------------------------------------------------------- log probabilities


def _check_logprobs(smla, x, tokens, top, scale=1.0, ids_too=True):
    torch = _torch()
    n, v = x.shape
    tok = torch.tensor(tokens, dtype=torch.int32, device="cuda")
    lp, ent = torch.full(tok.shape, 7.0, device="cuda"), torch.full((n,), 7.0, device="cuda")
    ids = torch.full((n, top), -7, dtype=torch.int32, device="cuda") if top else None
    alt = torch.full((n, top), 7.0, device="cuda") if top else None
    err = _i32([0])
    smla.token_logprobs(x, tok, lp, entropy=ent, top_ids=ids, top_logprobs=alt, scale=scale, error_word=err)
    x64 = x.double().cpu().numpy()
    want, went, wids, walt = PO.token_logprobs(x64, np.asarray(tokens), top, float(np.float32(scale)))
    outside = any(t != -1 and not 0 <= t < v for row in tokens for t in row)
    assert err.item() == (smla.SMLA_DEVERR_INDEX if outside else 0)
    # a thread adds up v / 256 terms one after another (2^-24 each); the exponentials are 2^-22 off, their arguments by
    # 2^-23 of their size, and so is the difference of a logit and the largest
    with np.errstate(invalid="ignore"):
        span = np.nan_to_num(np.abs(want), posinf=0, neginf=0)
        z = x64 * scale
        zmax = np.nan_to_num(np.abs(z), posinf=0, neginf=0).max(1)
    base = (v / 256 + 40) * 2.0 ** -24 + 2.0 ** -21
    tol = base + (2 * zmax[:, None] + span + 20) * 2.0 ** -22
    got = lp.double().cpu().numpy()
    assert np.array_equal(np.isfinite(got), np.isfinite(want)) and np.array_equal(np.isnan(got), np.isnan(want))
    f = np.isfinite(want)
    assert (np.abs(got - want)[f] <= tol[f]).all(), np.abs(got - want)[f].max()
    ge = ent.double().cpu().numpy()
    assert np.array_equal(np.isnan(ge), np.isnan(went))
    f = np.isfinite(went)
    # W / S: the terms' errors weigh with their distance from the largest, at most 60 where they count
    assert (np.abs(ge - went)[f] <= 2 * (base + 4 * 2.0 ** -22) * (went[f] + 16) + (2 * zmax[f] + 20) * 2.0 ** -22 * 4).all()
    if top and ids_too:
        assert np.array_equal(ids.cpu().numpy(), wids)
        ga = alt.double().cpu().numpy()
        f = np.isfinite(walt)
        assert np.array_equal(np.isfinite(ga), f)
        t2 = base + (2 * zmax[:, None] + np.abs(np.where(f, walt, 0)) + 20) * 2.0 ** -22
        assert (np.abs(ga - walt)[f] <= t2[f]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,v,g,k", [(1, 1, 1, 1), (2, 7, 2, 20), (1, 129280, 1, 20), (3, 32003, 1, 5), (40, 5001, 7, 64), (200, 999, 1, 33),
                                     (5, 2049, 0, 3), (4, 70001, 3, 0), (170, 16384, 1, 1),
                                     (700, 1862, 2, 20), (900, 4096, 1, 64), (64, 40001, 7, 20), (11, 70001, 1, 33)])
def test_logprobs(smla, dtype, n, v, g, k):
    torch = _torch()
    gen = torch.Generator().manual_seed(n * 1000 + v)
    x = (torch.randn((n, v), generator=gen) * 3).to(torch.float32 if dtype == "f32" else torch.bfloat16).cuda()
    tokens = torch.randint(0, v, (n, g), generator=gen).tolist() if g else [[] for _ in range(n)]
    _check_logprobs(smla, x, tokens, k, scale=1.0 if n % 2 else 0.7)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 160])
def test_logprobs_of_rows_that_fill_the_candidates(smla, dtype, n):
    torch = _torch()
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    v = 20011
    ramp = torch.arange(v, dtype=torch.float32) / v * 8
    some = torch.full((v,), -float("inf"))
    some[[5, 4000, 19000]] = torch.tensor([1.0, 2.0, 2.0])
    rows = [torch.zeros(v), ramp, ramp.flip(0), some, torch.where(torch.arange(v) % 2 == 0, 0.0, -0.0), -3e38 * (ramp / 8)]
    x = torch.stack([rows[i % 6] for i in range(6 if n == 1 else n)]).to(t).cuda()
    _check_logprobs(smla, x, [[i * 13 % v] for i in range(x.shape[0])], 20)
    _check_logprobs(smla, x[:1].contiguous(), [[3]], 64)


def test_logprobs_strides_and_tokens_outside(smla):
    torch = _torch()
    big = torch.randn((6, 3001), device="cuda")
    _check_logprobs(smla, big[:, 1:2999], [[-1, 0], [2997, 2998], [-2, 5], [1 << 30, 7], [3, -1], [0, 1]], 9)
    b16 = big.to(torch.bfloat16)
    for off in (1, 2, 3, 5, 7):
        _check_logprobs(smla, b16[:, off:off + 2900], [[0]] * 6, 4)
        _check_logprobs(smla, b16[:2, off:off + 5], [[4]] * 2, 4)


def test_logprobs_that_are_not_finite(smla):
    torch = _torch()
    x = torch.randn((4, 3000), device="cuda")
    x[0, 17] = float("nan")
    x[1, 2500] = float("inf")
    x[2] = -float("inf")
    _check_logprobs(smla, x, [[5], [5], [5], [5]], 4, ids_too=False)
    ids = torch.full((4, 4), -7, dtype=torch.int32, device="cuda")
    smla.token_logprobs(x, None, None, top_ids=ids)
    got = ids.cpu().numpy()
    assert ((got >= -1) & (got < 3000)).all() and got[1, 0] == 2500 and got[2].tolist() == [0, 1, 2, 3]
    assert all(len(set(r)) == 4 for r in got[1:].tolist())


def test_captured_on_another_stream(smla):
    torch = _torch()
    x = torch.randn((8, 4096), device="cuda").to(torch.bfloat16)
    w = torch.ones(4096, device="cuda").to(torch.bfloat16)
    y = torch.empty_like(x)
    lp, ids = torch.empty((8, 1), device="cuda"), torch.empty((8, 3), dtype=torch.int32, device="cuda")
    tok = _i32([[i] for i in range(8)])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            smla.add_rmsnorm(x, None, w, 1e-6, y=y)
            smla.token_logprobs(y, tok, lp, top_ids=ids)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    want = (y.clone(), lp.clone(), ids.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        smla.add_rmsnorm(x, None, w, 1e-6, y=y)
        smla.token_logprobs(y, tok, lp, top_ids=ids)
    for t in (y, lp, ids):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((y, lp, ids), want))
