"""Tree attention on the GPU against the float64 oracle, within bounds derived from the formula
(oracle.tree_oracle.error_bounds), at the sizes, masks and tables where it can go wrong."""
import math

import numpy as np
import pytest
import torch

import oracle as O
import oracle.tree_oracle as T
import sparse_mla_decode_smla_gb300 as smla

pytestmark = pytest.mark.gpu

FMT = {"bf16": 0, "fp8_ds": 1, "fp8_tensor": 2}
KV_SCALE = 0.5
SM = float(np.float32(1 / 24))


def _bits(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def rows_of_values(x, fmt):
    lat, rope = _bits(x[:, :512]), _bits(x[:, 512:])
    if fmt == "bf16":
        return O.pack_bf16(lat, rope)
    return O.pack_fp8_ds(lat, rope) if fmt == "fp8_ds" else O.pack_fp8_tensor(lat, rope, KV_SCALE)


class Batch:
    """A seeded batch: ragged contexts and nodes, shuffled pages, a random tree or a chain."""

    def __init__(self, fmt="fp8_ds", heads=16, ctx=(70,), nodes=(3,), page=64, tree=True, sink=False, seed=0, gain=1.0,
                 spare_rows=0, words=None, sm=SM, values=None):
        g = np.random.default_rng(seed)
        self.fmt, self.H, self.ctx, self.nodes, self.P, self.sm = fmt, heads, list(ctx), list(nodes), page, sm
        B = len(ctx)
        need = [-(-(c + n) // page) for c, n in zip(ctx, nodes)]
        self.pages, self.stride = sum(need) + 3, max(need) + 1
        perm = g.permutation(self.pages)
        self.table = np.full((B, self.stride), -1, dtype=np.int32)
        at = 0
        for r, k in enumerate(need):
            self.table[r, :k] = perm[at:at + k]
            at += k
        self.cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        self.tokens = int(self.cu[-1]) + spare_rows
        x = g.standard_normal((self.pages * page, 576)) * gain
        if values is not None:
            x = values(self, x)
        self.rows = rows_of_values(x, fmt)
        self.q = _bits(g.standard_normal((self.tokens, heads, 576)))
        self.mask = None
        if tree:
            W = words or -(-max(max(nodes), 1) // 32)
            self.mask = np.zeros((self.tokens, W), dtype=np.uint32)
            for r, n in enumerate(nodes):
                seen = []
                for i in range(n):
                    up = int(g.integers(-1, i)) if i else -1
                    seen.append((seen[up] if up >= 0 else 0) | 1 << i)
                    for w in range(W):
                        self.mask[self.cu[r] + i, w] = (seen[i] >> (32 * w)) & 0xFFFFFFFF
        self.sink = g.standard_normal(heads).astype(np.float32) if sink else None

    def slot(self, r, s):
        return int(self.table[r, s // self.P]) * self.P + s % self.P

    def oracle(self):
        return T.tree_decode(self.q, lambda i: self.rows[i], self.fmt, self.table, self.ctx, self.cu, self.mask, self.P, self.pages,
                             self.sm, self.sink, KV_SCALE if self.fmt == "fp8_tensor" else None)

    def to_gpu(self):
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
        W = 0 if self.mask is None else self.mask.shape[1]
        self.desc = smla.make_tree_desc(self.tokens, self.H, len(self.ctx), self.P, self.pages, self.stride, FMT[self.fmt], self.sm,
                                        mask_words=W, kv_scale=KV_SCALE)
        self.d_q = torch.from_numpy(self.q.view(np.int16)).cuda().view(torch.bfloat16)
        self.d_kv = torch.from_numpy(self.rows).cuda()
        self.d_table, self.d_ctx, self.d_cu = i32(self.table), i32(self.ctx), i32(self.cu)
        self.d_mask = None if self.mask is None else torch.from_numpy(self.mask.view(np.int32)).cuda()
        self.d_sink = None if self.sink is None else torch.from_numpy(self.sink).cuda()
        self.out = torch.full((self.tokens, self.H, 512), -77.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.tokens, self.H), -77.0, dtype=torch.float32, device="cuda")
        self.ws = torch.zeros(smla.tree_workspace_size(self.desc), dtype=torch.uint8, device="cuda")

    def call(self, stream=None, with_lse=True):
        smla.tree_decode(self.desc, self.d_q, self.d_kv, self.d_table, self.d_ctx, self.d_cu, self.d_mask, self.d_sink, self.out,
                         self.lse if with_lse else None, self.ws, stream)

    def run(self, err=0):
        self.to_gpu()
        self.call()
        assert smla.read_error(self.desc, self.ws) == err
        return self.out.double().cpu().numpy(), self.lse.double().cpu().numpy()

    def check(self, ref=None, got=None, err=0):
        got = got or self.run(err)
        ref = ref or self.oracle()
        real = ~np.isnan(ref["lse"][:, 0]) if ref.get("real") is None else ref["real"]
        b_out, b_lse = T.error_bounds(ref, self.fmt != "bf16")
        out, lse = got
        assert (out[~real] == -77).all() and (lse[~real] == -77).all()
        out, lse, ro, rl = out[real], lse[real], ref["out"][real], ref["lse"][real]
        assert np.array_equal(np.isneginf(lse), np.isneginf(rl))
        fin = np.isfinite(rl)
        assert np.isfinite(out).all()
        assert (np.abs(lse - rl)[fin] <= b_lse[real][fin]).all(), np.max((np.abs(lse - rl) / b_lse[real])[fin])
        assert (np.abs(out - ro) <= b_out[real]).all(), np.max(np.abs(out - ro) / b_out[real])


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("heads,nodes", [(1, (1, 2)), (16, (8, 5)), (48, (3, 7)), (64, (1, 1)), (80, (2, 9)), (128, (4, 1))])
def test_heads(fmt, heads, nodes):
    Batch(fmt, heads, ctx=(130, 77), nodes=nodes, sink=heads == 128, seed=heads).check()


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 32, 64, 128, 4096])
def test_pages(fmt, page):
    # contexts that end inside a page, at its end, at a tile's end, and none at all
    Batch(fmt, 16, ctx=(0, 1, 63, 64, 65, 200, 128), nodes=(3, 1, 2, 5, 1, 4, 64), page=page, seed=page).check()


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("tree", [True, False])
def test_single_tokens_and_chains(fmt, tree):
    Batch(fmt, 32, ctx=(0, 5, 127, 300, 64), nodes=(1, 1, 1, 1, 1), tree=tree, sink=True, seed=1).check()
    Batch(fmt, 32, ctx=(0, 5, 127), nodes=(70, 3, 40), tree=tree, seed=2).check()


@pytest.mark.parametrize("fmt", list(FMT))
def test_long_contexts_are_split_and_joined(fmt):
    # few rows over a long axis: many SMs share a row tile; lengths that are no multiple of anything
    b = Batch(fmt, 16, ctx=(7001, 3, 4099), nodes=(4, 2, 1), sink=True, seed=3)
    got = b.run()
    b.check(got=got)
    for _ in range(3):  # and every call gives the same bits
        b.call()
        torch.cuda.synchronize()
        assert np.array_equal(b.out.double().cpu().numpy(), got[0]) and np.array_equal(b.lse.double().cpu().numpy(), got[1])


def test_many_requests_some_without_nodes():
    g = np.random.default_rng(5)
    nodes = [int(x) for x in g.integers(0, 3, 300)]
    nodes[:40] = [0] * 40
    nodes[150:230] = [0] * 80
    b = Batch("fp8_ds", 16, ctx=[int(x) for x in g.integers(0, 90, 300)], nodes=nodes, page=16, seed=5, spare_rows=3)
    b.check()


@pytest.mark.parametrize("fmt", list(FMT))
def test_masks_that_leave_rows_empty(fmt):
    b = Batch(fmt, 16, ctx=(0, 0, 90), nodes=(5, 40, 6), seed=6, words=3)
    b.mask[:3] = 0                       # nothing at all: out 0, lse -inf
    b.mask[3, 0] = 1 << 0                # another node, not itself
    b.mask[4] = 0xFFFFFFFF               # bits past the last node are ignored
    b.mask[10] = 0
    b.mask[45:] = 0                      # only the context
    b.check()
    b = Batch(fmt, 16, ctx=(0,), nodes=(5,), seed=6, sink=True)
    b.mask[2] = 0                        # only the sink: out 0, lse = sink
    b.sink[3], b.sink[4] = -np.inf, 80.0
    b.check()


@pytest.mark.parametrize("fmt", ["bf16", "fp8_tensor", "fp8_ds"])
def test_what_is_hidden_never_counts(fmt):
    # non-finite keys: in slots past the last node, in the next request's rows of a shared page size,
    # and in a node that only one other node sees
    b = Batch(fmt, 16, ctx=(61, 30), nodes=(6, 3), page=16, seed=7)
    b.mask[:6, 0] = [1, 2, 4 | 1, 8, 16, 32 | 8]     # node 3 is seen by itself and node 5
    b.mask[6:, 0] = [1, 3, 7]
    clean = b.oracle()
    nan = {"bf16": np.array([0xC0, 0x7F], dtype=np.uint8), "fp8_tensor": np.array([0x7F], dtype=np.uint8),
           "fp8_ds": np.array([0x7F], dtype=np.uint8)}[fmt]
    used = {b.slot(r, s) for r in range(2) for s in range(b.ctx[r] + b.nodes[r])}
    for s in set(range(len(b.rows))) - used:
        b.rows[s] = np.resize(nan, b.rows.shape[1])
    got = b.run()
    b.check(clean, got)
    for d in (0, 300, 511):                          # a NaN and, in bf16, an infinity in node 3's latent
        rows = b.rows.copy()
        w = 2 if fmt == "bf16" else 1
        b.rows[b.slot(0, 61 + 3), w * d:w * d + w] = nan if d else (np.array([0x80, 0x7F], dtype=np.uint8) if w == 2 else nan)
        out, lse = b.run()
        b.rows = rows
        for t in range(9):
            if t in (3, 5):  # an infinity may leave a weight of zero
                assert (d == 0 and fmt == "bf16") or not np.isfinite(out[t]).any() and not np.isfinite(lse[t]).any(), t
            else:
                assert np.array_equal(out[t], got[0][t]) and np.array_equal(lse[t], got[1][t]), t


def test_pages_that_are_no_pages_are_skipped():
    for fmt in FMT:
        b = Batch(fmt, 16, ctx=(200, 100), nodes=(3, 2), page=16, seed=8)
        b.table[0, 2], b.table[1, 6] = -1, b.pages      # context; the nodes' own page
        b.check(err=smla.SMLA_DEVERR_PAGE)
        b = Batch(fmt, 16, ctx=(200, 100), nodes=(3, 2), page=128, seed=8)
        b.table[0] = b.pages + 5                          # every page of a request: its rows are empty
        b.check(err=smla.SMLA_DEVERR_PAGE)


def test_requests_that_do_not_fit_are_left_out():
    b = Batch("fp8_ds", 16, ctx=(70, 80, 90, 64), nodes=(3, 4, 40, 2), page=16, seed=9, words=2)
    good = b.oracle()
    for what in ("context", "long", "nodes", "order"):
        c, ref = Batch("fp8_ds", 16, ctx=(70, 80, 90, 64), nodes=(3, 4, 40, 2), page=16, seed=9, words=2), {**good}
        lost = np.zeros(49, dtype=bool)
        c.to_gpu()
        if what == "context":
            c.d_ctx[1] = -1
            lost[3:7] = True
        elif what == "long":
            c.d_ctx[0] = c.stride * c.P - 2
            lost[:3] = True
        elif what == "nodes":      # more than the mask's bits
            c.mask = np.ascontiguousarray(c.mask[:, :1])
            c.d_mask = torch.from_numpy(c.mask.view(np.int32)).cuda()
            c.desc.mask_words = 1
            lost[7:47] = True
        else:                      # more nodes than rows of q
            c.d_cu[4] = 60
            lost[47:] = True
        c.call()
        assert smla.read_error(c.desc, c.ws) == smla.SMLA_DEVERR_INDEX
        ref["real"] = ~lost
        c.check(ref, (c.out.double().cpu().numpy(), c.lse.double().cpu().numpy()))


@pytest.mark.parametrize("fmt", list(FMT))
def test_magnitudes(fmt):
    # large scores (a one-hot softmax), tiny ones, tiny and huge q
    for gain, sm in ((3.0, 1.0), (0.02, SM), (1.0, -SM), (1.0, 0.0)):
        Batch(fmt, 16, ctx=(150,), nodes=(4,), seed=10, gain=gain, sm=sm).check()
    for k in (2.0 ** -100, 2.0 ** 90):
        b = Batch(fmt, 16, ctx=(150,), nodes=(4,), seed=11)
        b.q = _bits(O.bf16_bits_to_f64(b.q) * k)
        b.sm = float(np.float32(SM / k))
        b.check()


def test_many_equal_small_weights_add_up():
    # one slot outweighs each of thousands of others by 2^14, together they count as much
    def values(b, x):
        x[:] = 0.0
        x[:, 0] = 1.0
        x[b.slot(0, 0), 0] = 15.0
        x[:, 100] = 1.0
        x[b.slot(0, 0), 100] = -1.0
        return x
    for fmt in FMT:
        b = Batch(fmt, 16, ctx=(8000,), nodes=(1,), seed=12, tree=False, values=values, sm=1.0)
        q = np.zeros((1, 16, 576))
        q[..., 0] = 0.6931
        b.q = _bits(q)
        b.check()


def test_scale_outside_the_window_is_flagged():
    b = Batch("fp8_ds", 16, ctx=(100,), nodes=(2,), seed=13)
    b.rows[b.slot(0, 17), 512:516] = np.frombuffer(np.float32(2.0 ** 9).tobytes(), dtype=np.uint8)
    b.to_gpu()
    b.call()
    assert smla.read_error(b.desc, b.ws) in (0, smla.SMLA_DEVERR_RANGE)  # a kernel that scales in fp32 need not flag


def test_no_lse_side_streams_and_a_graph():
    b = Batch("fp8_ds", 16, ctx=(2000, 10), nodes=(4, 2), seed=14)
    got = b.run()
    b.check(got=got)
    b.out.fill_(5)
    b.lse.fill_(-77)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b.call(stream=side, with_lse=False)
    side.synchronize()
    assert np.array_equal(b.out.double().cpu().numpy(), got[0]) and (b.lse == -77).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.call()
    # the lengths are read on the device: the same graph serves another batch of the same description
    b.ctx, b.nodes = [500, 1300], [1, 5]
    c = Batch("fp8_ds", 16, ctx=b.ctx, nodes=b.nodes, seed=15)
    b.d_ctx.copy_(torch.tensor(b.ctx, dtype=torch.int32))
    b.cu = np.array([0, 1, 6], dtype=np.int32)
    b.d_cu.copy_(torch.from_numpy(b.cu))
    b.mask[:] = c.mask
    b.d_mask.copy_(torch.from_numpy(b.mask.view(np.int32)))
    b.table[:] = np.random.default_rng(1).integers(0, b.pages, b.table.shape)
    b.d_table.copy_(torch.from_numpy(b.table))
    g.replay()
    assert smla.read_error(b.desc, b.ws) == 0
    b.check(got=(b.out.double().cpu().numpy(), b.lse.double().cpu().numpy()))


def test_two_streams_with_a_workspace_each():
    a, b = (Batch("bf16", 16, ctx=(3000,), nodes=(4,), seed=s) for s in (16, 17))
    ra, rb = a.run(), b.run()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        a.call(stream=s1)
        b.call(stream=s2)
    torch.cuda.synchronize()
    for x, r in ((a, ra), (b, rb)):
        assert np.array_equal(x.out.double().cpu().numpy(), r[0]) and np.array_equal(x.lse.double().cpu().numpy(), r[1])


def test_draft_verify_accept_fork():
    # the operators as they are used together: room for the draft, its keys written, the tree
    # attended, the accepted path compacted, the rest trimmed, a sample forked, and attended again
    g = np.random.default_rng(18)
    P, pages, stride, H = 16, 40, 8, 16
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    lens0, n = [37, 50, 0], 6
    cd = smla.make_cache_desc(1, 1, P, pages, 3, stride)
    kv = torch.zeros((pages * P, 656), dtype=torch.uint8, device="cuda")
    table, lens, refs = i32(np.full((3, stride), -1)), i32([0, 0, 0]), i32(np.zeros(pages))
    free, count, err = i32(np.arange(pages)), i32([pages]), i32([0])
    work, got = i32(np.zeros(6)), i32(np.zeros(3))
    tables = (table, lens, refs, free, count)
    smla.cache_resize(cd, *tables, i32([0, 1]), i32([x + n for x in lens0[:2]]), work, err)
    x = g.standard_normal((2, 60, 576)).astype(np.float32)

    def write(r, a, b):  # the rows of slots [a, b) of request r
        t = table[r].cpu().numpy()
        slots = torch.tensor([int(t[s // P]) * P + s % P for s in range(a, b)], device="cuda")
        v = torch.from_numpy(x[r, a:b]).cuda().to(torch.bfloat16)
        smla.pack_kv(1, 0, v[:, :512].contiguous(), v[:, 512:].contiguous(), slots, kv, pages * P)

    for r in range(2):
        write(r, 0, lens0[r] + n)
    mask = np.array([[1], [3], [5], [8 | 3], [16 | 5], [32 | 16 | 5]] * 2, dtype=np.uint32)

    def attend(ctx, cu, m, B, q):
        T_ = q.shape[0]
        d = smla.make_tree_desc(T_, H, B, P, pages, stride, 1, SM, mask_words=0 if m is None else 1)
        ws = torch.zeros(smla.tree_workspace_size(d), dtype=torch.uint8, device="cuda")
        out, lse = torch.empty((T_, H, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((T_, H), device="cuda")
        dm = None if m is None else torch.from_numpy(m.view(np.int32)).cuda()
        smla.tree_decode(d, torch.from_numpy(q.view(np.int16)).cuda().view(torch.bfloat16), kv, table, i32(ctx), i32(cu), dm, None,
                         out, lse, ws)
        assert smla.read_error(d, ws) == 0
        rows, t = kv.cpu().numpy(), table.cpu().numpy()
        ref = T.tree_decode(q, lambda i: rows[i], "fp8_ds", t, ctx, cu, m, P, pages, SM)
        bo, bl = T.error_bounds(ref, True)
        assert (np.abs(out.double().cpu().numpy() - ref["out"]) <= bo).all()
        assert (np.abs(lse.double().cpu().numpy() - ref["lse"]) <= bl).all()
        return out

    attend(lens0[:2], [0, 6, 12], mask, 2, _bits(g.standard_normal((12, H, 576))))
    before = [kv[[int(table[r, s // P]) * P + s % P for s in range(lens0[r] + n)]] for r in range(2)]
    paths = [[0, 2, 4, 5], [0, 1, 3]]
    new = i32([0, 0, 0])
    smla.cache_compact(cd, table, i32(lens0), i32([0, 4, 7, 7]), i32(sum(paths, [])), kv, new, err)
    smla.cache_resize(cd, *tables, i32([0, 1]), new[:2].contiguous(), work, err)
    smla.cache_fork(cd, *tables, i32([1]), i32([2]), got, kv, err)
    assert err.item() == 0 and lens.tolist() == [41, 53, 53] and count.item() == pages - 3 - 4 - 1
    for r, row in ((0, 0), (1, 1), (1, 2)):
        now = kv[[int(table[row, s // P]) * P + s % P for s in range(lens.tolist()[row])]]
        assert torch.equal(now[:lens0[r]], before[r][:lens0[r]])
        assert torch.equal(now[lens0[r]:], before[r][[lens0[r] + j for j in paths[r]]])
    # one more token each, its key the row after the context
    smla.cache_resize(cd, *tables, i32([0, 1, 2]), lens + 1, work, err)
    assert err.item() == 0
    t = table.cpu().numpy()
    ctx = [41, 53, 53]
    slots = torch.tensor([int(t[r, c // P]) * P + c % P for r, c in enumerate(ctx)], device="cuda")
    v = torch.randn(3, 576, device="cuda").to(torch.bfloat16)
    v[2] = v[1]
    smla.pack_kv(1, 0, v[:, :512].contiguous(), v[:, 512:].contiguous(), slots, kv, pages * P)
    q = _bits(g.standard_normal((3, H, 576)))
    q[2] = q[1]
    out = attend(ctx, [0, 1, 2, 3], None, 3, q)
    assert torch.equal(out[1], out[2])  # a fork answers as its source does


@pytest.mark.parametrize("fmt", list(FMT))
def test_long_chain_over_several_row_tiles(fmt):
    # a chunk of a prompt: many more nodes than a mask would hold, every key tile cut by the diagonal
    Batch(fmt, 3, ctx=(10, 0), nodes=(333, 130), page=32, tree=False, sink=True, seed=20).check()


def test_rows_before_the_first_node_and_odd_bounds():
    b = Batch("fp8_ds", 16, ctx=(70, 20), nodes=(3, 2), seed=21, spare_rows=7)
    # the nodes stand at rows 4..8 of q; the mask rows with them
    b.q[4:9], b.mask[4:9] = b.q[0:5].copy(), b.mask[0:5].copy()
    b.cu = (b.cu + 4).astype(np.int32)
    ref = b.oracle()
    out, lse = b.run()
    assert (out[:4] == -77).all() and (out[9:] == -77).all() and (lse[:4] == -77).all() and (lse[9:] == -77).all()
    b.check(ref, (out, lse))


@pytest.mark.parametrize("fmt", list(FMT))
def test_a_cache_past_four_gigabytes(fmt):
    # rows behind 4 GiB of others: 32-bit byte offsets would read elsewhere
    b = Batch(fmt, 16, ctx=(200, 90), nodes=(3, 2), page=64, seed=22)
    ref = b.oracle()
    R = b.rows.shape[1]
    far = (1 << 32) // (R * 64) + 5
    small = b.rows
    b.rows = np.zeros((1, R), dtype=np.uint8)
    table = b.table.copy()
    b.table = np.where(table >= 0, table + far, -1).astype(np.int32)
    pages = b.pages
    b.pages = pages + far
    b.to_gpu()
    kv = torch.zeros((b.pages * 64, R), dtype=torch.uint8, device="cuda")
    kv[far * 64:] = torch.from_numpy(small).cuda()
    b.d_kv = kv
    b.call()
    assert smla.read_error(b.desc, b.ws) == 0
    b.check(ref, (b.out.double().cpu().numpy(), b.lse.double().cpu().numpy()))


def test_one_row_tile_shared_by_every_sm():
    # one node over a long context: its 16 rows are split over the whole GPU
    b = Batch("fp8_tensor", 16, ctx=(20011,), nodes=(1,), seed=23, tree=False)
    b.check()


def test_queries_that_are_not_finite_stay_in_their_rows():
    for fmt in FMT:
        b = Batch(fmt, 16, ctx=(100,), nodes=(4,), seed=24)
        clean = b.run()
        b.q[1, 5, 7] = 0x7FC0        # NaN
        b.q[2, 3, 550] = 0x7F80      # infinity
        out, lse = b.run()
        assert np.isnan(out[1, 5]).all() and not np.isfinite(lse[2, 3])
        keep = np.ones((4, 16), dtype=bool)
        keep[1, 5] = keep[2, 3] = False
        assert np.array_equal(out[keep], clean[0][keep]) and np.array_equal(lse[keep], clean[1][keep])


def test_random_batches():
    g = np.random.default_rng(25)
    for n in range(24):
        B = int(g.integers(1, 9))
        Batch(["bf16", "fp8_ds", "fp8_tensor"][n % 3], int(g.integers(1, 129)), ctx=[int(x) for x in g.integers(0, 400, B)],
              nodes=[int(x) for x in g.integers(0, 12, B - 1)] + [1], page=1 << int(g.integers(0, 9)), tree=bool(g.integers(0, 2)),
              sink=bool(g.integers(0, 2)), seed=100 + n, spare_rows=int(g.integers(0, 3))).check()


@pytest.mark.parametrize("fmt", list(FMT))
def test_more_requests_than_threads(fmt):
    # every thread of the schedule counts several requests; and the largest number of them, hardly any with nodes
    g = np.random.default_rng(26)
    nodes = [int(x) for x in g.integers(0, 3, 2500)]
    Batch(fmt, 8, ctx=[int(x) for x in g.integers(0, 70, 2500)], nodes=nodes, page=16, seed=26, tree=fmt != "bf16").check()
    nodes = np.zeros(65536, dtype=int)
    nodes[g.choice(65536, 40, replace=False)] = 2
    nodes[-1] = 1
    Batch(fmt, 4, ctx=[int(x) for x in np.where(nodes > 0, 40, 0)], nodes=nodes.tolist(), page=32, seed=27).check()


@pytest.mark.parametrize("fmt", list(FMT))
def test_key_tiles_of_context_beside_tiles_with_nodes(fmt):
    # contexts that are whole key tiles, one slot less and one more: tiles without checks next to tiles with them, a missing
    # page inside one of the former, and rows of a tile that belong to no node
    b = Batch(fmt, 7, ctx=(128, 127, 129, 64, 192), nodes=(9, 3, 1, 64, 2), page=16, seed=28, sink=True)
    b.check()
    b.table[0, 3] = b.table[4, 11] = -1
    b.check(err=smla.SMLA_DEVERR_PAGE)


def _pair(fmt):
    """Two batches of one shape, and their results."""
    a = Batch(fmt, 16, ctx=(700, 40, 3), nodes=(6, 2, 4), page=16, seed=30, sink=True)
    b = Batch(fmt, 16, ctx=(40, 3, 700), nodes=(2, 4, 6), page=16, seed=31, sink=True)
    refs = []
    for x in (a, b):
        out, lse = x.run()
        x.check(None, (out, lse))
        refs.append((x.out.clone(), x.lse.clone()))
    assert a.desc.num_pages == b.desc.num_pages and a.desc.page_table_stride == b.desc.page_table_stride
    return a, b, refs


NAMES = ("d_q", "d_kv", "d_table", "d_ctx", "d_cu", "d_mask", "d_sink")


@pytest.mark.parametrize("fmt", list(FMT))
def test_inputs_written_just_before_the_call(fmt):
    # every input changes from call to call, by kernels and by copies, each of them last in turn; nothing waits in between
    a, b, refs = _pair(fmt)
    x = Batch(fmt, 16, ctx=(700, 40, 3), nodes=(6, 2, 4), page=16, seed=30, sink=True)
    x.to_gpu()
    got = []
    for i in range(42):
        src, order = (a, b)[i % 2], NAMES[i % 7:] + NAMES[:i % 7]
        for name in order:
            s, d = getattr(src, name), getattr(x, name)
            if i % 3 == 0:
                d.copy_(s)
            elif d.is_floating_point():
                torch.mul(s, 1, out=d)
            else:
                torch.bitwise_or(s, 0, out=d)
        x.call()
        got.append((x.out.clone(), x.lse.clone()))
    assert smla.read_error(x.desc, x.ws) == 0
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, refs[i % 2][0]) and torch.equal(l, refs[i % 2][1]), i


def test_graph_nodes_of_every_kind_before_the_call():
    # a captured call as the first node, behind a copy, behind a memset, behind a kernel, and behind two streams
    a, b, refs = _pair("fp8_ds")
    x = Batch("fp8_ds", 16, ctx=(700, 40, 3), nodes=(6, 2, 4), page=16, seed=30, sink=True)
    x.to_gpu()
    x.call()
    outs = [torch.zeros_like(x.out) for _ in range(5)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.call()
        outs[0].copy_(x.out)
        for name in NAMES:
            getattr(x, name).copy_(getattr(b, name))
        x.call()
        outs[1].copy_(x.out)
        x.out.zero_()
        x.call()
        torch.mul(x.out, 1, out=outs[2])
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for name in NAMES[:3]:
                getattr(x, name).copy_(getattr(a, name))
        for name in NAMES[3:]:
            getattr(x, name).copy_(getattr(a, name))
        torch.cuda.current_stream().wait_stream(side)
        x.call()
        outs[3].copy_(x.out)
        x.call()
        outs[4].copy_(x.out)
    for _ in range(3):
        for o in outs:
            o.fill_(-1)
        g.replay()
        torch.cuda.synchronize()
        for o, r in zip(outs, (0, 1, 1, 0, 0)):
            assert torch.equal(o, refs[r][0])
    assert smla.read_error(x.desc, x.ws) == 0


@pytest.mark.parametrize("fmt", list(FMT))
def test_row_tiles_that_start_inside_their_keys(fmt):
    # more row tiles than SMs and several a run: whole row tiles take their keys in a circle from inside the context, with nodes
    # of several key tiles, partly filled pages, and masks that hide the circle's start
    b = Batch(fmt, 128, ctx=(700, 330, 64), nodes=(96, 70, 65), page=16, seed=32, sink=True, spare_rows=1)
    b.check()
    b = Batch(fmt, 127, ctx=(190, 500), nodes=(130, 66), page=64, tree=False, seed=33)
    b.check()


def _scale_bytes(v):
    return torch.from_numpy(np.frombuffer(np.float32(v).tobytes(), dtype=np.uint8).copy()).cuda()


@pytest.mark.parametrize("heads", [1, 16, 64, 128])
def test_every_scale_outside_the_window_is_flagged(heads):
    # fp8_ds keys enter as f16 at every head count: block scales in [2^-15, 2^7], [2^-14, 2^7] where they are no powers of two.
    # Each of a row's four scales, in slots of every part of a key tile, of the context and of the nodes
    b = Batch("fp8_ds", heads, ctx=(130,), nodes=(3,), page=16, seed=40)
    b.to_gpu()
    up, down = (lambda x: float(np.nextafter(np.float32(x), np.float32(np.inf)))), 2.0 ** -14
    bad = [2.0 ** 8, up(2.0 ** 7), 2.0 ** -16, float(np.nextafter(np.float32(down), np.float32(0))), -2.0 ** 9, math.inf, math.nan]
    n = 0
    for s in (0, 5, 7, 8, 15, 16, 31, 32, 63, 64, 100, 127, 128, 129, 130, 132):
        for block in range(4):
            at = b.d_kv[b.slot(0, s), 512 + 4 * block:516 + 4 * block]
            old = at.clone()
            at.copy_(_scale_bytes(bad[n % len(bad)]))
            n += 1
            b.call()
            assert smla.read_error(b.desc, b.ws) == smla.SMLA_DEVERR_RANGE, (s, block, bad[(n - 1) % len(bad)])
            at.copy_(old)
    for s in (133, 140):  # past the last node: not a row of the call
        at = b.d_kv[b.slot(0, s), 512:516]
        at.copy_(_scale_bytes(math.nan))
    b.call()
    assert smla.read_error(b.desc, b.ws) == 0


@pytest.mark.parametrize("heads", [1, 16, 64])
def test_scales_at_the_edges_of_the_window(heads):
    # powers of two at both edges: the usual bounds
    for v, sm in ((2.0 ** 7, SM / 1024), (2.0 ** -15, SM)):
        b = Batch("fp8_ds", heads, ctx=(130,), nodes=(3,), page=16, seed=41, sm=float(np.float32(sm)))
        for s in (3, 70, 131):
            b.rows[b.slot(0, s), 512:528] = np.frombuffer(np.full(4, v, dtype=np.float32).tobytes(), dtype=np.uint8)
        b.check()
    # others: the scale and its product with the code are rounded to f16, 2^-11 relative each (together below 2^-10 * 1.001), and
    # products below 2^-14 to a multiple of 2^-24: half a step of it. A score moves by that of each key value, times |q|; an
    # output by the weights' change and by its own values'
    for v, sm in ((float(np.nextafter(np.float32(2.0 ** -14), np.float32(1))), SM), (0.71, SM), (127.9, SM / 1024)):
        b = Batch("fp8_ds", heads, ctx=(130,), nodes=(3,), page=16, seed=42, sm=float(np.float32(sm)))
        for s in range(133):
            b.rows[b.slot(0, s), 512:528] = np.frombuffer(np.full(4, v, dtype=np.float32).tobytes(), dtype=np.uint8)
        ref, (out, lse) = b.oracle(), b.run()
        b_out, b_lse = T.error_bounds(ref, True)
        t = ref["terms"]
        q1 = np.abs(O.bf16_bits_to_f64(b.q)).sum(-1)
        ds = 2.0 ** -10 * 1.001 * t["qk"] + abs(b.sm) * 2.0 ** -25 * q1
        assert (np.abs(lse - ref["lse"]) <= b_lse + ds).all()
        assert (np.abs(out - ref["out"]) <= (b_out + (2 * ds + 2.0 ** -10 * 1.001)[..., None] * t["A"] + 2.0 ** -25)).all()


@pytest.mark.parametrize("fmt", list(FMT))
def test_small_elements_of_a_query(fmt):
    # one element of 1 that meets zeros, 511 of 2^-18 (1 + 2^-7) that meet the largest codes: as f16 each of them is off by 2^-25,
    # all the same way; as bf16 (the BF16 cache) none is
    def values(b, x):
        x[:] = 224.0
        x[:, 0] = x[:, 512:] = 0.0
        return x
    b = Batch(fmt, 16, ctx=(1,), nodes=(1,), seed=43, tree=False, values=values, sm=1.0)
    q = np.full((1, 16, 576), 2.0 ** -18 * (1 + 2.0 ** -7))
    q[..., 0] = 1.0
    b.q = _bits(q)
    assert np.array_equal(O.bf16_bits_to_f64(b.q), q)
    b.check()


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("ctx,nodes,heads", [(7001, 4, 16), (9728, 1, 16), (9727, 1, 64), (20011, 2, 33)])
def test_no_slot_is_lost_where_runs_meet(fmt, ctx, nodes, heads):
    # the first and the last slot of every key tile in turn outweigh all others together: wherever the tile's work is cut, one
    # that were lost or counted twice would show in full. Odd tiles' first slots and even tiles' last slots in one call, the
    # others in the next: each marked slot has a value of its own dims
    for part in range(2):
        marks = [s for k in range(-(-(ctx + nodes) // 64)) for s in ((64 * k,) if (k + part) % 2 else (64 * k + 63,)) if s < ctx]

        def values(b, x):
            x *= 0.05
            x[:, 0] = 0.0
            for i, s in enumerate(marks):
                row = x[b.slot(0, s)]
                row[0] = 12.0
                row[1 + i % 500] += 1.0 if i < 500 else -1.0
            return x

        b = Batch(fmt, heads, ctx=(ctx,), nodes=(nodes,), seed=44 + part, tree=False, values=values, sm=1.0)
        b.q = _bits(O.bf16_bits_to_f64(b.q) * 0.02)
        b.q[..., 0] = 0x3F80  # 1: a marked slot counts e^12 of an unmarked one
        ref = b.oracle()
        # one mark less, or one twice, moves the log-sum-exp by 1 / len(marks): more than twice its bound
        b_lse = T.error_bounds(ref, fmt != "bf16")[1]
        assert (b_lse * 2 < 1 / len(marks)).all()
        b.check(ref)
