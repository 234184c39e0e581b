"""The cache's page operators on the GPU against their plain models, bit for bit: whole caches and
tables are compared, so a byte moved too much is found as well."""
import numpy as np
import pytest
import torch

import oracle.cache_pages_oracle as C
import sparse_mla_decode_smla_gb300 as smla

pytestmark = pytest.mark.gpu

FMT = {"bf16": 0, "fp8_ds": 1, "fp8_tensor": 2, "index_keys": 3}


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Pool:
    """A cache of L layers with its tables, on the GPU and as numpy arrays."""

    def __init__(self, fmt, L, page, lens, stride, pages, seed=0, gap=0):
        g = np.random.default_rng(seed)
        self.fmt, self.L, self.P, self.B, self.stride, self.pages = fmt, L, page, len(lens), stride, pages
        self.cache = g.integers(0, 256, (L, pages, C.page_bytes(fmt, page)), dtype=np.uint8)
        self.table = np.full((self.B, stride), -1, dtype=np.int32)
        perm = g.permutation(pages).astype(np.int32)
        self.lens, self.refs = np.array(lens, dtype=np.int32), np.zeros(pages, dtype=np.int32)
        at = 0
        for r, n in enumerate(lens):
            k = -(-n // page)
            self.table[r, :k] = perm[at:at + k]
            at += k
        self.refs[perm[:at]] = 1
        self.free = np.full(pages, -1, dtype=np.int32)
        self.free[:pages - at] = perm[at:]
        self.count = pages - at
        layer = pages * C.page_bytes(fmt, page)
        self.raw = torch.zeros((L, layer + gap), dtype=torch.uint8, device="cuda")
        self.raw[:, :layer] = torch.from_numpy(self.cache.reshape(L, -1)).cuda()
        self.desc = smla.make_cache_desc(FMT[fmt], L, page, pages, self.B, stride, layer + gap)
        self.d_table, self.d_lens, self.d_refs, self.d_free = (_dev(x) for x in (self.table, self.lens, self.refs, self.free))
        self.d_count, self.err = _dev([self.count]), torch.zeros(1, dtype=torch.int32, device="cuda")

    def tables(self):
        return self.d_table, self.d_lens, self.d_refs, self.d_free, self.d_count

    def fork(self, src, dst, stream=None):
        s, d = _dev(src), _dev(dst)
        got = torch.full((len(src),), -9, dtype=torch.int32, device="cuda")
        smla.cache_fork(self.desc, *self.tables(), s, d, got, self.raw, self.err, stream)
        e, self.count, pages = C.fork(self.cache, self.fmt, self.P, self.table, self.lens, self.refs, self.free, self.count, src, dst)
        torch.cuda.synchronize()
        assert got.tolist() == pages
        return e

    def resize(self, req, new, stream=None):
        r, n = _dev(req), _dev(new)
        work = torch.empty(2 * len(req), dtype=torch.int32, device="cuda")
        smla.cache_resize(self.desc, *self.tables(), r, n, work, self.err, stream)
        e, self.count = C.resize(self.P, self.table, self.lens, self.refs, self.free, self.count, req, new)
        torch.cuda.synchronize()
        return e

    def check(self, err=0):
        torch.cuda.synchronize()
        layer = self.cache[0].size
        assert np.array_equal(self.raw[:, :layer].cpu().numpy().reshape(self.cache.shape), self.cache)
        assert not self.raw[:, layer:].any()
        for name, d, a in (("table", self.d_table, self.table), ("lens", self.d_lens, self.lens), ("refs", self.d_refs, self.refs),
                           ("free", self.d_free, self.free)):
            assert np.array_equal(d.cpu().numpy(), a), name
        assert self.d_count.item() == self.count
        assert self.err.item() == err
        self.err.zero_()


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("page", [1, 2, 16, 64, 512])
def test_copy_pages(fmt, page):
    if fmt == "index_keys" and not 16 <= page <= 128:
        pytest.skip("index keys come in pages of 16 to 128 slots")
    for L, n, gap in ((1, 1, 0), (3, 5, 48)):
        p = Pool(fmt, L, page, [3], 4096, 14, seed=page, gap=gap)
        ids = np.random.default_rng(n).permutation(14)
        src, dst = ids[:n].tolist(), ids[n:2 * n].tolist()
        smla.cache_copy_pages(p.desc, _dev(src), _dev(dst), p.raw, p.err)
        C.copy_pages(p.cache, src, dst)
        p.check()


def test_copy_skips_and_flags():
    p = Pool("fp8_ds", 2, 16, [3], 4, 9)
    src, dst = [0, -1, 2, 5, 9, 3], [4, 1, -1, 5, 6, -7]
    smla.cache_copy_pages(p.desc, _dev(src), _dev(dst), p.raw, p.err)
    assert C.copy_pages(p.cache, src, dst) == C.ERR_PAGE
    p.check(C.ERR_PAGE)
    smla.cache_copy_pages(p.desc, _dev([8]), _dev([7]), p.raw)  # no error word
    C.copy_pages(p.cache, [8], [7])
    p.check()


def test_copy_past_four_gigabytes():
    # 32-bit offsets would wrap: the second layer starts past 4 GiB, and its last page past that
    page, pages = 64, 110000
    stride = pages * page * 656
    assert stride > 1 << 32
    raw = torch.zeros(2 * stride, dtype=torch.uint8, device="cuda")
    d = smla.make_cache_desc(1, 2, page, pages, 1, 1, stride)
    one = page * 656
    a = torch.randint(0, 256, (2, one), dtype=torch.uint8, device="cuda")
    for l in range(2):
        raw[l * stride + 7 * one:l * stride + 8 * one] = a[l]
    smla.cache_copy_pages(d, _dev([7]), _dev([pages - 1]), raw)
    torch.cuda.synchronize()
    for l in range(2):
        assert torch.equal(raw[l * stride + (pages - 1) * one:(l + 1) * stride], a[l])
    total = int(raw.view(torch.int64).ne(0).sum())
    assert total <= 4 * one // 8


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("page", [1, 8, 16, 64])
@pytest.mark.parametrize("L,gap", [(1, 0), (3, 16)])
def test_compact(fmt, page, L, gap):
    if fmt == "index_keys" and page < 16:
        pytest.skip("index keys come in pages of 16 to 128 slots")
    g = np.random.default_rng(page + L)
    lens = [0, 1, 2, 70, 333, 1500, 64, 129]
    p = Pool(fmt, L, page, lens, 1500 // page + 1, sum(-(-n // page) for n in lens) + 3, seed=5, gap=gap)
    starts, keep = [], []
    for n in lens:
        st = int(g.integers(0, n + 1)) if n < 1000 else 3
        rest = n - st
        keep.append(sorted(g.choice(rest, int(g.integers(0, rest + 1)), replace=False).tolist()) if rest else [])
        starts.append(st)
    keep[4] = list(range(len(keep[4])))  # already in place
    cu = np.concatenate([[0], np.cumsum([len(k) for k in keep])])
    flat = [x for k in keep for x in k]
    new = torch.full((len(lens),), -5, dtype=torch.int32, device="cuda")
    smla.cache_compact(p.desc, p.d_table, _dev(starts), _dev(cu), _dev(flat), p.raw, new, p.err)
    want = np.full(len(lens), -5)
    assert C.compact(p.cache, fmt, page, p.table, starts, cu, flat, want) == 0
    p.check()
    assert new.tolist() == want.tolist()


def test_compact_one_long_request_in_place():
    # every chunk's targets are sources of rows before them: a wrong order shows
    for fmt, keep in (("fp8_ds", list(range(1, 9000))), ("bf16", list(range(0, 9000, 2))), ("fp8_tensor", list(range(513, 9000)))):
        p = Pool(fmt, 1, 64, [9000], 141, 150, seed=1)
        smla.cache_compact(p.desc, p.d_table, _dev([0]), _dev([0, len(keep)]), _dev(keep), p.raw, None, p.err)
        C.compact(p.cache, fmt, 64, p.table, [0], [0, len(keep)], keep)
        p.check()


def test_compact_refuses_what_it_cannot_move():
    p = Pool("fp8_ds", 2, 4, [20, 20, 20, 20, 20], 5, 30, seed=3)
    table = p.table.copy()
    table[1, 2], table[2, 1] = 30, -1          # a page outside the cache, a page that is missing
    starts, cu = [0, 0, 0, -1, 4], [0, 3, 6, 9, 10, 14]
    keep = [5, 5, 7, 1, 8, 9, 2, 4, 5, 3, 1, 15, 16, 0]   # twice the same; bad pages; bad start; past the table; not ascending
    new = torch.full((5,), -5, dtype=torch.int32, device="cuda")
    smla.cache_compact(p.desc, _dev(table), _dev(starts), _dev(cu), _dev(keep), p.raw, new, p.err)
    want = np.full(5, -5)
    e = C.compact(p.cache, "fp8_ds", 4, table, starts, cu, keep, want)
    assert e == C.ERR_INDEX | C.ERR_PAGE
    p.check(e)
    assert new.tolist() == want.tolist()
    for bad in ([0, 3, 2, 3, 3, 3], [0, 99, 99, 99, 99, 99], [-1, 0, 0, 0, 0, 0]):
        smla.cache_compact(p.desc, p.d_table, _dev([0] * 5), _dev(bad), _dev([1, 2, 3]), p.raw, None, p.err)
        assert C.compact(p.cache, "fp8_ds", 4, p.table, [0] * 5, bad, [1, 2, 3]) == C.ERR_INDEX
        p.check(C.ERR_INDEX)


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("page", [1, 4, 16, 128])
def test_fork(fmt, page):
    if fmt == "index_keys" and page < 16:
        pytest.skip("index keys come in pages of 16 to 128 slots")
    lens = [0, 1, page, page + 1, 7 * page - 1, 300] + [0] * 8
    p = Pool(fmt, 3, page, lens, 300 // page + 7, sum(-(-n // page) for n in lens) + 9, seed=page, gap=32)
    assert p.fork([5, 1, 2, 0, 5, 3, 4, 5], [6, 7, 8, 9, 10, 11, 12, 13]) == 0
    p.check()
    # the copies let go, then the originals: the pages come back
    assert p.resize([13, 6, 8, 10], [0, 0, 0, 0]) == 0
    p.check()
    assert p.resize([5, 4, 12, 11], [1, 0, page, 0]) == 0
    p.check()


def test_fork_refusals():
    p = Pool("bf16", 2, 8, [9, 10, 16, 0, 0, 0, 0, 3], 2, 10, seed=4)  # two pages free
    assert p.count == 3
    e = p.fork([0, 0, 1, 99, 2, 3, 2], [3, 3, 7, 4, -1, 4, 5])
    # 3 twice; 7 holds slots; no request 99; no request -1; 3 is a source and so no target; 2 -> 5 shares pages
    assert e == C.ERR_INDEX
    p.check(e)
    e = p.fork([0, 1, 0, 7], [3, 4, 6, 99])
    p.check(e)
    assert p.resize([3, 4, 6, 5], [0, 0, 0, 0]) == 0
    p.check()
    q = Pool("bf16", 1, 8, [9, 16, 0, 0, 0, 0], 2, 5, seed=4)   # one page free, two forks that need one
    assert q.fork([0, 0, 1], [2, 3, 4]) == C.ERR_PAGE
    q.check(C.ERR_PAGE)


def test_resize_random_walk():
    g = np.random.default_rng(7)
    p = Pool("fp8_tensor", 1, 4, [0] * 40, 30, 500, seed=1)
    for _ in range(40):
        if g.random() < 0.7:
            n = int(g.integers(1, 41))
            ids = g.permutation(40)[:n]
            new = g.integers(0, 121, n) * (g.random(n) < 0.7)
            e = p.resize(ids.tolist(), new.tolist())
        else:
            ids = g.permutation(40)[:20]
            e = p.fork(ids[:10].tolist(), ids[10:].tolist())
        p.check(e)


def test_resize_refusals():
    p = Pool("bf16", 1, 4, [10, 11, 12, 0], 4, 12, seed=2)
    e = p.resize([0, 0, 1, 4], [0, 4, 17, 1])       # twice; too long; no such request
    assert e == C.ERR_INDEX
    p.check(e)
    assert p.resize([3, 2, 0], [16, 13, 0]) == 0     # grows on what the same call frees
    p.check()
    e = p.resize([0, 2, 1], [16, 16, 5])             # not enough for the first: it stays, the last still shrinks
    p.check(e)
    # a page that no request holds, and a table entry that is no page
    p.d_refs[int(p.table[1, 0])] = 0
    p.refs[int(p.table[1, 0])] = 0
    p.d_table[1, 1] = 77
    p.table[1, 1] = 77
    assert p.resize([1], [0]) == C.ERR_PAGE
    p.check(C.ERR_PAGE)


def test_resize_large_pool():
    g = np.random.default_rng(3)
    lens = g.integers(0, 40000, 96).tolist()
    p = Pool("fp8_tensor", 1, 1, [0] * 96, 40000, 4096, seed=1)
    del p
    pages = sum(-(-n // 16) for n in lens) + 1234
    B, stride = 96, 2500
    perm = g.permutation(pages).astype(np.int32)
    table, lens0 = np.full((B, stride), -1, dtype=np.int32), np.zeros(B, dtype=np.int32)
    refs, free, count = np.zeros(pages, dtype=np.int32), perm.copy(), pages
    d = smla.make_cache_desc(0, 1, 16, pages, B, stride)
    dv = [_dev(x) for x in (table, lens0, refs, free, [count])]
    err, work = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty(2 * B, dtype=torch.int32, device="cuda")
    order = g.permutation(B)
    for new in (np.array(lens)[order], np.where(g.random(B) < 0.5, 0, np.array(lens)[order] // 2), np.array(lens)[order]):
        smla.cache_resize(d, *dv, _dev(order), _dev(new), work, err)
        e, count = C.resize(16, table, lens0, refs, free, count, order.tolist(), new.tolist())
        assert e == 0 and err.item() == 0 and dv[4].item() == count
        for a, b in zip(dv, (table, lens0, refs, free)):
            assert np.array_equal(a.cpu().numpy(), b)


def test_streams_and_graphs():
    # on a side stream, and captured once and replayed: the same results as the calls made in turn
    p = Pool("fp8_ds", 2, 16, [40, 100, 0, 0], 8, 30, seed=9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert p.fork([0, 1], [2, 3], stream=side) == 0
    p.check()
    ids, up, down = _dev([0, 1]), _dev([60, 100]), _dev([40, 100])
    work = torch.empty(4, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        smla.cache_resize(p.desc, *p.tables(), ids, up, work, p.err)
        smla.cache_resize(p.desc, *p.tables(), ids, down, work, p.err)
    for _ in range(3):
        g.replay()
        for new in ([60, 100], [40, 100]):
            e, p.count = C.resize(p.P, p.table, p.lens, p.refs, p.free, p.count, [0, 1], new)
            assert e == 0
        p.check()


def test_resize_of_more_pages_than_a_round_of_marks():
    # over a million pages: the freed ones still come back in ascending order over all of them
    pages, B, stride = 2_300_001, 3, 1_200_000
    g = np.random.default_rng(5)
    perm = g.permutation(pages).astype(np.int32)
    lens = np.array([1_150_000, 700_000, 400_000], dtype=np.int32)
    table = np.full((B, stride), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(lens):
        table[r, :n] = perm[at:at + n]
        at += n
    refs = np.zeros(pages, dtype=np.int32)
    refs[perm[:at]] = 1
    free = np.full(pages, -1, dtype=np.int32)
    free[:pages - at] = perm[at:]
    d = smla.make_cache_desc(0, 1, 1, pages, B, stride)
    dv = [_dev(x) for x in (table, lens, refs, free, [pages - at])]
    work, err = torch.empty(4, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    smla.cache_resize(d, *dv, _dev([2, 0]), _dev([5, 100]), work, err)
    assert err.item() == 0
    gone = np.sort(np.concatenate([table[2, 5:400_000], table[0, 100:1_150_000]]))
    got = dv[3].cpu().numpy()
    assert dv[4].item() == pages - at + len(gone)
    assert np.array_equal(got[:pages - at], free[:pages - at])
    assert np.array_equal(got[pages - at:pages - at + len(gone)], gone) and (got[pages - at + len(gone):] == -1).all()
    left = dv[2].cpu().numpy()
    refs[gone] = 0
    assert np.array_equal(left, refs)


@pytest.mark.parametrize("fmt", ["bf16", "index_keys"])
def test_compact_many_layers_and_chunks(fmt):
    # more layers than a CTA takes together, rows of one chunk and of several in one call
    g = np.random.default_rng(3)
    lens = [40, 900, 17, 0, 260] * 12
    p = Pool(fmt, 40, 16, lens, 60, sum(-(-n // 16) for n in lens) + 1, seed=7)
    keep = [sorted(g.choice(n, n * 2 // 3, replace=False).tolist()) if n else [] for n in lens]
    cu = np.concatenate([[0], np.cumsum([len(k) for k in keep])])
    flat = [x for k in keep for x in k]
    smla.cache_compact(p.desc, p.d_table, _dev([0] * 60), _dev(cu), _dev(flat), p.raw, None, p.err)
    C.compact(p.cache, fmt, 16, p.table, [0] * 60, cu, flat)
    p.check()


def test_resize_in_one_launch_over_a_large_pool():
    # few requests (one launch) over a pool of several rounds of marks, the widest page table rows count
    pages, B, stride = 1_000_003, 65536, 12
    g = np.random.default_rng(6)
    ids = g.choice(B, 300, replace=False)
    table, lens = np.full((B, stride), -1, dtype=np.int32), np.zeros(B, dtype=np.int32)
    refs, free = np.zeros(pages, dtype=np.int32), g.permutation(pages).astype(np.int32)
    count = pages
    d = smla.make_cache_desc(0, 1, 4, pages, B, stride)
    dv = [_dev(x) for x in (table, lens, refs, free, [count])]
    err, work = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty(600, dtype=torch.int32, device="cuda")
    for new in (g.integers(0, 49, 300), g.integers(0, 49, 300) * (g.random(300) < 0.5), np.full(300, 48), np.zeros(300, dtype=int)):
        smla.cache_resize(d, *dv, _dev(ids), _dev(new), work, err)
        e, count = C.resize(4, table, lens, refs, free, count, ids.tolist(), new.tolist())
        assert e == 0 and err.item() == 0 and dv[4].item() == count
        for a, b in zip(dv, (table, lens, refs, free)):
            assert np.array_equal(a.cpu().numpy(), b)


def test_forks_follow_resizes_without_a_pause():
    # calls queued one behind another, none waited for: each sees what the one before did
    for lens in ([100, 37, 0, 0, 0, 0], [2000, 1999, 0, 0, 0, 0]):
        p = Pool("fp8_tensor", 2, 1 if lens[0] == 100 else 2, lens, 1100, 4096, seed=11)
        work, got = torch.empty(12, dtype=torch.int32, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")
        a, b, z, grow = _dev([0, 1, 1, 0]), _dev([2, 3, 4, 5]), _dev([0, 0, 0, 0]), _dev([lens[0] + 3, lens[1] + 70])
        two = _dev([0, 1])
        for _ in range(30):
            smla.cache_fork(p.desc, *p.tables(), a, b, got, p.raw, p.err)
            smla.cache_resize(p.desc, *p.tables(), b, z, work, p.err)
            smla.cache_resize(p.desc, *p.tables(), two, grow, work, p.err)
            smla.cache_resize(p.desc, *p.tables(), two, _dev(lens[:2]), work, p.err)
        for _ in range(30):
            _, p.count, _ = C.fork(p.cache, p.fmt, p.P, p.table, p.lens, p.refs, p.free, p.count, [0, 1, 1, 0], [2, 3, 4, 5])
            for ids, new in (([2, 3, 4, 5], [0] * 4), ([0, 1], grow.tolist()), ([0, 1], lens[:2])):
                _, p.count = C.resize(p.P, p.table, p.lens, p.refs, p.free, p.count, ids, new)
        p.check()


@pytest.mark.parametrize("stride", [8, 2048])  # one launch; three
def test_resize_releases_a_page_more_often_than_it_is_held(stride):
    # 64 requests hold page 7 by their tables, three by its count, and two of them page 5, which is free by its count: three
    # releases count, page 7 is listed once, and every order of the others ends the same
    B, pages, P = 64, 16, 16
    d = smla.make_cache_desc(1, 1, P, pages, B, stride)
    for seed in range(20):
        g = np.random.default_rng(seed)
        table, lens = np.full((B, stride), -1, dtype=np.int32), np.full(B, P, dtype=np.int32)
        table[:, 0] = 7
        two = g.choice(B, 2, replace=False)
        table[two, 1], lens[two] = 5, 2 * P
        refs, free = np.zeros(pages, dtype=np.int32), np.full(pages, -1, dtype=np.int32)
        refs[7] = 3
        free[:14] = [p for p in range(16) if p not in (5, 7)]
        dv = [_dev(x) for x in (table, lens, refs, free, [14])]
        err, work = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty(2 * B, dtype=torch.int32, device="cuda")
        ids = g.permutation(B)
        smla.cache_resize(d, *dv, _dev(ids), _dev(np.zeros(B, dtype=int)), work, err)
        e, count = C.resize(P, table, lens, refs, free, 14, ids.tolist(), [0] * B)
        assert e == C.ERR_PAGE == err.item() and dv[4].item() == count == 15 and free[14] == 7
        for a, b in zip(dv, (table, lens, refs, free)):
            assert np.array_equal(a.cpu().numpy(), b)


def test_compact_leaves_out_a_length_past_int32():
    p = Pool("fp8_ds", 1, 4, [8, 8], 2, 6, seed=4)
    new = torch.full((2,), -5, dtype=torch.int32, device="cuda")
    for start, n in ((2**31 - 3, 3), (2**31 - 1, 1), (2**31 - 1, 0)):
        starts, cu, keep = [start, 0], [0, n, n + 1], list(range(1, n + 1)) + [2]
        want = np.full(2, -5)
        smla.cache_compact(p.desc, p.d_table, _dev(starts), _dev(cu), _dev(keep), p.raw, new.fill_(-5), p.err)
        e = C.compact(p.cache, "fp8_ds", 4, p.table, starts, cu, keep, want)
        assert e == (C.ERR_INDEX if n else 0)
        p.check(e)
        assert new.tolist() == want.tolist() == ([-5, 1] if n else [2**31 - 1, 1])


@pytest.mark.parametrize("big", [False, True])  # one launch a resize; three
@pytest.mark.parametrize("captured", [False, True])
def test_calls_behind_writes_of_what_they_read(captured, big):
    # tables, lists and rows change just before each call, by kernels and by copies, and nothing waits in between; the same
    # captured into a graph
    lens = [2000, 1999, 0, 0, 0, 0] if big else [100, 37, 0, 0, 0, 0]
    p = Pool("fp8_ds", 2, 1 if big else 4, lens, 17000 if big else 70, 11000 if big else 100, seed=12)
    h_src, h_dst, h_req, h_new, h_start, h_cu, h_keep = ([0, 1], [2, 3], [0, 1, 2, 3], [lens[0] + 9, 20, 0, 41], [30] + [0] * 5,
                                                         [0] + [2] * 6, [1, 3])
    a, b = [int(p.table[0, 0])], [int(p.free[0])]
    first = [x.clone() for x in (p.raw, *p.tables())] + [_dev(x) for x in (h_src, h_dst, h_req, h_new, h_start, h_cu, h_keep, a, b)]
    src, dst, req, new, start, cu, keep, d_a, d_b = (torch.empty_like(x) for x in first[6:])
    state = [p.raw, *p.tables(), src, dst, req, new, start, cu, keep, d_a, d_b]
    new_lens, got, work = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (6, 2, 8))

    def write(i, names):
        for k in names:
            if i % 2:
                state[k].copy_(first[k])
            else:
                torch.bitwise_or(first[k], 0, out=state[k])

    def once(i):
        write(i, [(k + i) % 15 for k in range(15)])
        smla.cache_copy_pages(p.desc, d_a, d_b, p.raw, p.err)
        write(i, [6, 7])
        smla.cache_fork(p.desc, *p.tables(), src, dst, got, p.raw, p.err)
        write(i, [8, 9])
        smla.cache_resize(p.desc, *p.tables(), req, new, work, p.err)
        write(i, [10, 11, 12])
        smla.cache_compact(p.desc, p.d_table, start, cu, keep, p.raw, new_lens, p.err)

    once(0)
    C.copy_pages(p.cache, a, b)
    e, p.count, pages = C.fork(p.cache, "fp8_ds", p.P, p.table, p.lens, p.refs, p.free, p.count, h_src, h_dst)
    assert e == 0 and got.tolist() == pages
    e, p.count = C.resize(p.P, p.table, p.lens, p.refs, p.free, p.count, h_req, h_new)
    lens_after = np.zeros(6, dtype=int)
    assert e == 0 and C.compact(p.cache, "fp8_ds", p.P, p.table, h_start, h_cu, h_keep, lens_after) == 0
    p.check()
    assert new_lens.tolist() == lens_after.tolist()
    want = [x.clone() for x in (*state, got, new_lens)]
    marks = []
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            once(0)
            once(1)
        for _ in range(4):
            g.replay()
            marks.append([x.clone() for x in (*state, got, new_lens)])
    else:
        for i in range(30):
            once(i)
            marks.append([x.clone() for x in (*state, got, new_lens)])
    torch.cuda.synchronize()
    assert p.err.item() == 0
    for m in marks:
        for x, y in zip(m, want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("stride", [8, 40000])  # one launch; three
@pytest.mark.parametrize("entry", [-1, -7, 40, 2**31 - 1, -2**31])
def test_resize_over_a_free_list_entry_that_is_no_page(stride, entry):
    # the request that takes it keeps -1 there, the others get their pages
    p = Pool("fp8_tensor", 1, 4, [9, 0, 2], stride, 40, seed=13)
    p.free[p.count - 2] = p.free[1] = entry
    p.d_free.copy_(_dev(p.free))
    assert p.resize([1, 2, 0], [11, 6, 20]) == C.ERR_PAGE
    assert p.table[1, :4].tolist().count(-1) == 2 and p.lens.tolist() == [20, 11, 6]
    p.check(C.ERR_PAGE)
    assert p.resize([0, 1, 2], [0, 0, 0]) == C.ERR_PAGE  # the entry without a page is met again
    p.check(C.ERR_PAGE)


@pytest.mark.parametrize("bad", [-1, -5, 30, 2**31 - 1, -2**31])
@pytest.mark.parametrize("fmt,page", [("bf16", 4), ("index_keys", 16)])
def test_fork_of_a_source_whose_pages_are_none(fmt, page, bad):
    # the last page, partly filled, is none: the fork is refused and changes nothing, those behind it take what it would have
    # taken; a full page that is none is passed on
    lens = [2 * page + 3, 3 * page, page + 1, 5, 0, 0, 0, 0]
    p = Pool(fmt, 2, page, lens, 6, 30, seed=14, gap=16)
    p.table[0, 2] = p.table[1, 1] = bad
    p.d_table.copy_(_dev(p.table))
    count = p.count
    assert p.fork([0, 1, 2, 3], [4, 5, 6, 7]) == C.ERR_PAGE
    assert p.lens.tolist()[4:] == [0, 3 * page, page + 1, 5] and p.count == count - 2 and p.table[5, 1] == bad
    p.check(C.ERR_PAGE)


@pytest.mark.parametrize("entry", [-1, -7, 12, 2**31 - 1, -2**31])
def test_fork_over_a_free_list_entry_that_is_no_page(entry):
    # the fork whose turn it is is refused, the entry leaves the list, and the next fork takes the one before it
    p = Pool("fp8_ds", 2, 4, [3, 6, 0, 0, 0, 0], 3, 12, seed=15)
    p.free[p.count - 2] = entry
    p.d_free.copy_(_dev(p.free))
    count, third = p.count, int(p.free[p.count - 3])
    assert p.fork([0, 1, 0], [2, 3, 4]) == C.ERR_PAGE
    assert p.count == count - 3 and p.lens.tolist() == [3, 6, 3, 0, 3, 0] and p.table[4, 0] == third
    p.check(C.ERR_PAGE)


@pytest.mark.parametrize("n,short", [(1025, 1), (3000, 1300), (3000, 0), (2048, 1)])
def test_resize_of_lists_longer_than_a_batch(n, short):
    # the plan takes 1024 requests at a time: places, shortage and refusals carry over from one batch to the next. `short`: how
    # many of the last requests that grow find no page left
    g = np.random.default_rng(n + short)
    B, stride, P = n + 50, 8, 4
    ids = g.permutation(B)[:n]
    new = g.integers(1, stride * P + 1, n)
    need = -(-new // P)
    pages = int(need[:n - short].sum()) + (int(need[n - short]) - 1 if short else 17)
    p = Pool("fp8_tensor", 1, P, [0] * B, stride, pages, seed=16)
    e = p.resize(ids.tolist(), new.tolist())
    assert e == (C.ERR_PAGE if short else 0) and np.count_nonzero(p.lens) == n - short
    p.check(e)
    # some shrink, some grow on what those free, in another order; one twice, no such request, too long, in the second batch
    order, new = g.permutation(ids), g.integers(0, stride * P + 1, n)
    order[-1], order[n - 3], new[n - 4] = order[3], B, stride * P + 1
    e = p.resize(order.tolist(), new.tolist())
    assert e & C.ERR_INDEX
    p.check(e)
    assert p.resize(ids.tolist(), [0] * n) == 0 and p.count == pages
    p.check()


@pytest.mark.parametrize("n,short", [(1025, 1), (1025, 0), (2600, 1500), (2600, 3)])
def test_fork_of_lists_longer_than_a_batch(n, short):
    g = np.random.default_rng(n + short)
    live = [9, 3, 8, 1, 14, 4, 0]
    B, used = n + len(live) + 5, sum(-(-x // 4) for x in live)
    src = g.integers(0, len(live), n)
    src[-1] = 0
    need = np.array([live[s] % 4 != 0 for s in src])
    last = np.flatnonzero(need)
    pages = used + len(last) - short + (0 if short else 9)
    p = Pool("fp8_tensor", 2, 4, live + [0] * (B - len(live)), 4, pages, seed=17)
    dst = g.permutation(np.arange(len(live), B))[:n]
    e = p.fork(src.tolist(), dst.tolist())
    assert e == (C.ERR_PAGE if short else 0)
    p.check(e)
    # refusals behind the first batch: a target twice, one that is a source, no such request; the others are taken
    assert p.resize(dst.tolist(), [0] * n) == 0
    src[1024], dst[n - 1] = dst[5], dst[2]
    src[7] = -1
    e = p.fork(src.tolist(), dst.tolist())
    assert e & C.ERR_INDEX
    p.check(e)


def test_resize_refusals_in_three_launches():
    p = Pool("bf16", 1, 4, [10, 11, 12, 0], 40000, 12, seed=2)
    e = p.resize([0, 0, 1, 4], [0, 4, 160001, 1])       # twice; too long; no such request
    assert e == C.ERR_INDEX
    p.check(e)
    e = p.resize([3, -1, 3, 2], [4, 0, 0, -1])          # twice, apart; no such request; a negative length
    assert e == C.ERR_INDEX
    p.check(e)
    assert p.resize([3, 2, 0], [16, 13, 0]) == 0         # grows on what the same call frees
    p.check()
    e = p.resize([0, 2, 1], [16, 160000, 5])             # not enough from the second on: it stays, the last still shrinks
    assert e == C.ERR_PAGE
    p.check(e)
    # a page that no request holds, and a table entry that is no page
    p.d_refs[int(p.table[1, 0])] = 0
    p.refs[int(p.table[1, 0])] = 0
    p.d_table[1, 1] = 77
    p.table[1, 1] = 77
    assert p.resize([1, 0], [0, 3]) == C.ERR_PAGE
    p.check(C.ERR_PAGE)


def test_resize_random_walk_in_three_launches():
    g = np.random.default_rng(18)
    p = Pool("fp8_tensor", 1, 4, [0] * 40, 70000, 500, seed=1)
    for _ in range(25):
        n = int(g.integers(1, 41))
        ids = g.permutation(40)[:n]
        if g.random() < 0.3:
            ids[-1] = ids[0]
        new = g.integers(0, 121, n) * (g.random(n) < 0.7)
        e = p.resize(ids.tolist(), new.tolist())
        p.check(e)


def test_resize_of_the_longest_list():
    # 65,536 requests take a page each and give it back; the last ones find none
    B = n = 65536
    pages = B - 7
    g = np.random.default_rng(19)
    ids, free = g.permutation(B).astype(np.int32), g.permutation(pages).astype(np.int32)
    d = smla.make_cache_desc(0, 1, 2, pages, B, 3)
    dv = [_dev(x) for x in (np.full((B, 3), -1), np.zeros(B), np.zeros(pages), free, [pages])]
    work, err = torch.empty(2 * n, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    smla.cache_resize(d, *dv, _dev(ids), _dev(np.ones(n)), work, err)
    table, lens, refs = np.full((B, 3), -1), np.zeros(B), np.ones(pages)
    table[ids[:pages], 0], lens[ids[:pages]] = free[::-1], 1
    assert err.item() == C.ERR_PAGE and dv[4].item() == 0
    for a, b in zip(dv, (table, lens, refs, np.full(pages, -1))):
        assert np.array_equal(a.cpu().numpy(), b)
    err.zero_()
    smla.cache_resize(d, *dv, _dev(ids[::-1].copy()), _dev(np.zeros(n)), work, err)
    assert err.item() == 0 and dv[4].item() == pages
    for a, b in zip(dv, (np.full((B, 3), -1), np.zeros(B), np.zeros(pages), np.arange(pages))):
        assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("L", [1, 9])
def test_compact_one_long_list_among_short_ones(fmt, L):
    # few kept rows a request on average, the form for short lists, and one request of several chunks: on its own, and in front
    # of and behind requests of one row and of none
    g = np.random.default_rng(20 + L)
    for B, at, n in ((64, 0, 1400), (64, 63, 1400), (200, 77, 4500)):
        lens = [int(x) for x in g.integers(0, 3, B)]
        lens[at] = n
        p = Pool(fmt, L, 16, lens, -(-n // 16), sum(-(-x // 16) for x in lens) + 2, seed=21, gap=16)
        keep = [list(range(x - 1, x)) if x else [] for x in lens]
        keep[at] = sorted(g.choice(n, n * 9 // 10, replace=False).tolist())
        flat = sum(keep, [])
        assert 256 < len(keep[at]) and len(flat) <= 24 * B
        cu = np.concatenate([[0], np.cumsum([len(k) for k in keep])])
        new, want = torch.full((B,), -5, dtype=torch.int32, device="cuda"), np.full(B, -5)
        smla.cache_compact(p.desc, p.d_table, _dev([0] * B), _dev(cu), _dev(flat), p.raw, new, p.err)
        assert C.compact(p.cache, fmt, 16, p.table, [0] * B, cu, flat, want) == 0
        p.check()
        assert new.tolist() == want.tolist()


@pytest.mark.parametrize("fmt", ["bf16", "fp8_ds"])
def test_compact_refusals_in_a_list_of_several_chunks(fmt):
    # in the form for short lists and in the other one: entries that break the order, at a chunk's start too, pages that are none
    # and slots past the table are left where they are, the others move
    g = np.random.default_rng(22)
    for B in (1, 120):
        lens = [2600] + [0] * (B - 1)
        p = Pool(fmt, 2, 16, lens, 163, 170, seed=23)
        keep = sorted(g.choice(2599, 2300, replace=False).tolist())
        for k in (64, 128, 255, 256, 448, 512, 1000, 1792):
            keep[k] = keep[k - 1] if k % 3 else 0
        keep[-1] = 5000
        table = p.table.copy()
        table[0, [9, 40, 100]] = [-1, 170, 2**31 - 1]
        cu = [0] + [len(keep)] * B
        smla.cache_compact(p.desc, _dev(table), _dev([0] * B), _dev(cu), _dev(keep), p.raw, None, p.err)
        e = C.compact(p.cache, fmt, 16, table, [0] * B, cu, keep)
        assert e == C.ERR_INDEX | C.ERR_PAGE
        p.check(e)
