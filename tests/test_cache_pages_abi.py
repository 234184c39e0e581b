"""The tree and cache page calls refuse bad arguments on the host (CPU only), and the page
oracle's own pins."""
import ctypes
import os

import numpy as np
import pytest

import oracle.cache_pages_oracle as C
import sparse_mla_decode_smla_gb300 as smla
from sparse_mla_decode_smla_gb300 import _build

P = ctypes.c_void_p
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "smla.h")


@pytest.fixture(scope="module")
def L():
    _build.build()
    return smla.lib()


def _tree(**kw):
    d = smla.make_tree_desc(8, 16, 2, 64, 16, 4, smla.SMLA_KV_FP8_DS, 1 / 24)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _tree_status(L, d, q=16, kv=16, pt=16, ctx=16, cu=16, mask=None, sink=None, out=16, lse=None, ws=256, nbytes=1 << 30):
    return L.smla_tree_decode(ctypes.byref(d) if d is not None else None, P(q), P(kv), P(pt), P(ctx), P(cu), P(mask), P(sink),
                              P(out), P(lse), P(ws), nbytes, None)


def test_layouts_match_the_header():
    assert ctypes.sizeof(smla.smla_tree_desc) == 56
    assert smla.smla_tree_desc.num_pages.offset == 16 and smla.smla_tree_desc.mask_words.offset == 40
    assert ctypes.sizeof(smla.smla_cache_desc) == 40
    assert smla.smla_cache_desc.num_pages.offset == 24 and smla.smla_cache_desc.layer_stride.offset == 32


@pytest.mark.parametrize("field,value,status", [
    ("num_tokens", 0, 2), ("num_heads", 0, 2), ("num_heads", 129, 2), ("num_requests", 0, 2), ("num_requests", 65537, 2),
    ("page_size", 48, 2), ("page_size", 8192, 2), ("page_size", 0, 2), ("num_pages", 0, 2), ("num_pages", 1 << 25, 2),
    ("num_pages", 1 << 62, 2), ("page_table_stride", 0, 2), ("kv_format", 3, 4), ("sm_scale", float("nan"), 2),
    ("mask_words", -1, 2), ("mask_words", 2049, 2), ("num_tokens", 1 << 30, 2)])
def test_tree_desc_rules(L, field, value, status):
    assert _tree_status(L, _tree(**{field: value})) == status
    n = ctypes.c_size_t(7)
    assert L.smla_tree_workspace_size(ctypes.byref(_tree(**{field: value})), ctypes.byref(n)) == status
    assert n.value == 0


def test_tree_pointers_and_mask(L):
    assert _tree_status(L, None) == 1
    for k in ("q", "kv", "pt", "ctx", "cu", "out", "ws"):
        assert _tree_status(L, _tree(), **{k: 0}) == 1, k
        assert _tree_status(L, _tree(), **{k: 258}) == 3, k
    for k in ("sink", "lse"):
        assert _tree_status(L, _tree(), **{k: 18}) == 3, k
    assert _tree_status(L, _tree(), mask=16) == 2               # a mask without mask_words
    assert _tree_status(L, _tree(mask_words=1)) == 2            # mask_words without a mask
    assert _tree_status(L, _tree(mask_words=1), mask=18) == 3
    d = _tree()
    d.reserved[2] = 1
    assert _tree_status(L, d) == 2
    assert _tree_status(L, _tree(kv_format=smla.SMLA_KV_FP8_TENSOR, kv_scale=0.0)) == 2
    assert L.smla_tree_workspace_size(ctypes.byref(_tree()), None) == 1


def _cache(**kw):
    d = smla.make_cache_desc(smla.SMLA_KV_FP8_DS, 2, 64, 16, 4, 8)
    for k, v in kw.items():
        setattr(d, k, v)
    return ctypes.byref(d)


def _calls(L, d, a=16, kv=16, n=2):
    """Every page call with the same description and plain pointers `a` and `kv`."""
    return {
        "copy": L.smla_cache_copy_pages(d, P(a), P(16), n, P(kv), None, None),
        "compact": L.smla_cache_compact(d, P(a), P(16), P(16), P(16), n, P(kv), None, None, None),
        "fork": L.smla_cache_fork(d, P(a), P(16), P(16), P(16), P(16), P(16), P(16), n, P(16), P(kv), None, None),
        "resize": L.smla_cache_resize(d, P(a), P(16), P(16), P(16), P(16), P(16), P(16), n, P(16), None, None),
    }


@pytest.mark.parametrize("field,value,status", [
    ("kv_format", 4, 4), ("kv_format", -1, 4), ("num_layers", 0, 2), ("page_size", 3, 2), ("page_size", 8192, 2),
    ("num_requests", 0, 2), ("num_requests", 65537, 2), ("page_table_stride", 0, 2), ("reserved", 1, 2), ("num_pages", 0, 2),
    ("num_pages", 1 << 31, 2), ("layer_stride", 16 * 64 * 656 - 16, 2), ("layer_stride", 16 * 64 * 656 + 8, 2)])
def test_cache_desc_rules(L, field, value, status):
    assert set(_calls(L, _cache(**{field: value})).values()) == {status}


def test_cache_pointers_and_counts(L):
    assert set(_calls(L, None).values()) == {1}
    assert set(_calls(L, _cache(), a=0).values()) == {1}
    assert set(_calls(L, _cache(), a=18).values()) == {3}
    assert set(_calls(L, _cache(), n=-1).values()) == {2}
    got = _calls(L, _cache(), kv=24)
    assert [got[k] for k in ("copy", "compact", "fork")] == [3, 3, 3]
    got = _calls(L, _cache(), kv=0)
    assert [got[k] for k in ("copy", "compact", "fork")] == [1, 1, 1]
    got = _calls(L, _cache(), n=5)                        # more than the four requests
    assert got["fork"] == 2 and got["resize"] == 2
    assert _calls(L, _cache(), n=17)["copy"] == 2         # more than the sixteen pages
    got = _calls(L, _cache(), n=0)
    assert got["copy"] == 0 and got["fork"] == 0 and got["resize"] == 0
    # the index keys come in pages of 16 to 128 slots
    assert set(_calls(L, _cache(kv_format=smla.SMLA_CACHE_INDEX_KEYS, page_size=8)).values()) == {2}


def test_without_a_device_the_calls_say_so(L):
    n = ctypes.c_size_t(0)
    if L.smla_tree_workspace_size(ctypes.byref(_tree()), ctypes.byref(n)) != 8:
        pytest.skip("an sm_103 device is present")
    assert _tree_status(L, _tree()) == 8
    assert set(_calls(L, _cache()).values()) == {8}


def test_oracle_compact_keeps_rows_in_order():
    g = np.random.default_rng(1)
    for fmt in ("bf16", "fp8_ds", "fp8_tensor", "index_keys"):
        Pg = 16
        cache = g.integers(0, 256, (2, 5, C.page_bytes(fmt, Pg)), dtype=np.uint8)
        table = np.array([[3, 0, 4]])
        flat = [C.row_get(cache, fmt, Pg, table[0, s // Pg], s % Pg) for s in range(48)]
        keep = sorted(g.choice(30, 11, replace=False).tolist())
        assert C.compact(cache, fmt, Pg, table, [7], [0, 11], keep) == 0
        now = [C.row_get(cache, fmt, Pg, table[0, s // Pg], s % Pg) for s in range(48)]
        for k, j in enumerate(keep):
            assert np.array_equal(now[7 + k], flat[7 + j])
        for s in list(range(7)) + list(range(18, 48)):
            assert np.array_equal(now[s], flat[s])


def test_oracle_pages_are_conserved():
    # random forks and resizes: every page is either free or held, as often as its refcount says
    g = np.random.default_rng(2)
    Pg, pages, B, stride = 4, 40, 6, 8
    cache = g.integers(0, 256, (1, pages, 4 * 576), dtype=np.uint8)
    table, lens = np.full((B, stride), -1), np.zeros(B, dtype=int)
    refs, free, count = np.zeros(pages, dtype=int), np.arange(pages), pages
    refused = 0
    for _ in range(300):
        if g.random() < 0.6:
            ids = g.permutation(B)[:g.integers(1, B + 1)]
            e, count = C.resize(Pg, table, lens, refs, free, count, ids, g.integers(0, stride * Pg + 1, len(ids)))
        else:
            ids = g.permutation(B)[:4]
            e, count, _p = C.fork(cache, "fp8_tensor", Pg, table, lens, refs, free, count, ids[:2], ids[2:])
        refused += e != 0
        held = np.zeros(pages, dtype=int)
        for r in range(B):
            used = -(-lens[r] // Pg)
            assert (table[r, used:] == -1).all()
            np.add.at(held, table[r, :used], 1)
        assert np.array_equal(held, refs)
        assert sorted(free[:count]) == sorted(np.flatnonzero(refs == 0)) and (free[count:] == -1).all()
    assert refused


def test_oracle_resize_leaves_slots_without_a_page_where_the_list_holds_none():
    table, lens, refs = np.full((2, 4), -1), np.zeros(2, dtype=int), np.zeros(6, dtype=int)
    free = np.array([0, 77, -3, 5, -1, -1])
    e, count = C.resize(4, table, lens, refs, free, 4, [0, 1], [9, 3])
    assert e == C.ERR_PAGE and count == 0 and (free == -1).all()
    assert table.tolist() == [[5, -1, -1, -1], [0, -1, -1, -1]] and lens.tolist() == [9, 3] and refs.tolist() == [1, 0, 0, 0, 0, 1]


def test_oracle_fork_refuses_a_last_page_that_is_none_and_passes_full_ones_on():
    cache = np.arange(2 * 6 * 4 * 576, dtype=np.int64).astype(np.uint8).reshape(2, 6, -1)
    before = cache.copy()
    table = np.array([[0, 9, -1], [1, -1, -1], [-1, -1, -1], [-1, -1, -1], [-1, -1, -1]])
    lens, refs = np.array([7, 4, 0, 0, 0]), np.array([1, 1, 0, 0, 0, 0])
    free = np.array([2, 3, 4, 5, -1, -1])
    e, count, pages = C.fork(cache, "fp8_tensor", 4, table, lens, refs, free, 4, [0, 1], [2, 3])
    assert e == C.ERR_PAGE and count == 4 and pages == [-2, -1] and free.tolist() == [2, 3, 4, 5, -1, -1]
    assert table[2].tolist() == [-1] * 3 and table[3].tolist() == [1, -1, -1] and lens.tolist() == [7, 4, 0, 4, 0]
    table[1, 0] = 9  # a full page that is none
    e, count, pages = C.fork(cache, "fp8_tensor", 4, table, lens, refs, free, 4, [1], [4])
    assert e == C.ERR_PAGE and pages == [-1] and table[4].tolist() == [9, -1, -1] and refs.tolist() == [1, 2, 0, 0, 0, 0]
    assert np.array_equal(cache, before)


def test_header_says_that_a_refused_fork_may_take_a_bad_entry_off_the_list():
    # the model: an entry that is no page leaves the list with the fork that it refuses; the next fork takes the one before it
    cache = np.zeros((1, 6, 4 * 576), dtype=np.uint8)
    table, lens = np.array([[0], [-1], [-1], [-1]]), np.array([3, 0, 0, 0])
    refs, free = np.array([1, 0, 0, 0, 0, 0]), np.array([1, 2, -6, 3, -1, -1])
    e, count, pages = C.fork(cache, "fp8_tensor", 4, table, lens, refs, free, 4, [0, 0, 0], [1, 2, 3])
    assert e == C.ERR_PAGE and count == 1 and pages == [3, -2, 2] and free.tolist() == [1, -1, -1, -1, -1, -1]
    assert lens.tolist() == [3, 3, 0, 3] and table[2, 0] == -1
    text = " ".join(open(HEADER).read().replace("*", " ").split())
    assert "refused and changed nothing" not in text and "the entry leaves the list all the same" in text


def test_header_says_that_tree_attention_has_the_scale_window_at_every_head_count():
    text = " ".join(open(HEADER).read().replace("*", " ").split())
    assert "fp8_ds with 64+ heads (smla_tree_decode: with any number)" in text and "here with any number of heads" in text


def test_header_gives_the_error_of_small_elements_of_a_query():
    text = " ".join(open(HEADER).read().replace("*", " ").split())
    tree = text[text.index("Attention of all nodes over their contexts"):]
    assert "q exactly" not in tree and "elements below 2^-17 of their row's largest, which keep 2^-25 of it" in tree
