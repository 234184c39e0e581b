"""The calls around a prompt refuse bad arguments on the host (CPU only)."""
import ctypes

import pytest

import sparse_mla_decode_smla_gb300 as smla
from sparse_mla_decode_smla_gb300 import _build

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    _build.build()
    return smla.lib()


def _ref(d):
    return ctypes.byref(d) if d is not None else None


def test_layouts_match_the_header():
    assert ctypes.sizeof(smla.smla_read_desc) == 64 and smla.smla_read_desc.kv_scale.offset == 48
    assert ctypes.sizeof(smla.smla_norm_desc) == 40 and smla.smla_norm_desc.rms_eps.offset == 28
    assert ctypes.sizeof(smla.smla_prompt_desc) == 104 and smla.smla_prompt_desc.q_token_stride.offset == 48
    assert ctypes.sizeof(smla.smla_logprob_desc) == 48 and smla.smla_logprob_desc.scale.offset == 32


# ---------------------------------------------------------------- cache rows


def _read(L, d, kv=16, pt=16, starts=16, cu=16, lat=16, rope=16, err=None):
    return L.smla_cache_read(_ref(d), P(kv), P(pt), P(starts), P(cu), P(lat), P(rope), P(err), None)


def _read_desc(**kw):
    d = smla.make_read_desc(smla.SMLA_KV_FP8_DS, 64, 16, 2, 4, 100)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("field,value,status", [
    ("kv_format", 3, 4), ("kv_format", -1, 4), ("page_size", 48, 2), ("page_size", 0, 2), ("page_size", 8192, 2), ("num_pages", 0, 2),
    ("num_pages", 1 << 31, 2), ("num_requests", 0, 2), ("num_requests", 65537, 2), ("page_table_stride", 0, 2), ("num_rows", -1, 2),
    ("num_rows", 1 << 31, 2), ("latent_stride", 504, 2), ("latent_stride", 516, 2), ("rope_stride", 56, 2), ("rope_stride", 68, 2)])
def test_read_rules(L, field, value, status):
    assert _read(L, _read_desc(**{field: value})) == status


def test_read_pointers(L):
    assert _read(L, None) == 1
    for k in ("kv", "pt", "starts", "cu", "lat", "rope"):
        assert _read(L, _read_desc(), **{k: 0}) == 1, k
        assert _read(L, _read_desc(), **{k: 18}) == 3, k
    assert _read(L, _read_desc(), err=18) == 3
    d = _read_desc()
    d.reserved[1] = 1
    assert _read(L, d) == 2
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert _read(L, _read_desc(kv_format=smla.SMLA_KV_FP8_TENSOR, kv_scale=s)) == 2
    assert _read(L, _read_desc(num_rows=0), lat=0) == 0  # nothing to do


# ---------------------------------------------------------------- attention


def _attn(L, d, q=16, k=16, v=16, rope=16, cq=16, ck=16, prefix=None, slopes=None, sink=None, out=16, lse=None, ws=256, nbytes=1 << 40):
    return L.smla_prompt_attention(_ref(d), P(q), P(k), P(v), P(rope), P(cq), P(ck), P(prefix), P(slopes), P(sink), P(out), P(lse),
                                   P(ws), nbytes, None)


def _attn_desc(**kw):
    d = smla.make_prompt_desc(8, 16, 4, 2, 2, 64, 192 ** -0.5)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("field,value,status", [
    ("num_tokens", -1, 2), ("num_tokens", 1 << 30, 2), ("num_keys", 0, 2), ("num_heads", 0, 2), ("num_heads", 5, 2), ("num_heads", 2048, 2),
    ("num_kv_heads", 0, 2), ("num_kv_heads", 3, 2), ("num_requests", 0, 2), ("num_requests", 65537, 2), ("rope_dim", 32, 4),
    ("rope_dim", 128, 4), ("causal", 2, 4), ("sm_scale", 0.0, 2), ("sm_scale", -0.1, 2), ("sm_scale", float("nan"), 2),
    ("sm_scale", 3e38, 2), ("softcap", -1.0, 2), ("softcap", float("inf"), 2), ("softcap", float("nan"), 2), ("softcap", 1e-40, 2),
    ("q_token_stride", 4, 2), ("q_token_stride", 772, 2), ("q_head_stride", 128, 2), ("k_token_stride", 120, 2), ("k_head_stride", 132, 2),
    ("v_token_stride", 0, 2), ("v_head_stride", -128, 2), ("rope_token_stride", 56, 2), ("v_token_stride", 1 << 40, 2)])
def test_attention_rules(L, field, value, status):
    d = _attn_desc(**{field: value})
    assert _attn(L, d) == status
    n = ctypes.c_size_t(7)
    assert L.smla_prompt_workspace_size(ctypes.byref(d), ctypes.byref(n)) == status and n.value == 0


def test_attention_pointers(L):
    assert _attn(L, None) == 1
    for k in ("q", "k", "v", "cq", "ck", "out", "ws"):
        assert _attn(L, _attn_desc(), **{k: 0}) == 1, k
        assert _attn(L, _attn_desc(), **{k: 258}) == 3, k
    for k in ("prefix", "slopes", "sink", "lse", "rope"):
        assert _attn(L, _attn_desc(), **{k: 18}) == 3, k
    assert _attn(L, _attn_desc(), rope=0) == 2                     # a RoPE part without its keys
    assert _attn(L, _attn_desc(rope_dim=0)) == 2                   # and the other way round
    assert _attn(L, _attn_desc(num_tokens=0), q=0) == 0
    d = _attn_desc()
    d.reserved[2] = 1
    assert _attn(L, d) == 2
    assert L.smla_prompt_workspace_size(ctypes.byref(_attn_desc()), None) == 1


# ---------------------------------------------------------------- the norm


def _norm(L, d, x=16, res=16, w=16, sum_=16, y=16, codes=16, scales=16):
    return L.smla_add_rmsnorm(_ref(d), P(x), P(res), P(w), P(sum_), P(y), P(codes), P(scales), None)


def _norm_desc(**kw):
    d = smla.smla_norm_desc(n=4, x_stride=512, dim=512, group=128, scale_mode=0, rms_eps=1e-6)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("field,value,status", [
    ("n", -1, 2), ("n", 1 << 31, 2), ("dim", 0, 2), ("dim", 516, 2), ("dim", 32776, 2), ("x_stride", 504, 2), ("x_stride", 516, 2),
    ("group", 64, 4), ("scale_mode", 2, 4), ("rms_eps", -1e-6, 2), ("rms_eps", float("nan"), 2), ("rms_eps", float("inf"), 2)])
def test_norm_rules(L, field, value, status):
    assert _norm(L, _norm_desc(**{field: value})) == status


def test_norm_pointers(L):
    assert _norm(L, None) == 1
    assert _norm(L, _norm_desc(), x=0) == 1 and _norm(L, _norm_desc(), w=0) == 1
    assert _norm(L, _norm_desc(), codes=0) == 1 and _norm(L, _norm_desc(), scales=0) == 1  # together or not at all
    assert _norm(L, _norm_desc(), sum_=0, y=0, codes=0, scales=0) == 1
    for k, v in (("x", 24), ("res", 24), ("w", 24), ("sum_", 24), ("y", 24), ("codes", 20), ("scales", 18)):
        assert _norm(L, _norm_desc(), **{k: v}) == 3, k
    assert _norm(L, _norm_desc(n=0), x=0) == 0
    d = _norm_desc()
    d.reserved[1] = 1
    assert _norm(L, d) == 2


# ---------------------------------------------------------------- log probabilities


def _lp(L, d, x=16, tok=16, lp=16, ent=16, ids=16, alt=16, err=None):
    return L.smla_token_logprobs(_ref(d), P(x), P(tok), P(lp), P(ent), P(ids), P(alt), P(err), None)


def _lp_desc(**kw):
    d = smla.smla_logprob_desc(n=4, row_stride=1000, vocab=1000, given=1, top=5, logits_format=1, scale=1.0)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("field,value,status", [
    ("n", -1, 2), ("n", 1 << 31, 2), ("vocab", 0, 2), ("vocab", (1 << 24) + 1, 2), ("row_stride", 999, 2), ("row_stride", 1 << 31, 2),
    ("given", -1, 2), ("given", 1025, 2), ("top", -1, 2), ("top", 65, 2), ("logits_format", 2, 4), ("logits_format", -1, 4),
    ("scale", 0.0, 2), ("scale", -1.0, 2), ("scale", float("nan"), 2), ("scale", float("inf"), 2)])
def test_logprob_rules(L, field, value, status):
    assert _lp(L, _lp_desc(**{field: value})) == status


def test_logprob_pointers(L):
    assert _lp(L, None) == 1
    for k in ("x", "tok", "lp", "ids"):
        assert _lp(L, _lp_desc(), **{k: 0}) == 1, k
    for k in ("x", "tok", "lp", "ent", "ids", "alt", "err"):
        assert _lp(L, _lp_desc(), **{k: 18}) == 3, k
    assert _lp(L, _lp_desc(logits_format=0), x=17) == 3
    assert _lp(L, _lp_desc(n=0), x=0) == 0
    d = _lp_desc()
    d.reserved[2] = 1
    assert _lp(L, d) == 2
