"""The Python calls around a prompt refuse tensors of types and strides that the library would read as something else (CPU only)."""
import pytest
import torch

import sparse_mla_decode_smla_gb300 as smla
from sparse_mla_decode_smla_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    smla.lib()


def _refused(status, f, *args, **kw):
    with pytest.raises(smla.SmlaError) as e:
        f(*args, **kw)
    assert e.value.status == status


def _lp(**kw):
    a = dict(logits=torch.zeros(4, 100), tokens=torch.zeros(4, 2, dtype=torch.int32), logprobs=torch.zeros(4, 2), entropy=torch.zeros(4),
             top_ids=torch.zeros(4, 3, dtype=torch.int32), top_logprobs=torch.zeros(4, 3))
    a.update(kw)
    return a


@pytest.mark.parametrize("dtype", [torch.float16, torch.int32, torch.int16, torch.float64, torch.uint8])
def test_logits_of_another_type(dtype):
    _refused(4, smla.token_logprobs, **_lp(logits=torch.zeros(4, 100, dtype=dtype)))


def test_logits_whose_elements_do_not_follow_one_another():
    for t in (torch.zeros(100, 4).t(), torch.zeros(4, 200)[:, ::2], torch.zeros(4, 1).expand(4, 100), torch.zeros(1, 200)[:, ::2]):
        _refused(2, smla.token_logprobs, **_lp(logits=t))


@pytest.mark.parametrize("name,wrong", [("tokens", torch.int64), ("tokens", torch.float32), ("logprobs", torch.bfloat16), ("entropy", torch.float64),
                                        ("top_ids", torch.int64), ("top_logprobs", torch.float16)])
def test_the_rest_of_the_log_probabilities(name, wrong):
    _refused(4, smla.token_logprobs, **_lp(**{name: _lp()[name].to(wrong)}))
    wide = torch.zeros(8, 6, dtype=_lp()[name].dtype)
    shape = _lp()[name].shape
    _refused(2, smla.token_logprobs, **_lp(**{name: wide[:4, :shape[1]] if len(shape) == 2 else wide[::2, 0]}))


def _norm(**kw):
    bf = torch.bfloat16
    a = dict(x=torch.zeros(4, 256, dtype=bf), residual=torch.zeros(4, 256, dtype=bf), weight=torch.zeros(256, dtype=bf), eps=1e-6,
             residual_out=torch.zeros(4, 256, dtype=bf), y=torch.zeros(4, 256, dtype=bf), codes=torch.zeros(4, 256, dtype=torch.uint8),
             scales=torch.zeros(4, 2))
    a.update(kw)
    return a


@pytest.mark.parametrize("name", ["x", "residual", "weight", "residual_out", "y", "codes", "scales"])
def test_the_norm(name):
    t = _norm()[name]
    for wrong in (torch.float16, torch.float64):
        _refused(4, smla.add_rmsnorm, **_norm(**{name: t.to(wrong)}))
    wide = torch.zeros([2 * n for n in t.shape], dtype=t.dtype)
    _refused(2, smla.add_rmsnorm, **_norm(**{name: wide[tuple(slice(0, 2 * n, 2) for n in t.shape)]}))
    if t.dim() == 2:
        _refused(2, smla.add_rmsnorm, **_norm(**{name: torch.zeros(t.shape[::-1], dtype=t.dtype).t()}))


def test_a_scale_whose_product_with_log2_e_is_not_finite():
    for scale in (2.4e38, 3e38, 3.4e38):
        _refused(2, smla.token_logprobs, **_lp(scale=scale), stream=0)
