"""Calls on one stream take effect in order, also where a kernel may start before the one ahead of it has ended.

A kernel launched with programmatic serialization that never waits (griddepcontrol.wait) can end while the kernel ahead of
it still runs, and what follows waits for it alone: so each of them waits somewhere."""
import os
import re

import numpy as np
import pytest
import torch

import sparse_mla_decode_smla_gb300 as smla
import workloads as W

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_mla_decode_smla_gb300", "csrc")


def _bodies(text):
    """name -> body of every __global__ function of a source file."""
    out = {}
    for m in re.finditer(r"__global__\b[^;{]*?(\w+)\s*\((?:[^()]|\([^()]*\))*\)\s*\{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        out[m.group(1)] = text[m.end():i]
    return out


def test_every_kernel_that_may_start_early_waits():
    seen = []
    for f in sorted(os.listdir(CSRC)):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, f)).read())
        if "programmaticStreamSerializationAllowed" not in text:
            continue
        for name, body in _bodies(text).items():
            if re.search(name + r"(<[^<>]*>)?\s*<<<", text):
                continue  # a plain launch: ordered behind everything before it
            seen.append(name)
            assert "pdl_wait()" in body, (f, name)
    assert {"decode_hg_kernel", "decode_hg_f8_kernel", "merge_kernel", "tree_decode_kernel", "tree_join_kernel",
            "cache_copy_kernel", "cache_compact_kernel", "cache_fork_kernel", "cache_resize_kernel"} <= set(seen)


def _tail_decode(fmt, fp8_q):
    """A decode whose last items run as a launch of their own that overlaps the first one's end: 81 tokens of 128 heads."""
    from sparse_mla_decode_smla_gb300.runner import DeviceDecode
    base = W.WORKLOADS[2] if fmt == "fp8_ds" else W.EXTRA_WORKLOADS[1]
    p = W.make_problem(W.small_variant(base, num_requests=81, ctx_lo=600, ctx_hi=900, topk=512))
    assert p.w.num_heads == 128 and p.w.num_tokens == 81 and p.w.kv_format == fmt
    dd = DeviceDecode(p)
    if fp8_q:
        dd.q = W.q_to_e4m3(p.q, W.Q_SCALE_FP8).cuda().contiguous()
        dd.desc.q_format, dd.desc.q_scale = smla.SMLA_Q_FP8_E4M3, W.Q_SCALE_FP8
    plan = smla.plan_launches(dd.desc, torch.cuda.get_device_properties(0).multi_processor_count)
    assert plan.num_launches == 2
    return dd


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,fp8_q", [("fp8_ds", False), ("fp8_tensor", False), ("fp8_tensor", True)])
@pytest.mark.parametrize("captured", [False, True])
def test_page_calls_behind_a_decode_of_two_launches(fmt, fp8_q, captured):
    dd = _tail_decode(fmt, fp8_q)
    dd.run()
    torch.cuda.synchronize()
    want, kv = dd.out.clone(), dd.kv.clone()
    n = want.numel() * 2 // 1152  # the outputs as cache rows: 81 x 128 x 1024 bytes
    both = torch.zeros((2 * n, 1152), dtype=torch.uint8, device="cuda")
    dd.out = both[:n].view(torch.bfloat16).view(want.shape)
    d_out = smla.make_cache_desc(smla.SMLA_KV_BF16, 1, 1, 2 * n, 1, 1)
    slots = kv.shape[0]
    d_kv = smla.make_cache_desc(smla.runner.FMT[fmt], 1, 1, slots, 1, 1)
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    src, dst, err = i32(np.arange(n)), i32(np.arange(n, 2 * n)), i32([0])
    kv_src, kv_dst = i32(np.full(slots - 1, slots - 1)), i32(np.arange(slots - 1))

    def once():
        dd.run()
        smla.cache_copy_pages(d_out, src, dst, both, err)          # reads what the decode wrote
        both[:n].zero_()
        dd.run()
        smla.cache_copy_pages(d_kv, kv_src, kv_dst, dd.kv, err)    # writes over what the decode reads

    def check():
        torch.cuda.synchronize()
        assert torch.equal(both[n:].view(torch.int16), want.view(torch.int16).view(n, 576))
        assert torch.equal(dd.out.view(torch.int16), want.view(torch.int16))
        assert (dd.kv == kv[-1]).all() and err.item() == 0
        both.zero_()
        dd.kv.copy_(kv)

    if not captured:
        for _ in range(10):
            once()
            check()
        return
    once()
    check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        once()
    for _ in range(10):
        g.replay()
        check()
