"""The operators around a prompt, as cases that can be run and timed.

Each case is one operator at one size. With `own` false, run() computes it from elementary torch
operations (the plain form); with `own` true it makes the library's calls.

* attention: attention of packed prompts (a document mask) over per-head keys and values, with the RoPE
  part of the keys shared by all heads; causal over a longer context, with a visible prefix, scores
  capped by a tanh, a bias by distance, a sink; and its form for single tokens.
* read: rows of the paged latent cache read back as bf16, the context that a prompt's chunk needs.
* norm: the residual's addition, the root-mean-square norm, and its output in bf16 and in E4M3 with scales.
* logprobs: log probabilities of given tokens, the entropy, and the most likely alternatives.
"""
import math
import random

import numpy as np
import torch

own = False

ROW_BYTES = {"bf16": 1152, "fp8_ds": 656, "fp8_tensor": 576}
FORMAT = {"bf16": 0, "fp8_ds": 1, "fp8_tensor": 2}
KV_SCALE = 0.75


def listed():
    return [
        # one user's short first prompt, one tensor-parallel shard of 16 heads: latency
        dict(name="attn_1x24_H16", op="attention", requests=1, q_lo=24, q_hi=24, past_lo=0, past_hi=0, heads=16, kv_heads=16, rope=64,
             causal=True, prefix=False, cap=0.0, bias=False, sink=False),
        # a batch of ragged documents packed behind one another
        dict(name="attn_docs_13_H32", op="attention", requests=13, q_lo=1, q_hi=1700, past_lo=0, past_hi=0, heads=32, kv_heads=32, rope=64,
             causal=True, prefix=False, cap=0.0, bias=False, sink=True),
        # chunks of two long prompts over what was read before, scores capped
        dict(name="attn_chunk_2x1024_past12k_H16_cap", op="attention", requests=2, q_lo=900, q_hi=1024, past_lo=6000, past_hi=12000,
             heads=16, kv_heads=16, rope=64, causal=True, prefix=False, cap=30.0, bias=False, sink=False),
        # one long prompt
        dict(name="attn_1x8191_H32", op="attention", requests=1, q_lo=8191, q_hi=8191, past_lo=0, past_hi=0, heads=32, kv_heads=32,
             rope=64, causal=True, prefix=False, cap=0.0, bias=False, sink=False),
        # prompts with an instruction that every token sees, a bias by distance, grouped heads without a RoPE part
        dict(name="attn_prefix_4x2k_H32x8_bias", op="attention", requests=4, q_lo=800, q_hi=2100, past_lo=0, past_hi=0, heads=32,
             kv_heads=8, rope=0, causal=True, prefix=True, cap=0.0, bias=True, sink=False),
        # single tokens of a batch over ragged contexts, grouped heads, scores capped
        dict(name="attn_token_32x1_past16k_H64x8_cap", op="attention", requests=32, q_lo=1, q_hi=1, past_lo=700, past_hi=16000, heads=64,
             kv_heads=8, rope=0, causal=True, prefix=False, cap=50.0, bias=False, sink=False),
        # the short context of three chats
        dict(name="read_fp8ds_3_ctx200", op="read", requests=3, ctx_lo=20, ctx_hi=200, page=64, format="fp8_ds"),
        # the contexts of a batch of long prompts
        dict(name="read_fp8ds_24_ctx32k", op="read", requests=24, ctx_lo=4096, ctx_hi=32768, page=64, format="fp8_ds"),
        # a decode step of a small batch: hidden states with the residual, E4M3 in blocks of 128
        dict(name="norm_7_D7168_block", op="norm", rows=7, dim=7168, residual=True, group=128, pow2=True, y=True),
        # a long prompt's hidden states, one scale a token
        dict(name="norm_16384_D7168_row", op="norm", rows=16384, dim=7168, residual=True, group=0, pow2=False, y=True),
        # a small batch's sampled tokens
        dict(name="logprobs_5_V32003_f32", op="logprobs", rows=5, vocab=32003, given=1, top=5, dtype="f32"),
        # the tokens of scored prompts, bf16 logits full of ties
        dict(name="logprobs_1024_V129280_bf16", op="logprobs", rows=1024, vocab=129280, given=1, top=20, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "read", "norm", "logprobs"])
    if op == "attention":
        rope = rng.choice([64, 64, 0])
        kv = rng.choice([1, 2, 4, 5, 8, 16, 16, 32])
        heads = kv * (1 if rope and rng.random() < 0.7 else rng.choice([1, 2, 3, 4, 8]))
        token = rng.random() < 0.3
        hi = 1 if token else _log(rng, 2, 8192)
        past = _log(rng, 16, 65536) if token else rng.choice([0, 0, _log(rng, 1, 16384)])
        c = dict(op=op, requests=_log(rng, 1, 96), q_lo=_log(rng, 1, hi), q_hi=hi, past_lo=past // rng.randint(1, 8), past_hi=past,
                 heads=heads, kv_heads=kv, rope=rope, causal=rng.random() < 0.85, prefix=rng.random() < 0.25,
                 cap=rng.choice([0.0, 0.0, 30.0, 50.0]), bias=rng.random() < 0.25, sink=rng.random() < 0.25)
        while c["requests"] * c["q_hi"] * (c["q_hi"] + c["past_hi"]) * heads > 2.1e9 or \
                c["requests"] * (c["q_hi"] + c["past_hi"]) * (kv * 256 + 64) > 1.1e9:
            if c["requests"] > 1:
                c["requests"] = c["requests"] * 2 // 3
            else:
                c["q_hi"] = max(1, c["q_hi"] * 2 // 3)
                c["q_lo"] = min(c["q_lo"], c["q_hi"])
                c["past_hi"] = c["past_hi"] * 2 // 3
                c["past_lo"] = min(c["past_lo"], c["past_hi"])
        return c
    if op == "read":
        hi = _log(rng, 2, 65536)
        c = dict(op=op, requests=_log(rng, 1, 128), ctx_lo=_log(rng, 1, hi), ctx_hi=hi, page=rng.choice([1, 4, 16, 32, 64, 64, 128, 256]),
                 format=rng.choice(["bf16", "fp8_ds", "fp8_ds", "fp8_tensor"]))
        while c["requests"] * c["ctx_hi"] > 450000:
            c["requests"] = max(1, c["requests"] * 2 // 3)
        return c
    if op == "norm":
        dim = 8 * _log(rng, 8, 2048)
        return dict(op=op, rows=max(1, min(_log(rng, 1, 32768), 16384 * 7168 // dim)), dim=dim, residual=rng.random() < 0.7,
                    group=rng.choice([128, 128, 0]), pow2=rng.random() < 0.6, y=rng.random() < 0.5)
    v = _log(rng, 500, 200000)
    return dict(op=op, rows=max(1, min(_log(rng, 1, 4096), 1024 * 129280 // v)), vocab=v, given=rng.choice([1, 1, 2, 7]),
                top=rng.choice([0, 1, 5, 20, 20, 33]), dtype=rng.choice(["f32", "bf16"]))


def _lens(case):
    """The requests' queries and keys: ragged, the same for every seed."""
    r = random.Random("%s %s %s" % (case["requests"], case.get("q_hi"), case.get("ctx_hi", case.get("past_hi"))))
    if case["op"] == "read":
        return [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["requests"])]
    nq = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["requests"])]
    nk = [n + r.randint(case["past_lo"], case["past_hi"]) for n in nq]
    pre = [r.randint(0, n) if case["prefix"] else 0 for n in nk]
    return nq, nk, pre


def work(case):
    op = case["op"]
    if op == "read":
        return {"bytes": sum(_lens(case)) * (ROW_BYTES[case["format"]] + 1152), "flops": 0}
    if op == "norm":
        n, d = case["rows"], case["dim"]
        one = 2 + (4 if case["residual"] else 0) + (2 if case["y"] else 0) + 1
        return {"bytes": n * d * one + 4 * n * (-(-d // 128) if case["group"] else 1), "flops": 0}
    if op == "logprobs":
        return {"bytes": case["rows"] * (case["vocab"] * (4 if case["dtype"] == "f32" else 2) + 8 * case["given"] + 8 * case["top"] + 4),
                "flops": 0}
    nq, nk, pre = _lens(case)
    pairs = 0
    for a, b, p in zip(nq, nk, pre):
        if case["causal"]:
            i = np.arange(a, dtype=np.int64) + b - a + 1
            pairs += int(np.maximum(i, p).sum())
        else:
            pairs += a * b
    d, h, hk = 128 + case["rope"], case["heads"], case["kv_heads"]
    return {"bytes": sum(nq) * h * (2 * d + 256 + 4) + sum(nk) * (hk * 512 + 2 * case["rope"]), "flops": 2 * (d + 128) * h * pairs}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dev, op = "cuda", case["op"]
    s = {"case": dict(case)}
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    bf = lambda *n: torch.randn(n, generator=gen, device=dev, dtype=torch.float32).to(torch.bfloat16)  # noqa: E731
    if op == "attention":
        nq, nk, pre = _lens(case)
        T, N, H, HK, rope = sum(nq), sum(nk), case["heads"], case["kv_heads"], case["rope"]
        q = torch.randn((T, H, 128 + rope), generator=gen, device=dev)
        s["q"] = (q * torch.linspace(0.5, 3.0, H, device=dev)[None, :, None]).to(torch.bfloat16)
        # keys and values as one up-projection of the latents writes them
        s["kv"] = bf(N, HK, 256)
        s["k"], s["v"] = s["kv"][..., :128], s["kv"][..., 128:]
        s["rope"] = bf(N, rope) if rope else None
        s["cu_q"], s["cu_k"] = i32([0] + list(np.cumsum(nq))), i32([0] + list(np.cumsum(nk)))
        s["pre"] = i32(pre) if case["prefix"] else None
        s["slopes"] = torch.exp2(-8.0 * (torch.arange(H, device=dev, dtype=torch.float32) + 1) / H) if case["bias"] else None
        s["sink"] = torch.randn((H,), generator=gen, device=dev) if case["sink"] else None
        s["out"] = torch.empty((T, H, 128), dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty((T, H), dtype=torch.float32, device=dev)
        s["max_q"], s["max_k"], s["scale"] = max(nq), max(nk), float(np.float32((128 + rope) ** -0.5))
        return s
    if op == "read":
        ctx, P, fmt = _lens(case), case["page"], case["format"]
        need = [-(-c // P) for c in ctx]
        s["stride"], s["pool"] = max(need), sum(need) + 2
        perm = torch.randperm(s["pool"], generator=gen, device=dev).to(torch.int32)
        n = torch.tensor(need, device=dev)
        k = torch.arange(s["stride"], device=dev)
        pos = (torch.cumsum(n, 0) - n)[:, None] + k
        s["table"] = torch.where(k < n[:, None], perm[pos.clamp(max=s["pool"] - 1)], torch.full_like(perm[:1], -1)).contiguous()
        rows = s["pool"] * P
        s["kv"] = torch.empty((rows, ROW_BYTES[fmt]), dtype=torch.uint8, device=dev)
        for a in range(0, rows, 1 << 18):
            m = min(1 << 18, rows - a)
            x = torch.randn((m, 576), generator=gen, device=dev)
            if fmt == "bf16":
                s["kv"][a:a + m] = x.to(torch.bfloat16).view(torch.uint8)
            elif fmt == "fp8_tensor":
                s["kv"][a:a + m] = (x / KV_SCALE).to(torch.float8_e4m3fn).view(torch.uint8)
            else:
                b = x[:, :512].reshape(m, 4, 128)
                sc = b.abs().amax(-1) / 448
                s["kv"][a:a + m, :512] = (b / sc[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(m, 512)
                s["kv"][a:a + m, 512:528] = sc.view(torch.uint8)
                s["kv"][a:a + m, 528:] = x[:, 512:].to(torch.bfloat16).contiguous().view(torch.uint8)
        s["starts"], s["cu"] = i32([0] * len(ctx)), i32([0] + list(np.cumsum(ctx)))
        s["latent"] = torch.empty((sum(ctx), 512), dtype=torch.bfloat16, device=dev)
        s["rope"] = torch.empty((sum(ctx), 64), dtype=torch.bfloat16, device=dev)
        s["err"] = torch.zeros(1, dtype=torch.int32, device=dev)
        return s
    if op == "norm":
        n, d = case["rows"], case["dim"]
        x = torch.randn((n, d), generator=gen, device=dev)
        big = torch.rand((d,), generator=gen, device=dev) < 0.01  # a few channels are far larger than the others
        s["x"] = (x * torch.where(big, 30.0, 1.0)).to(torch.bfloat16)
        s["res"] = (torch.randn((n, d), generator=gen, device=dev) * 3).to(torch.bfloat16) if case["residual"] else None
        s["w"] = (1 + 0.2 * torch.randn((d,), generator=gen, device=dev)).to(torch.bfloat16)
        s["sum"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["y"] = torch.empty_like(s["x"]) if case["y"] else None
        s["codes"] = torch.empty((n, d), dtype=torch.uint8, device=dev)
        s["scales"] = torch.empty((n, -(-d // 128) if case["group"] else 1), dtype=torch.float32, device=dev)
        return s
    n, v, g, k = case["rows"], case["vocab"], case["given"], case["top"]
    x = torch.empty((n, v), dtype=torch.float32 if case["dtype"] == "f32" else torch.bfloat16, device=dev)
    x.normal_(0.0, 3.0, generator=gen)
    s["x"] = x
    s["tokens"] = torch.randint(0, v, (n, g), generator=gen, device=dev, dtype=torch.int32)
    s["lp"] = torch.empty((n, g), device=dev)
    s["ent"] = torch.empty((n,), device=dev)
    s["ids"] = torch.empty((n, k), dtype=torch.int32, device=dev)
    s["alt"] = torch.empty((n, k), device=dev)
    s["err"] = torch.zeros(1, dtype=torch.int32, device=dev)
    return s


# ---------------------------------------------------------------- plain forms


def _attention_plain(s):
    c = s["case"]
    H, HK, N, L = c["heads"], c["kv_heads"], s["max_q"], s["max_k"]
    g = H // HK
    cq, ck = s["cu_q"].long(), s["cu_k"].long()
    nq, nk = cq[1:] - cq[:-1], ck[1:] - ck[:-1]
    i, j = torch.arange(N, device="cuda"), torch.arange(L, device="cuda")
    rows = (cq[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    keys = (ck[:-1, None] + j).clamp(max=s["k"].shape[0] - 1)
    B, real = rows.shape[0], i < nq[:, None]
    pos = nk[:, None] - nq[:, None] + i
    if c["causal"]:
        lim = torch.minimum(pos + 1, nk[:, None])
        if s["pre"] is not None:
            lim = torch.maximum(lim, torch.minimum(s["pre"].long(), nk)[:, None])
    else:
        lim = nk[:, None].expand(-1, N)
    hide = j >= lim[..., None]  # [B, N, L]
    q = s["q"][rows].float().reshape(B, N, HK, g, -1).permute(0, 2, 3, 1, 4).reshape(B, HK, g * N, -1)
    k = s["k"][keys].float().permute(0, 2, 3, 1)  # [B, HK, 128, L]
    x = torch.matmul(q[..., :128], k)
    if s["rope"] is not None:
        x += torch.matmul(q[..., 128:].reshape(B, HK * g * N, -1), s["rope"][keys].float().transpose(1, 2)).reshape(x.shape)
    x = x.mul_(s["scale"]).reshape(B, HK, g, N, L)
    if c["cap"]:
        x.div_(c["cap"]).tanh_().mul_(c["cap"])
    if s["slopes"] is not None:
        x -= s["slopes"].reshape(HK, g, 1, 1) * (pos[..., None] - j).abs().float()[:, None, None]
    x.masked_fill_(hide[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    if s["sink"] is not None:
        m = torch.maximum(m, s["sink"].reshape(HK, g, 1, 1))
    x.sub_(m).exp_()
    den = x.sum(-1)
    if s["sink"] is not None:
        den = den + torch.exp(s["sink"].reshape(HK, g, 1) - m[..., 0])
    o = torch.matmul(x.reshape(B, HK, g * N, L), s["v"][keys].float().permute(0, 2, 1, 3)).reshape(B, HK, g, N, 128)
    o = o / den.clamp(min=1e-37)[..., None]
    s["out"][rows[real]] = o.permute(0, 3, 1, 2, 4).reshape(B, N, H, 128)[real].to(torch.bfloat16)
    s["lse"][rows[real]] = (torch.log(den) + m[..., 0]).permute(0, 3, 1, 2).reshape(B, N, H)[real]
    return {"out": s["out"], "lse": s["lse"]}


def _read_plain(s):
    c = s["case"]
    P, cu = c["page"], s["cu"].long()
    k = torch.arange(s["latent"].shape[0], device="cuda")
    r = torch.searchsorted(cu, k, right=True) - 1
    slot = s["starts"].long()[r] + k - cu[r]
    raw = s["kv"][s["table"].long()[r, slot // P] * P + slot % P]
    if c["format"] == "bf16":
        x = raw.view(torch.bfloat16)
        lat, rope = x[:, :512], x[:, 512:]
    elif c["format"] == "fp8_tensor":
        x = raw.view(torch.float8_e4m3fn).float() * KV_SCALE
        lat, rope = x[:, :512], x[:, 512:]
    else:
        lat = raw[:, :512].contiguous().view(torch.float8_e4m3fn).float().reshape(-1, 4, 128)
        lat = (lat * raw[:, 512:528].contiguous().view(torch.float32)[..., None]).reshape(-1, 512)
        rope = raw[:, 528:].contiguous().view(torch.bfloat16)
    s["latent"].copy_(lat)
    s["rope"].copy_(rope)
    return {"latent": s["latent"], "rope": s["rope"]}


def _norm_plain(s):
    c = s["case"]
    n, d = s["x"].shape
    h = s["x"].float()
    out = {}
    if s["res"] is not None:
        h = h + s["res"].float()
        s["sum"].copy_(h)
        out["sum"] = s["sum"]
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * s["w"].float()
    if s["y"] is not None:
        s["y"].copy_(y)
        out["y"] = s["y"]
    G = 128 if c["group"] else d
    b = torch.nn.functional.pad(y, (0, -d % G)).reshape(n, -1, G)
    amax = b.abs().amax(-1)
    scale = amax / 448
    if c["pow2"]:
        frac, e = torch.frexp(scale)
        scale = torch.ldexp(torch.ones_like(scale), e - (frac == 0.5).int())
    scale = torch.where(amax == 0, torch.ones_like(scale), scale)
    code = (b / scale[..., None]).clamp(-448, 448).reshape(n, -1)[:, :d].to(torch.float8_e4m3fn)
    s["codes"].copy_(code.view(torch.uint8))
    s["scales"].copy_(scale)
    out["codes"], out["scales"] = s["codes"].view(torch.float8_e4m3fn), s["scales"]
    return out


def _logprobs_plain(s):
    x = s["x"].float() + 0.0
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    log_z = torch.log(z)
    s["lp"].copy_(torch.gather(x, 1, s["tokens"].long()) - m - log_z)
    s["ent"].copy_((log_z - torch.where(e > 0, e * (x - m), e).sum(-1, keepdim=True) / z)[:, 0])
    k = s["case"]["top"]
    if k:
        val, idx = torch.sort(x, dim=-1, descending=True, stable=True)
        s["ids"].copy_(idx[:, :k])
        s["alt"].copy_(val[:, :k] - m - log_z)
    return {"logprobs": s["lp"], "entropy": s["ent"], "ids": s["ids"], "alternatives": s["alt"]}


def run(s):
    c, op = s["case"], s["case"]["op"]
    if own:
        import sparse_mla_decode_smla_gb300 as smla
        if op == "attention":
            if "desc" not in s:
                s["desc"] = smla.make_prompt_desc(s["q"].shape[0], s["k"].shape[0], c["heads"], c["kv_heads"], c["requests"], c["rope"],
                                                  s["scale"], causal=c["causal"], softcap=c["cap"], q_strides=s["q"].stride()[:2],
                                                  k_strides=s["k"].stride()[:2], v_strides=s["v"].stride()[:2])
                s["ws"] = torch.zeros(smla.prompt_workspace_size(s["desc"]), dtype=torch.uint8, device="cuda")
            smla.prompt_attention(s["desc"], s["q"], s["k"], s["v"], s["rope"], s["cu_q"], s["cu_k"], s["pre"], s["slopes"], s["sink"],
                                  s["out"], s["lse"], s["ws"])
            return {"out": s["out"], "lse": s["lse"]}
        if op == "read":
            if "desc" not in s:
                s["desc"] = smla.make_read_desc(FORMAT[c["format"]], c["page"], s["pool"], c["requests"], s["stride"],
                                                s["latent"].shape[0], kv_scale=KV_SCALE)
            smla.cache_read(s["desc"], s["kv"], s["table"], s["starts"], s["cu"], s["latent"], s["rope"], s["err"])
            return {"latent": s["latent"], "rope": s["rope"]}
        if op == "norm":
            smla.add_rmsnorm(s["x"], s["res"], s["w"], 1e-6, residual_out=s["sum"], y=s["y"], codes=s["codes"], scales=s["scales"],
                             group=c["group"], scale_mode=smla.SMLA_SCALE_POW2 if c["pow2"] else smla.SMLA_SCALE_FP32)
            out = {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"]}
            if s["y"] is not None:
                out = {"y": s["y"], **out}
            return {"sum": s["sum"], **out} if s["sum"] is not None else out
        smla.token_logprobs(s["x"], s["tokens"], s["lp"], entropy=s["ent"], top_ids=s["ids"], top_logprobs=s["alt"], error_word=s["err"])
        return {"logprobs": s["lp"], "entropy": s["ent"], "ids": s["ids"], "alternatives": s["alt"]}
    if op == "attention":
        return _attention_plain(s)
    if op == "read":
        return _read_plain(s)
    if op == "norm":
        return _norm_plain(s)
    return _logprobs_plain(s)


# ---------------------------------------------------------------- 64 bits


def _attention_exact(case, s):
    nq, nk, pre = _lens(case)
    H, HK = case["heads"], case["kv_heads"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    t0 = k0 = 0
    for a, b, p in zip(nq, nk, pre):
        where = torch.arange(b - a, b, device="cuda", dtype=torch.float64)
        key_at = torch.arange(b, device="cuda", dtype=torch.float64)
        step = max(1, (1 << 27) // max(1, b))
        for h in range(H):
            key = s["k"][k0:k0 + b, h // (H // HK)].double()
            if case["rope"]:
                key = torch.cat([key, s["rope"][k0:k0 + b].double()], 1)
            val = s["v"][k0:k0 + b, h // (H // HK)].double()
            for u in range(0, a, step):
                e = min(a, u + step)
                z = (s["q"][t0 + u:t0 + e, h].double() @ key.T) * s["scale"]
                if case["cap"]:
                    z = case["cap"] * torch.tanh(z / case["cap"])
                far = where[u:e, None] - key_at[None, :]
                if case["bias"]:
                    z = z - float(s["slopes"][h]) * far.abs()
                if case["causal"]:
                    z = z.masked_fill((far < 0) & (key_at >= p)[None, :], -math.inf)
                if case["sink"]:
                    z = torch.cat([z, s["sink"][h].double().expand(e - u, 1)], 1)
                total = torch.logsumexp(z, 1)
                lse[t0 + u:t0 + e, h] = total
                out[t0 + u:t0 + e, h] = torch.exp(z[:, :b] - total[:, None]) @ val
        t0, k0 = t0 + a, k0 + b
    return {"out": out, "lse": lse}


def _read_exact(case, s):
    P, fmt, parts = case["page"], case["format"], []
    for r, c in enumerate(_lens(case)):
        local = torch.arange(c, device="cuda")
        parts.append(s["kv"][s["table"][r].to(torch.int64)[torch.div(local, P, rounding_mode="floor")] * P + local.remainder(P)])
    raw = torch.cat(parts)
    if fmt == "bf16":
        x = raw.view(torch.bfloat16).double()
    elif fmt == "fp8_tensor":
        x = raw.view(torch.float8_e4m3fn).double() * KV_SCALE
    else:
        x = torch.empty((raw.shape[0], 576), dtype=torch.float64, device="cuda")
        sc = raw[:, 512:528].contiguous().view(torch.float32).double()
        for b in range(4):
            x[:, 128 * b:128 * b + 128] = raw[:, 128 * b:128 * b + 128].contiguous().view(torch.float8_e4m3fn).double() * sc[:, b:b + 1]
        x[:, 512:] = raw[:, 528:].contiguous().view(torch.bfloat16).double()
    return {"latent": x[:, :512].contiguous(), "rope": x[:, 512:].contiguous()}


def _norm_exact(case, s):
    n, d = s["x"].shape
    h = s["x"].double()
    out = {}
    if case["residual"]:
        h = h + s["res"].double()
        out["sum"] = h
    y = h / torch.sqrt(h.square().sum(1, keepdim=True) / d + 1e-6) * s["w"].double()
    if case["y"]:
        out["y"] = y
    group = 128 if case["group"] else d
    at = torch.arange(d, device="cuda") // group
    amax = torch.zeros((n, -(-d // group)), dtype=torch.float64, device="cuda").scatter_reduce_(1, at.expand(n, -1), y.abs(), "amax")
    scale = amax / 448
    if case["pow2"]:
        scale = torch.exp2(torch.ceil(torch.log2(scale)))
    scale = torch.where(amax > 0, scale, torch.ones_like(scale))
    # the codes are the nearest E4M3 values of this
    out["codes"], out["scales"] = y / scale[:, at], scale
    return out


def _logprobs_exact(case, s):
    n, k, t = case["rows"], case["top"], s["tokens"].to(torch.int64)
    lp = torch.empty(s["lp"].shape, dtype=torch.float64, device="cuda")
    ent = torch.empty((n,), dtype=torch.float64, device="cuda")
    ids = torch.empty((n, k), dtype=torch.int32, device="cuda")
    alt = torch.empty((n, k), dtype=torch.float64, device="cuda")
    for a in range(0, n, 64):
        x = s["x"][a:a + 64].double()
        full = x - torch.logsumexp(x, 1, keepdim=True)
        lp[a:a + 64] = torch.gather(full, 1, t[a:a + 64])
        ent[a:a + 64] = -(torch.exp(full) * full).sum(1)
        order = torch.argsort(-x, dim=1, stable=True)[:, :k]
        ids[a:a + 64] = order.to(torch.int32)
        alt[a:a + 64] = torch.gather(full, 1, order)
    return {"logprobs": lp, "entropy": ent, "ids": ids, "alternatives": alt}


def exact(case, seed):
    if case["op"] == "attention" and work(case)["flops"] > 3e12:
        return None
    s = prepare(case, seed)
    return {"attention": _attention_exact, "read": _read_exact, "norm": _norm_exact, "logprobs": _logprobs_exact}[case["op"]](case, s)
