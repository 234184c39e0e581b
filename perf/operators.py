"""The operators around a drafted tree over the paged latent cache, as cases that can be run and timed.

Each case is one operator at one size. With `own` false, run() computes it from elementary torch
operations (the plain form); with `own` true it makes the library's calls.

* tree: attention of the drafted nodes of every request over its cached context and over the
  nodes each of them sees (an ancestor mask, or a chain), with the rows of one paged latent cache.
* copy: whole pages copied inside the cache, every layer at once.
* compact: rows that are kept move together, in place, every layer at once.
* fork: the dead beams' rows are emptied, and live requests are forked into them: full pages
  shared, the last partly filled page copied.
* resize: requests grow and shrink; pages come from the free list and go back to it.
"""
import math
import random

import numpy as np
import torch

own = False

ROW_BYTES = {"bf16": 1152, "fp8_ds": 656, "fp8_tensor": 576}
FORMAT = {"bf16": 0, "fp8_ds": 1, "fp8_tensor": 2}
SM_SCALE = float(np.float32(1.0 / math.sqrt(576)))
KV_SCALE = 0.75


def listed():
    return [
        # two users' first drafts on a short prompt, one tensor-parallel shard of 16 heads: latency
        dict(name="tree_bf16_2x8_H16_ctx256", op="tree", requests=2, nodes=8, heads=16, ctx_lo=40, ctx_hi=256, page=64,
             format="bf16", tree=True, sink=False),
        # plain single-token decode of a batch over ragged contexts, dense, per-tensor FP8 cache
        dict(name="token_fp8t_64x1_H64_ctx32k", op="tree", requests=64, nodes=1, heads=64, ctx_lo=1024, ctx_hi=32768,
             page=64, format="fp8_tensor", tree=False, sink=False),
        # a chain of four MTP tokens on four very long documents, 16 heads: few rows, a long axis
        dict(name="chain_bf16_4x4_H16_ctx128k", op="tree", requests=4, nodes=4, heads=16, ctx_lo=100001, ctx_hi=131072,
             page=32, format="bf16", tree=False, sink=True),
        # verification of wide draft trees of a batch, all 128 heads, FP8 block-scaled cache, sink
        dict(name="tree_fp8ds_16x64_H128_ctx16k", op="tree", requests=16, nodes=64, heads=128, ctx_lo=4096, ctx_hi=16384,
             page=64, format="fp8_ds", tree=True, sink=True),
        # four pages of one layer's cache copied before they are written (copy on write)
        dict(name="copy_fp8ds_L1_n4", op="copy", layers=1, count=4, page=64, format="fp8_ds"),
        # a batch of shared prefixes made private in every layer
        dict(name="copy_fp8ds_L32_n256", op="copy", layers=32, count=256, page=64, format="fp8_ds"),
        # the accepted path of every drafted tree becomes context, every layer
        dict(name="compact_accept_64x64_L32", op="compact", requests=64, nodes=64, layers=32, ctx_lo=100, ctx_hi=2000, page=64,
             format="fp8_ds", evict=False),
        # half of the slots of long contexts are evicted
        dict(name="compact_evict_16_ctx16k_L4", op="compact", requests=16, nodes=0, layers=4, ctx_lo=4096, ctx_hi=16384, page=64,
             format="fp8_ds", evict=True),
        # one user's beams: four live ones forked into four dead ones' rows
        dict(name="fork_4x1_ctx300_L1", op="fork", requests=4, children=1, layers=1, ctx_lo=100, ctx_hi=300, page=16, format="bf16"),
        # a batch of prompts, each forked into three samples, every layer
        dict(name="fork_32x3_ctx8k_L8", op="fork", requests=32, children=3, layers=8, ctx_lo=512, ctx_hi=8192, page=64,
             format="fp8_ds"),
        # room for eight drafted tokens per request, given back after the verification
        dict(name="resize_draft_64_ctx8k", op="resize", requests=64, ctx_lo=512, ctx_hi=8192, page=16, grow=8, preempt=False),
        # a quarter of a large batch is preempted and later restored
        dict(name="resize_preempt_512_ctx64k", op="resize", requests=512, ctx_lo=1024, ctx_hi=65536, page=32, grow=0, preempt=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "copy", "compact", "fork", "resize"])
    fmt = rng.choice(["bf16", "fp8_ds", "fp8_tensor"])
    page = rng.choice([1, 4, 16, 32, 64, 64, 128, 256])
    if op == "tree":
        tree = rng.random() < 0.6
        hi = _log(rng, 2, 131072)
        c = dict(op=op, requests=_log(rng, 1, 128), nodes=_log(rng, 1, 64), heads=16 * rng.randint(1, 8), ctx_lo=_log(rng, 1, hi),
                 ctx_hi=hi, page=page, format=fmt, tree=tree, sink=rng.random() < 0.5)
        while work(c)["flops"] > 2.0e12 or c["requests"] * c["ctx_hi"] > 2.2e6 or \
                c["requests"] * c["nodes"] * c["heads"] * c["ctx_hi"] > 2.2e9:
            if c["ctx_hi"] >= 64 * c["requests"]:
                c["ctx_hi"] = c["ctx_hi"] * 2 // 3
                c["ctx_lo"] = min(c["ctx_lo"], c["ctx_hi"])
            else:
                c["requests"] = max(1, c["requests"] * 2 // 3)
        return c
    if op == "copy":
        c = dict(op=op, layers=_log(rng, 1, 61), count=_log(rng, 1, 2000), page=page, format=fmt)
        while c["layers"] * c["count"] * page * ROW_BYTES[fmt] > 340e6:
            c["count"] = max(1, c["count"] * 2 // 3)
            c["layers"] = max(1, c["layers"] * 9 // 10)
        return c
    if op == "compact":
        evict = rng.random() < 0.4
        hi = _log(rng, 2, 16384)
        c = dict(op=op, requests=_log(rng, 1, 128), nodes=0 if evict else rng.randint(2, 64), layers=_log(rng, 1, 48),
                 ctx_lo=_log(rng, 1, hi), ctx_hi=hi, page=page, format=fmt, evict=evict)
        while c["requests"] * c["layers"] * (c["ctx_hi"] + c["nodes"] + page) * ROW_BYTES[fmt] > 600e6:
            c["requests"] = max(1, c["requests"] * 2 // 3)
            c["layers"] = max(1, c["layers"] * 9 // 10)
        return c
    if op == "fork":
        hi = _log(rng, 2, 8192)
        c = dict(op=op, requests=_log(rng, 1, 64), children=rng.randint(1, 7), layers=_log(rng, 1, 48), ctx_lo=_log(rng, 1, hi),
                 ctx_hi=hi, page=page, format=fmt)
        while c["requests"] * c["layers"] * (c["ctx_hi"] + 8 * page) * ROW_BYTES[fmt] > 600e6:
            c["requests"] = max(1, c["requests"] * 2 // 3)
            c["layers"] = max(1, c["layers"] * 9 // 10)
        return c
    hi = _log(rng, 2, 65536)
    c = dict(op=op, requests=_log(rng, 1, 512), ctx_lo=_log(rng, 1, hi), ctx_hi=hi, page=max(4, page), grow=rng.randint(1, 64),
             preempt=rng.random() < 0.5)
    while c["requests"] * (c["ctx_hi"] // c["page"] + 1) > 1.1e6:
        c["requests"] = max(1, c["requests"] * 2 // 3)
    return c


def _lens(case):
    """The contexts' lengths, and the requests' node counts: ragged, the same for every seed."""
    r = random.Random("%s %s %s" % (case["requests"], case["ctx_lo"], case["ctx_hi"]))
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["requests"])]
    n = case.get("nodes", 0)
    nodes = [r.randint(max(1, n // 2), n) if n else 0 for _ in range(case["requests"])]
    return ctx, nodes


def work(case):
    op = case["op"]
    if op == "copy":
        return {"bytes": 2 * case["layers"] * case["count"] * case["page"] * ROW_BYTES[case["format"]], "flops": 0}
    ctx, nodes = _lens(case)
    if op == "tree":
        rows, h = sum(nodes), case["heads"]
        seen = sum(n * c + (n * (n + 1) // 2 if not case["tree"] else n * n) for n, c in zip(nodes, ctx))
        b = sum(n + c for n, c in zip(nodes, ctx)) * ROW_BYTES[case["format"]] + rows * h * (576 * 2 + 512 * 2 + 4)
        return {"bytes": b, "flops": 2 * 1088 * h * seen}
    if op == "compact":
        moved = sum(c // 2 for c in ctx) if case["evict"] else sum(max(1, n // 4) for n in nodes)
        return {"bytes": 2 * moved * case["layers"] * ROW_BYTES[case["format"]] + 4 * moved, "flops": 0}
    if op == "fork":
        rows = sum(c % case["page"] for c in ctx) * case["children"]
        pages = sum(-(-c // case["page"]) for c in ctx) * case["children"]
        return {"bytes": 2 * rows * case["layers"] * ROW_BYTES[case["format"]] + 32 * pages, "flops": 0}
    p, g = case["page"], case["grow"]
    if case["preempt"]:
        pages = sum(-(-c // p) for c in ctx[: max(1, len(ctx) // 4)])
    else:
        pages = sum(-(-(c + g) // p) - -(-c // p) for c in ctx)
    return {"bytes": 2 * (pages * 16 + 8 * len(ctx)), "flops": 0}


def _tables(lens, page, gen, spare, stride):
    """A page table over shuffled physical pages: (table [B, stride], pages used, pool size)."""
    need = [-(-n // page) for n in lens]
    total = sum(need)
    pool = total + spare
    perm = torch.randperm(pool, generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    n = torch.tensor(need, device="cuda")
    k = torch.arange(stride, device="cuda")
    used = k < n[:, None]
    pos = (torch.cumsum(n, 0) - n)[:, None] + k
    table = torch.where(used, perm[pos.clamp(max=pool - 1)], torch.full_like(perm[:1], -1))
    return table.contiguous(), perm, total, pool


def _rows(fmt, n, gen):
    """n cache rows of this format as bytes: latents and RoPE parts of unit size."""
    out = torch.empty((n, ROW_BYTES[fmt]), dtype=torch.uint8, device="cuda")
    step = 1 << 18
    for a in range(0, n, step):
        m = min(step, n - a)
        x = torch.randn((m, 576), generator=gen, device="cuda")
        if fmt == "bf16":
            out[a:a + m] = x.to(torch.bfloat16).view(torch.uint8)
        elif fmt == "fp8_tensor":
            out[a:a + m] = (x / KV_SCALE).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            amax = x[:, :512].reshape(m, 4, 128).abs().amax(-1)
            scale = torch.exp2(torch.ceil(torch.log2(amax / 448)))
            out[a:a + m, :512] = (x[:, :512].reshape(m, 4, 128) / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(m, 512)
            out[a:a + m, 512:528] = scale.view(torch.uint8)
            out[a:a + m, 528:] = x[:, 512:].to(torch.bfloat16).contiguous().view(torch.uint8)
    return out


def _tree_masks(nodes, rng):
    """Ancestor masks of random trees: a node hangs below one of the nodes before it or below the context."""
    words = -(-max(nodes) // 32)
    rows = []
    for n in nodes:
        seen = []
        for i in range(n):
            p = rng.randint(max(-1, i - 9), i - 1)
            seen.append((seen[p] if p >= 0 else 0) | (1 << i))
        rows += [[(m >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for m in seen]
    a = np.array(rows, dtype=np.uint32).view(np.int32).reshape(-1, words)
    return torch.from_numpy(a).cuda(), words


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rng = random.Random(int(seed))
    op, dev = case["op"], "cuda"
    s = {"case": dict(case)}
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    if op == "copy":
        L, n, P, R = case["layers"], case["count"], case["page"], ROW_BYTES[case["format"]]
        pool = 2 * n + 3
        s["kv"] = torch.randint(0, 256, (L, pool, P, R), generator=gen, device=dev, dtype=torch.uint8)
        perm = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
        s["src"], s["dst"], s["pool"] = perm[:n].contiguous(), perm[n:2 * n].contiguous(), pool
        s["err"] = torch.zeros(1, dtype=torch.int32, device=dev)
        return s
    ctx, nodes = _lens(case)
    B, P = case["requests"], case["page"]
    if op == "tree":
        lens = [c + n for c, n in zip(ctx, nodes)]
        s["stride"] = -(-max(lens) // P)
        s["table"], _, _, s["pool"] = _tables(lens, P, gen, 2, s["stride"])
        s["kv"] = _rows(case["format"], s["pool"] * P, gen)
        T, H = sum(nodes), case["heads"]
        q = torch.randn((T, H, 576), generator=gen, device=dev)
        s["q"] = (q * torch.linspace(0.5, 4.0, H, device=dev)[None, :, None]).to(torch.bfloat16)
        s["ctx"], s["cu"] = i32(ctx), i32([0] + list(np.cumsum(nodes)))
        s["mask"], s["words"] = _tree_masks(nodes, rng) if case["tree"] else (None, 0)
        s["sink"] = torch.randn((H,), generator=gen, device=dev) if case["sink"] else None
        s["out"] = torch.empty((T, H, 512), dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty((T, H), dtype=torch.float32, device=dev)
        s["max_nodes"], s["max_len"] = max(nodes), max(lens)
        return s
    s["err"] = torch.zeros(1, dtype=torch.int32, device=dev)
    if op == "compact":
        L, R = case["layers"], ROW_BYTES[case["format"]]
        if case["evict"]:
            lens, starts = ctx, [0] * B
            keep = [sorted(rng.sample(range(c), c - c // 2)) for c in ctx]
        else:
            lens, starts = [c + n for c, n in zip(ctx, nodes)], ctx
            keep = [sorted(rng.sample(range(n), max(1, n // 4))) for n in nodes]
        s["stride"] = -(-max(lens) // P)
        s["table"], _, _, s["pool"] = _tables(lens, P, gen, 1, s["stride"])
        s["kv"] = torch.randint(0, 256, (L, s["pool"], P, R), generator=gen, device=dev, dtype=torch.uint8)
        s["starts"], s["keep"] = i32(starts), i32([x for k in keep for x in k])
        s["cu"] = i32([0] + list(np.cumsum([len(k) for k in keep])))
        s["lens"] = torch.zeros(B, dtype=torch.int32, device=dev)
        return s
    if op == "fork":
        C, L, R = case["children"], case["layers"], ROW_BYTES[case["format"]]
        s["stride"] = -(-max(ctx) // P)
        spare = B * C + 5
        parents, perm, used, s["pool"] = _tables(ctx, P, gen, spare, s["stride"])
        s["table"] = torch.cat([parents, torch.full((B * C, s["stride"]), -1, dtype=torch.int32, device=dev)]).contiguous()
        s["kv"] = torch.randint(0, 256, (L, s["pool"], P, R), generator=gen, device=dev, dtype=torch.uint8)
        s["lens"] = i32(ctx + [0] * (B * C))
        order = list(range(B, B + B * C))
        rng.shuffle(order)
        s["dst_ids"], s["src_ids"] = i32(order), i32([i % B for i in range(B * C)])
        s["zeros"] = torch.zeros(B * C, dtype=torch.int32, device=dev)
        s["pages"] = torch.empty(B * C, dtype=torch.int32, device=dev)
        s["work"] = torch.empty(2 * B * C, dtype=torch.int32, device=dev)
    else:
        g = case["grow"]
        s["stride"] = -(-(max(ctx) + g) // P)
        spare = 0 if case["preempt"] else sum(-(-(c + g) // P) - -(-c // P) for c in ctx)
        s["table"], perm, used, s["pool"] = _tables(ctx, P, gen, spare + 7, s["stride"])
        s["lens"] = i32(ctx)
        ids = list(range(B))
        rng.shuffle(ids)
        if case["preempt"]:  # the first quarter of the requests, in a drawn order
            ids = [i for i in ids if i < max(1, B // 4)]
            first, then = [0] * len(ids), [ctx[i] for i in ids]
        else:
            first, then = [ctx[i] + g for i in ids], [ctx[i] for i in ids]
        s["ids"], s["first"], s["then"] = i32(ids), i32(first), i32(then)
        s["work"] = torch.empty(2 * len(ids), dtype=torch.int32, device=dev)
    s["refs"] = torch.zeros(s["pool"], dtype=torch.int32, device=dev)
    s["refs"][perm[:used].long()] = 1
    s["free"] = torch.full((s["pool"],), -1, dtype=torch.int32, device=dev)
    s["free"][: s["pool"] - used] = perm[used:]
    s["nfree"] = i32([s["pool"] - used])
    return s


# ---------------------------------------------------------------- plain forms


def _keys(kv, slots, fmt):
    r = kv[slots.reshape(-1)]
    if fmt == "bf16":
        k = r.view(torch.bfloat16).float()
    elif fmt == "fp8_tensor":
        k = r.view(torch.float8_e4m3fn).float() * KV_SCALE
    else:
        lat = r[:, :512].contiguous().view(torch.float8_e4m3fn).float().reshape(-1, 4, 128)
        sc = r[:, 512:528].contiguous().view(torch.float32)
        k = torch.cat([(lat * sc[..., None]).reshape(-1, 512), r[:, 528:].contiguous().view(torch.bfloat16).float()], 1)
    return k.reshape(*slots.shape, 576)


def _visible(s):
    """[B, max_nodes, max_len] whether a node of a request sees a slot, and the nodes' rows of q."""
    ctx, cu, N, Lm = s["ctx"].long(), s["cu"].long(), s["max_nodes"], s["max_len"]
    n = cu[1:] - cu[:-1]
    node = torch.arange(N, device="cuda")
    slot = torch.arange(Lm, device="cuda")
    tok = (cu[:-1, None] + node).clamp(max=s["q"].shape[0] - 1)
    j = slot[None, :] - ctx[:, None]  # the node of a slot
    if s["mask"] is None:
        see = j[:, None, :] <= node[None, :, None]
    else:
        bits = s["mask"][tok]  # [B, N, W]
        word = (j.clamp(0, 32 * s["words"] - 1) // 32)[:, None, :].expand(-1, N, -1)
        see = ((torch.gather(bits, 2, word) >> (j.clamp(min=0) % 32)[:, None, :]) & 1).bool() | (j < 0)[:, None, :]
    see = see & (j < n[:, None])[:, None, :]
    return see, tok, (node < n[:, None]), slot


def _tree_plain(s):
    c = s["case"]
    P, H, N = c["page"], c["heads"], s["max_nodes"]
    see, tok, real, slot = _visible(s)
    page = s["table"].long()[:, slot // P].clamp(min=0)
    k = _keys(s["kv"], page * P + slot % P, c["format"])  # [B, L, 576]
    B, Lm = k.shape[:2]
    q = s["q"][tok].float().reshape(B, N * H, 576)
    x = torch.matmul(q, k.transpose(1, 2)).mul_(SM_SCALE).reshape(B, N, H, Lm)
    x.masked_fill_(~see[:, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    if s["sink"] is not None:
        m = torch.maximum(m, s["sink"][None, None, :, None])
    x.sub_(m).exp_()
    den = x.sum(-1)
    if s["sink"] is not None:
        den = den + torch.exp(s["sink"] - m[..., 0])
    o = torch.matmul(x.reshape(B, N * H, Lm), k[..., :512]).reshape(B, N, H, 512) / den.clamp(min=1e-37)[..., None]
    s["out"][tok[real]] = o[real].to(torch.bfloat16)
    s["lse"][tok[real]] = (torch.log(den) + m[..., 0])[real]
    return {"out": s["out"], "lse": s["lse"]}


def _compact_plain(s):
    P, starts, cu, keep = s["case"]["page"], s["starts"].long(), s["cu"].long(), s["keep"].long()
    k = torch.arange(keep.shape[0], device="cuda")
    r = torch.searchsorted(cu, k, right=True) - 1
    src, dst = starts[r] + keep, starts[r] + k - cu[r]
    slot = lambda x: s["table"][r, x // P].long() * P + x % P  # noqa: E731
    flat = s["kv"].view(s["kv"].shape[0], -1, s["kv"].shape[-1])
    flat[:, slot(dst)] = flat[:, slot(src)]
    s["lens"].copy_(s["starts"] + s["cu"][1:] - s["cu"][:-1])
    return {"kv": s["kv"], "lens": s["lens"]}


def _resize_plain(s, ids, new):
    """Pages that no request holds any more go to the end of the free list in ascending order; then the
    requests that grow take pages off its end, in the order of the list."""
    P, stride, dev = s["case"]["page"], s["stride"], "cuda"
    ids, new = ids.long(), new.long()
    old_p, new_p = (s["lens"][ids].long() + P - 1) // P, (new + P - 1) // P
    k = torch.arange(stride, device=dev)
    rows = s["table"][ids].long()
    gone = (k >= new_p[:, None]) & (k < old_p[:, None])
    pool = s["pool"]
    held = torch.cat([s["refs"], s["refs"].new_zeros(1)])
    less = torch.zeros(pool + 1, dtype=torch.int32, device=dev)
    less.index_add_(0, torch.where(gone, rows, pool).reshape(-1), gone.reshape(-1).int())
    now = held - less
    now[pool] = 0
    freed = ((held > 0) & (now == 0))[:pool]
    count = s["nfree"].long()
    at = torch.where(freed, count + torch.cumsum(freed, 0) - 1, pool)
    free = torch.cat([s["free"], s["free"].new_zeros(1)])
    free[at] = torch.arange(pool, device=dev, dtype=torch.int32)
    count = count + freed.sum()
    need = (new_p - old_p).clamp(min=0)
    before = torch.cumsum(need, 0) - need
    taken = (k >= old_p[:, None]) & (k < new_p[:, None])
    pos = torch.where(taken, count - 1 - (before[:, None] + k - old_p[:, None]), pool)
    page = free[pos].long()
    s["table"][ids] = torch.where(taken, page, torch.where(gone, -1, rows)).int()
    now.index_add_(0, torch.where(taken, page, pool).reshape(-1), taken.reshape(-1).int())
    free[pos] = -1
    s["refs"].copy_(now[:pool])
    s["free"].copy_(free[:pool])
    s["nfree"].copy_(count - need.sum())
    s["lens"][ids] = new.int()


def _fork_plain(s, src, dst):
    P, stride, dev = s["case"]["page"], s["stride"], "cuda"
    src, dst = src.long(), dst.long()
    n = s["lens"][src].long()
    full, part = n // P, n % P
    k = torch.arange(stride, device=dev)
    rows = s["table"][src].long()
    shared = k < full[:, None]
    need = (part > 0).long()
    pos = s["nfree"].long() - 1 - (torch.cumsum(need, 0) - need)
    pos = torch.where(need > 0, pos, s["pool"])
    free = torch.cat([s["free"], s["free"].new_zeros(1)])
    page = free[pos].long()
    last = (k == full[:, None]) & (need > 0)[:, None]
    s["table"][dst] = torch.where(shared, rows, torch.where(last, page[:, None], -1)).int()
    s["pages"].copy_(torch.where(need > 0, page, -1))
    refs = torch.cat([s["refs"], s["refs"].new_zeros(1)])
    refs.index_add_(0, torch.where(shared, rows, s["pool"]).reshape(-1), shared.reshape(-1).int())
    refs.index_add_(0, torch.where(need > 0, page, s["pool"]), need.int())
    s["refs"].copy_(refs[:-1])
    free[pos] = -1
    s["free"].copy_(free[:-1])
    s["nfree"].sub_(need.sum().int())
    s["lens"][dst] = n.int()
    old = rows.gather(1, torch.where(need > 0, full, full - 1)[:, None])[:, 0]
    row = torch.arange(P, device=dev)
    into = torch.where(need > 0, page, old)[:, None] * P + row
    move = (row < part[:, None])
    flat = s["kv"].view(s["kv"].shape[0], -1, s["kv"].shape[-1])
    # rows that do not move are copied onto themselves
    flat[:, into.reshape(-1)] = flat[:, torch.where(move, old[:, None] * P + row, into).reshape(-1)]


def _pages(s):
    return {"table": s["table"], "lens": s["lens"], "refs": s["refs"], "free": s["free"], "nfree": s["nfree"]}


def run(s):
    c, op = s["case"], s["case"]["op"]
    if own:
        import sparse_mla_decode_smla_gb300 as smla
        if op == "tree":
            if "desc" not in s:
                s["desc"] = smla.make_tree_desc(s["q"].shape[0], c["heads"], c["requests"], c["page"], s["pool"], s["stride"],
                                                FORMAT[c["format"]], SM_SCALE, mask_words=s["words"], kv_scale=KV_SCALE)
                s["ws"] = torch.zeros(smla.tree_workspace_size(s["desc"]), dtype=torch.uint8, device="cuda")
            smla.tree_decode(s["desc"], s["q"], s["kv"], s["table"], s["ctx"], s["cu"], s["mask"], s["sink"], s["out"], s["lse"],
                             s["ws"])
            return {"out": s["out"], "lse": s["lse"]}
        if "desc" not in s:
            kv = s.get("kv")
            s["desc"] = smla.make_cache_desc(FORMAT[c.get("format", "bf16")], kv.shape[0] if kv is not None else 1, c["page"], s["pool"],
                                             s["table"].shape[0] if "table" in s else 1, s.get("stride", 1))
        d = s["desc"]
        if op == "copy":
            smla.cache_copy_pages(d, s["src"], s["dst"], s["kv"], s["err"])
            return {"kv": s["kv"]}
        if op == "compact":
            smla.cache_compact(d, s["table"], s["starts"], s["cu"], s["keep"], s["kv"], s["lens"], s["err"])
            return {"kv": s["kv"], "lens": s["lens"]}
        if op == "fork":
            smla.cache_resize(d, s["table"], s["lens"], s["refs"], s["free"], s["nfree"], s["dst_ids"], s["zeros"], s["work"],
                              s["err"])
            smla.cache_fork(d, s["table"], s["lens"], s["refs"], s["free"], s["nfree"], s["src_ids"], s["dst_ids"],
                            s["pages"], s["kv"], s["err"])
            return {"kv": s["kv"], "pages": s["pages"], **_pages(s)}
        smla.cache_resize(d, s["table"], s["lens"], s["refs"], s["free"], s["nfree"], s["ids"], s["first"], s["work"],
                          s["err"])
        smla.cache_resize(d, s["table"], s["lens"], s["refs"], s["free"], s["nfree"], s["ids"], s["then"], s["work"], s["err"])
        return _pages(s)
    if op == "tree":
        return _tree_plain(s)
    if op == "copy":
        s["kv"][:, s["dst"].long()] = s["kv"][:, s["src"].long()]
        return {"kv": s["kv"]}
    if op == "compact":
        return _compact_plain(s)
    if op == "fork":
        _resize_plain(s, s["dst_ids"], s["zeros"])
        _fork_plain(s, s["src_ids"], s["dst_ids"])
        return {"kv": s["kv"], "pages": s["pages"], **_pages(s)}
    _resize_plain(s, s["ids"], s["first"])
    _resize_plain(s, s["ids"], s["then"])
    return _pages(s)


def exact(case, seed):
    """The attention in 64 bits, a node at a time over its own list of slots (the other operators move whole
    numbers: nothing to compute)."""
    if case["op"] != "tree":
        return None
    if work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    ctx, nodes = _lens(case)
    P, H, fmt = case["page"], case["heads"], case["format"]
    out = torch.zeros((sum(nodes), H, 512), dtype=torch.float64, device="cuda")
    lse = torch.full((sum(nodes), H), -math.inf, dtype=torch.float64, device="cuda")
    t = 0
    for r, (c, n) in enumerate(zip(ctx, nodes)):
        local = torch.arange(c + n, device="cuda")
        raw = s["kv"].reshape(-1, ROW_BYTES[fmt])[s["table"][r].to(torch.int64)[torch.div(local, P, rounding_mode="floor")] * P + local.remainder(P)]
        if fmt == "bf16":
            key = raw.view(torch.bfloat16).double()
        elif fmt == "fp8_tensor":
            key = raw.view(torch.float8_e4m3fn).double() * KV_SCALE
        else:
            key = torch.empty((c + n, 576), dtype=torch.float64, device="cuda")
            scales = raw[:, 512:528].contiguous().view(torch.float32).double()
            for b in range(4):
                key[:, 128 * b:128 * b + 128] = raw[:, 128 * b:128 * b + 128].contiguous().view(torch.float8_e4m3fn).double() * scales[:, b:b + 1]
            key[:, 512:] = raw[:, 528:].contiguous().view(torch.bfloat16).double()
        sees = np.zeros((n, n), dtype=bool)
        if s["mask"] is None:
            sees = np.tril(np.ones((n, n), dtype=bool))
        else:
            w = s["mask"][t:t + n].cpu().numpy().view(np.uint32)
            for i in range(n):
                for j in range(n):
                    sees[i, j] = bool((int(w[i, j // 32]) >> (j % 32)) & 1)
        hidden = torch.zeros((n, c + n), dtype=torch.bool, device="cuda")
        hidden[:, c:] = ~torch.from_numpy(sees).cuda()
        step = max(1, (1 << 28) // (H * (c + n)))
        for a in range(0, n, step):
            e = min(n, a + step)
            z = (s["q"][t + a:t + e].double().reshape(-1, 576) @ key.T).reshape(e - a, H, c + n) * SM_SCALE
            z = z.masked_fill(hidden[a:e, None, :], -math.inf)
            if s["sink"] is not None:
                z = torch.cat([z, s["sink"].double()[None, :, None].expand(e - a, H, 1)], 2)
            lse[t + a:t + e] = torch.logsumexp(z, 2)
            w = torch.exp(z - lse[t + a:t + e, :, None])[..., :c + n]
            out[t + a:t + e] = (w.reshape(-1, c + n) @ key[:, :512]).reshape(e - a, H, 512)
        t += n
    return {"out": out, "lse": lse}
