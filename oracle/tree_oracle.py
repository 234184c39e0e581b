"""Float64 oracle of tree attention: a node of a request attends the request's context slots and
the nodes it sees. Scores, softmax, sink and values are smla_oracle.attend's; this module adds
the list of slots a node sees and the error bounds of a 16-bit tensor-core evaluation."""
from __future__ import annotations

import numpy as np

from . import smla_oracle as O


def node_sees(i: int, j: int, mask_row) -> bool:
    """Whether node i sees node j: bit j of its mask row (32-bit words), or j <= i without a mask."""
    if mask_row is None:
        return j <= i
    return bool((int(mask_row[j // 32]) >> (j % 32)) & 1)


def slots_seen(ctx: int, n: int, i: int, mask_row) -> list:
    """Request-local slots node i of n sees behind a context of ctx slots, ascending."""
    return list(range(ctx)) + [ctx + j for j in range(n) if node_sees(i, j, mask_row)]


def tree_decode(q_bits, rows_of, kv_format: str, page_table, ctx, cu, mask, page_size: int, num_pages: int,
                sm_scale: float, sink=None, kv_scale=None):
    """q_bits [T, H, 576] bf16 patterns; rows_of(physical slots) -> cache rows [n, R]; mask [T, W]
    uint32 or None. Returns dict(out, lse, terms) with NaN rows for the rows of no node; terms
    holds what error_bounds needs, per token and head."""
    T, H, _ = q_bits.shape
    out, lse = np.full((T, H, O.LATENT), np.nan), np.full((T, H), np.nan)
    terms = dict(A=np.zeros((T, H, O.LATENT)), qk=np.zeros((T, H)), small=np.zeros((T, H)), n=np.zeros((T, H)),
                 vmax=np.zeros((T, H)), smax=np.zeros((T, H)))
    for r in range(len(ctx)):
        n = int(cu[r + 1]) - int(cu[r])
        for i in range(n):
            t = int(cu[r]) + i
            phys = []
            for s in slots_seen(int(ctx[r]), n, i, None if mask is None else mask[t]):
                page = int(page_table[r, s // page_size])
                if 0 <= page < num_pages:
                    phys.append(page * page_size + s % page_size)
            keys = (O.dequant_rows(rows_of(np.asarray(phys, dtype=np.int64)), kv_format, kv_scale) if phys
                    else np.zeros((0, O.DIM)))
            q = O.bf16_bits_to_f64(q_bits[t])
            out[t], lse[t], _ = O.attend(q, keys, sm_scale, sink)
            if not phys:
                continue
            s = float(sm_scale) * (q @ keys.T)
            with np.errstate(invalid="ignore"):
                w = np.exp(s - lse[t][:, None])
                terms["A"][t] = w @ np.abs(keys[:, :O.LATENT])
                terms["qk"][t] = abs(sm_scale) * (np.abs(q) @ np.abs(keys).T).max(1)
                terms["small"][t] = abs(sm_scale) * np.abs(q).max(1) * np.abs(keys).sum(1).max()
                terms["smax"][t] = np.abs(s).max(1)
            terms["n"][t] = len(phys)
            terms["vmax"][t] = np.abs(keys[:, :O.LATENT]).max()
    return dict(out=out, lse=lse, terms=terms)


def error_bounds(ref, f16: bool):
    """(out, lse) bounds on the distance of a tensor-core evaluation from `ref`.

    Scores: 36 accumulations of 16 exact products, each within 2^-23 of the absolute sum, a second
    rounding for the stacked halves' sum, and q's f16 conversion (2^-25 of the row's largest; none
    in bf16): ds. Exponent: its fp32 argument (2^-23 of the largest |s| log2 e, twice) and the
    exponential (2^-21). Probabilities: half a step of f16 (2^-11) or bf16 (2^-8), and 2^-25 / 2^6
    of the largest for those below f16's normal range. Sums over n slots, in any order: n - 1
    additions within 2^-24 each, and a few rescales. Output: half a step of bf16, 2^-8 relative."""
    t = ref["terms"]
    ds = (36 + 2) * 2.0 ** -23 * 2 * t["qk"] + (2.0 ** -24 * t["small"] if f16 else 0.0)
    ex = 2.0 ** -21 + 4 * 2.0 ** -23 * 1.4427 * t["smax"]
    sums = (t["n"] + 8) * 2.0 ** -24
    p = 2.0 ** -11 if f16 else 2.0 ** -8
    rel = 2 * (ds + ex) + sums + p
    out = 2.0 ** -8 * np.abs(ref["out"]) + rel[..., None] * t["A"] * 1.01
    if f16:
        out = out + (t["n"] * 2.0 ** -31 * t["vmax"])[..., None]
    out = out + 1e-30
    lse = ds + ex + sums + 2.0 ** -22 * np.abs(np.where(np.isfinite(ref["lse"]), ref["lse"], 0.0)) + 1e-6
    return out, lse
