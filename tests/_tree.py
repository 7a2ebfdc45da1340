"""Plain fp64 form of tree attention, and the tolerances that follow from the kernels' roundings."""
from __future__ import annotations

import math
import random

import torch


def random_tree(rng: random.Random, n: int, shape: str) -> list[int]:
    if shape == "chain":
        return [i - 1 for i in range(n)]
    if shape == "roots":
        return [-1] * n
    return [-1 if i == 0 or rng.random() < 0.1 else rng.randrange(i) for i in range(n)]


def lines_of(parents) -> list[list[int]]:
    """For each node, itself and then its ancestors up to the root."""
    lines = []
    for i, p in enumerate(parents):
        lines.append([i] if p < 0 else [i] + lines[p])
    return lines


def tree_reference(q, kd, vd, k, v, lens, parents, counts, policy, scale=None, kept=None):
    """(out, lse, mean of |v| under the softmax weights), all fp64, rows behind counts[b] zero.

    q [B, T, Hq, d]; kd, vd [B, T, Hkv, d]; k, v dense [B, Hkv, Lmax, d]; policy[b * Hkv + h] =
    (kind, sink, window); kept[(b, h)]: cached positions a retrieval head sees beyond the local rule."""
    B, T, Hq, D = q.shape
    Hkv = kd.shape[2]
    g = Hq // Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    dev = q.device
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device=dev)
    lse = torch.zeros(B, T, Hq, dtype=torch.float64, device=dev)
    mag = torch.zeros(B, T, Hq, D, dtype=torch.float64, device=dev)
    for b in range(B):
        n, L = counts[b], lens[b]
        if n == 0:
            continue
        lines = lines_of(parents[b][:n])
        pos = torch.tensor([L + len(x) - 1 for x in lines], device=dev)
        anc = torch.zeros(n, n, dtype=torch.bool)
        for i, x in enumerate(lines):
            anc[i, x] = True
        j = torch.cat([torch.arange(L, device=dev), pos])  # positions of the cache, then of the nodes
        known = torch.cat([torch.ones(n, L, dtype=torch.bool, device=dev), anc.to(dev)], 1)
        for h in range(Hkv):
            kind, s, w = policy[b * Hkv + h][:3]
            see = known
            if kind in ("local", "retrieval"):
                rule = (j < s)[None] | (j[None] > (pos - w)[:, None])
                if kind == "retrieval":
                    rule[:, :L] |= kept[(b, h)].to(dev)[None, :L]
                see = known & rule
            kk = torch.cat([k[b, h, :L].double(), kd[b, :n, h].double()])
            vv = torch.cat([v[b, h, :L].double(), vd[b, :n, h].double()])
            sc = torch.einsum("tgd,jd->tgj", q[b, :n, h * g:(h + 1) * g].double(), kk) * scale
            sc = sc.masked_fill(~see[:, None], -math.inf)
            p = torch.softmax(sc, -1)
            out[b, :n, h * g:(h + 1) * g] = p @ vv
            mag[b, :n, h * g:(h + 1) * g] = p @ vv.abs()
            lse[b, :n, h * g:(h + 1) * g] = torch.logsumexp(sc, -1)
    return out, lse, mag


def assert_tree_close(out, lse, ref, pages: str):
    """Element by element, against the bound of the roundings the kernels make.

    P is rounded to the operand type of P V (bf16: 2^-8 relative, f16 next to E4M3 pages: 2^-11, fp32
    pages: not at all), the result to the output's type (bf16: 2^-8).  Scores are fp32 sums of d products:
    an error of at most d 2^-23 sum|q k| scale, for normal q and k below 1.2e-4 (tensor cores, d = 128) and
    6.1e-5 (fp32 FMA, half an ulp a step); it enters the weights once above and once below the fraction
    line; the exponential adds at most 7.8e-5 twice and the row sums 2^-24 a term: below 6e-4, and
    1.5e-4 for fp32 pages, of the weighted mean of |v| in all."""
    o_ref, l_ref, mag = ref
    p_round = {"bf16": 2.0 ** -8, "e4m3": 2.0 ** -11, "f32": 0.0}[pages]
    o_round = 2.0 ** -24 if pages == "f32" else 2.0 ** -8
    slack = 1.5e-4 if pages == "f32" else 6e-4
    err = (out.double() - o_ref).abs()
    bound = p_round * mag * 1.01 + o_round * (o_ref.abs() + p_round * mag) + slack * mag
    worst = (err - bound).max().item()
    assert worst <= 0, (worst, err.max().item())
    l_err = (lse.double() - l_ref).abs().max().item()
    assert l_err <= (7e-5 if pages == "f32" else 3e-4), l_err
