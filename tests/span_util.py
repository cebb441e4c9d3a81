"""64-bit forms of the span operators and of the cache reader, and device copies of their inputs."""
from __future__ import annotations

import numpy as np
import torch

from sparse_mla_decode_fp8_b200 import workloads as W
from tests import independent

SPAN, PAGE = 64, 256


def dev(a: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def dev_bf16(bits: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


def paged(seq_lens, seed: int, extra_pages: int = 2, outliers: float = 0.05, garbage: bool = True):
    """(cache, block_table) of requests of these lengths: latents N(0, 1), some rows 20 times larger,
    in pages drawn without replacement; every other byte of the pool is 0xFF (e4m3 NaN, bf16 NaN,
    scale NaN), so that whatever reads a token it should not shows it."""
    rng = np.random.default_rng(seed)
    need = [max(1, -(-max(int(n), 0) // PAGE)) for n in seq_lens]
    pages = sum(need) + extra_pages
    perm = rng.permutation(pages).astype(np.int32)
    table = np.full((len(need), max(need)), -1, np.int32)
    cache = np.full((pages, W.PAGE_BYTES), 0xFF if garbage else 0, np.uint8)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
        n = max(int(seq_lens[b]), 0)
        if n:
            lat = rng.standard_normal((n, 512), dtype=np.float32)
            lat[rng.random(n) < outliers] *= 20.0
            t = np.arange(n)
            W.write_tokens(cache, table[b, t // PAGE].astype(np.int64), t % PAGE, lat)
    return cache, table


def latents(cache, table, b, pos) -> np.ndarray:
    """fp64 latents of positions of request b."""
    pos = np.asarray(pos, np.int64)
    return independent.token_latents(cache, table[b, pos // PAGE], pos % PAGE)


def span_mean(cache, table, seq_lens, b, j) -> np.ndarray:
    pos = np.arange(j * SPAN, min((j + 1) * SPAN, int(seq_lens[b])))
    return latents(cache, table, b, pos).mean(axis=0)


def scores(q, keys, table, seq_lens, sm_scale, num_pages=None) -> np.ndarray:
    """fp64 [B, 4 max_blocks]: q [B, 64, 512] and keys [pages, 4, 512] as fp64 values."""
    B, blocks = table.shape
    pages = keys.shape[0] if num_pages is None else num_pages
    out = np.zeros((B, 4 * blocks))
    for b in range(B):
        j = np.arange(min(-(-max(int(seq_lens[b]), 0) // SPAN), 4 * blocks))
        page = table[b, j // 4]
        j, page = j[(page >= 0) & (page < pages)], page[(page >= 0) & (page < pages)]
        if not len(j):
            continue
        x = sm_scale * (q[b] @ keys[page, j % 4].T)
        p = np.exp(x - x.max(axis=1, keepdims=True))
        out[b, j] = (p / p.sum(axis=1, keepdims=True)).sum(axis=0)
    return out


def select(score_rows, seq_lens, nsel, first, last):
    """(spans [B, nsel], tokens [B, 64 nsel]) by sorting."""
    B, width = score_rows.shape
    spans = np.full((B, nsel), -1, np.int64)
    idx = np.full((B, nsel * SPAN), -1, np.int64)
    for b in range(B):
        n = min(width, -(-max(int(seq_lens[b]), 0) // SPAN))
        s = np.where(np.isnan(score_rows[b, :n]), -np.inf, score_rows[b, :n]).astype(np.float64)
        kept = (np.arange(n) < first) | (np.arange(n) >= n - last)
        order = sorted(range(n), key=lambda j: (not kept[j], -s[j], j))
        chosen = np.sort(np.array(order[:nsel], np.int64))
        spans[b, :len(chosen)] = chosen
        for i, j in enumerate(chosen):
            t = np.arange(j * SPAN, (j + 1) * SPAN)
            idx[b, i * SPAN:(i + 1) * SPAN] = np.where(t < seq_lens[b], t, -1)
    return spans, idx


def attention(q, cache, table, b, pos, sm_scale):
    """fp64 attention of q [64, 512] over the listed positions of request b (with multiplicity):
    (out, lse, weighted mean of |k|, largest sum |q k| sm_scale over the tokens)."""
    if not len(pos):
        z = np.zeros((64, 512))
        return z, np.full(64, -np.inf), z, 0.0
    k = latents(cache, table, b, pos)
    s = sm_scale * (q @ k.T)
    m = s.max(axis=1, keepdims=True)
    p = np.exp(s - m)
    total = p.sum(axis=1, keepdims=True)
    size = abs(sm_scale) * float((np.abs(q) @ np.abs(k).T).max())
    return p @ k / total, (m + np.log(total))[:, 0], p @ np.abs(k) / total, size


def check_decode(out, lse, q, cache, table, positions, sm_scale):
    """decode_spans' results against attention() over positions[b], with the bounds its arithmetic gives.

    Scores: 512 exact bf16 products added in fp32, each addition off by at most 2^-23 of the largest
    partial sum (the tensor core may truncate): |ds| <= 512 2^-23 size.  A weight's relative error is then
    at most e = |ds| (of the token and of the reference m, which cancels in O and LSE up to rounding)
    + 2^-21 (exp2 and the product with log2 e).  Weights enter P V as bf16, half a step 2^-8 each; the
    sum over n tokens adds n 2^-23 of sum p |k|; the output is rounded once, 2^-8 of |O|."""
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, pos in enumerate(positions):
        o, l, mean_abs, size = attention(q[b], cache, table, b, pos, sm_scale)
        if not len(pos):
            assert not out[b].any() and np.isneginf(lse[b]).all(), b
            continue
        n = len(pos)
        e = 512 * 2.0 ** -23 * size + 2.0 ** -21
        off = np.abs(out[b] - o)
        bound = mean_abs * (2.0 ** -8 * (1 + 2 * e) + 2 * e + (n + 16) * 2.0 ** -23) + 2.0 ** -8 * (np.abs(o) + off)
        assert (off <= bound).all(), (b, float((off - bound).max()))
        assert (np.abs(lse[b] - l) <= e + (n + 16) * 2.0 ** -24 + 2.0 ** -21 * (1 + np.abs(l))).all(), b
