"""Definitions of the MXFP4 operators and of scored routing in 64 bits, for their tests."""
import numpy as np
import torch

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def quantised(x):
    """(values [rows, K], scale bytes [rows, K/32]) of a matrix, in float64: per 32 elements the scale
    2^(floor(log2 amax) - 2), elements to the nearest E2M1 value, ties to the even code."""
    x = np.asarray(x, np.float64).reshape(x.shape[0], -1, 32)
    amax = np.abs(x).max(-1)
    bad = ~np.isfinite(amax)
    _, e = np.frexp(np.where(bad | (amax == 0), 4.0, amax))  # mantissa in [1/2, 1)
    byte = np.where(bad, 255, np.maximum(e - 3 + 127, 0))
    scale = np.exp2(byte - 127.0)[..., None]
    a = np.abs(np.where(bad[..., None], 0, x)) / scale
    dist = np.abs(a[..., None] - E2M1)
    n = dist.argmin(-1)  # the lower of two as near; the even one of a tie between n and n + 1:
    up = np.minimum(n + 1, 7)
    n = np.where((np.take_along_axis(dist, up[..., None], -1)[..., 0] == dist.min(-1)) & (n % 2 == 1), up, n)
    v = np.copysign(E2M1[n] * scale, x)
    v[np.broadcast_to(bad[..., None], v.shape)] = np.nan
    return v.reshape(x.shape[0], -1), byte.astype(np.uint8)


def values(codes, scales):
    """The values of MXFP4 rows (uint8 tensors, scales in rows), as a float64 tensor."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    v = torch.tensor(np.concatenate([E2M1, -E2M1]), device=codes.device)[n]
    s = torch.exp2(scales.double() - 127)
    s[scales == 255] = float("nan")
    return v * s.repeat_interleave(32, -1)


def tile_index(rows, K):
    """Byte of the scale of (row, block of 32) among tiles, and the size of the tiles."""
    chunks = -(-K // 128)
    r, j = np.meshgrid(np.arange(rows), np.arange(K // 32), indexing="ij")
    at = ((r // 128) * chunks + j // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + j % 4
    return at, -(-rows // 128) * chunks * 512


def random_mx(rows, K, seed=0, lo=118, hi=122):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (rows, K // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(lo, hi, (rows, K // 32), generator=g, dtype=torch.uint8)
    return codes.cuda(), scales.cuda()


def selected(logits, bias, k, score="sigmoid", n_group=1, topk_group=1, group_top=2, renorm=True,
             scale=1.0):
    """(topk_idx, topk_w) by the formulas, float64. A NaN ranks below every number, ties go to the
    lower index; without a bias experts rank by their logits."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            e = np.exp(-np.abs(l))
            s = np.where(l < 0, e, 1.0) / (1.0 + e)
        else:
            e = np.exp(l - np.fmax.reduce(l, axis=1, keepdims=True))
            s = e / e.sum(1, keepdims=True)
        c = s if bias is None else s + np.asarray(bias, np.float64)
        rank = l if bias is None else c


        def sorted_desc(v):  # NaN last, told apart from -inf
            key = np.lexsort((np.arange(v.shape[-1]) + 0 * v, np.where(np.isnan(v), 0, -v), np.isnan(v)),
                             axis=-1)
            return key

        if n_group > 1 and topk_group < n_group:
            per = E // n_group
            by = c if group_top == 2 else (rank if bias is None else c)
            by = by.reshape(T, n_group, per)
            top = np.take_along_axis(by, sorted_desc(by)[..., :group_top], -1).sum(-1)
            keep = sorted_desc(top)[:, :topk_group]
            mask = np.zeros((T, n_group), bool)
            np.put_along_axis(mask, keep, True, -1)
            mask = np.repeat(mask, per, -1)
        else:
            mask = np.ones((T, E), bool)
        idx = np.empty((T, k), np.int64)
        for t in range(T):
            e_in = np.flatnonzero(mask[t])
            idx[t] = e_in[sorted_desc(rank[t, e_in])[:k]]
        at = np.take_along_axis(s, idx, 1)
        if renorm:
            if score == "softmax":
                li = np.take_along_axis(l, idx, 1)
                at = np.exp(li - np.fmax.reduce(li, axis=1, keepdims=True))
            tot = at.sum(1, keepdims=True)
            at = np.where(tot == 0, 0.0, at / tot)
    return idx, at * scale
