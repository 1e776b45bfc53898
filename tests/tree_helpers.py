"""64-bit references for the draft-tree operators (rope-append, tree attention,
acceptance), on torch tensors of any device; nothing here calls the library."""
import math

import numpy as np
import torch

import oracle

D = 128


def rotation(seed, device="cpu"):
    """R = H diag(s) / sqrt(128) in 64 bits."""
    i = np.arange(D)
    pop = np.array([[bin(a & b).count("1") for b in i] for a in i])
    H = 1.0 - 2.0 * (pop % 2)
    return torch.from_numpy(H * oracle.signs(seed)[None].astype(np.float64) / math.sqrt(D)).to(device)


def dequantised(blocks):
    """[..., 66] uint8 -> [..., 128] float64 in the rotated domain."""
    scale = blocks[..., :2].contiguous().view(torch.float16).double()
    idx = torch.stack((blocks[..., 2:] & 15, blocks[..., 2:] >> 4), -1).flatten(-2)
    return scale * (2.0 * idx.double() - 15.0) / 15.0


def tokens_of(cache, b, g, n, table=None):
    """Blocks [n][66] of sequence b, KV head g."""
    if table is None:
        return cache[b, g, :n]
    size = cache.shape[2]
    pages = table[b, : (n + size - 1) // size].long().to(cache.device)
    return cache[pages, g].reshape(-1, cache.shape[3])[:n]


def tree_attention(q, kc, vc, ctx, n_nodes, mask, scale, seed, table=None):
    """(out [B][T][Hq][128], eps [B][T][Hq], amp [B][T][Hq][1]) in 64 bits.
    eps: the largest change of a visible logit when every rotated query channel
    is off by its relative half step of fp16, 2^-11; amp: the softmax-weighted
    mean of |v| over the visible tokens, per rotated channel's largest."""
    B, T, Hq, _ = q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    R = rotation(seed, q.device)
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    eps = torch.zeros(q.shape[:3], dtype=torch.float64, device=q.device)
    amp = torch.zeros((*q.shape[:3], 1), dtype=torch.float64, device=q.device)
    for b in range(B):
        c, n = int(ctx[b]), int(n_nodes[b])
        if n == 0:
            continue
        m = mask if mask.dim() == 1 else mask[b]
        see = torch.ones((n, c + n), dtype=torch.bool, device=q.device)
        see[:, c:] = (m[:n, None] >> torch.arange(n, device=q.device)) & 1 == 1
        for g in range(Hkv):
            k = dequantised(tokens_of(kc, b, g, c + n, table))
            v = dequantised(tokens_of(vc, b, g, c + n, table))
            for h in range(g * G, (g + 1) * G):
                qr = q[b, :n, h].double() @ R.T
                s = (qr @ k.nan_to_num(0.0).T * scale).masked_fill(~see, -math.inf)
                top = s.amax(-1, keepdim=True).clamp(min=-1e300)
                p = (s - top).exp()
                p = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
                out[b, :n, h] = p @ v.nan_to_num(0.0) @ R
                e = (qr.abs() @ k.nan_to_num(0.0).abs().T * abs(scale)).masked_fill(~see, 0.0)
                eps[b, :n, h] = e.amax(-1) * 2.0 ** -11
                # a change of the rotated output by x changes each output channel
                # by at most sum_d |x_d| / sqrt(128)
                amp[b, :n, h, 0] = (p @ v.nan_to_num(0.0).abs()).sum(-1) / math.sqrt(D)
    return out, eps, amp


def check_tree(got, want, eps, amp):
    """Per element, and in the 2-norm.

    bf16 outputs: each softmax weight is off by its fp16 rounding (2^-11) and by
    what the fp16 rounding of the query does to its logit (a factor within
    e^(+-eps)), numerator and denominator alike; fp32 sums and exponentials add
    some 2^-18.  With x = e^eps (1 + 2^-11) - 1 + 2^-18 the output moves by at
    most 2 x amp, and is then rounded to bf16 (half a step: 2^-8 relative).
    fp16 outputs: queries and weights go in as pairs of fp16 terms (2^-21 and
    eps 2^-10), so x = e^(eps 2^-10) (1 + 2^-21) - 1 + 2^-18, and the rounding
    is 2^-11 relative (2^-25 absolute among the subnormals).
    2-norm: the rounding alone is within that half step; the rest may take as
    much again."""
    half = torch.finfo(got.dtype).eps / 2
    fp16 = got.dtype == torch.float16
    x = torch.expm1(eps * (2.0 ** -10 if fp16 else 1.0))[..., None]
    x = x * (1 + 2.0 ** -11) + (2.0 ** -21 if fp16 else 2.0 ** -11) + 2.0 ** -18
    bound = 2 * x * amp + half * (want.abs() + 2 * x * amp) + 2.0 ** -25
    err = (got.double() - want).abs()
    over = err - bound
    at = int(over.argmax())
    assert bool((over <= 0).all()), (
        f"element {at}: {float(got.flatten()[at])} for {float(want.flatten()[at])}, "
        f"off {float(err.flatten()[at]):.3e}, bound {float(bound.flatten()[at]):.3e}")
    rel = float((got.double() - want).norm() / want.norm().clamp(min=1e-300))
    print(f"tree rel-L2 {rel:.2e} ({got.dtype}), worst share of its bound "
          f"{float((err / bound.clamp(min=1e-300)).max()):.2f}")
    assert rel <= 2 * half or float(want.norm()) == 0.0, rel


def rope(x, positions, inv_freq, interleaved):
    """x [n][H][128] float32 (numpy) rotated as the library defines it: cos and
    sin in 64 bits rounded to binary32, then single binary32 operations."""
    x = np.array(x, np.float32)
    h = len(inv_freq)
    theta = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(theta).astype(np.float32)[:, None], np.sin(theta).astype(np.float32)[:, None]
    a, b = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    x1, x2 = x[..., a].copy(), x[..., b].copy()
    x[..., a] = x1 * c - x2 * s
    x[..., b] = x2 * c + x1 * s
    return x


def encoded(rows, seed):
    """[n][H][128] float32 -> the oracle's blocks [n][H][66]."""
    n, H, _ = rows.shape
    cap = (n + 7) // 8 * 8
    cache = np.zeros((1, H, cap, 66), np.uint8)
    oracle.quantize_append(np.ascontiguousarray(rows)[None], np.zeros(1, np.int32), cap, seed, cache)
    return cache[0, :, :n].transpose(1, 0, 2)


def random_tree(rng, T, kind="random"):
    """Parents of T nodes in an order in which a parent precedes its children."""
    if kind == "chain":
        return np.arange(T) - 1
    if kind == "star":
        return np.full(T, -1)
    return np.array([-1 if i == 0 or rng.random() < 0.1 else rng.integers(max(0, i - 6), i) for i in range(T)])
