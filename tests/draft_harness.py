"""Shared set-up of the drafted-token tests: trees, a float64 restatement of the tree
attention over an oracle cache, and its error bound."""

from __future__ import annotations

import numpy as np
import torch

from tests.gpu_harness import D

H16 = 2.0 ** -11   # half a step of fp16, relative
HBF = 2.0 ** -8    # half a step of bf16, relative


def parents(rng, t, width):
    """A random tree: node i hangs on one of the `width` nodes before it (1: a chain)."""
    p = np.full(t, -1, np.int32)
    for i in range(1, t):
        p[i] = max(0, i - 1 - rng.integers(0, width))
    return p


def ancestors(parent, n):
    see = np.zeros((n, n), bool)
    for i in range(n):
        j = i
        while j >= 0:
            see[i, j] = True
            j = parent[j]
    return see


def tree_reference(cache, q, k, v, parent, n):
    """float64 attention of the first n nodes over an OracleCache and their ancestors.
    q [t, Hq, d], k, v [t, Hkv, d] (bf16-exact). Returns (o, bound) [n, Hq, d]: bound is the
    worst case of the kernel's roundings before its bf16 output.

    The roundings (the fp32 sums add about 2^-20 of the same terms, covered by 2^-18): a
    score s = sum_i q~_i k_i, k_i = s c + z, has q~ rounded to fp16 and (with many query
    rows) the products s c as well, so |ds| <= 2^-11 sum |q~_i| (|k_i| + |s c|), and scores
    off by at most D change a softmax average of v by at most (e^(2D) - 1) sum p |v|.
    Probabilities are rounded once, their products with the value scales or the values
    themselves once more, and a sum may be normalised by unrounded ones (3 * 2^-11 of
    sum p |v|); the un-rotation rounds its two operands to fp16 (2 * 2^-11 of
    sum_k |x_k| |R_ck|)."""
    hkv = cache.k.shape[1]
    g = q.shape[1] // hkv
    see = ancestors(parent, n)
    out = np.zeros((n, q.shape[1], D))
    bound = np.zeros_like(out)
    lo, hi = cache.int2_lo, cache.int2_hi
    for h in range(hkv):
        kh, vh = cache.raw_kv(h)
        if hi > lo:   # the INT2 keys as the kernel sees them
            zero = np.repeat(cache.k_zero[:, h].astype(np.float64), cache.group, axis=-1)
            kr = kh[lo:hi] @ cache.r_k[h]
            kr = np.abs(kr) + np.abs(kr - zero)
        vr = vh[lo:hi] @ cache.r_v[h]
        kk = np.concatenate([kh, k[:n, h]])
        vv = np.concatenate([vh, v[:n, h]])
        for m in range(g):
            j = h * g + m
            s = q[:n, j] @ kk.T / np.sqrt(D)
            s[:, len(kh):][~see] = -np.inf
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            out[:, j] = p @ vv
            ds = 0.0
            if hi > lo:
                qr = np.abs(q[:n, j] @ cache.r_k[h])
                ds = (H16 + 2.0 ** -18) * (qr @ kr.T).max(1, keepdims=True) / np.sqrt(D)
            spread = p @ np.abs(vv)
            e = (np.expm1(2 * ds) + 3 * H16 + 2.0 ** -18) * spread
            if hi > lo:
                mass = p[:, lo:hi] @ np.abs(vr)          # also bounds the INT2 value sums
                zero = np.abs(vr).max() * p[:, lo:hi].sum(1, keepdims=True)
                e = e + (2 * H16 * (mass + zero)) @ np.abs(cache.r_v[h]).T
            bound[:, j] = e
    return out, bound


def check_rows(got, want, bound):
    """Elementwise against the bound plus the bf16 output rounding, and in norm against the
    attention tolerance 2e-3 plus that rounding."""
    got = np.asarray(got, np.float64)
    assert np.isfinite(got).all()
    limit = bound + HBF * (np.abs(want) + bound)
    worst = np.abs(got - want) - limit
    assert (worst <= 0).all(), "off by %g over the bound" % worst.max()
    rel = np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-300)
    assert rel <= 2e-3 + HBF, rel


def draft(layer, bsz, t, stream):
    """Drafted q [B, t, Hq, d], k, v [B, t, Hkv, d]: bf16-exact float32 and device bf16 copies."""
    layer.stream_id = 700 + stream
    k, v = layer.draw(bsz * t)
    q = layer.queries(bsz * t, 300 + stream)
    shape = lambda x, h: x.reshape(bsz, t, h, D)  # noqa: E731
    host = (shape(q, layer.hq).numpy(), shape(k, layer.hkv).numpy(), shape(v, layer.hkv).numpy())
    dev = tuple(torch.from_numpy(x).to(torch.bfloat16).cuda().contiguous() for x in host)
    return host, dev


def tree_call(layer, dev, parent, length=None, o=None, workspace=None, stream=None):
    q, k, v = dev
    b, t = q.shape[:2]
    if o is None:
        o = torch.full_like(q, float("nan"))
    if workspace is None:
        workspace = torch.empty(layer.ctx.tree_attn_workspace_bytes(b, t), dtype=torch.uint8, device="cuda")
    layer.ctx.tree_attn(q, k, v, parent, layer.cache.page_table[:b].contiguous(), layer.cache.state[:b], o, b, t,
                        workspace, draft_len=length, stream=stream)
    return o
