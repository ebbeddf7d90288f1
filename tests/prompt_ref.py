"""Batches of new tokens over a cache, and the append and causal-attention rules in
64 bits, for the tests of tri_append and tri_prefill_attention.

A cache is held here as flat rows [records, d]; ``rec[r]`` lists the record of every
slot of row r (layer, sequence, KV head), -1 where its table names no block."""
from __future__ import annotations

import math

import numpy as np
import torch

import kv_cache_compression_calib_b200 as tri

DTYPE = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}


def bytes_of(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


class Batch:
    """new[s] tokens of sequence s behind old[s] cached slots.  ``row_len`` (one length
    per row) replaces new + old.  Records outside the rows hold ``junk``."""

    def __init__(self, new, old, L=1, hq=4, h=2, d=128, elem="bf16", layout="paged", bs=16, pad=0, il=False, theta=1e4,
                 seed=0, dev="cpu", row_len=None, extra_blocks=3, junk=float("nan"), amp=1.0, v_mean=0.0):
        g = torch.Generator().manual_seed(seed)
        S = len(new)
        self.new, self.S, self.L, self.hq, self.h, self.d, self.elem, self.bs, self.dev = new, S, L, hq, h, d, elem, bs, dev
        self.layout, self.il, self.theta = layout, il, theta
        self.m = tri.model(L, hq, h, theta, d, tri.TRI_ROPE_INTERLEAVED if il else tri.TRI_ROPE_HALF)
        self.T = sum(new) + pad
        self.tok = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        lens = row_len if row_len is not None else [new[s] + old[s] for _ in range(L) for s in range(S) for _ in range(h)]
        self.row_off_np = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        self.total = int(self.row_off_np[-1])
        if layout == "paged":
            need = [max((int(lens[(l * S + s) * h + x]) + bs - 1) // bs for l in range(L) for x in range(h)) for s in range(S)]
            self.nb = sum(need) + extra_blocks
            perm = torch.randperm(self.nb, generator=g).int().numpy()
            self.table_np = np.full((S, max(max(need), 1)), -1, np.int32)
            at = 0
            for s, n in enumerate(need):
                self.table_np[s, :n] = perm[at:at + n]
                at += n
            self.shape = (L, self.nb, bs, h, d)
        else:
            self.shape = (self.total + 5, d)  # records behind the last row
        self.amp = amp
        n = int(np.prod(self.shape[:-1]))
        K, V = (amp * torch.randn(n, d, generator=g) for _ in range(2))
        V = V / amp + v_mean
        used = np.zeros(n, bool)
        for r in range(len(lens)):
            rec = self.rec(r)
            used[rec[rec >= 0]] = True
        free = torch.as_tensor(~used)
        K[free], V[free] = junk, junk
        self.K, self.V = (x.to(DTYPE[elem]).view(self.shape).to(dev) for x in (K, V))
        self.pos = torch.full(self.shape[:-1], -7, dtype=torch.int32, device=dev)
        self.q = (amp * torch.randn(L, self.T, hq, d, generator=g)).to(torch.bfloat16).to(dev)
        self.row_off = torch.as_tensor(self.row_off_np).to(dev)
        self.tok_off = torch.as_tensor(self.tok).to(dev)
        self.g = g

    def rec(self, r):
        """Records of row r's slots."""
        n = int(self.row_off_np[r + 1] - self.row_off_np[r])
        if self.layout == "contig":
            return np.arange(self.row_off_np[r], self.row_off_np[r + 1])
        l, s, x = r // (self.S * self.h), (r // self.h) % self.S, r % self.h
        j = np.arange(n)
        bi = np.minimum(j // self.bs, self.table_np.shape[1] - 1)
        blk = np.where(j // self.bs < self.table_np.shape[1], self.table_np[s, bi], -1).astype(np.int64)
        ok = (blk >= 0) & (blk < self.nb)
        return np.where(ok, ((l * self.nb + blk) * self.bs + j % self.bs) * self.h + x, -1)

    def kv(self):
        e = tri.elem_type_of(self.K)
        if self.layout == "contig":
            return tri.kv_contig(self.S, self.row_off, self.total, e)
        return tri.kv_paged(self.S, self.row_off, self.total, torch.as_tensor(self.table_np).to(self.dev), self.bs, self.nb, e)

    def rows64(self, t):
        return t.double().view(-1, self.d)


def attend64(b, scale):
    """(out, lse, mag) fp64 [L][T][Hq][d], [L][T][Hq]: mag = sum_j w_j |v_j| of the softmax
    weights w, the scale of the result's error.  Rows behind the last token are NaN."""
    G = b.hq // b.h
    out = torch.full((b.L, b.T, b.hq, b.d), math.nan, dtype=torch.float64, device=b.dev)
    mag, lse = out.clone(), out[..., 0].clone()
    K, V = b.rows64(b.K), b.rows64(b.V)
    for l in range(b.L):
        for s, n in enumerate(b.new):
            for x in range(b.h):
                rec = torch.as_tensor(b.rec((l * b.S + s) * b.h + x)).to(b.dev)
                N = len(rec)
                for i in range(n):
                    seen = rec[:max(0, N - n + i + 1)]
                    seen = seen[seen >= 0]
                    t, hs = int(b.tok[s]) + i, slice(x * G, (x + 1) * G)
                    if len(seen) == 0:
                        out[l, t, hs], mag[l, t, hs], lse[l, t, hs] = 0, 0, -math.inf
                        continue
                    k, v = K[seen], V[seen]
                    sc = scale * (b.q[l, t, hs].double() @ k.T)
                    w = torch.softmax(sc, -1)
                    out[l, t, hs], mag[l, t, hs] = w @ v, w @ v.abs()
                    lse[l, t, hs] = torch.logsumexp(sc, -1)
    return out, lse, mag


def attend64_rows(b, scale):
    """attend64 with a row's tokens at once, for larger batches."""
    G = b.hq // b.h
    out = torch.full((b.L, b.T, b.hq, b.d), math.nan, dtype=torch.float64, device=b.dev)
    mag, lse = out.clone(), out[..., 0].clone()
    K, V = b.K.view(-1, b.d), b.V.view(-1, b.d)
    rows = lambda t, r: bytes_of(t)[r].view(t.dtype).double()  # noqa: E731
    for l in range(b.L):
        for s, n in enumerate(b.new):
            if n == 0:
                continue
            t = slice(int(b.tok[s]), int(b.tok[s]) + n)
            for x in range(b.h):
                rec = torch.as_tensor(b.rec((l * b.S + s) * b.h + x)).to(b.dev)
                N, hs = len(rec), slice(x * G, (x + 1) * G)
                q = b.q[l, t, hs].double()
                seen = torch.arange(N, device=b.dev) <= (N - n + torch.arange(n, device=b.dev))[:, None]
                seen = (seen & (rec >= 0))[:, None]
                k, v = rows(K, rec.clamp(min=0)), rows(V, rec.clamp(min=0))
                sc = torch.where(seen, scale * torch.einsum("igd,jd->igj", q, k), -math.inf)
                lse[l, t, hs] = torch.logsumexp(sc, -1)
                w = torch.exp(sc - lse[l, t, hs][..., None].clamp(min=-1e300))
                v = torch.where(seen.any(0).any(0)[:, None], v, 0.0)
                out[l, t, hs] = torch.einsum("igj,jd->igd", w, v)
                mag[l, t, hs] = torch.einsum("igj,jd->igd", w, v.abs())
    return out, lse, mag


def score_error(b, scale):
    """Bound of a score's fp32 error: d products summed in fp32, 4 d 2^-24 of scale |q| . |k|
    (at most scale * ||q|| ||k||, the largest of the batch)."""
    qn = b.q.double().norm(dim=-1).max().item()
    K = b.rows64(b.K)
    kn = 0.0
    for r in range(b.L * b.S * b.h):
        rec = b.rec(r)
        rec = torch.as_tensor(rec[rec >= 0]).to(b.dev)
        if len(rec):
            kn = max(kn, K[rec].norm(dim=-1).nan_to_num(0.0).max().item())
    return 4 * b.d * 2.0 ** -24 * scale * qn * kn


def turned64(x, pos, theta, il):
    """Pairs of x [..., T, heads, d] turned by pos [T] * theta^(-2f/d), fp64."""
    d = x.shape[-1]
    z = x.double()
    re, im = (z[..., 0::2], z[..., 1::2]) if il else (z[..., :d // 2], z[..., d // 2:])
    f = np.arange(d // 2, dtype=np.longdouble)
    w = np.longdouble(theta) ** (-2 * f / d)
    a = np.asarray(pos.cpu().numpy(), dtype=np.longdouble)[:, None] * w
    c = torch.as_tensor(np.cos(a).astype(np.float64)).to(x.device)[:, None]
    s = torch.as_tensor(np.sin(a).astype(np.float64)).to(x.device)[:, None]
    r, i = re * c - im * s, re * s + im * c
    return torch.stack((r, i), -1).flatten(-2) if il else torch.cat((r, i), -1)
