"""Paged caches on the GPU with host copies, for the tests of the cache's calls."""
import numpy as np
import torch

import bit_affine_quantized_gb300 as bq
from oracle import kv_oracle as KO

BF16 = 2.0 ** -8   # half a step of bf16, relative to a value
F32 = 2.0 ** -24


def bf16(x):
    """The nearest bf16 values, in float64."""
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).double().numpy()


def f64(t):
    return t.detach().cpu().double().numpy()


def dev(x, dtype=torch.bfloat16):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dtype).cuda()


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


class Cache:
    """A cache whose sequences' first lengths[s] positions hold rows of bell-shaped values; what no sequence
    looks at holds NaN (8 bits: any codes with the scale NaN), and table entries behind them name no page."""

    def __init__(self, seed, lengths, heads, D, page, bits8, spare=2, room=1):
        g = np.random.default_rng(seed)
        self.heads, self.D, self.page, self.bits8 = heads, D, page, bits8
        lengths = np.asarray(lengths)
        need = (lengths + room + page - 1) // page
        n, width = len(lengths), int(max(need.max(), 1))
        n_pages = int(need.sum()) + spare
        order = g.permutation(n_pages)
        self.table = np.where(g.random((n, width)) < 0.5, -1, 1 << 30).astype(np.int32)
        self.k, self.v = np.full((2, n_pages, heads, page, D), np.nan)
        self.ks, self.vs = np.full((2, n_pages, heads, page), np.nan)
        if bits8:
            self.k, self.v = g.integers(-127, 128, self.k.shape) * 1.0, g.integers(-127, 128, self.k.shape) * 1.0
        at = 0
        for s, L in enumerate(lengths):
            self.table[s, :need[s]] = order[at:at + need[s]]
            at += need[s]
            for j in range(int(need[s])):
                rows, p = min(page, int(L) - j * page), self.table[s, j]
                if rows <= 0:
                    continue
                for x, sc in ((self.k, self.ks), (self.v, self.vs)):
                    v = g.standard_normal((heads, rows, D)) * np.exp(g.standard_normal((heads, rows, 1)) * 0.5)
                    if bits8:
                        q, m = KO.quantise(v)
                        x[p, :, :rows], sc[p, :, :rows] = q, m.astype(np.float32)
                    else:
                        x[p, :, :rows] = bf16(v)
        self.upload()

    def upload(self):
        kind = torch.int8 if self.bits8 else torch.bfloat16
        self.dk, self.dv = dev(self.k, kind), dev(self.v, kind)
        self.dks, self.dvs = (dev(self.ks, torch.float32), dev(self.vs, torch.float32)) if self.bits8 else (None, None)
        self.dtable = i32(self.table)
        self.c = bq.make_kv_cache(self.dk, self.dv, self.dtable, self.dks, self.dvs)

    def rows(self, seq, pos):
        """Keys and values [T, heads, D] of positions, from the host copy."""
        return (KO.rows(self.k, self.ks if self.bits8 else None, self.table, self.page, seq, pos),
                KO.rows(self.v, self.vs if self.bits8 else None, self.table, self.page, seq, pos))
