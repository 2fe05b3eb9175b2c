"""Paged caches and tolerances shared by the tests of the rotation, the cache append and the decode."""
import numpy as np
import torch

import oracle

E4M3 = torch.float8_e4m3fn


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def bf16(g, *shape):
    return torch.randn(shape, generator=g).to(torch.bfloat16)


class Paged:
    """Sequences of the given lengths in shuffled pages (CPU tensors). Every slot
    that holds no token is NaN, and every table entry behind a sequence's last
    page is out of range: reading either shows. A table has a spare column."""

    def __init__(self, lens, page_size, H_kv, d, *, e4m3=False, heads_first=False, seed=0,
                 k_scale=1.0, v_scale=1.0, spare_pages=3, data=None):
        g = torch.Generator().manual_seed(seed)
        per = [-(-n // page_size) for n in lens]
        self.lens, self.page_size = list(lens), page_size
        self.n_pages = sum(per) + spare_pages
        order = torch.randperm(self.n_pages, generator=g).tolist()
        self.rows = []  # pages of each sequence
        for n in per:
            self.rows.append(order[:n])
            order = order[n:]
        self.table = torch.full((len(lens), max(per) + 1), 1 << 30, dtype=torch.int32)
        self.table[:, 1::2] = -7
        for b, r in enumerate(self.rows):
            self.table[b, :len(r)] = torch.tensor(r, dtype=torch.int32)
        self.seq_lens = torch.tensor(lens, dtype=torch.int32)
        self.k_scale, self.v_scale = k_scale, v_scale
        shape = (self.n_pages, page_size, H_kv, d)
        if heads_first:
            shape = (self.n_pages, H_kv, page_size, d)
        dtype = E4M3 if e4m3 else torch.bfloat16
        self.k = torch.full(shape, float("nan"), dtype=torch.float32)
        self.v = torch.full(shape, float("nan"), dtype=torch.float32)
        self.heads_first = heads_first
        kk, vv = self.pages(self.k), self.pages(self.v)
        for b, n in enumerate(lens):
            if n:
                p = torch.arange(n)
                at = torch.tensor(self.rows[b])[p // page_size], p % page_size
                k, v = (bf16(g, n, H_kv, d), bf16(g, n, H_kv, d)) if data is None else data[b]
                kk[at] = (k.float() / k_scale).clamp(-448, 448) if e4m3 else k.float()
                vv[at] = (v.float() / v_scale).clamp(-448, 448) if e4m3 else v.float()
        self.k, self.v = self.k.to(dtype), self.v.to(dtype)

    def pages(self, t):
        """[n_pages, page_size, H_kv, d] view of a page tensor."""
        return t.transpose(1, 2) if self.heads_first else t

    def on_gpu(self, eba):
        self.gk, self.gv = self.k.cuda(), self.v.cuda()
        self.gtable, self.glens = self.table.cuda(), self.seq_lens.cuda()
        return eba.PagedCache(self.pages(self.gk), self.pages(self.gv), self.k_scale, self.v_scale)

    def contents(self, k=None, v=None):
        """The sequences' keys and values as float64 [n_b, H_kv, d] lists (what the
        stored elements stand for)."""
        k = np64(self.pages(self.k if k is None else k)) * np.float64(np.float32(self.k_scale))
        v = np64(self.pages(self.v if v is None else v)) * np.float64(np.float32(self.v_scale))
        return ([oracle.gather(k, r, n) for r, n in zip(self.rows, self.lens)],
                [oracle.gather(v, r, n) for r, n in zip(self.rows, self.lens)])


def decode_tolerances(q, keys, values, scale, o, lse, e4m3):
    """Bounds of |O - exact| [B, H, d] and |lse - exact| [B, H] by arithmetic.

    Scores: d products added in fp32, off by at most d 2^-24 sum |q k| scale (and
    as much again for the scaling, the base-2 reference and the exponential's own
    2^-22). A weight's relative error e is that plus its rounding for the product
    with V (two bf16 terms, the second at most 2^-7 of the weight: half a step of
    it, 2^-15; fp16: 2^-11) plus fp32 sums over the keys (blocks of 16, then one addition a block
    and one a part: n / 16 + 64 roundings at most). The weighted mean then moves
    by at most 2 e max |v|, and the bf16 output by half a step, 2^-8 |O|."""
    q = np64(q) if isinstance(q, torch.Tensor) else q
    B, H, d = q.shape
    to, tl = np.zeros_like(o), np.zeros_like(lse)
    for b in range(B):
        n, hk = keys[b].shape[:2]
        if n == 0:
            continue
        for h in range(H):
            g = h // (H // hk)
            big = (np.abs(keys[b][:, g]) @ np.abs(q[b, h])).max() * scale
            score = 2 * d * 2.0 ** -24 * big + 2.0 ** -20
            weight = score + (2.0 ** -11 if e4m3 else 2.0 ** -15) + (n / 16 + 64) * 2.0 ** -24
            to[b, h] = 2.0 ** -8 * np.abs(o[b, h]) + 2 * weight * np.abs(values[b][:, g]).max()
            tl[b, h] = score + (n / 16 + 64) * 2.0 ** -24 + 2.0 ** -22 * abs(lse[b, h])
    return to, tl


def axes_of(plan):
    return [a for a, n in enumerate(plan.axis_pairs) for _ in range(n)]


def rope_exact(x, pos, plan, inverse=False):
    """oracle.rope of [T, H, d] rows with a plan's axes and frequencies."""
    pos = np.asarray(pos).reshape(plan.n_axes, -1)
    return oracle.rope(x, pos, axes_of(plan), plan.frequencies, plan.pairing == "interleaved", inverse)


def rope_tolerance(x, exact, plan):
    """Half a bf16 step of the result (2^-8) and the fp32 rotation: the angle to
    2^-32 turns, its float half turns to 2^-25, sine and cosine to 2 ulp and three
    roundings, together below 2^-20 of |x| + |y| for a pair."""
    x = np.abs(np64(x))
    n = plan.n_pairs
    both = x.copy()
    if plan.pairing == "interleaved":
        both[..., 0:2 * n:2] += x[..., 1:2 * n:2]
        both[..., 1:2 * n:2] += x[..., 0:2 * n:2]
    else:
        both[..., :n] += x[..., n:2 * n]
        both[..., n:2 * n] += x[..., :n]
    return 2.0 ** -8 * np.abs(exact) + 2.0 ** -20 * both
