"""Inputs and 64-bit references of the paged-cache tests (torch, any device)."""
import math

import torch

import block_sparse_long_qsa_b200 as qsa


def half_step(dt) -> float:
    """Largest relative error of one rounding to dt."""
    return torch.finfo(dt).eps / 2


# -------------------------------------------------------------- norm and rotation
def inv_freq64(rope_dim, theta, factor=0.0, original=262144.0, fast=32.0, slow=1.0):
    half = rope_dim // 2
    f = [theta ** (-i / half) for i in range(half)]
    if factor <= 1.0:
        return torch.tensor(f, dtype=torch.float64), 1.0
    turns = lambda i: original * f[i] / (2 * math.pi)  # noqa: E731
    ends = [half * math.log(original / (2 * math.pi * n)) / math.log(theta) for n in (fast, slow)]
    lo, hi = max(math.floor(ends[0]), 0), min(math.ceil(ends[1]), rope_dim - 1)
    # the ends are where the count of turns crosses the two betas
    for i in range(half):
        assert (turns(i) >= fast * (1 - 1e-9)) == (i <= ends[0] + 1e-9)
    out = []
    for i in range(half):
        t = min(max((i - lo) / (hi - lo), 0.0), 1.0)
        out.append((1 - t) * f[i] + t * f[i] / factor)
    return torch.tensor(out, dtype=torch.float64), 0.1 * math.log(factor) + 1


def axes_of_pairs(p):
    half, n = p.rope_dim // 2, list(p.rope_section)
    if p.rope_axes == 1:
        return [0] * half
    if not p.rope_interleaved:
        return [0] * n[0] + [1] * n[1] + [2] * n[2]
    left, out = [None, n[1], n[2]], []
    for i in range(half):
        a = i % 3
        if a and left[a] > 0:
            left[a] -= 1
            out.append(a)
        else:
            out.append(0)
    return out


def norm_rope64(p, x, weight, positions):
    """x [T][H][D]; positions int [axes][T].  (value, size of the terms of each value)."""
    y = x.double()
    if weight is not None:
        w = weight.double() + (1 if p.norm_zero_centred else 0)
        y = y / (y.square().mean(-1, keepdim=True) + float(p.norm_eps)).sqrt() * w
    if p.rope_dim == 0:
        return y, y.abs()
    f, factor = inv_freq64(p.rope_dim, p.rope_theta, p.yarn_factor, p.yarn_original_max, p.yarn_beta_fast,
                           p.yarn_beta_slow)
    a = positions.double()[axes_of_pairs(p)].t() * f.to(x.device)         # [T][half]
    h = p.rope_dim // 2
    z = torch.complex(y[..., :h], y[..., h:2 * h]) * torch.polar(torch.full_like(a, factor), a)[:, None]
    size = factor * (y[..., :h].abs() + y[..., h:2 * h].abs())
    return torch.cat([z.real, z.imag, y[..., 2 * h:]], -1), torch.cat([size, size, y[..., 2 * h:].abs()], -1)


def check_norm_rope(got, want, size, dt):
    """One rounding to dt, and fp32 arithmetic before it: the sum of squares (13
    roundings, halved by the root), root and reciprocal (4 half steps), weights
    and products (4), the angle (a rounding of at most one half turn: pi), sine
    and cosine (4), rotation (3): below 32 half steps of 2^-24 of the terms."""
    err = (got.double() - want).abs()
    tol = half_step(dt) * want.abs() + 2.0 ** -19 * size + 2.0 ** -25 * (dt == torch.float16)
    assert bool((err <= tol).all()), float((err - tol).max())


# ------------------------------------------------------------------------- cache
class Cache:
    """A pool of pages in one of three layouts, every slot NaN until it is
    written, with a table whose unneeded entries name no page."""

    def __init__(self, p, lens, page, dtype, device, layout="token", seed=0, extra_pages=2, needed=None):
        g = torch.Generator().manual_seed(seed)
        self.p, self.page, self.lens = p, page, lens
        H, D = p.n_kv_heads, p.head_dim
        needed = needed or [range(-(-n // page)) for n in lens]
        n_pages = sum(len(x) for x in needed) + extra_pages
        ids = torch.randperm(n_pages, generator=g).tolist()
        table = torch.full((len(lens), max(1, max(-(-n // page) for n in lens)) + 1), -7, dtype=torch.int32)
        for b, need in enumerate(needed):
            for j in need:
                table[b, j] = ids.pop()
        self.spare = ids
        if layout == "token":
            pool = torch.full((2, n_pages, page, H, D), float("nan"), dtype=dtype)
            k, v = pool.to(device)
        elif layout == "head":
            pool = torch.full((2, n_pages, H, page, D), float("nan"), dtype=dtype)
            k, v = pool.to(device).transpose(2, 3)
        else:                                       # K and V of a page side by side, a gap behind the rows
            pool = torch.full((n_pages, 2, page, H, D + 8), float("nan"), dtype=dtype).to(device)
            k, v = pool[:, 0, ..., :D], pool[:, 1, ..., :D]
        self.k, self.v = k, v
        self.table = table.to(device)
        self.kv = qsa.PagedKV(k, v, self.table)

    def slots(self, b, keys):
        t = self.table[b].long()[keys // self.page]
        return t, keys % self.page

    def fill(self, b, lo, hi, k, v):
        keys = torch.arange(lo, hi, device=self.k.device)
        pg, sl = self.slots(b, keys)
        self.k[pg, sl], self.v[pg, sl] = k, v

    def rows(self, b, keys):
        pg, sl = self.slots(b, keys)
        return self.k[pg, sl].double(), self.v[pg, sl].double()


def visible(p, pos):
    keys = torch.arange(pos + 1)
    if p.window:
        keys = keys[(keys > pos - p.window) | (keys < p.n_sinks)]
    return keys


def needed_pages(p, first, last, page):
    """Pages that hold a key some token at positions first .. last sees."""
    return sorted({int(j) // page for pos in {first, last} for j in visible(p, pos)} |
                  {j // page for j in range(max(0, first - p.window + 1) if p.window else 0, last + 1)})


def attend64(p, q, k, v):
    """q [H][D], keys [n][Hk][D] all visible.  (out, lse, bound of out's error, of lse's)."""
    H, D = q.shape
    per = H // p.n_kv_heads
    k, v = k.repeat_interleave(per, 1), v.repeat_interleave(per, 1)
    scale = float(p.softmax_scale) or D ** -0.5
    q = q.double()
    s = torch.einsum("hd,nhd->hn", q, k) * scale
    # a score of D products in fp32: at most 2 D half steps of the terms
    delta = (torch.einsum("hd,nhd->hn", q.abs(), k.abs()) * scale).amax(1) * 2 * D * 2.0 ** -24
    lse = torch.logsumexp(s, 1)
    w = (s - lse[:, None]).exp()
    n = k.shape[0]
    return torch.einsum("hn,nhd->hd", w, v), lse, torch.einsum("hn,nhd->hd", w, v.abs()), delta, n


def check_row(got, got_lse, ref, dt):
    """Weights rounded to dt and shifted by the scores' error, sums of n terms in
    fp32, one rounding of the result."""
    want, lse, size, delta, n = ref
    tol = half_step(dt) * want.abs() + (half_step(dt) + 2 * delta[:, None] + (n + 64) * 2.0 ** -23) * size
    tol = tol + 2.0 ** -25 * (dt == torch.float16)
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), (float(err.max()), float((err - tol).max()))
    if got_lse is not None:
        e = (got_lse.double() - lse).abs()
        assert bool((e <= delta + (n + 64) * 2.0 ** -23 + 2.0 ** -22 * lse.abs()).all()), float(e.max())
