"""Shared pieces of the cache and attention tests: the 8-bit format and the
attention itself in 64 bits, written out plainly on the CPU, paged caches laid
out by hand, and how far a result of given types may be from the definition."""
from __future__ import annotations

import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step of each type
U32 = 2.0 ** -24


def e4m3_exponent(amax: float) -> int:
    """The smallest e >= -126 with amax <= 448 * 2^e."""
    e = -126
    while amax > math.ldexp(448.0, e):
        e += 1
    return e


def e4m3_round(x: torch.Tensor) -> torch.Tensor:
    """Nearest e4m3 value, ties to even, of float64 values of magnitude <= 448; NaN and infinities become NaN."""
    ok = torch.isfinite(x)
    y = torch.where(ok, x, torch.zeros_like(x))
    f = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(f - 3)
    r = torch.round(y / step) * step  # round() takes ties to even
    return torch.where(ok, r, torch.full_like(r, math.nan))


def quantise(x: torch.Tensor):
    """Rows [..., D] -> (e4m3 values float64 [..., D], scale bytes [...])."""
    x = x.double()
    flat = x.reshape(-1, x.shape[-1])
    q, s = torch.empty_like(flat), torch.empty(flat.shape[0], dtype=torch.uint8)
    for i, row in enumerate(flat):
        fin = row[torch.isfinite(row)]
        e = e4m3_exponent(float(fin.abs().max()) if fin.numel() else 0.0)
        q[i] = e4m3_round(row * math.ldexp(1.0, -e))
        s[i] = e + 127
    return q.reshape(x.shape), s.reshape(x.shape[:-1])


def dequantise(q: torch.Tensor, s: torch.Tensor) -> torch.Tensor:
    return q.double() * torch.exp2(s.double() - 127.0)[..., None]


def attend(q, k, v, limits, scale, u_prob, u_out, lift=0):
    """q [R, Hq, D] float64 against k, v [L, Hkv, D]; row i sees tokens t < limits[i].
    Returns (out, lse, out_tol, lse_tol).

    The tolerances count roundings only.  A score is a sum of D products in 32
    bits, scaled and shifted by the maximum: off by at most es = (D + 8) U32
    scale sum|q k|, and the shift by 2 U32 |s - m| <= 4 U32 max|s|.  A
    probability then is off by that much relative, plus the exponential's few
    32-bit steps, and by u_prob from its rounding to 16 bits; the sums of L
    terms in 32 bits by L U32.  All of them weigh |v|: out is off by at most
    (u_prob + 2 (es + ...)) sum p|v|, and by u_out |out| from its own rounding.
    A float16 probability below 2^-14 is off by up to 2^-25 absolute instead,
    against a sum of at least 1 in the same units (of 2^lift, where the largest
    probability is held as 2^lift at least)."""
    R, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = torch.zeros(R, Hq, D, dtype=torch.float64)
    lse = torch.full((R, Hq), -math.inf, dtype=torch.float64)
    tol = torch.zeros(R, Hq, D, dtype=torch.float64)
    lse_tol = torch.zeros(R, Hq, dtype=torch.float64)
    for i in range(R):
        n = int(limits[i])
        if n <= 0:
            continue
        kk, vv = k[:n].repeat_interleave(G, 1), v[:n].repeat_interleave(G, 1)  # [n, Hq, D]
        s = torch.einsum("hd,nhd->hn", q[i], kk) * scale
        z = torch.logsumexp(s, 1)
        p = torch.exp(s - z[:, None])
        out[i] = torch.einsum("hn,nhd->hd", p, vv)
        lse[i] = z
        es = (D + 8) * U32 * scale * torch.einsum("hd,nhd->hn", q[i].abs(), kk.abs()).max(1).values
        es = es + 4 * U32 * s.abs().max(1).values + 8 * U32
        A = torch.einsum("hn,nhd->hd", p, vv.abs())
        small = 2.0 ** (-25 - lift) * vv.abs().sum(0) / torch.exp(z - s.max(1).values)[:, None] if u_prob == U[torch.float16] else 0.0
        tol[i] = (u_prob + 2 * (es + n * U32))[:, None] * A + small + u_out * out[i].abs()
        lse_tol[i] = es + n * U32 + 4 * U32 * z.abs()
    return out, lse, tol * 1.01 + 1e-30, lse_tol * 1.01 + 1e-30


def check(name, got, want, tol):
    """got within tol of want, element by element, NaN and infinities in the same places."""
    got = got.double().cpu()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    odd = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{name}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{name}: infinities differ"
    far = torch.where(odd, torch.zeros_like(want), (got - want).abs() - tol)
    worst = float(far.max()) if far.numel() else 0.0
    assert worst <= 0, f"{name}: off by {worst} more than its tolerance at {int(far.argmax())} of {far.numel()}"


class Paged:
    """A paged cache built by hand: request b holds tokens [0, lens[b]); every
    other slot holds NaN (and the scale of an unused slot is anything)."""

    def __init__(self, lens, Hkv, D, page, dtype, cache, seed, width=None, spare=2):
        g = torch.Generator().manual_seed(seed)
        self.page, self.Hkv, self.D, self.cache = page, Hkv, D, cache
        need = [-(-max(n, 0) // page) for n in lens]
        self.width = width or max(1, max(need))
        n_pages = sum(need) + spare
        order = torch.randperm(n_pages, generator=g).tolist()
        self.table = torch.full((len(lens), self.width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            n = min(n, self.width)
            self.table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += need[b]
        shape = (n_pages, Hkv, page, D)
        e4 = cache == torch.float8_e4m3fn
        self.buf, self.scale, self.tokens = {}, {"k": None, "v": None}, {"k": [], "v": []}
        for n in ("k", "v"):
            pool = torch.full(shape, math.nan, dtype=torch.float32)
            byte = torch.randint(0, 256, shape[:3], generator=g).to(torch.uint8)
            for b, ln in enumerate(lens):
                x = (torch.randn((max(ln, 0), Hkv, D), generator=g) * (1.5 if n == "k" else 1.0)).to(dtype).float()
                if e4:
                    q, s = quantise(x) if ln > 0 else (x.double(), torch.zeros((0, Hkv), dtype=torch.uint8))
                    x = dequantise(q, s) if ln > 0 else x.double()
                for t in range(max(ln, 0)):
                    pi = t // page
                    if pi >= self.width:
                        break
                    pg = int(self.table[b, pi])
                    pool[pg, :, t % page] = (q[t] if e4 else x[t]).float()
                    if e4:
                        byte[pg, :, t % page] = s[t]
                self.tokens[n].append(x.double())
            self.buf[n] = pool.to(cache)
            if e4:
                self.scale[n] = byte

    def on(self, dev):
        d = dict(k_cache=self.buf["k"].to(dev), v_cache=self.buf["v"].to(dev), page_table=self.table.to(dev))
        if self.scale["k"] is not None:
            d.update(k_scale=self.scale["k"].to(dev), v_scale=self.scale["v"].to(dev))
        return d


def offsets(rows, lead=0):
    off = [lead]
    for r in rows:
        off.append(off[-1] + r)
    return torch.tensor(off, dtype=torch.int32)


def far_inputs(rows, keys, Hq, Hkv, D, dtype, seed):
    """q, k, v and a scale whose scores are exact in 32 bits: multiples of 2^30
    for rows 0, 3, .., of 8 for rows 1, 4, .. and zeros for the others."""
    g = torch.Generator().manual_seed(seed)
    q, k = torch.zeros(rows, Hq, D), torch.zeros(keys, Hkv, D)
    q[0::3, :, 0], q[1::3, :, 0] = 2.0 ** 15, 2.0 ** -12
    k[:, :, 0] = 2.0 ** 8 * torch.randint(-7, 8, (keys, Hkv), generator=g).float()
    v = torch.randn(keys, Hkv, D, generator=g)
    return q.to(dtype), k.to(dtype), v.to(dtype), 128.0


def far_tolerances(out, lse, tol, lse_tol, v, u_out):
    """Tolerances of rows 0, 3, ..: a score is exact, and a step of it is 2^30, so
    a probability is 1 or 0; what is left is the sum of at most n equal terms,
    its division, and the roundings of the results."""
    n = v.shape[0]
    tol[0::3] = (n + 4) * U32 * v.abs().max() + u_out * out[0::3].abs()
    lse_tol[0::3] = 8 * U32 * lse[0::3].abs()
    return tol, lse_tol
