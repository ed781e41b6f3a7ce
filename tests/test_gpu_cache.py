"""dspark_kv_write and dspark_kv_read, bit for bit: placement, the 8-bit format
against its definition in 64 bits, slots and rows that must stay as they were."""
import math

import pytest
import torch

from attendkit import dequantise, offsets, quantise

pytestmark = pytest.mark.gpu

BF, FH, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


def _ds():
    import draft_sampling_verification_02_amd as ds
    ds.load_library()
    return ds


def _bits(t):
    t = t.cpu()
    return t.view(torch.uint8) if t.element_size() == 1 else t.view(torch.int16)


def _setup(rows, past, Hkv, D, page, dtype, cache, seed, width, lead, tail, wide):
    g = torch.Generator().manual_seed(seed)
    need = [max(0, -(-(r + p) // page)) if p >= 0 else 0 for r, p in zip(rows, past)]
    n_pages = sum(need) + 2
    order = torch.randperm(n_pages, generator=g).tolist()
    width = width or max(1, max(need))
    table = torch.full((len(rows), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        m = min(n, width)
        table[b, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
        at += n
    N = lead + sum(rows) + tail
    x = (torch.randn((N, 2 * Hkv + wide, D), generator=g) * torch.exp(2 * torch.randn((N, 1, 1), generator=g))).to(dtype)
    e4 = cache == E4
    fill = lambda: torch.full((n_pages, Hkv, page, D), 3.0).to(cache)
    caches = {"k": fill(), "v": fill()}
    scales = {n: torch.full((n_pages, Hkv, page), 77, dtype=torch.uint8) if e4 else None for n in ("k", "v")}
    return table, x, caches, scales


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FH, FH), (BF, E4), (FH, E4)])
@pytest.mark.parametrize("Hkv,D,page", [(1, 64, 16), (2, 128, 32), (5, 64, 64), (8, 128, 16), (3, 256, 1024)])
def test_rows_land_in_their_slots_and_nowhere_else(dtype, cache, Hkv, D, page):
    for rows, past, width, lead, tail in [
            ([1] * 9, [0, 1, 15, 16, 17, 31, 100, 5, 63], None, 0, 0),
            ([3, 0, 17, 1, 40, 2], [14, 3, 0, -1, 30, -9], None, 2, 3),
            ([5, 30], [60, 10], 3 if page < 64 else 1, 0, 1)]:
        ds = _ds()
        print(f"cache: {dtype} {cache} Hkv={Hkv} D={D} page={page} rows={rows}", flush=True)
        table, x, caches, scales = _setup(rows, past, Hkv, D, page, dtype, cache, 7, width, lead, tail, 1)
        k, v = x[:, :Hkv], x[:, Hkv:2 * Hkv]
        off = offsets(rows, lead)
        one_each = lead == tail == 0 and all(r == 1 for r in rows)
        xd = x.cuda()
        dev = {n: caches[n].cuda() for n in caches}
        dsc = {n: None if scales[n] is None else scales[n].cuda() for n in scales}
        ds.dspark_kv_write(xd[:, :Hkv], xd[:, Hkv:2 * Hkv], dev["k"], dev["v"],
                           torch.tensor(past, dtype=torch.int32, device="cuda"), table.cuda(),
                           row_offsets=None if one_each else off.cuda(), k_scale=dsc["k"], v_scale=dsc["v"])
        torch.cuda.synchronize()
        written = {}
        for n, src in (("k", k), ("v", v)):
            if cache == E4:
                q, s = quantise(src)
                vals = q.to(torch.float32).to(E4)
            for b in range(len(rows)):
                for i in range(rows[b]):
                    t, r = past[b] + i, lead + sum(rows[:b]) + i
                    if past[b] < 0 or t // page >= table.shape[1]:
                        continue
                    pg = int(table[b, t // page])
                    if cache == E4:
                        caches[n][pg, :, t % page] = vals[r]
                        scales[n][pg, :, t % page] = s[r]
                        written[(n, r)] = dequantise(q[r], s[r])
                    else:
                        caches[n][pg, :, t % page] = src[r]
                        written[(n, r)] = src[r].double()
            assert torch.equal(_bits(dev[n]), _bits(caches[n])), n
            if cache == E4:
                assert torch.equal(dsc[n].cpu(), scales[n]), n
        # and back
        out = {n: torch.full((x.shape[0], Hkv, D), 9.0, dtype=dtype, device="cuda") for n in ("k", "v")}
        ds.dspark_kv_read(dev["k"], dev["v"], table.cuda(), x.shape[0], row_offsets=None if one_each else off.cuda(),
                          first=torch.tensor(past, dtype=torch.int32, device="cuda"), k_scale=dsc["k"],
                          v_scale=dsc["v"], dtype=dtype, out=out)
        torch.cuda.synchronize()
        top = torch.finfo(dtype).max
        for n in ("k", "v"):
            for r in range(x.shape[0]):
                inside = lead <= r < lead + sum(rows)
                want = written.get((n, r))
                if want is None:
                    want = torch.full((Hkv, D), 0.0 if inside else 9.0, dtype=torch.float64)
                assert torch.equal(out[n][r].cpu(), want.clamp(-top, top).to(dtype)), (n, r)


@pytest.mark.parametrize("dtype", [BF, FH])
def test_8_bit_format_over_the_whole_range(dtype):
    # every finite exponent of the type, zeros, ties, the type's largest and smallest values, bad values
    ds = _ds()
    tiny, top = torch.finfo(dtype).tiny, torch.finfo(dtype).max
    g = torch.Generator().manual_seed(11)
    D = 64
    exps = torch.arange(-133 if dtype == BF else -24, 128 if dtype == BF else 16)
    base = torch.randn((len(exps), D), generator=g).double() * torch.exp2(exps.double())[:, None]
    rows = [base.clamp(-top, top)]
    rows.append(torch.zeros(1, D, dtype=torch.float64))
    rows.append(torch.full((1, D), top, dtype=torch.float64))
    rows.append(torch.full((1, D), tiny, dtype=torch.float64))
    for a in (448.0, 449.0, 447.0, 1.75, 1.7578125, 0.875):
        r = torch.linspace(-a, a, D, dtype=torch.float64)[None]
        rows.append(r)
    ties = torch.tensor([17.0, 19.0, 18.0, 2.0 ** -10, 3 * 2.0 ** -10, 5 * 2.0 ** -10, 232.0, 248.0] * 8)[None].double()
    ties[0, 0] = 448.0
    rows.append(ties)
    x = torch.cat(rows).to(dtype)
    bad = torch.randn((4, D), generator=g).to(dtype)
    bad[0, 3], bad[1, 5], bad[2, 7] = math.nan, math.inf, -math.inf
    bad[3] = math.nan
    x = torch.cat([x, bad])[:, None]  # one head
    N = x.shape[0]
    page = 16
    n_pages = -(-N // page)
    kc, vc = (torch.zeros((n_pages, 1, page, D), device="cuda").to(E4) for _ in range(2))
    ks, vs = (torch.zeros((n_pages, 1, page), dtype=torch.uint8, device="cuda") for _ in range(2))
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda")[None]
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    ds.dspark_kv_write(x.cuda(), (-x).contiguous().cuda(), kc, vc, zero, table, row_offsets=off, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    q, s = quantise(x)
    for cache, sc, sign in ((kc, ks, 1.0), (vc, vs, -1.0)):
        got = cache.float().cpu().reshape(-1, 1, D)[:N]
        want = (sign * q).float()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        ok = ~torch.isnan(want)
        assert torch.equal(got[ok], want[ok])
        assert torch.equal(sc.cpu().reshape(-1, 1)[:N], s)
    # the definition's own bound: half a step of e4m3, 2^-4, or half its smallest step
    back = dequantise(q, s)[:-4]
    err = (back - x[:-4].double()).abs()
    bound = torch.maximum(x[:-4].double().abs() * 2.0 ** -4, 2.0 ** -10 * torch.exp2(s[:-4].double() - 127)[..., None])
    assert bool((err <= bound).all())
    r = ds.dspark_kv_read(kc, vc, table, N, row_offsets=off, k_scale=ks, v_scale=vs, dtype=dtype)
    torch.cuda.synchronize()
    want = dequantise(q, s).clamp(-top, top).to(dtype)
    for got, w in ((r["k"].cpu(), want), (r["v"].cpu(), -want)):
        assert torch.equal(torch.isnan(got), torch.isnan(w))
        assert torch.equal(got[~torch.isnan(w)], w[~torch.isnan(w)])


def test_many_rows_of_many_requests():
    # the wide workgroups: rows of several requests in one
    ds = _ds()
    g = torch.Generator().manual_seed(2)
    rows = [int(r) for r in torch.randint(0, 40, (700,), generator=g)]
    past = [int(p) for p in torch.randint(0, 50, (700,), generator=g)]
    Hkv, D, page = 2, 128, 16
    N = sum(rows)
    need = [-(-(r + p) // page) for r, p in zip(rows, past)]
    width, n_pages = max(need), sum(need)
    order = torch.randperm(n_pages, generator=g).to(torch.int32)
    table = torch.full((700, width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    k, v = (torch.randn((N, Hkv, D), generator=g).to(BF) for _ in range(2))
    kc, vc = (torch.zeros((n_pages, Hkv, page, D), dtype=BF) for _ in range(2))
    kd, vd = kc.cuda(), vc.cuda()
    off = offsets(rows)
    pd = torch.tensor(past, dtype=torch.int32, device="cuda")
    ds.dspark_kv_write(k.cuda(), v.cuda(), kd, vd, pd, table.cuda(), row_offsets=off.cuda())
    req = torch.repeat_interleave(torch.arange(700), torch.tensor(rows))
    pos = torch.arange(N) - off[req].long() + torch.tensor(past)[req]
    pg = table[req, pos // page].long()
    kc[pg, :, pos % page] = k
    vc[pg, :, pos % page] = v
    assert torch.equal(kd.cpu(), kc) and torch.equal(vd.cpu(), vc)
    r = ds.dspark_kv_read(kd, vd, table.cuda(), N, row_offsets=off.cuda(), first=pd)
    assert torch.equal(r["k"].cpu(), k) and torch.equal(r["v"].cpu(), v)


@pytest.mark.parametrize("cache", [BF, E4])
@pytest.mark.parametrize("low,high", [(-5, 200), (-2 ** 31, 2 ** 31 - 1)])
def test_offsets_outside_the_rows_count_as_clamped(low, high, cache):
    # requests that start before the first row or end behind the last: rows go
    # where they go with the offsets clamped into [0, n_rows], in a write, a
    # read and an attention over the cache
    ds = _ds()
    Hkv, D, page, n = 2, 64, 16, 12
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((n, Hkv, D), generator=g).to(BF).cuda() for _ in range(2))
    q = torch.randn((n, 2 * Hkv, D), generator=g).to(BF).cuda()
    past = torch.tensor([4, 30, 0, 9], dtype=torch.int32, device="cuda")
    table = torch.randperm(16, generator=g).to(torch.int32).view(4, 4).cuda()
    results = []
    for off in ([low, 3, 9, 9, high], [0, 3, 9, 9, n]):
        off = torch.tensor(off, dtype=torch.int32, device="cuda")
        kc, vc = (torch.full((16, Hkv, page, D), 3.0, device="cuda").to(cache) for _ in range(2))
        sc = {x: torch.full((16, Hkv, page), 77, dtype=torch.uint8, device="cuda") for x in ("k_scale", "v_scale")} if cache == E4 else {}
        ds.dspark_kv_write(k, v, kc, vc, past, table, row_offsets=off, **sc)
        back = ds.dspark_kv_read(kc, vc, table, n, row_offsets=off, first=past, **sc)
        att = ds.dspark_paged_attention(q, kc, vc, past, table, row_offsets=off, lse=True, **sc)
        torch.cuda.synchronize()
        results.append([_bits(kc), _bits(vc), _bits(back["k"]), _bits(back["v"]), _bits(att["out"]), att["lse"].cpu()]
                       + [x.cpu() for x in sc.values()])
    for a, b in zip(*results):
        assert torch.equal(a, b)
    if cache == BF:
        assert torch.equal(back["k"], k) and torch.equal(back["v"], v)
