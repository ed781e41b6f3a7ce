"""dspark_rotary and dspark_kv_append against their definition in 64 bits: norms,
both kinds of pairs, part of a head turned, positions near and far, ragged and
inactive requests, rows and slots that must stay as they were."""
import math

import pytest
import torch

from attendkit import U, U32, check, dequantise, e4m3_exponent, offsets, quantise

pytestmark = pytest.mark.gpu

BF, FH, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
EPS = 1e-5


def _ds():
    import draft_sampling_verification_02_amd as ds
    ds.load_library()
    return ds


def _bits(t):
    t = t.cpu()
    return t.contiguous().view(torch.uint8)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def turned(x, pos, freq, weight, neighbours):
    """x [n, H, D] in 64 bits -> (values, magnitudes that an error is relative to).

    In 32 bits a sum of D squares is off by at most D U32, its root by half that,
    and root, product and weight by 4 U32; the angle by 2^-21 and its cosine and
    sine by 2 U32; the two products and their sum by 3 U32 of the magnitudes."""
    x = x.double()
    n, H, D = x.shape
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.double().cpu()
    mag = x.abs()
    if freq is None:
        return x, mag
    rot = 2 * freq.numel()
    a = pos.double()[:, None, None] * freq.double().cpu()
    i = torch.arange(rot // 2)
    first, second = (2 * i, 2 * i + 1) if neighbours else (i, i + rot // 2)
    y, big = x.clone(), mag.clone()
    u, v = x[..., first], x[..., second]
    y[..., first], y[..., second] = u * a.cos() - v * a.sin(), v * a.cos() + u * a.sin()
    big[..., first] = big[..., second] = u.abs() + v.abs()
    return y, big


def slack(mag, D):
    return (D / 2 + 9) * U32 * mag + 2.0 ** -21 * mag


def tolerance(want, mag, D, dtype):
    tol = slack(mag, D) + U[dtype] * (want.abs() + slack(mag, D)) + 1e-30
    return tol + (2.0 ** -25 if dtype == FH else 0.0)


def _freq(rot, theta=10000.0):
    return (theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float() if rot else None


def _positions(rows, first, lead, tail):
    pos = [-1] * lead
    for r, f in zip(rows, first):
        pos += [f + i if f >= 0 else -1 for i in range(r)]
    return torch.tensor(pos + [-1] * tail)


LAYOUTS = [
    ([1] * 5, [0, 1, 17, 100000, 7], 0, 0),
    ([3, 0, 17, 1, 40, 2], [14, 3, 0, -1, 1 << 20, -9], 2, 3),
    ([2, 1], [(1 << 31) - 1, 1 << 30], 0, 1),
]


@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("Hq,Hkv,D,rot,neighbours,norm", [
    (4, 1, 64, 64, False, None), (3, 3, 64, 32, True, "row"), (8, 2, 128, 128, False, "row"), (5, 1, 128, 112, True, "f32"),
    (1, 2, 128, 16, False, "q"), (2, 1, 256, 256, True, None), (6, 2, 256, 240, False, "f32"), (4, 4, 128, 0, False, "k"),
])
def test_rows_are_normed_and_turned(dtype, Hq, Hkv, D, rot, neighbours, norm):
    ds = _ds()
    g = torch.Generator().manual_seed(Hq * D + rot)
    freq = _freq(rot)
    wt = torch.float32 if norm == "f32" else dtype
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=g)).to(wt) for _ in range(2))
    wq = wq if norm in ("row", "f32", "q") else None
    wk = wk if norm in ("row", "f32", "k") else None
    dev = lambda t: None if t is None else t.cuda()
    for rows, first, lead, tail in LAYOUTS:
        print(f"rotary: {dtype} {Hq}/{Hkv} D={D} rot={rot} {neighbours} {norm} {rows}", flush=True)
        n = lead + sum(rows) + tail
        x = torch.randn((n, Hq + Hkv + 1, D), generator=g).to(dtype)
        one_each = lead == tail == 0 and all(r == 1 for r in rows)
        xd = x.cuda()
        out = {"q": torch.full((n, Hq, D), 9.0, dtype=dtype, device="cuda"),
               "k": torch.full((n, Hkv + 2, D), 9.0, dtype=dtype, device="cuda")[:, :Hkv]}
        kw = dict(row_offsets=None if one_each else offsets(rows, lead).cuda(), first=_i32(first), q_norm=dev(wq),
                  k_norm=dev(wk), eps=EPS, neighbours=neighbours)
        ds.dspark_rotary(xd[:, :Hq], xd[:, Hq:Hq + Hkv], dev(freq), out=out, **kw)
        pos = _positions(rows, first, lead, tail)
        for name, src, w in (("q", x[:, :Hq], wq), ("k", x[:, Hq:Hq + Hkv], wk)):
            want, mag = turned(src, pos, freq, w, neighbours)
            tol = tolerance(want, mag, D, dtype)
            if w is None and rot < D:
                tol[..., rot:] = 0  # as they were
            want[pos < 0], tol[pos < 0] = 9.0, 0.0
            check(name, out[name], want, tol)
        new = ds.dspark_rotary(xd[:, :Hq], xd[:, Hq:Hq + Hkv], dev(freq), **kw)
        for name in ("q", "k"):
            live = (pos >= 0).cuda()
            assert torch.equal(_bits(new[name][live]), _bits(out[name][live]))
            assert not new[name][~live].any()
        # in place, in slices of the wider rows; a part of the heads alone
        y = xd.clone()
        ds.dspark_rotary(y[:, :Hq], y[:, Hq:Hq + Hkv], dev(freq), out={"q": y[:, :Hq], "k": y[:, Hq:Hq + Hkv]}, **kw)
        whole = xd.clone()
        whole[live, :Hq], whole[live, Hq:Hq + Hkv] = out["q"][live], out["k"][live]
        assert torch.equal(_bits(y), _bits(whole))
        alone = ds.dspark_rotary(None, xd[:, Hq:Hq + Hkv], dev(freq), **kw)
        assert set(alone) == {"k"} and torch.equal(_bits(alone["k"][live]), _bits(out["k"][live]))
        alone = ds.dspark_rotary(xd[:, :Hq], None, dev(freq), **kw)
        assert set(alone) == {"q"} and torch.equal(_bits(alone["q"][live]), _bits(out["q"][live]))


def test_a_call_without_positions_starts_at_zero():
    ds = _ds()
    x = torch.randn(7, 4, 64, device="cuda").to(BF)
    freq = _freq(64).cuda()
    a = ds.dspark_rotary(x[:, :3], x[:, 3:], freq, row_offsets=_i32([0, 7]))
    b = ds.dspark_rotary(x[:, :3], x[:, 3:], freq, first=_i32(list(range(7))))
    assert torch.equal(a["q"], b["q"]) and torch.equal(a["k"], b["k"])
    assert torch.equal(a["q"][0], x[0, :3])


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (0, 1, 64), (3, 1, 256), (40, 40, 64)])
def test_many_rows_are_what_few_rows_are(Hq, Hkv, D):
    ds = _ds()
    heads = Hq + Hkv
    n = 3000 + (1 << 23) // (heads * D) // 2
    print(f"rotary: {n} rows of {Hq}/{Hkv} D={D}", flush=True)
    x = torch.randn(n, heads, D, device="cuda").to(BF)
    w = torch.randn(D, device="cuda").to(BF)
    freq = _freq(D).cuda()
    q, k = (x[:, :Hq] if Hq else None), x[:, Hq:]
    cuts = [0, 1, 40, n // 3, n - 2, n]
    big = ds.dspark_rotary(q, k, freq, row_offsets=_i32(cuts), q_norm=w, k_norm=w)
    for a, b in zip(cuts, cuts[1:]):
        for at in sorted({a, max(a, b - 50), (a + b) // 2}):
            m = min(50, b - at)
            small = ds.dspark_rotary(None if q is None else q[at:at + m], k[at:at + m], freq, row_offsets=_i32([0, m]),
                                     first=_i32([at - a]), q_norm=w, k_norm=w)
            for name in small:
                assert torch.equal(small[name], big[name][at:at + m]), (name, a, at)


def test_bad_values_stay_in_their_heads():
    ds = _ds()
    x = torch.randn(6, 4, 128, device="cuda").to(BF)
    x[1, 2, 100], x[3, 0, 5], x[4, 1, 127] = math.inf, math.nan, -math.inf
    freq, w = _freq(64).cuda(), torch.ones(128, device="cuda", dtype=BF)
    for weight in (None, w):
        y = ds.dspark_rotary(x, None, freq, row_offsets=_i32([0, 6]), first=_i32([3]), q_norm=weight)["q"]
        clean = torch.nan_to_num(x, nan=1.0, posinf=1.0, neginf=1.0)
        z = ds.dspark_rotary(clean, None, freq, row_offsets=_i32([0, 6]), first=_i32([3]), q_norm=weight)["q"]
        bad = {(1, 2), (3, 0), (4, 1)}
        for r in range(6):
            for h in range(4):
                if (r, h) not in bad:
                    assert torch.equal(y[r, h], z[r, h])
                else:
                    assert not torch.isfinite(y[r, h]).all()
        if weight is None:
            assert y[1, 2, 100] == math.inf and y[4, 1, 127] == -math.inf
            assert int((~torch.isfinite(y[1, 2])).sum()) == 1 and int(torch.isnan(y[3, 0]).sum()) == 2


def _cache_of(rows, past, Hkv, D, page, cache, width, g):
    need = [max(0, -(-(r + p) // page)) if p >= 0 else 0 for r, p in zip(rows, past)]
    n_pages = sum(need) + 2
    order = torch.randperm(n_pages, generator=g).tolist()
    width = width or max(1, max(need))
    table = torch.full((len(rows), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :min(n, width)] = torch.tensor(order[at:at + min(n, width)], dtype=torch.int32)
        at += n
    fill = lambda: torch.full((n_pages, Hkv, page, D), 3.0).to(cache).cuda()
    scale = lambda: torch.full((n_pages, Hkv, page), 77, dtype=torch.uint8, device="cuda") if cache == E4 else None
    return table.cuda(), {"k": fill(), "v": fill()}, {"k": scale(), "v": scale()}


APPENDS = [
    ([1] * 9, [0, 1, 15, 16, 17, 31, 100, 5, 63], None, 0, 0),
    ([3, 0, 17, 1, 40, 2], [14, 3, 0, -1, 30, -9], None, 2, 3),
    ([5, 30], [60, 10], 3, 0, 1),
]


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FH, FH), (BF, E4), (FH, E4)])
@pytest.mark.parametrize("Hq,Hkv,D,page,rot,neighbours,norm", [
    (4, 1, 64, 16, 64, False, True), (2, 2, 128, 32, 64, True, False), (0, 8, 128, 16, 128, False, True),
    (3, 3, 256, 16, 256, False, True), (5, 5, 64, 64, 48, True, True)])
def test_rows_are_turned_into_their_slots(dtype, cache, Hq, Hkv, D, page, rot, neighbours, norm):
    ds = _ds()
    for rows, past, width, lead, tail in APPENDS:
        print(f"append: {dtype} {cache} {Hq}/{Hkv} D={D} page={page} rot={rot} {rows}", flush=True)
        g = torch.Generator().manual_seed(D + rot)
        table, caches, scales = _cache_of(rows, past, Hkv, D, page, cache, width, g)
        n = lead + sum(rows) + tail
        x = (torch.randn((n, Hq + 2 * Hkv, D), generator=g) * torch.exp(2 * torch.randn((n, 1, 1), generator=g))).to(dtype)
        freq = _freq(rot)
        wq, wk = ((1 + 0.3 * torch.randn(D, generator=g)).to(dtype) for _ in range(2)) if norm else (None, None)
        one_each = lead == tail == 0 and all(r == 1 for r in rows)
        xd, off, ln = x.cuda(), None if one_each else offsets(rows, lead).cuda(), _i32(past)
        dev = lambda t: None if t is None else t.cuda()
        turn = dict(q_norm=dev(wq), k_norm=dev(wk), eps=EPS, neighbours=neighbours)
        sc = dict(k_scale=scales["k"], v_scale=scales["v"])
        q, k, v = xd[:, :Hq] if Hq else None, xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:]
        # the reference: turned rows, then the write that is tested bit for bit elsewhere
        table2, c2, s2 = _cache_of(rows, past, Hkv, D, page, cache, width, torch.Generator().manual_seed(D + rot))
        kt = ds.dspark_rotary(q, k, freq.cuda(), row_offsets=off, first=ln, **turn)
        ds.dspark_kv_write(kt["k"], v, c2["k"], c2["v"], ln, table, row_offsets=off, k_scale=s2["k"], v_scale=s2["v"])
        out = {"q": torch.full((n, Hq, D), 9.0, dtype=dtype, device="cuda")} if Hq else None
        r = ds.dspark_kv_append(q, k, v, freq.cuda(), caches["k"], caches["v"], ln, table, row_offsets=off, out=out, **sc,
                                **turn)
        torch.cuda.synchronize()
        pos = _positions(rows, past, lead, tail)
        if Hq:
            live = (pos >= 0).cuda()
            assert torch.equal(_bits(r["q"][live]), _bits(kt["q"][live])) and bool((r["q"][~live] == 9).all())
        assert torch.equal(_bits(caches["v"]), _bits(c2["v"]))
        if cache != E4:
            assert torch.equal(_bits(caches["k"]), _bits(c2["k"]))
            continue
        assert torch.equal(scales["v"], s2["v"])
        # slots that no row names are as they were; the rows' are the nearest values of their 32-bit heads
        want, mag = turned(x[:, Hq:Hq + Hkv], pos, freq, wk, neighbours)
        err = slack(mag, D)
        named = torch.zeros(scales["k"].shape, dtype=torch.bool)
        raw, byte = caches["k"].float().cpu().double(), scales["k"].cpu()
        for b in range(len(rows)):
            for i in range(rows[b]):
                t, row = past[b] + i, lead + sum(rows[:b]) + i
                if past[b] < 0 or t // page >= table.shape[1]:
                    continue
                pg = int(table[b, t // page])
                named[pg, :, t % page] = True
                got = dequantise(raw[pg, :, t % page], byte[pg, :, t % page])
                for h in range(Hkv):
                    top = float(want[row, h].abs().max())
                    e = int(byte[pg, h, t % page]) - 127
                    slip = float(err[row, h].max())
                    assert e4m3_exponent(max(top - slip, 0.0)) <= e <= e4m3_exponent(top + slip)
                    step = torch.maximum(want[row, h].abs() * 2.0 ** -4, torch.tensor(math.ldexp(2.0 ** -10, e)))
                    assert bool(((got[h] - want[row, h]).abs() <= step * 1.01 + 2 * err[row, h]).all()), (row, h)
        fresh = torch.full_like(caches["k"].float().cpu(), 3.0).to(E4)
        assert torch.equal(_bits(caches["k"])[~named], _bits(fresh)[~named])
        assert bool((byte[~named] == 77).all())


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (BF, E4), (FH, E4)])
def test_append_without_norm_and_rotation_is_the_write(dtype, cache):
    ds = _ds()
    g = torch.Generator().manual_seed(3)
    rows, past, Hkv, D, page = [4, 1, 33], [0, 40, 9], 2, 128, 16
    n = sum(rows)
    x = (torch.randn((n, 2 * Hkv, D), generator=g) * torch.exp(8 * torch.randn((n, 1, 1), generator=g))).clamp(-6e4, 6e4).to(dtype)
    x[3, 1, 7], x[9, 3, 0], x[20, 0, 3] = math.inf, math.nan, -math.inf
    x[11] = 0
    x = x.cuda()
    off, ln = offsets(rows).cuda(), _i32(past)
    got = _cache_of(rows, past, Hkv, D, page, cache, None, torch.Generator().manual_seed(1))
    want = _cache_of(rows, past, Hkv, D, page, cache, None, torch.Generator().manual_seed(1))
    r = ds.dspark_kv_append(None, x[:, :Hkv], x[:, Hkv:], None, got[1]["k"], got[1]["v"], ln, got[0], row_offsets=off,
                            k_scale=got[2]["k"], v_scale=got[2]["v"])
    assert r == {}
    ds.dspark_kv_write(x[:, :Hkv], x[:, Hkv:], want[1]["k"], want[1]["v"], ln, want[0], row_offsets=off,
                       k_scale=want[2]["k"], v_scale=want[2]["v"])
    for m in ("k", "v"):
        assert torch.equal(_bits(got[1][m]), _bits(want[1][m]))
        if cache == E4:
            assert torch.equal(got[2][m], want[2][m])


def test_long_prompts_are_what_short_calls_are():
    ds = _ds()
    Hq, Hkv, D, page, n = 8, 2, 128, 16, 9000
    x = torch.randn(n, Hq + 2 * Hkv, D, device="cuda").to(BF)
    w, freq = torch.randn(D, device="cuda"), _freq(D).cuda()
    for cache in (BF, E4):
        whole, parts = (_cache_of([n], [100], Hkv, D, page, cache, None, torch.Generator().manual_seed(1)) for _ in range(2))
        def append(c, a, b, past):
            return ds.dspark_kv_append(x[a:b, :Hq], x[a:b, Hq:Hq + Hkv], x[a:b, Hq + Hkv:], freq, c[1]["k"], c[1]["v"],
                                       _i32([past]), c[0], row_offsets=_i32([0, b - a]), k_norm=w, k_scale=c[2]["k"],
                                       v_scale=c[2]["v"])["q"]
        q = append(whole, 0, n, 100)
        qs = torch.cat([append(parts, a, min(a + 700, n), 100 + a) for a in range(0, n, 700)])
        assert torch.equal(q, qs)
        for m in ("k", "v"):
            assert torch.equal(_bits(whole[1][m]), _bits(parts[1][m]))
