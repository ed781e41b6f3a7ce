"""dspark_paged_attention against the definition in 64 bits: lengths around every
tile, unit and page border, masks that leave rows empty, NaN in every unused
slot, shared and missing pages, split and whole walks, all types."""
import math

import pytest
import torch

from attendkit import U, Paged, attend, check, dequantise, far_inputs, far_tolerances, offsets, quantise

pytestmark = pytest.mark.gpu

BF, FH, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


def _ds():
    import draft_sampling_verification_02_amd as ds
    ds.load_library()
    return ds


def _expect(pg, q, rows, lens, G, causal, scale, dtype, off0=0, table_tokens=None):
    """Whole expected output [N, Hq, D] (rows of no request NaN) and its tolerances."""
    N, Hq, D = q.shape
    out = torch.full((N, Hq, D), math.nan, dtype=torch.float64)
    lse = torch.full((N, Hq), math.nan, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    # over 8 bits: bfloat16 probabilities, with a second term beside float16 rows
    up = (U[BF] if dtype == BF else U[BF] ** 2) if pg.cache == E4 else U[dtype]
    at = off0
    for b, (r, past) in enumerate(zip(rows, lens)):
        total = past + r if past >= 0 else 0
        if table_tokens is not None:
            total = min(total, table_tokens)
        lim = [0 if past < 0 else (min(past + i + 1, total) if causal else total) for i in range(r)]
        o = attend(q[at:at + r].double(), pg.tokens["k"][b], pg.tokens["v"][b], lim, scale, up, U[dtype])
        out[at:at + r], lse[at:at + r], tol[at:at + r], ltol[at:at + r] = o
        at += r
    return out, lse, tol, ltol


def _run(rows, lens, Hkv, G, D, page, dtype=BF, cache=BF, causal=True, width=None, max_rows=None, seed=0, lead=0,
         tail=0, wide_q=False):
    ds = _ds()
    print(f"paged: rows={rows[:6]} lens={lens[:6]} Hkv={Hkv} G={G} D={D} page={page} {dtype} {cache} causal={causal} "
          f"width={width}", flush=True)
    total = [max(0, p + r) if p >= 0 else 0 for p, r in zip(lens, rows)]
    pg = Paged(total, Hkv, D, page, dtype, cache, seed, width)
    N = lead + sum(rows) + tail
    g = torch.Generator().manual_seed(seed + 1)
    full = (torch.randn((N, Hkv * G + (3 if wide_q else 0), D), generator=g)).to(dtype)
    q = full[:, :Hkv * G]
    scale = D ** -0.5
    dev = pg.on("cuda")
    qd = full.cuda()[:, :Hkv * G]
    out = {"out": torch.full((N, Hkv * G, D), 7.0, dtype=dtype, device="cuda"),
           "lse": torch.full((N, Hkv * G), 7.0, device="cuda")}
    off = None if lead == tail == 0 and all(r == 1 for r in rows) else offsets(rows, lead).cuda()
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    r = ds.dspark_paged_attention(qd, dev["k_cache"], dev["v_cache"], cl, dev["page_table"], row_offsets=off,
                                  k_scale=dev.get("k_scale"), v_scale=dev.get("v_scale"), causal=causal,
                                  max_rows=max_rows, out=out)
    torch.cuda.synchronize()
    want, wlse, tol, ltol = _expect(pg, q, rows, lens, G, causal, scale, dtype, lead, pg.width * page)
    own = slice(lead, lead + sum(rows))
    check("out", r["out"][own], want[own], tol[own])
    check("lse", r["lse"][own], wlse[own], ltol[own])
    for n in ("out", "lse"):
        for other in (r[n][:lead], r[n][lead + sum(rows):]):
            assert bool((other == 7.0).all()), f"{n}: rows of no request were written"
    return r, dev, qd, off, cl


EDGES = [0, 1, 15, 16, 30, 31, 32, 33, 63, 64, 126, 127, 128, 129, 255, 256, 257]


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FH, FH), (BF, E4), (FH, E4)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_single_rows_at_every_border(dtype, cache, D):
    _run([1] * len(EDGES), EDGES, 2, 4, D, 16, dtype, cache)


@pytest.mark.parametrize("width", [None, 200])
@pytest.mark.parametrize("page", [16, 32, 64, 1024])
def test_pages_and_table_widths(page, width):
    # a wide table takes the split walk whatever the lengths
    _run([1, 1, 1, 1], [0, 700, 1024, 37], 1, 2, 64, page, width=width)


@pytest.mark.parametrize("cache", [BF, E4])
@pytest.mark.parametrize("G", [1, 2, 3, 5, 8, 16, 17, 64])
def test_group_sizes(G, cache):
    _run([1, 1, 1], [5, 600, 250], 2, G, 64, 16, cache=cache, width=40)


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FH, FH), (BF, E4), (FH, E4)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_verify_rows(dtype, cache, D, causal):
    # the anchor and up to five drafts a request, over borders
    _run([6, 1, 3, 6, 5, 2, 4], [0, 31, 30, 124, 127, 509, 1], 2, 4, D, 16, dtype, cache, causal, width=36, max_rows=6)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("max_rows", [1, 3, 8, 40])
def test_any_max_rows_gives_the_same_result(max_rows, D):
    # the hint picks a kernel; requests with more rows take several query groups
    _run([9, 1, 0, 17, 33], [100, 3, 50, 0, 300], 2, 3, D, 32, max_rows=max_rows, width=20)


def test_more_requests_than_threads():
    rows = [1 + (i % 3) for i in range(600)]
    lens = [(i * 37) % 90 for i in range(600)]
    _run(rows, lens, 1, 2, 64, 16, width=64, max_rows=3)


def test_requests_without_rows_and_out_of_the_call():
    # a negative cache length takes a request out: zeros, lse -inf
    _run([2, 0, 1, 3, 0, 1], [40, 10, -1, -5, -1, 0], 2, 2, 128, 16, width=40, lead=2, tail=3)
    _run([1, 1, 1], [-1, 20, -1], 2, 2, 64, 16)


def test_rows_of_wider_tensors():
    _run([2, 3, 1], [40, 0, 333], 2, 4, 128, 16, wide_q=True, width=40)


def test_tokens_past_the_table_are_left_out():
    _run([4, 1], [62, 500], 1, 4, 64, 16, width=4)


def test_one_long_request_is_split_and_joined():
    _run([1], [9000], 1, 4, 128, 64, cache=E4)
    _run([2], [5003], 2, 8, 64, 16, max_rows=2)


def test_very_uneven_lengths():
    _run([1] * 24, [3] * 11 + [6000] + [40] * 12, 2, 4, 128, 16)


def test_missing_pages_and_shared_pages():
    ds = _ds()
    Hkv, G, D, page = 2, 2, 64, 16
    lens, rows = [100, 70, 40], [1, 1, 1]
    for cache in (BF, E4):
        pg = Paged([l + 1 for l in lens], Hkv, D, page, BF, cache, 5, width=40)
        n_pages = pg.buf["k"].shape[0]
        gone = {0: [1, 4], 1: [0], 2: [0, 1, 2]}  # request 2 keeps nothing
        for b, ps in gone.items():
            for j, i in enumerate(ps):
                pg.table[b, i] = [-7, n_pages, 2 ** 31 - 1][j % 3]
        q = torch.randn((3, Hkv * G, D), generator=torch.Generator().manual_seed(1)).to(BF)
        dev = pg.on("cuda")
        r = ds.dspark_paged_attention(q.cuda(), dev["k_cache"], dev["v_cache"],
                                      torch.tensor(lens, dtype=torch.int32, device="cuda"), dev["page_table"],
                                      k_scale=dev.get("k_scale"), v_scale=dev.get("v_scale"), lse=True)
        torch.cuda.synchronize()
        for b in range(3):
            keep = [t for t in range(lens[b] + 1) if t // page not in gone[b]]
            o, z, tol, lt = attend(q[b:b + 1].double(), pg.tokens["k"][b][keep], pg.tokens["v"][b][keep], [len(keep)],
                                   D ** -0.5, U[BF], U[BF])
            check("out", r["out"][b:b + 1], o, tol)
            check("lse", r["lse"][b:b + 1], z, lt)
    # two requests on the same pages see the same tokens
    pg = Paged([90], Hkv, D, page, BF, BF, 6)
    pg.table = pg.table.repeat(2, 1)
    dev = pg.on("cuda")
    q2 = q[:1].repeat(2, 1, 1).cuda()
    r = ds.dspark_paged_attention(q2, dev["k_cache"], dev["v_cache"], torch.tensor([89, 89], dtype=torch.int32, device="cuda"),
                                  dev["page_table"])
    assert torch.equal(r["out"][0], r["out"][1])


@pytest.mark.parametrize("cache", [BF, E4])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_nan_and_infinities_of_later_rows_stay_out_of_earlier_ones(bad, cache):
    # the last of four rows' own token is bad: rows 0..2 must not see it
    ds = _ds()
    Hkv, G, D, page, past = 1, 2, 64, 16, 45
    pg = Paged([past + 4], Hkv, D, page, BF, cache, 8, width=40)
    t = past + 3
    pgid = int(pg.table[0, t // page])
    for n in ("k", "v"):
        # e4m3 has no infinity: NaN stands for it
        x = bad if cache == BF else math.nan
        pg.buf[n][pgid, :, t % page] = torch.full((Hkv, D), x).to(cache)
    q = torch.randn((4, Hkv * G, D), generator=torch.Generator().manual_seed(2)).to(BF)
    dev = pg.on("cuda")
    r = ds.dspark_paged_attention(q.cuda(), dev["k_cache"], dev["v_cache"],
                                  torch.tensor([past], dtype=torch.int32, device="cuda"), dev["page_table"],
                                  row_offsets=torch.tensor([0, 4], dtype=torch.int32, device="cuda"),
                                  k_scale=dev.get("k_scale"), v_scale=dev.get("v_scale"), lse=True)
    torch.cuda.synchronize()
    o, z, tol, lt = attend(q[:3].double(), pg.tokens["k"][0], pg.tokens["v"][0], [past + 1, past + 2, past + 3],
                           D ** -0.5, U[BF], U[BF])
    check("out", r["out"][:3], o, tol)
    check("lse", r["lse"][:3], z, lt)
    if bad != bad or cache == E4:
        assert bool(torch.isnan(r["out"][3]).all())


def test_page_offsets_past_4_gib():
    # a cache larger than 4 GiB whose used pages lie at its end
    ds = _ds()
    Hkv, G, D, page = 8, 2, 128, 64
    n_pages = (5 << 30) // (Hkv * page * D * 2)
    L = 150
    kc = torch.zeros((n_pages, Hkv, page, D), dtype=BF, device="cuda")
    vc = torch.zeros((n_pages, Hkv, page, D), dtype=BF, device="cuda")
    ids = [n_pages - 1, n_pages - 2, n_pages - 3]
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((L, Hkv, D), generator=g).to(BF) for _ in range(2))
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, L], dtype=torch.int32, device="cuda")
    ds.dspark_kv_write(k.cuda(), v.cuda(), kc, vc, zero, table, row_offsets=off)
    back = ds.dspark_kv_read(kc, vc, table, L, row_offsets=off)
    assert torch.equal(back["k"].cpu(), k) and torch.equal(back["v"].cpu(), v)
    q = torch.randn((1, Hkv * G, D), generator=g).to(BF)
    r = ds.dspark_paged_attention(q.cuda(), kc, vc, zero + (L - 1), table, lse=True)
    torch.cuda.synchronize()
    o, z, tol, lt = attend(q.double(), k.double(), v.double(), [L], D ** -0.5, U[BF], U[BF])
    check("out", r["out"], o, tol)
    check("lse", r["lse"], z, lt)


def test_same_bits_on_every_call_streams_and_graph_replays():
    # two calls, a call on a side stream, and a captured call replayed after the
    # lengths grew: the capture follows the device arrays
    ds = _ds()
    rows, lens = [1, 1, 1, 1], [400, 3, 900, 77]
    pg = Paged([l + 9 for l in lens], 2, 64, 16, BF, BF, 4, width=70)
    dev = pg.on("cuda")
    q = torch.randn((4, 8, 64), generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def call(**kw):
        return ds.dspark_paged_attention(q, dev["k_cache"], dev["v_cache"], cl, dev["page_table"], lse=True, **kw)

    a, b = call(), call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = call(stream=side)
    torch.cuda.synchronize()
    for r in (b, c):
        assert torch.equal(a["out"], r["out"]) and torch.equal(a["lse"], r["lse"])
    out = call()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call(out=out)
    for step in range(4):
        cl += 1
        eager = call()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager["out"], out["out"]) and torch.equal(eager["lse"], out["lse"]), step


def test_two_calls_at_once_on_two_streams():
    ds = _ds()
    rows, lens = [3, 1, 2, 6], [700, 30, 2000, 5]
    pg = Paged([l + r for l, r in zip(lens, rows)], 2, 128, 16, BF, BF, 4)
    dev = pg.on("cuda")
    q = torch.randn((sum(rows) + 4, 8, 128), generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    off = offsets(rows, lead=1).cuda()

    def call(**kw):
        return ds.dspark_paged_attention(q, dev["k_cache"], dev["v_cache"], cl, dev["page_table"], row_offsets=off,
                                         lse=True, max_rows=6, **kw)

    want = call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            got.append(call(stream=s))
        torch.cuda.synchronize()
        for r in got:
            assert torch.equal(r["out"], want["out"]) and torch.equal(r["lse"], want["lse"])
            assert bool((r["out"][:1] == 0).all()) and bool((r["out"][13:] == 0).all())


@pytest.mark.parametrize("width", [None, 80])  # walked whole, and split and joined
@pytest.mark.parametrize("rows,G", [([1, 1], 4), ([12, 3], 5)])
@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_infinities_reach_rows_that_hardly_weigh_them(width, rows, G, dtype, D):
    # scores spread over some 60 units, so that most probabilities are far below
    # float16's smallest value: a visible infinity still makes its channel
    # infinite, and infinities of both signs make it NaN
    ds = _ds()
    Hkv, page, lens = 2, 16, [700, 333]
    print(f"paged: rows={rows} G={G} D={D} {dtype} width={width}", flush=True)
    pg = Paged([p + r for p, r in zip(lens, rows)], Hkv, D, page, dtype, dtype, 8, width=width)
    marks = [(3, 5, math.inf), (300, 9, -math.inf), (81, 9, math.inf), (20, D - 1, math.inf), (75, 11, math.nan)]
    for b, last in enumerate([lens[0] + rows[0] - 1, lens[1]]):
        for t, c, x in marks + [(last, 13, -math.inf)]:  # seen by the last row only, and by all rows but those before the newest
            pg.buf["v"][int(pg.table[b, t // page]), :, t % page, c] = x
            pg.tokens["v"][b][t, :, c] = 0.0
    q = (8.0 / 1.5 * torch.randn((sum(rows), Hkv * G, D), generator=torch.Generator().manual_seed(2))).to(dtype)
    dev = pg.on("cuda")
    off = None if rows == [1, 1] else offsets(rows).cuda()
    r = ds.dspark_paged_attention(q.cuda(), dev["k_cache"], dev["v_cache"], torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                  dev["page_table"], row_offsets=off, lse=True)
    torch.cuda.synchronize()
    out, lse, tol, lt = _expect(pg, q, rows, lens, G, True, D ** -0.5, dtype)
    for t, c, x in marks:
        out[:, :, c] += x  # inf - inf is NaN
    out[rows[0] - 1:, :, 13] = -math.inf
    check("out", r["out"], out, tol)
    check("lse", r["lse"], lse, lt)


@pytest.mark.parametrize("rows,past", [(1, 300), (3, 5000), (40, 700), (40, 2000)])
@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FH, FH), (BF, E4), (FH, E4)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scores_far_from_zero(rows, past, dtype, cache, D):
    # scores of 2^30 and more beside ordinary ones: half a step of a 32-bit
    # maximum is more than the range of the probabilities
    ds = _ds()
    page, Hkv, L = 16, 2, past + rows
    pages = -(-L // page)
    q, k, v, scale = far_inputs(rows, pages * page, 6, Hkv, D, dtype, D + rows)
    paged = lambda x: x.reshape(pages, page, *x.shape[1:]).transpose(1, 2).contiguous().cuda()
    if cache == E4:
        (kq, ks), (vq, vs) = quantise(k), quantise(v)
        k, v = dequantise(kq, ks), dequantise(vq, vs)
        args = dict(k_cache=paged(kq.float().to(E4)), v_cache=paged(vq.float().to(E4)), k_scale=paged(ks), v_scale=paged(vs))
    else:
        args = dict(k_cache=paged(k), v_cache=paged(v))
    r = ds.dspark_paged_attention(q.cuda(), cache_len=torch.tensor([past], dtype=torch.int32, device="cuda"),
                                  page_table=torch.arange(pages, dtype=torch.int32, device="cuda")[None],
                                  row_offsets=offsets([rows]).cuda(), scale=scale, lse=True, **args)
    torch.cuda.synchronize()
    up = (U[BF] if dtype == BF else U[BF] ** 2) if cache == E4 else U[dtype]
    o, z, tol, lt = attend(q.double(), k[:L].double(), v[:L].double(), [past + i + 1 for i in range(rows)], scale, up, U[dtype])
    tol, lt = far_tolerances(o, z, tol, lt, v, U[dtype])
    check("out", r["out"], o, tol)
    check("lse", r["lse"], z, lt)


@pytest.mark.parametrize("rows,past", [(1, 700), (1, 9000), (9, 500), (9, 9000)])  # walked whole, and split and joined
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_small_float16_probabilities_count(rows, past, D):
    # one key stands 26 powers of two above all others, whose values alone make
    # the output: each is below float16's smallest half step beside the first one's 1
    ds = _ds()
    g = torch.Generator().manual_seed(D)
    page, L = 16, past + rows
    pages = -(-L // page)
    q = 0.01 * torch.randn((rows, 4, D), generator=g)
    q[:, :, 0] = 4.0
    k = 0.05 * torch.randn((pages * page, 2, D), generator=g)
    k[:, :, 0] = 0.0
    k[0, :, 0] = 26.0 * math.log(2.0) / 4.0
    v = 64.0 + 64.0 * torch.rand((pages * page, 2, D), generator=g)
    v[0] = 0.0
    q, k, v = q.to(FH), k.to(FH), v.to(FH)
    kc, vc = (x.reshape(pages, page, 2, D).transpose(1, 2).contiguous().cuda() for x in (k, v))
    r = ds.dspark_paged_attention(q.cuda(), kc, vc, torch.tensor([past], dtype=torch.int32, device="cuda"),
                                  torch.arange(pages, dtype=torch.int32, device="cuda")[None], row_offsets=offsets([rows]).cuda(),
                                  scale=1.0, lse=True)
    torch.cuda.synchronize()
    o, z, tol, lt = attend(q.double(), k[:L].double(), v[:L].double(), [past + i + 1 for i in range(rows)], 1.0, U[FH], U[FH],
                           lift=14)
    assert bool((tol < 0.01 * o.abs()).all())
    check("out", r["out"], o, tol)
    check("lse", r["lse"], z, lt)
