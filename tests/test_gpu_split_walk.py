"""dspark_paged_attention where the table is longer than 1024 tokens, so that
requests are cut into units, partials are left in the workspace and joined: all
types and head sizes, masks that leave rows empty, several query groups a
request, rows of no request, missing pages, NaN and infinities behind the mask,
and more requests than a workgroup has threads.  Every call is checked to have
taken the joining path."""
import math

import pytest
import torch

from attendkit import U, Paged, attend, check
from test_gpu_paged_attention import _expect, _run

pytestmark = pytest.mark.gpu

BF, FH, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
TYPES = [(BF, BF), (FH, FH), (BF, E4), (FH, E4)]
WIDE = 80  # pages of 16: 1280 tokens


def _ds():
    import draft_sampling_verification_02_amd as ds
    ds.load_library()
    return ds


@pytest.fixture(autouse=True)
def joined():
    """The test's calls launched paged_join as often as paged_attention."""
    ds = _ds()
    ds.dspark_profile_reset()
    ds.dspark_profile_enable(True)
    try:
        yield
        torch.cuda.synchronize()
        ds.dspark_profile_collect()
    finally:
        ds.dspark_profile_enable(False)
    launched = ds.dspark_profile_read()
    ds.dspark_profile_reset()
    assert launched["paged_attention"][0] > 0 and launched["paged_join"][0] == launched["paged_attention"][0], launched


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_verify_rows(dtype, cache, D, causal):
    _run([6, 1, 3, 0, 6, 2], [700, 255, 1200, 40, 509, 1], 2, 4, D, 16, dtype, cache, causal, width=WIDE, max_rows=6,
         lead=2, tail=3)


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FH, E4)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("max_rows", [1, 3, 8, 40])
def test_several_query_groups_a_request(max_rows, D, dtype, cache):
    _run([9, 1, 0, 17, 33], [800, 3, 50, 0, 600], 1, 3, D, 32, dtype, cache, max_rows=max_rows, width=WIDE // 2)


@pytest.mark.parametrize("G", [1, 5, 16, 17])
def test_group_sizes(G):
    _run([1, 1, 1], [5, 1100, 650], 2, G, 64, 16, width=WIDE)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_requests_without_rows_and_out_of_the_call(dtype, cache):
    _run([2, 0, 1, 3, 0, 1], [740, 10, -1, -5, -1, 1000], 2, 2, 128, 16, dtype, cache, width=WIDE, lead=2, tail=3)


@pytest.mark.parametrize("max_rows", [1, 3])
def test_more_requests_than_threads(max_rows):
    rows = [1 + (i % 3) for i in range(600)]
    lens = [1100 if i % 75 == 3 else (i * 37) % 90 for i in range(600)]
    _run(rows, lens, 1, 2, 64, 16, width=WIDE, max_rows=max_rows)


def test_tokens_past_the_table_are_left_out():
    _run([4, 1], [1278, 5000], 1, 4, 64, 16, width=WIDE)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_missing_pages(dtype, cache, D):
    # pages missing in one half of a tile, in both, over whole units, and all of a request's
    ds = _ds()
    Hkv, G, page, lens = 2, 2, 16, [900, 400, 40]
    pg = Paged([n + 1 for n in lens], Hkv, D, page, dtype, cache, 5, width=WIDE)
    n_pages = pg.buf["k"].shape[0]
    gone = {0: [1, 4, 6, 7] + list(range(16, 41)), 1: [0, 25], 2: [0, 1, 2]}
    for b, ps in gone.items():
        for j, i in enumerate(ps):
            pg.table[b, i] = [-7, n_pages, 2 ** 31 - 1][j % 3]
    q = torch.randn((3, Hkv * G, D), generator=torch.Generator().manual_seed(1)).to(dtype)
    dev = pg.on("cuda")
    r = ds.dspark_paged_attention(q.cuda(), dev["k_cache"], dev["v_cache"], torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                  dev["page_table"], k_scale=dev.get("k_scale"), v_scale=dev.get("v_scale"), lse=True)
    torch.cuda.synchronize()
    up = (U[BF] if dtype == BF else U[BF] ** 2) if cache == E4 else U[dtype]
    for b in range(3):
        keep = [t for t in range(lens[b] + 1) if t // page not in gone[b]]
        o, z, tol, lt = attend(q[b:b + 1].double(), pg.tokens["k"][b][keep], pg.tokens["v"][b][keep], [len(keep)], D ** -0.5,
                               up, U[dtype])
        check("out", r["out"][b:b + 1], o, tol)
        check("lse", r["lse"][b:b + 1], z, lt)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_bad_values_stay_behind_the_mask(bad, dtype, cache, D):
    # 40 rows over two tiles; from the 20th on their own tokens are bad
    ds = _ds()
    Hkv, G, page, past, n, first = 1, 2, 16, 1100, 40, 20
    pg = Paged([past + n], Hkv, D, page, dtype, cache, 8, width=WIDE)
    x = bad if cache != E4 else math.nan  # e4m3 has no infinity: NaN stands for it
    for t in range(past + first, past + n):
        for name in ("k", "v"):
            pg.buf[name][int(pg.table[0, t // page]), :, t % page] = torch.full((Hkv, D), x).to(cache)
    q = torch.randn((n, Hkv * G, D), generator=torch.Generator().manual_seed(2)).to(dtype)
    dev = pg.on("cuda")
    r = ds.dspark_paged_attention(q.cuda(), dev["k_cache"], dev["v_cache"], torch.tensor([past], dtype=torch.int32, device="cuda"),
                                  dev["page_table"], row_offsets=torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                                  k_scale=dev.get("k_scale"), v_scale=dev.get("v_scale"), lse=True)
    torch.cuda.synchronize()
    want = _expect(pg, q, [n], [past], G, True, D ** -0.5, dtype)
    for name, w, tol in (("out", want[0], want[2]), ("lse", want[1], want[3])):
        check(name, r[name][:first], w[:first], tol[:first])
    if x != x:
        assert bool(torch.isnan(r["out"][first:]).all())


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dtype", [BF, FH])
def test_one_bad_value_reaches_exactly_the_rows_that_see_it(bad, dtype):
    # a channel of one V row: seen by the rows from the 9th on, and by all of a second request from the middle of its past
    ds = _ds()
    Hkv, G, D, page, lens, rows = 2, 3, 128, 16, [1000, 900], [12, 3]
    pg = Paged([p + r for p, r in zip(lens, rows)], Hkv, D, page, dtype, dtype, 8, width=WIDE)
    for b, t in ((0, 1008), (1, 333)):
        pg.buf["v"][int(pg.table[b, t // page]), :, t % page, 7] = bad
        pg.tokens["v"][b][t, :, 7] = 0.0
    q = torch.randn((15, Hkv * G, D), generator=torch.Generator().manual_seed(2)).to(dtype)
    dev = pg.on("cuda")
    r = ds.dspark_paged_attention(q.cuda(), dev["k_cache"], dev["v_cache"], torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                  dev["page_table"], row_offsets=torch.tensor([0, 12, 15], dtype=torch.int32, device="cuda"),
                                  lse=True)
    torch.cuda.synchronize()
    out, lse, tol, lt = _expect(pg, q, rows, lens, G, True, D ** -0.5, dtype)
    out[8:, :, 7] = bad
    check("out", r["out"], out, tol)
    check("lse", r["lse"], lse, lt)
