"""dspark_prompt_attention against the definition in 64 bits: packed sequences of
every length around the tile borders, prefixes, grouped heads, rows that see
nothing, NaN and infinities in masked places, all types."""
import math

import pytest
import torch

from attendkit import U, attend, check, far_inputs, far_tolerances, offsets

pytestmark = pytest.mark.gpu

BF, FH = torch.bfloat16, torch.float16


def _ds():
    import draft_sampling_verification_02_amd as ds
    ds.load_library()
    return ds


def _run(rows, keys, Hkv, G, D, dtype=BF, causal=True, seed=0, lead=0, tail=0, klead=0, fused=False, scale=None, poke=None):
    """keys None: the same rows.  poke(k, v) may change the keys and values in place."""
    ds = _ds()
    print(f"prompt: rows={rows[:6]} keys={None if keys is None else keys[:6]} Hkv={Hkv} G={G} D={D} {dtype} "
          f"causal={causal}", flush=True)
    g = torch.Generator().manual_seed(seed)
    N = lead + sum(rows) + tail
    if keys is None:
        M, klead = N, lead
    else:
        M = klead + sum(keys) + tail
    Hq = Hkv * G
    if fused:
        x = torch.randn((N, Hq + 2 * Hkv, D), generator=g).to(dtype)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        xd = x.cuda()
        qd, kd, vd = xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:]
    else:
        q = torch.randn((N, Hq, D), generator=g).to(dtype)
        k, v = ((torch.randn((M, Hkv, D), generator=g) * 1.3).to(dtype) for _ in range(2))
        if poke:
            poke(k, v)
        qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    s = D ** -0.5 if scale is None else scale
    out = {"out": torch.full((N, Hq, D), 7.0, dtype=dtype, device="cuda"), "lse": torch.full((N, Hq), 7.0, device="cuda")}
    r = ds.dspark_prompt_attention(qd, kd, vd, offsets(rows, lead).cuda(),
                                   kv_offsets=None if keys is None else offsets(keys, klead).cuda(), scale=scale,
                                   causal=causal, out=out)
    torch.cuda.synchronize()
    at, kat = lead, klead
    for b, n in enumerate(rows):
        L = n if keys is None else keys[b]
        lim = [min(L, max(0, L - n + i + 1)) if causal else L for i in range(n)]
        o, z, tol, lt = attend(q[at:at + n].double(), k[kat:kat + L].double(), v[kat:kat + L].double(), lim, s, U[dtype],
                               U[dtype])
        check(f"out of {b}", r["out"][at:at + n], o, tol)
        check(f"lse of {b}", r["lse"][at:at + n], z, lt)
        at, kat = at + n, kat + L
    for n in ("out", "lse"):
        for other in (r[n][:lead], r[n][at:]):
            assert bool((other == 7.0).all()), f"{n}: rows of no sequence were written"
    return r


@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_packed_lengths_around_every_border(dtype, D, causal):
    _run([1, 2, 7, 0, 31, 32, 33, 63, 64, 65, 0, 127, 129], None, 2, 4, D, dtype, causal, lead=3, tail=5)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 8, 33])
def test_group_sizes(G):
    _run([70, 1, 130], None, 2, G, 64)


@pytest.mark.parametrize("Hkv", [1, 3, 8])
def test_wide_batches_take_wide_workgroups(Hkv):
    # enough queries for every workgroup width
    for n in (60, 300, 700):
        _run([n, n // 3, 5, n], None, Hkv, 4, 64, seed=n)
    _run([500, 9, 333], None, Hkv, 8, 128)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_behind_a_prefix(D, causal):
    _run([1, 5, 64, 17, 3], [200, 5, 65, 400, 0], 2, 4, D, causal=causal, klead=2, tail=1)


def test_few_rows_behind_a_long_prefix():
    _run([3], [5000], 1, 4, 128)
    _run([18, 1, 40], [2100, 3000, 41], 2, 8, 64)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_prompts_of_few_heads_are_cut_and_joined(D, causal):
    # blocks near the diagonal's start have fewer parts than the plan, one sequence has a single tile
    _run([700, 3, 1301], None, 1, 3, D, causal=causal, seed=D, lead=2, tail=3)


def test_more_rows_than_keys_leave_rows_empty():
    _run([40, 70, 3], [10, 0, 3], 2, 2, 64)


def test_slices_of_a_fused_projection():
    _run([100, 1, 60], None, 2, 4, 128, fused=True)


def test_scales():
    _run([50], None, 1, 2, 64, scale=0.5)
    _run([50], None, 1, 2, 64, scale=1e-6)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_bad_values_stay_behind_the_mask(bad, D):
    # sequence 1's rows are bad, and the last rows of sequence 0: rows before
    # them, and sequences 0 and 2 beside them, must not see them
    ds = _ds()
    n = [70, 30, 50]
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn((sum(n), h, D), generator=g).to(BF) for h in (4, 2, 2))
    first = 61  # first bad row of sequence 0
    for x in (k, v):
        x[first:100] = bad
    r = ds.dspark_prompt_attention(q.cuda(), k.cuda(), v.cuda(), offsets(n).cuda(), lse=True)
    torch.cuda.synchronize()
    o, z, tol, lt = attend(q[:first].double(), k.double(), v.double(), [i + 1 for i in range(first)], D ** -0.5, U[BF], U[BF])
    check("out before", r["out"][:first], o, tol)
    check("lse before", r["lse"][:first], z, lt)
    o, z, tol, lt = attend(q[100:].double(), k[100:].double(), v[100:].double(), [i + 1 for i in range(50)], D ** -0.5, U[BF], U[BF])
    check("out after", r["out"][100:], o, tol)
    check("lse after", r["lse"][100:], z, lt)
    if bad != bad:
        assert bool(torch.isnan(r["out"][first:100]).all())


def test_values_of_one_bad_value_reach_exactly_the_rows_that_see_it():
    # an infinite value: the rows that see it are infinite in that channel only
    ds = _ds()
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn((40, h, 64), generator=g).to(BF) for h in (2, 1, 1))
    v[23, 0, 5] = math.inf
    r = ds.dspark_prompt_attention(q.cuda(), k.cuda(), v.cuda(), offsets([40]).cuda())
    torch.cuda.synchronize()
    v[23, 0, 5] = 0.0
    o, _, tol, _ = attend(q.double(), k.double(), v.double(), [i + 1 for i in range(40)], 0.125, U[BF], U[BF])
    o[23:, :, 5] = math.inf
    check("out", r["out"], o, tol)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_bad_values_where_the_keys_are_cut(D):
    # the diagonal lies in the last part: an infinite value there, NaN past the sequence's end
    ds = _ds()
    n, L = 18, 2000
    g = torch.Generator().manual_seed(6)
    q, k, v = (torch.randn((m, h, D), generator=g).to(BF) for m, h in ((n, 4), (L + 20, 1), (L + 20, 1)))
    seen = L - n + 7  # rows from 7 on see it
    v[seen, 0, 5] = -math.inf
    k[L:], v[L:] = math.nan, math.nan
    r = ds.dspark_prompt_attention(q.cuda(), k.cuda(), v.cuda(), offsets([n]).cuda(),
                                   kv_offsets=torch.tensor([0, L], dtype=torch.int32, device="cuda"), lse=True)
    torch.cuda.synchronize()
    v[seen, 0, 5] = 0.0
    o, z, tol, lt = attend(q.double(), k[:L].double(), v[:L].double(), [L - n + i + 1 for i in range(n)], D ** -0.5, U[BF],
                           U[BF])
    o[7:, :, 5] = -math.inf
    check("out", r["out"], o, tol)
    check("lse", r["lse"], z, lt)


def test_a_captured_call_with_cut_keys_follows_its_offsets():
    ds = _ds()
    g = torch.Generator().manual_seed(7)
    q, k, v = (torch.randn((m, h, 128), generator=g).to(BF).cuda() for m, h in ((40, 8), (3000, 1), (3000, 1)))
    off, kvoff = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 20, 40], [0, 1500, 3000]))
    res = ds.dspark_prompt_attention(q, k, v, off, kv_offsets=kvoff, lse=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ds.dspark_prompt_attention(q, k, v, off, kv_offsets=kvoff, lse=True, out=res)
    for a, b in (([0, 20, 40], [0, 1500, 3000]), ([0, 3, 40], [0, 2900, 3000]), ([0, 0, 40], [0, 10, 3000]),
                 ([0, 39, 40], [0, 70, 71]), ([0, 20, 40], [0, 1500, 3000])):
        off.copy_(torch.tensor(a, dtype=torch.int32))
        kvoff.copy_(torch.tensor(b, dtype=torch.int32))
        want = ds.dspark_prompt_attention(q, k, v, off, kv_offsets=kvoff, lse=True)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(res["out"], want["out"]) and torch.equal(res["lse"], want["lse"])
        for i in range(2):
            rows, keys = a[i + 1] - a[i], b[i + 1] - b[i]
            lim = [min(keys, max(0, keys - rows + j + 1)) for j in range(rows)]
            o, z, tol, lt = attend(q[a[i]:a[i + 1]].cpu().double(), k[b[i]:b[i + 1]].cpu().double(),
                                   v[b[i]:b[i + 1]].cpu().double(), lim, 128 ** -0.5, U[BF], U[BF])
            check(f"out {a} {i}", res["out"][a[i]:a[i + 1]], o, tol)
            check(f"lse {a} {i}", res["lse"][a[i]:a[i + 1]], z, lt)


def test_same_bits_on_every_call_stream_and_graph_replay():
    ds = _ds()
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn((300, h, 128), generator=g).to(BF).cuda() for h in (8, 2, 2))
    off = offsets([120, 100, 80]).cuda()
    a = ds.dspark_prompt_attention(q, k, v, off, lse=True)
    b = ds.dspark_prompt_attention(q, k, v, off, lse=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = ds.dspark_prompt_attention(q, k, v, off, lse=True, stream=side)
    torch.cuda.synchronize()
    for r in (b, c):
        assert torch.equal(a["out"], r["out"]) and torch.equal(a["lse"], r["lse"])
    out = ds.dspark_prompt_attention(q, k, v, off, lse=True)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        ds.dspark_prompt_attention(q, k, v, off, out=out)
    for split in ([40, 200, 60], [300, 0, 0], [1, 1, 298]):
        off.copy_(offsets(split).cuda())
        eager = ds.dspark_prompt_attention(q, k, v, off, lse=True)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager["out"], out["out"]) and torch.equal(eager["lse"], out["lse"]), split


def test_two_calls_at_once_and_new_outputs_on_the_calls_stream():
    # two streams, each with its own results and workspace, while both run; the
    # zeros of rows that no sequence owns come from the call's own stream
    ds = _ds()
    g = torch.Generator().manual_seed(6)
    q, k, v = (torch.randn((600, h, 64), generator=g).to(BF).cuda() for h in (4, 1, 1))
    off = offsets([100, 300], lead=50).cuda()
    want = ds.dspark_prompt_attention(q, k, v, off, lse=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            got.append(ds.dspark_prompt_attention(q, k, v, off, lse=True, stream=s))
        torch.cuda.synchronize()
        for r in got:
            assert torch.equal(r["out"], want["out"]) and torch.equal(r["lse"], want["lse"])
            assert bool((r["out"][:50] == 0).all()) and bool((r["out"][450:] == 0).all())


def test_a_reused_result_gains_the_lse_it_lacks():
    ds = _ds()
    torch.manual_seed(5)
    off = torch.tensor([0, 70, 100], dtype=torch.int32, device="cuda")
    q, k = (torch.randn(101, h, 64, device="cuda").to(torch.bfloat16) for h in (8, 2))
    want = ds.dspark_prompt_attention(q, k, k, off, lse=True)
    res = ds.dspark_prompt_attention(q, k, k, off)
    assert "lse" not in res
    again = ds.dspark_prompt_attention(q, k, k, off, lse=True, out=res)
    assert again is res and torch.equal(res["lse"][:100], want["lse"][:100]) and torch.equal(res["out"], want["out"])
    assert bool((res["lse"][100] == 0).all())


# (rows, keys, Hkv, G, rows of V, counted from the last key, that hold the bad value)
STRADDLING = [
    ([200], None, 1, 1, [100, 10]),                 # 128 rows a block: the four waves end in three tiles
    ([70, 200, 130], None, 2, 3, [100, 40, 10]),    # a block's rows start anywhere
    ([200, 90], [216, 107], 1, 4, [70, 33]),        # 32 rows a block behind a prefix that is no multiple of them
    ([150], [3000], 1, 1, [100, 10]),               # cut keys, the diagonal over several tiles
]


@pytest.mark.parametrize("rows,keys,Hkv,G,back", STRADDLING)
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_bad_values_of_later_tiles_leave_earlier_rows_alone(rows, keys, Hkv, G, back, bad, dtype, D):
    # channel 5 of some V rows is bad: the rows that see one have that channel
    # bad and nothing else, the rows before them nothing at all
    ds = _ds()
    lens = keys or rows
    print(f"prompt: rows={rows} keys={keys} Hkv={Hkv} G={G} D={D} {dtype} bad={bad}", flush=True)
    need = ds.dspark_prompt_attention_workspace_size(len(rows), sum(rows), sum(lens), Hkv * G, Hkv, D)
    assert (need > 256) == (max(lens) >= 3000)  # the last case is cut and joined
    g = torch.Generator().manual_seed(D)
    q = torch.randn((sum(rows), Hkv * G, D), generator=g).to(dtype)
    k, v = (torch.randn((sum(lens), Hkv, D), generator=g).to(dtype) for _ in range(2))
    clean, at = v.clone(), 0
    for L in lens:
        at += L
        for x in back:
            if x <= L:
                v[at - x, :, 5], clean[at - x, :, 5] = bad, 0.0
    r = ds.dspark_prompt_attention(q.cuda(), k.cuda(), v.cuda(), offsets(rows).cuda(),
                                   kv_offsets=None if keys is None else offsets(keys).cuda(), lse=True)
    torch.cuda.synchronize()
    at = kat = 0
    for b, (n, L) in enumerate(zip(rows, lens)):
        o, z, tol, lt = attend(q[at:at + n].double(), k[kat:kat + L].double(), clean[kat:kat + L].double(),
                               [L - n + i + 1 for i in range(n)], D ** -0.5, U[dtype], U[dtype])
        first = max(0, n - max(x for x in back if x <= L))  # the first row that sees a bad one
        o[first:, :, 5] = bad
        check(f"out of {b}", r["out"][at:at + n], o, tol)
        check(f"lse of {b}", r["lse"][at:at + n], z, lt)
        at, kat = at + n, kat + L


@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_blocks_with_different_numbers_of_parts_are_joined(dtype, D, causal):
    # 2400 rows of one and two heads: the first blocks of a causal prompt have
    # one part, the last ones all; a short sequence beside it has a single tile
    ds = _ds()
    for G, rows in ((1, [2390, 5]), (2, [3, 2400])):
        N, lead = sum(rows) + 3, 1
        assert ds.dspark_prompt_attention_workspace_size(2, N, N, G, 1, D) > 256, "the keys are cut"
        print(f"prompt: rows={rows} G={G} D={D} {dtype} causal={causal}", flush=True)
        g = torch.Generator().manual_seed(D + G)
        q, k, v = (torch.randn((N, h, D), generator=g).to(dtype) for h in (G, 1, 1))
        out = {"out": torch.full((N, G, D), 7.0, dtype=dtype, device="cuda"), "lse": torch.full((N, G), 7.0, device="cuda")}
        r = ds.dspark_prompt_attention(q.cuda(), k.cuda(), v.cuda(), offsets(rows, lead).cuda(), causal=causal, out=out)
        torch.cuda.synchronize()
        at = lead
        for n in rows:
            pick = sorted({i for i in (0, 1, 2, 4, 62, 63, 64, 65, 126, 127, 128, 129, 700, 1023, 1024, 1500, 2000, 2303,
                                       n - 65, n - 64, n - 2, n - 1) if 0 <= i < n})
            lim = [i + 1 if causal else n for i in pick]
            own = slice(at, at + n)
            o, z, tol, lt = attend(q[own][pick].double(), k[own].double(), v[own].double(), lim, D ** -0.5, U[dtype], U[dtype])
            check("out", r["out"][own][pick], o, tol)
            check("lse", r["lse"][own][pick], z, lt)
            assert bool(torch.isfinite(r["out"][own]).all())
            at += n
        for n in ("out", "lse"):
            assert bool((r[n][:lead] == 7.0).all()) and bool((r[n][at:] == 7.0).all())


@pytest.mark.parametrize("rows,keys,Hkv,G", [([300], None, 1, 1), ([90, 200], None, 2, 3), ([50], [3000], 1, 4)])
@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_infinities_reach_rows_that_hardly_weigh_them(rows, keys, Hkv, G, dtype, D):
    # scores spread over some 60 units, so that most probabilities are far below
    # float16's smallest value: a visible infinity still makes its channel
    # infinite, and infinities of both signs make it NaN
    ds = _ds()
    lens = keys or rows
    print(f"prompt: rows={rows} keys={keys} Hkv={Hkv} G={G} D={D} {dtype}", flush=True)
    need = ds.dspark_prompt_attention_workspace_size(len(rows), sum(rows), sum(lens), Hkv * G, Hkv, D)
    assert (need > 256) == (max(lens) >= 3000)
    g = torch.Generator().manual_seed(D)
    q = torch.randn((sum(rows), Hkv * G, D), generator=g).to(dtype)
    k, v = (torch.randn((sum(lens), Hkv, D), generator=g).to(dtype) for _ in range(2))
    marks = [(3, 5, math.inf), (70, 9, -math.inf), (81, 9, math.inf), (20, D - 1, math.inf), (75, 11, math.nan)]  # token, channel, value
    clean, at = v.clone(), 0
    for L in lens:
        for t, c, x in marks:
            v[at + t, :, c], clean[at + t, :, c] = x, 0.0
        at += L
    scale = 8.0 * D ** -0.5
    r = ds.dspark_prompt_attention(q.cuda(), k.cuda(), v.cuda(), offsets(rows).cuda(),
                                   kv_offsets=None if keys is None else offsets(keys).cuda(), scale=scale, lse=True)
    torch.cuda.synchronize()
    at = kat = 0
    for b, (n, L) in enumerate(zip(rows, lens)):
        o, z, tol, lt = attend(q[at:at + n].double(), k[kat:kat + L].double(), clean[kat:kat + L].double(),
                               [L - n + i + 1 for i in range(n)], scale, U[dtype], U[dtype])
        for t, c, x in marks:
            first = max(0, n - L + t)  # the first row that sees token t
            o[first:, :, c] += x  # inf - inf is NaN
        check(f"out of {b}", r["out"][at:at + n], o, tol)
        check(f"lse of {b}", r["lse"][at:at + n], z, lt)
        at, kat = at + n, kat + L


@pytest.mark.parametrize("rows,keys,G", [(200, 200, 1), (70, 90, 3), (40, 3000, 2)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scores_far_from_zero(rows, keys, G, causal, dtype, D):
    # scores of 2^30 and more beside ordinary ones: half a step of a 32-bit
    # maximum is more than the range of the probabilities
    ds = _ds()
    q, k, v, scale = far_inputs(rows, keys, G, 1, D, dtype, D + rows)
    need = ds.dspark_prompt_attention_workspace_size(1, rows, keys, G, 1, D)
    assert (need > 256) == (keys >= 3000)
    r = ds.dspark_prompt_attention(q.cuda(), k.cuda(), v.cuda(), offsets([rows]).cuda(), kv_offsets=offsets([keys]).cuda(),
                                   scale=scale, causal=causal, lse=True)
    torch.cuda.synchronize()
    o, z, tol, lt = attend(q.double(), k.double(), v.double(), [keys - rows + i + 1 if causal else keys for i in range(rows)],
                           scale, U[dtype], U[dtype])
    tol, lt = far_tolerances(o, z, tol, lt, v, U[dtype])
    check("out", r["out"], o, tol)
    check("lse", r["lse"], z, lt)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("keys", [150, 700, 4100])  # walked by one workgroup, cut and joined
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_small_float16_probabilities_count(D, keys, causal):
    # one key stands 26 powers of two above all others, whose values
    # alone make the output: each is below float16's smallest half step beside
    # the first one's 1
    ds = _ds()
    g = torch.Generator().manual_seed(D)
    rows = 40
    need = ds.dspark_prompt_attention_workspace_size(1, rows, keys, 2, 1, D)
    assert (need > 256) == (keys >= 700)
    q = 0.01 * torch.randn((rows, 2, D), generator=g)
    q[:, :, 0] = 4.0
    k = 0.05 * torch.randn((keys, 1, D), generator=g)
    k[:, :, 0] = 0.0
    k[0, :, 0] = 26.0 * math.log(2.0) / 4.0
    v = 64.0 + 64.0 * torch.rand((keys, 1, D), generator=g)
    v[0] = 0.0
    q, k, v = q.to(FH), k.to(FH), v.to(FH)
    r = ds.dspark_prompt_attention(q.cuda(), k.cuda(), v.cuda(), offsets([rows]).cuda(), kv_offsets=offsets([keys]).cuda(),
                                   scale=1.0, causal=causal, lse=True)
    torch.cuda.synchronize()
    o, z, tol, lt = attend(q.double(), k.double(), v.double(), [keys - rows + i + 1 if causal else keys for i in range(rows)],
                           1.0, U[FH], U[FH], lift=11)
    assert bool((tol < 0.01 * o.abs()).all())
    check("out", r["out"], o, tol)
    check("lse", r["lse"], z, lt)
