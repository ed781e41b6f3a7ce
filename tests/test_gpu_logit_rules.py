"""dspark_logit_rules against its definition in 64 bits: texts, drafts, penalties,
biases and masks together and alone, odd vocabularies, padded rows, and ids and
indexes outside their ranges."""
import math

import pytest
import torch

from attendkit import U32, offsets

pytestmark = pytest.mark.gpu

BF, FH, F32 = torch.bfloat16, torch.float16, torch.float32


def _ds():
    import draft_sampling_verification_02_amd as ds
    ds.load_library()
    return ds


def make(seed, V, rows, text, gamma, n_bias, n_masks, lead=0, tail=0, penalties=True, wild=True):
    g = torch.Generator().manual_seed(seed)
    B, n = len(rows), lead + sum(rows) + tail
    ids = lambda *s: (V * torch.rand(s, generator=g) ** 3).to(torch.int32).clamp(max=V - 1)
    c = dict(V=V, rows=rows, lead=lead, n=n, row_offsets=offsets(rows, lead))
    c["history"], c["drafts"] = ids(B, text), ids(B, gamma) if gamma else None
    c["history_len"] = torch.randint(0, text + 1, (B,), generator=g, dtype=torch.int32)
    c["history_len"][0] = text
    c["prompt_len"] = (c["history_len"] * torch.rand(B, generator=g)).to(torch.int32)
    if wild and text > 3:  # ids outside the vocabulary, a length past the buffer, a negative one
        c["history"][:, 1::7] = V
        c["history"][:, 2::9] = -3
        c["history_len"][-1] = text + 100 if B > 1 else text
        if B > 2:
            c["history_len"][1], c["prompt_len"][2] = -5, text + 9
    pick = lambda v: torch.tensor(v)[torch.randint(0, len(v), (B,), generator=g)]
    c["repetition"] = c["frequency"] = c["presence"] = None
    if penalties:
        c["repetition"], c["frequency"], c["presence"] = pick([1.0, 1.3, 0.8]), pick([0.0, 0.4]), pick([0.0, 0.6, -0.3])
    c["bias_offsets"] = c["bias_ids"] = c["bias_values"] = None
    if n_bias:
        nb = [0 if b % 4 == 3 else n_bias for b in range(B)]
        c["bias_offsets"] = offsets(nb)
        c["bias_ids"] = ids(sum(nb))
        c["bias_ids"][1::5] = c["bias_ids"][0]  # the same token again and again
        if wild:
            c["bias_ids"][3::11] = V + 5
            c["bias_ids"][4::13] = -1
        c["bias_values"] = torch.randn(sum(nb), generator=g)
    c["masks"] = c["mask_index"] = None
    if n_masks:
        words = (V + 31) // 32 + (1 if wild else 0)
        c["masks"] = torch.randint(-2 ** 31, 2 ** 31, (n_masks, words), generator=g).to(torch.int32)
        c["masks"][0] = 0
        c["masks"][0, (V - 1) // 32] = -2 ** 31 if (V - 1) % 32 == 31 else 1 << ((V - 1) % 32)
        c["mask_index"] = torch.randint(-1, n_masks + (1 if wild else 0), (n,), generator=g, dtype=torch.int32)
    return c


ARGS = ("history", "history_len", "prompt_len", "drafts", "repetition", "frequency", "presence", "bias_offsets", "bias_ids",
        "bias_values", "masks", "mask_index")


def want(c, logits):
    """(values, tolerance): each of a quotient, a product, the sums and the subtraction is off by U32 of its size."""
    V, out = c["V"], logits.double().clone()
    tol = torch.zeros_like(out)
    at = c["lead"]
    for b, r in enumerate(c["rows"]):
        text = c["history"][b][:max(int(c["history_len"][b]), 0)].tolist() if c["history"] is not None else []
        p = int(c["prompt_len"][b]) if c["prompt_len"] is not None else 0
        rho, phi, pi = (1.0 if n == "repetition" and c[n] is None else 0.0 if c[n] is None else float(c[n][b])
                        for n in ("repetition", "frequency", "presence"))
        for j in range(r):
            row = at + j
            said = text[max(p, 0):] + (c["drafts"][b, :j].tolist() if c["drafts"] is not None else [])
            seen = {t for t in text + said if 0 <= t < V}
            count = {}
            for t in said:
                count[t] = count.get(t, 0) + 1
            for t in seen:
                z = float(out[row, t])
                z = z / rho if z > 0 else z * rho
                n = count.get(t, 0)
                cut = phi * n + (pi if n else 0.0)
                if rho != 1.0 or cut != 0.0:
                    tol[row, t] = 3 * U32 * (abs(z) + abs(phi) * n + abs(pi)) if math.isfinite(z) else 0
                out[row, t] = z - cut
            if c["bias_offsets"] is not None:
                for e in range(int(c["bias_offsets"][b]), int(c["bias_offsets"][b + 1])):
                    t, x = int(c["bias_ids"][e]), float(c["bias_values"][e])
                    if 0 <= t < V:
                        out[row, t] += x
                        if math.isfinite(float(out[row, t])):
                            tol[row, t] += U32 * (abs(float(out[row, t])) + 40 * abs(x))  # up to 40 of a token are added
            if c["masks"] is not None and 0 <= int(c["mask_index"][row]) < c["masks"].shape[0]:
                bits = c["masks"][int(c["mask_index"][row])]
                v = torch.arange(V)
                forbidden = ((bits[v // 32] >> (v % 32)) & 1) == 0
                out[row, forbidden] = -math.inf
                tol[row, forbidden] = 0
        at += r
    return out, tol * 1.01


def compare(got, w, tol):
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(w))
    odd = ~torch.isfinite(w)
    assert torch.equal(got[odd & ~torch.isnan(w)], w[odd & ~torch.isnan(w)])
    assert bool(torch.isfinite(got[~odd]).all())
    assert bool(((got - w).abs() <= tol)[~odd].all()), float((got - w).abs()[~odd].max())


def call(c, logits, **kw):
    dev = {n: None if c[n] is None else c[n].cuda() for n in ARGS}
    return _ds().dspark_logit_rules(logits, row_offsets=c["row_offsets"].cuda(), **dev, **kw)


SHAPES = [
    # V, rows, text, gamma, biases, masks, lead, tail
    (1000, [1, 3, 0, 6, 2], 50, 5, 12, 3, 0, 0),
    (4099, [2, 1, 1], 300, 1, 40, 2, 1, 2),
    (12928, [4] * 9, 700, 3, 5, 1, 0, 1),
    (50257, [1, 5], 3000, 4, 30, 2, 0, 0),
    (20000, [2, 1], 30000, 3, 9, 2, 0, 0),
    (20001, [2, 1], 25000, 3, 9, 2, 0, 1),
    (151936, [2] * 10, 20000, 1, 7, 2, 0, 0),
    (151937, [1] * 10, 700, 1, 7, 2, 0, 0),
    (33, [2, 2, 2], 9, 2, 3, 4, 0, 0),
    (1, [1, 2], 4, 1, 2, 1, 0, 0),
]


@pytest.mark.parametrize("dtype", [BF, FH, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_all_rules_together(dtype, shape):
    V, rows, text, gamma, nb, nm, lead, tail = shape
    print(f"rules: {dtype} {shape}", flush=True)
    c = make(V + len(rows), V, rows, text, gamma, nb, nm, lead, tail)
    x = (3 * torch.randn((c["n"], V), generator=torch.Generator().manual_seed(5))).to(dtype)
    x.view(-1)[::97] = -math.inf
    w, tol = want(c, x)
    out = torch.full((c["n"], V), 7.0, device="cuda")
    r = call(c, x.cuda(), out=out)
    assert r is out
    own = torch.zeros(c["n"], dtype=torch.bool)
    own[lead:lead + sum(rows)] = True
    w[~own], tol[~own] = 7.0, 0.0
    compare(r, w, tol)
    new = call(c, x.cuda())
    assert torch.equal(new[own.cuda()], r[own.cuda()]) and not new[~own.cuda()].any()
    # rows with room behind them, on both sides
    pad = torch.full((c["n"], V + 5), 6e4, dtype=dtype)
    pad[:, :V] = x
    wide = torch.full((c["n"], V + 3), 7.0, device="cuda")
    call(c, pad.cuda()[:, :V], out=wide[:, :V])
    assert torch.equal(wide[:, :V], r) and bool((wide[:, V:] == 7).all())
    if dtype == F32:
        y = x.cuda()
        call(c, y, out=y)
        assert torch.equal(y[own.cuda()], r[own.cuda()]) and torch.equal(y[~own.cuda()].cpu(), x[~own])


@pytest.mark.parametrize("part", ["none", "text", "repetition", "frequency", "presence", "drafts", "biases", "masks"])
def test_each_rule_alone(part):
    V = 5000
    c = make(3, V, [1, 4, 2], 80, 3, 9, 2)
    keep = {"none": (), "text": ("history", "history_len"), "repetition": ("history", "history_len", "prompt_len", "repetition"),
            "frequency": ("history", "history_len", "prompt_len", "frequency"),
            "presence": ("history", "history_len", "presence"), "drafts": ("drafts", "repetition", "frequency", "presence"),
            "biases": ("bias_offsets", "bias_ids", "bias_values"), "masks": ("masks", "mask_index")}[part]
    for n in ARGS:
        if n not in keep:
            c[n] = None
    x = torch.randn((c["n"], V), generator=torch.Generator().manual_seed(5)).to(BF)
    x[0, 5], x[2, 77] = math.nan, math.inf
    w, tol = want(c, x)
    r = call(c, x.cuda())
    compare(r, w, tol)
    if part in ("none", "text"):
        assert torch.equal(r.cpu()[1:2], x[1:2].float())


def test_one_row_a_request_and_many_of_them():
    ds = _ds()
    V, B = 129280, 40
    c = make(8, V, [1] * B, 100, 0, 6, 5)
    x = (3 * torch.randn((B, V), device="cuda")).to(BF)
    dev = {n: None if c[n] is None else c[n].cuda() for n in ARGS}
    a = ds.dspark_logit_rules(x, **dev)
    w, tol = want(c, x.cpu())
    compare(a, w, tol)
    for b in (0, 7, 39):  # few slices, small ones: the same bits
        one = {n: t if n in ("masks", "bias_ids", "bias_values") or t is None
               else t[b:b + 2] if n == "bias_offsets" else t[b:b + 1] for n, t in dev.items()}
        assert torch.equal(ds.dspark_logit_rules(x[b:b + 1], **one)[0], a[b])


def test_a_bias_list_with_one_token_only():
    # added in the order of the list: the sum in 32 bits, step by step
    V, n = 300, 1500
    g = torch.Generator().manual_seed(2)
    values = torch.randn(n, generator=g) * torch.exp(3 * torch.randn(n, generator=g))
    ids = torch.full((n,), 17, dtype=torch.int32)
    ids[::50] = 18
    acc = {17: torch.zeros(()), 18: torch.zeros(())}
    for i, x in zip(ids.tolist(), values):
        acc[i] = acc[i] + x
    r = _ds().dspark_logit_rules(torch.zeros(1, V, device="cuda"), bias_offsets=torch.tensor([0, n], dtype=torch.int32).cuda(),
                                 bias_ids=ids.cuda(), bias_values=values.cuda()).cpu()
    assert float(r[0, 17]) == float(acc[17]) and float(r[0, 18]) == float(acc[18]) and int((r != 0).sum()) == 2


def test_a_captured_call_follows_its_inputs():
    ds = _ds()
    V, rows = 9000, [3, 1, 4]
    cases = [make(s, V, rows, 200, 3, 20, 3) for s in range(4)]
    x = [torch.randn((8, V), generator=torch.Generator().manual_seed(s)).to(BF) for s in range(4)]
    live = {n: cases[0][n].cuda() for n in ARGS}
    lx, off, out = x[0].cuda(), cases[0]["row_offsets"].cuda(), torch.zeros(8, V, device="cuda")
    ds.dspark_logit_rules(lx, row_offsets=off, out=out, **live)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ds.dspark_logit_rules(lx, row_offsets=off, out=out, **live)
    for k in (1, 2, 3, 0):
        for n in ARGS:
            live[n].copy_(cases[k][n])
        lx.copy_(x[k])
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        w, tol = want(cases[k], x[k])
        compare(out, w, tol)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_an_infinite_frequency_bans_what_was_generated_and_that_alone(dtype):
    # c = 0 takes no part in frequency * c: tokens of the prompt keep what the repetition makes of them
    V, off = 70, torch.tensor([0, 2], dtype=torch.int32).cuda()
    history = torch.tensor([[3, 5, 5, 9, 11, -1, V, 69]], dtype=torch.int32).cuda()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()
    f32 = lambda *v: torch.tensor(v).cuda()
    x = torch.randn((2, V), generator=torch.Generator().manual_seed(1)).to(dtype)
    x[:, 3], x[:, 5], x[:, 9], x[0, 40] = 2.0, -3.0, -math.inf, math.inf
    for sign in (1.0, -1.0):
        r = _ds().dspark_logit_rules(x.cuda(), row_offsets=off, history=history, history_len=i32(8), prompt_len=i32(4),
                                     drafts=i32(20).reshape(1, 1), repetition=f32(2.0), frequency=f32(sign * math.inf),
                                     presence=f32(0.5)).cpu()
        for j in range(2):
            for t in range(V):
                z = float(x[j, t])
                if t in (3, 5, 9):
                    z = z / 2 if z > 0 else z * 2
                if t in (11, 69) or (t == 20 and j == 1):
                    z = -sign * math.inf
                assert float(r[j, t]) == z, (j, t, float(r[j, t]), z)


def _bias_call(V, B, ids, values, dtype=BF):
    n = ids.numel()
    off = (torch.arange(B + 1) * n).to(torch.int32).cuda()
    dev = ids.repeat(B).cuda(), values.repeat(B).cuda()
    x = torch.zeros((B, V), dtype=dtype, device="cuda")
    return lambda: _ds().dspark_logit_rules(x, bias_offsets=off, bias_ids=dev[0], bias_values=dev[1])


@pytest.mark.parametrize("V,B,text", [(2500, 2, 0), (2500, 2, 30000), (160000, 10, 0), (160000, 10, 20000)])
@pytest.mark.parametrize("kinds", [1, 2, 40, 2000])
def test_biases_of_few_tokens_are_added_in_the_order_of_their_list(V, B, text, kinds):
    # of each choice of the slices; the repeated ones lie in one part of the list, in several, and next to each other
    g = torch.Generator().manual_seed(kinds)
    n = 3001
    names = torch.randperm(V, generator=g)[:kinds]
    ids = names[torch.randint(0, kinds, (n,), generator=g)].to(torch.int32)
    ids[1000:1100], ids[5::97], ids[7::89] = int(names[0]), -1, V
    values = torch.randn(n, generator=g) * torch.exp(3 * torch.randn(n, generator=g))
    want = torch.zeros(V)
    for t, x in zip(ids.tolist(), values):
        if 0 <= t < V:
            want[t] = want[t] + x
    off = (torch.arange(B + 1) * n).to(torch.int32).cuda()
    kw = {} if not text else dict(history=torch.zeros((B, text), dtype=torch.int32, device="cuda"),
                                  history_len=torch.zeros(B, dtype=torch.int32, device="cuda"))
    r = _ds().dspark_logit_rules(torch.zeros((B, V), device="cuda"), bias_offsets=off, bias_ids=ids.repeat(B).cuda(),
                                 bias_values=values.repeat(B).cuda(), **kw).cpu()
    for b in range(B):
        assert torch.equal(r[b], want)


def test_a_list_of_one_token_takes_about_as_long_as_one_of_many():
    # a repeated token costs a pass over its part of the list, not a turn of the workgroup for each of its entries
    V, n = 1000, 16384
    g = torch.Generator().manual_seed(3)

    def us(ids):
        call = _bias_call(V, 1, ids.to(torch.int32), torch.ones(n))
        best = math.inf
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            call()
            b.record()
            torch.cuda.synchronize()
            best = min(best, 1000 * a.elapsed_time(b))
        return best

    many, one = us(torch.randint(0, V, (n,), generator=g) + V), us(torch.full((n,), 17))  # (ids past V: the scan alone)
    print(f"biases: {n} of other tokens {many:.0f} us, of one token {one:.0f} us", flush=True)
    # 64 parts of the list.  The scan of one: an exchange and two loads; its sums: at most 64 steps of two LDS reads and
    # four sums beside that, 2 us at 2 GHz.  One entry a turn instead is 16384 turns of three barriers, more than 2 ms.
    assert one < 8 * many + 200
