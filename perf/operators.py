"""The attention operators around a draft-and-verify round, as workloads.

The target forward of a round attends, for every request, from its 1 + ell_b
rows (the anchor and the drafts) over that request's key-value cache; a prompt
attends over itself; the cache is paged and may be held in 8 bits.  Four
operators: writing rows into the paged cache, reading rows back out of it,
attention of a few new rows a request over it, and causal attention over
whole packed prompts.

Each case runs either in its plain form (elementary torch operations in 32
bits) or, where ``own`` is true, through the library's entry points.

The 8-bit cache holds e4m3 values with one power-of-two scale for each (token,
head): the smallest 2^e, e >= -126, with max|x| <= 448 * 2^e.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
DEV = "cuda"
E4M3_MAX = 448.0


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decoding step of a moderate batch: one new row a request goes into the cache (latency)
        dict(name="write_decode", op="write", B=64, lo=1, hi=1, past=4096, Hkv=8, D=128, page=16,
             dtype="bf16", cache="bf16", shape=1),
        # a verify step at the headline batch: 1 + ell rows a request, ell up to 5, quantised and read back
        dict(name="write_verify_e4m3", op="write", B=256, lo=1, hi=6, past=2048, Hkv=8, D=128, page=16,
             dtype="bf16", cache="e4m3", shape=2),
        # prompts of ragged lengths enter an 8-bit cache and are read back
        dict(name="write_prompts_e4m3", op="write", B=9, lo=100, hi=8001, past=0, Hkv=8, D=128, page=64,
             dtype="bf16", cache="e4m3", shape=3),
        # a few short cached prefixes are gathered for requests that share them (latency)
        dict(name="read_short_e4m3", op="read", B=3, lo=1, hi=130, past=0, Hkv=4, D=64, page=32,
             dtype="f16", cache="e4m3", shape=4),
        # long cached prefixes are gathered to be continued by a prompt pass
        dict(name="read_prefixes", op="read", B=16, lo=1, hi=16001, past=0, Hkv=8, D=128, page=16,
             dtype="bf16", cache="bf16", shape=5),
        # one request, one new token, a short cache: the smallest step there is
        dict(name="decode_one", op="paged", B=1, lo=1, hi=1, past_lo=500, past=520, Hq=32, Hkv=8, D=128, page=16,
             dtype="bf16", cache="bf16", shape=6),
        # one new token for each request of the headline batch, ragged caches
        dict(name="decode_batch", op="paged", B=256, lo=1, hi=1, past_lo=16, past=8192, Hq=32, Hkv=8, D=128, page=16,
             dtype="bf16", cache="bf16", shape=7),
        # a few requests with very long 8-bit caches
        dict(name="decode_long_e4m3", op="paged", B=4, lo=1, hi=1, past_lo=60000, past=131000, Hq=64, Hkv=8, D=128,
             page=64, dtype="bf16", cache="e4m3", shape=8),
        # the verify forward of the headline batch: 1 + ell rows a request, ell up to 5
        dict(name="verify_batch", op="paged", B=256, lo=1, hi=6, past_lo=16, past=4096, Hq=32, Hkv=8, D=128, page=16,
             dtype="bf16", cache="bf16", shape=9),
        # short packed prompts, float16, narrow heads
        dict(name="prompts_short", op="prompt", B=32, lo=1, hi=200, prefix=0, Hq=16, Hkv=4, D=64, dtype="f16",
             shape=10),
        # an ordinary packed batch of prompts
        dict(name="prompts_packed", op="prompt", B=16, lo=100, hi=4100, prefix=0, Hq=32, Hkv=8, D=128, dtype="bf16",
             shape=11),
        # one long prompt
        dict(name="prompt_long", op="prompt", B=1, lo=16384, hi=16384, prefix=0, Hq=32, Hkv=8, D=128, dtype="bf16",
             shape=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "paged", "paged", "prompt", "prompt"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    c = dict(op=op, Hkv=Hkv, D=D, dtype=dtype, shape=rng.randrange(1 << 30))
    if op == "prompt":
        c["Hq"] = Hkv * rng.choice([1, 2, 3, 4, 8])
        hi = _log_int(rng, 1, 8000)
        c["B"] = _log_int(rng, 1, max(1, min(64, 16000 // hi)))
        c["lo"] = rng.choice([1, hi])
        c["hi"] = hi
        c["prefix"] = rng.choice([0, 0, _log_int(rng, 1, 4000)])  # cached tokens in front of the rows
        # keep a drawn case below the largest listed one
        while c["B"] * c["Hq"] * c["D"] * c["hi"] * (c["hi"] / 2 + c["prefix"]) > 4.0e11:
            c["hi"] = max(1, c["hi"] // 2)
            c["lo"] = min(c["lo"], c["hi"])
        return c
    c["cache"] = rng.choice([dtype, "e4m3"])
    c["page"] = rng.choice([16, 32, 64, 128])
    row_bytes = Hkv * D * 4
    if op == "paged":
        c["Hq"] = Hkv * rng.choice([1, 2, 3, 4, 8, 16])
        c["lo"], c["hi"] = 1, rng.choice([1, 1, 1, 5, 6, 9, 17])
        c["B"] = _log_int(rng, 1, 300)
        c["past"] = _log_int(rng, 1, max(1, min(131000, int(4.0e9 / row_bytes / c["B"]))))
        c["past_lo"] = rng.choice([0, c["past"] // 2])
        return c
    c["B"] = _log_int(rng, 1, 256)
    c["lo"], c["hi"] = 1, _log_int(rng, 1, max(1, min(16000, int(1.0e9 / row_bytes / c["B"]))))
    c["past"] = _log_int(rng, 1, 4000) if op == "write" else 0
    return c


# -------------------------------------------------------- lengths and layouts

def _lengths(case):
    """(rows, past) of every request: fixed by the case."""
    r = random.Random(case["shape"])
    rows = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    if case["op"] == "prompt":
        past = [r.randint(0, case["prefix"]) for _ in rows]
    else:
        past = [r.randint(case.get("past_lo", 0), case["past"]) for _ in rows]
    return rows, past


def _offsets(lens):
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    return off


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _values(g, shape, dtype, std=1.0):
    """Normal values with a few loud channels, as keys and values have."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
    loud = torch.exp(0.3 * torch.randn(shape[-1], generator=g, device=DEV))
    return (x * (std * loud)).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    rows, past = _lengths(case)
    B, Hkv, D, dt = case["B"], case["Hkv"], case["D"], DTYPES[case["dtype"]]
    off = _offsets(rows)
    N = off[-1]
    st = dict(case=case, rows=rows, past=past, off=off, offsets=_i32(off), N=N)
    if case["op"] == "prompt":
        Hq = case["Hq"]
        kv_off = _offsets([r + p for r, p in zip(rows, past)])
        st["kv_off"], st["same"] = kv_off, not any(past)
        st["kv_offsets"] = _i32(kv_off)
        if st["same"]:
            # q, k, v as a fused projection leaves them: slices of one row
            qkv = _values(g, (N, Hq + 2 * Hkv, D), dt)
            st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        else:
            st["q"] = _values(g, (N, Hq, D), dt)
            kv = _values(g, (kv_off[-1], 2 * Hkv, D), dt)
            st["k"], st["v"] = kv[:, :Hkv], kv[:, Hkv:]
        return st
    ps = case["page"]
    total = [r + p for r, p in zip(rows, past)]
    need = [-(-t // ps) for t in total]
    width = max(need) + 1
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device=DEV).tolist()
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (width - n))
        at += n
    st["page_table"] = _i32(table)
    st["cache_len"] = _i32(past)
    shape = (n_pages, Hkv, ps, D)
    if case["op"] == "write":
        kv = _values(g, (N, 2 * Hkv, D), dt)
        st["k"], st["v"] = kv[:, :Hkv], kv[:, Hkv:]
    else:
        k, v = _values(g, shape, dt), _values(g, shape, dt)
        if case["cache"] == "e4m3":
            st["k_cache"], st["k_scale"] = _quantise(k)
            st["v_cache"], st["v_scale"] = _quantise(v)
        else:
            st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"] = k, v, None, None
    if case["op"] == "write":
        e4 = case["cache"] == "e4m3"
        for n in ("k", "v"):
            st[n + "_cache"] = torch.zeros(shape, dtype=torch.float8_e4m3fn if e4 else dt, device=DEV)
            st[n + "_scale"] = torch.zeros(shape[:3], dtype=torch.uint8, device=DEV) if e4 else None
    if case["op"] == "paged":
        st["q"] = _values(g, (N, case["Hq"], D), dt)
    return st


# ------------------------------------------------------------ the plain forms

def _quantise(x):
    """e4m3 values and the byte e + 127 of their scale, over the last axis."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))  # amax = m 2^e, m in [1/2, 1)
    e = torch.where(m <= 0.875, e - 9, e - 8)  # 448 = 0.875 * 2^9
    e = torch.where(m == 0, torch.full_like(e, -126), e).clamp(min=-126)
    q = torch.ldexp(x, -e.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q, (e + 127).to(torch.uint8)


def _dequantise(q, s):
    x = q.float()
    return x if s is None else torch.ldexp(x, (s.to(torch.int32) - 127).unsqueeze(-1))


def _places(st, rows_at):
    """Page and slot of every row; rows_at is the position of each request's first row."""
    i = torch.arange(st["N"], device=DEV, dtype=torch.int32)
    b = torch.searchsorted(st["offsets"][1:], i, right=True)
    pos = (i - st["offsets"][b] + rows_at[b]).long()
    ps = st["case"]["page"]
    return st["page_table"][b, pos // ps].long(), pos % ps


def _plain_write(st):
    page, slot = _places(st, st["cache_len"])
    for n in ("k", "v"):
        x, scale = st[n], st[n + "_scale"]
        if scale is not None:
            x, s = _quantise(x)
            scale[page, :, slot] = s
            st[n + "_cache"].view(torch.uint8)[page, :, slot] = x.view(torch.uint8)
        else:
            st[n + "_cache"][page, :, slot] = x


def _plain_read(st, rows_at):
    page, slot = _places(st, rows_at)
    dt = DTYPES[st["case"]["dtype"]]
    out = {}
    for n in ("k", "v"):
        cache, scale = st[n + "_cache"], st[n + "_scale"]
        if scale is None:
            out[n] = cache[page, :, slot]
        else:
            q = cache.view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn)
            x = _dequantise(q, scale[page, :, slot])
            top = torch.finfo(dt).max
            out[n] = x.clamp(-top, top).to(dt)
    return out


def _attend(q, k, v, first, scale):
    """q [R, Hq, D] at positions first, first + 1, ... over k, v [L, Hkv, D] in float32."""
    R, Hq, D = q.shape
    L, Hkv = k.shape[:2]
    qh = q.transpose(0, 1).reshape(Hkv, Hq // Hkv * R, D).contiguous()
    kt = k.permute(1, 2, 0).contiguous()
    s = torch.matmul(qh, kt).view(Hkv, Hq // Hkv, R, L) * scale
    hidden = torch.arange(L, device=DEV)[None, :] > first + torch.arange(R, device=DEV)[:, None]
    s = s.masked_fill(hidden, float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(Hkv, -1, L), v.transpose(0, 1).contiguous()).view(Hkv, -1, R, D) / l
    return o.reshape(Hq, R, D).transpose(0, 1), (m + torch.log(l)).view(Hq, R).t()


def _plain_paged(st):
    c = st["case"]
    ps, scale = c["page"], 1.0 / math.sqrt(c["D"])
    out = torch.empty_like(st["q"])
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float32, device=DEV)
    for b in range(c["B"]):
        r0, r1, L = st["off"][b], st["off"][b + 1], st["past"][b] + st["rows"][b]
        pages = st["page_table"][b, :-(-L // ps)].long()
        kv = []
        for n in ("k", "v"):
            x, s = st[n + "_cache"].view(torch.uint8)[pages].view(st[n + "_cache"].dtype), st[n + "_scale"]
            x = _dequantise(x, None if s is None else s[pages])
            kv.append(x.transpose(1, 2).reshape(-1, c["Hkv"], c["D"])[:L])
        o, z = _attend(st["q"][r0:r1].float(), kv[0], kv[1], st["past"][b], scale)
        out[r0:r1] = o.to(out.dtype)
        lse[r0:r1] = z
    return {"out": out, "lse": lse}


_CHUNK = 1 << 28  # scores held at once


def _plain_prompt(st):
    c = st["case"]
    scale = 1.0 / math.sqrt(c["D"])
    out = torch.empty(st["q"].shape, dtype=st["q"].dtype, device=DEV)
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float32, device=DEV)
    for b in range(c["B"]):
        r0, r1 = st["off"][b], st["off"][b + 1]
        k0, k1 = st["kv_off"][b], st["kv_off"][b + 1]
        k, v = st["k"][k0:k1].float(), st["v"][k0:k1].float()
        step = max(1, _CHUNK // (c["Hq"] * (k1 - k0)))
        for a in range(r0, r1, step):
            e = min(r1, a + step)
            first = st["past"][b] + a - r0
            seen = first + e - a  # keys past the last row of the chunk take no part
            o, z = _attend(st["q"][a:e].float(), k[:seen], v[:seen], first, scale)
            out[a:e] = o.to(out.dtype)
            lse[a:e] = z
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------------ run

def _first_rows(st):
    """Read cases start at position 0; rows just written start behind the past."""
    if st["case"]["op"] == "write":
        return st["cache_len"]
    if "zero" not in st:
        st["zero"] = torch.zeros_like(st["cache_len"])
    return st["zero"]


def run(state):
    st, c = state, state["case"]
    if own:
        import draft_sampling_verification_02_amd as ds
        if c["op"] == "prompt":
            r = ds.dspark_prompt_attention(st["q"], st["k"], st["v"], st["offsets"],
                                           kv_offsets=None if st["same"] else st["kv_offsets"], lse=True,
                                           out=st.get("res"))
            st["res"] = r
            return {"out": r["out"], "lse": r["lse"]}
        scales = dict(k_scale=st["k_scale"], v_scale=st["v_scale"])
        if c["op"] == "paged":
            r = ds.dspark_paged_attention(st["q"], st["k_cache"], st["v_cache"], st["cache_len"], st["page_table"],
                                          row_offsets=None if c["hi"] == 1 else st["offsets"],
                                          max_rows=c["hi"], lse=True, out=st.get("res"), **scales)
            st["res"] = r
            return {"out": r["out"], "lse": r["lse"]}
        if c["op"] == "write":
            ds.dspark_kv_write(st["k"], st["v"], st["k_cache"], st["v_cache"], st["cache_len"], st["page_table"],
                               row_offsets=None if c["hi"] == 1 else st["offsets"], **scales)
            if c["cache"] != "e4m3":
                return {"k": st["k_cache"], "v": st["v_cache"]}
        r = ds.dspark_kv_read(st["k_cache"], st["v_cache"], st["page_table"], st["N"], row_offsets=st["offsets"],
                              first=_first_rows(st), dtype=DTYPES[c["dtype"]], out=st.get("res"), **scales)
        st["res"] = r
        return {"k": r["k"], "v": r["v"]}
    if c["op"] == "prompt":
        return _plain_prompt(st)
    if c["op"] == "paged":
        return _plain_paged(st)
    if c["op"] == "write":
        _plain_write(st)
        if c["cache"] != "e4m3":
            return {"k": st["k_cache"], "v": st["v_cache"]}
    # an 8-bit cache is judged by the values it stands for: the rows just written, read back
    return _plain_read(st, _first_rows(st))


def work(case):
    rows, past = _lengths(case)
    N, Hkv, D = sum(rows), case["Hkv"], case["D"]
    index = 4 * (case["B"] + 1)
    if case["op"] == "prompt":
        Hq = case["Hq"]
        pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(rows, past))
        keys = N + sum(past)
        return {"bytes": N * Hq * D * 2 * 2 + keys * Hkv * D * 2 * 2 + N * Hq * 4 + index,
                "flops": 4 * pairs * Hq * D}
    elt = D + 1 if case["cache"] == "e4m3" else 2 * D  # bytes of one (token, head)
    if case["op"] == "paged":
        Hq = case["Hq"]
        keys = sum(n + p for n, p in zip(rows, past))
        pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(rows, past))
        table = 4 * sum(-(-(n + p) // case["page"]) for n, p in zip(rows, past))
        return {"bytes": keys * Hkv * elt * 2 + N * Hq * D * 2 * 2 + N * Hq * 4 + table + 2 * index,
                "flops": 4 * pairs * Hq * D}
    moved = 2 * N * Hkv * (2 * D + elt) + 2 * index  # rows in one type read, in the other written
    if case["op"] == "write" and case["cache"] == "e4m3":
        moved *= 2  # and read back
    return {"bytes": moved, "flops": 0}


# ------------------------------------------------- the definitions in 64 bits

def _exact_round(x, top):
    """x to the nearest e4m3 value times a power of two, over the last axis, in 64 bits."""
    amax = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -140) / E4M3_MAX))
    e = torch.where(amax > E4M3_MAX * torch.exp2(e), e + 1, e)
    e = torch.where(amax <= E4M3_MAX * torch.exp2(e - 1), e - 1, e).clamp(min=-126.0)
    y = x * torch.exp2(-e)
    f = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))  # exponent, subnormals at -6
    step = torch.exp2(f - 3)
    return (torch.round(y / step) * step * torch.exp2(e)).clamp(-top, top)


def _exact_softmax(q, k, v, first, scale):
    """One key-value head: q [R, G, D], k and v [L, D], all float64."""
    R, G, D = q.shape
    s = (q.reshape(R * G, D) @ k.t().contiguous()).view(R, G, -1) * scale
    at = torch.arange(k.shape[0], device=q.device)
    s = torch.where((at[None, :] <= first + torch.arange(R, device=q.device)[:, None])[:, None, :], s, -math.inf)
    z = torch.logsumexp(s, -1)
    return (torch.exp(s - z[..., None]).view(R * G, -1) @ v).view(R, G, D), z


def exact(case, seed):
    st = prepare(case, seed)
    rows, past, Hkv, D, dt = st["rows"], st["past"], case["Hkv"], case["D"], DTYPES[case["dtype"]]
    top = torch.finfo(dt).max
    if case["op"] in ("write", "read"):
        if case["op"] == "write" and case["cache"] != "e4m3" and st["N"] > 2000:
            return None  # row by row: too slow for many rows
        ps = case["page"]
        out = {}
        for n in ("k", "v"):
            if case["op"] == "write" and case["cache"] == "e4m3":
                out[n] = _exact_round(st[n].double(), top)
            elif case["op"] == "write":
                x = st[n + "_cache"].double()
                for b, (r, p) in enumerate(zip(rows, past)):
                    for i in range(r):
                        page = int(st["page_table"][b, (p + i) // ps])
                        x[page, :, (p + i) % ps] = st[n][st["off"][b] + i].double()
                out[n] = x
            else:
                parts = []
                for b, r in enumerate(rows):
                    pages = st["page_table"][b, :(r + ps - 1) // ps].long()
                    parts.append(_exact_gather(st, n, pages)[:r].clamp(-top, top))
                out[n] = torch.cat(parts)
        return out
    Hq = case["Hq"]
    G, scale = Hq // Hkv, 1.0 / math.sqrt(D)
    out = torch.empty((st["N"], Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.empty((st["N"], Hq), dtype=torch.float64, device=DEV)
    for b, (r, p) in enumerate(zip(rows, past)):
        r0, L = st["off"][b], r + p
        if case["op"] == "prompt":
            k, v = (st[n][st["kv_off"][b]:st["kv_off"][b + 1]].double() for n in ("k", "v"))
        else:
            pages = st["page_table"][b, :(L + case["page"] - 1) // case["page"]].long()
            k, v = (_exact_gather(st, n, pages)[:L] for n in ("k", "v"))
        step = max(1, (1 << 27) // (G * L))
        for h in range(Hkv):
            kh, vh = k[:, h].contiguous(), v[:, h].contiguous()
            for a in range(0, r, step):
                e = min(r, a + step)
                o, z = _exact_softmax(st["q"][r0 + a:r0 + e, h * G:(h + 1) * G].double(), kh, vh, p + a, scale)
                out[r0 + a:r0 + e, h * G:(h + 1) * G] = o
                lse[r0 + a:r0 + e, h * G:(h + 1) * G] = z
    return {"out": out, "lse": lse}


def _exact_gather(st, n, pages):
    cache = st[n + "_cache"]
    if cache.dtype == torch.float8_e4m3fn:
        x = cache.view(torch.uint8)[pages].view(torch.float8_e4m3fn).to(torch.float32).double()
        x = x * torch.exp2(st[n + "_scale"][pages].double() - 127.0)[..., None]
    else:
        x = cache[pages].double()
    return x.permute(0, 2, 1, 3).reshape(-1, x.shape[1], x.shape[3])
