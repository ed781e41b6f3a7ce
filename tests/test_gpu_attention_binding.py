"""The binding's two ways into the cache and attention entry points -- the
compiled marshalling module, and the checks in Python that word the errors --
accept the same calls, refuse the same calls and give the same results."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, FH, E4, I32 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.int32


def _ds():
    import draft_sampling_verification_02_amd as ds
    ds.load_library()
    return ds


def _t(*shape, dtype=BF, seed=1):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) if dtype.is_floating_point else torch.zeros(shape)
    return x.to(dtype).cuda()


def _i(*values, dtype=I32):
    return torch.tensor(values, dtype=dtype, device="cuda")


# a call of each entry point that takes the short way: its arguments
def _cache():
    return dict(k_cache=_t(9, 2, 16, 64), v_cache=_t(9, 2, 16, 64, seed=2), page_table=torch.arange(9, dtype=I32, device="cuda").view(3, 3))


def _write():
    return dict(k=_t(3, 2, 64), v=_t(3, 2, 64, seed=3), cache_len=_i(0, 5, 16), **_cache())


def _read():
    return dict(n_rows=3, dtype=BF, first=_i(0, 5, 16), out={"k": _t(3, 2, 64), "v": _t(3, 2, 64)}, **_cache())


def _results(q, workspace_bytes):
    return {"out": torch.zeros_like(q), "lse": torch.zeros(q.shape[:2], device="cuda"),
            "workspace": torch.empty(workspace_bytes, dtype=torch.uint8, device="cuda")}


def _paged():
    q = _t(3, 4, 64)
    return dict(q=q, cache_len=_i(0, 5, 16), out=_results(q, _ds().dspark_paged_attention_workspace_size(1, 4, 2, 64)), **_cache())


def _prompt():
    q = _t(3, 4, 64)
    return dict(q=q, k=_t(3, 2, 64), v=_t(3, 2, 64, seed=3), row_offsets=_i(0, 1, 3),
                out=_results(q, _ds().dspark_prompt_attention_workspace_size(2, 3, 3, 4, 2, 64)))


CALLS = {"dspark_kv_write": _write, "dspark_kv_read": _read, "dspark_paged_attention": _paged, "dspark_prompt_attention": _prompt}

# changes to the arguments, made one at a time; a function takes the arguments it changes
ROWS = {
    "float32": lambda: _t(3, 2, 64, dtype=torch.float32), "8 bits": lambda: _t(3, 2, 64, dtype=E4), "heads": lambda: _t(3, 3, 64),
    "head size": lambda: _t(3, 2, 128), "fewer rows": lambda: _t(2, 2, 64), "transposed": lambda: _t(3, 64, 2).transpose(1, 2),
    "every other channel": lambda: _t(3, 2, 128)[:, :, ::2], "every other head": lambda: _t(3, 4, 64)[:, ::2],
    "two dimensions": lambda: _t(3, 128), "none": lambda: None, "host": lambda: _t(3, 2, 64).cpu(), "no rows": lambda: _t(0, 2, 64),
    "broadcast": lambda: _t(1, 2, 64).expand(3, 2, 64), "unaligned": lambda: _t(3 * 128 + 1)[1:].view(3, 2, 64),
    "of wider rows": lambda: _t(3, 5, 64)[:, 1:3], "float16": lambda: _t(3, 2, 64, dtype=FH),
}
INTS = {"none": lambda: None, "longer": lambda: _i(0, 1, 2, 3, 3), "shorter": lambda: _i(0, 1), "int64": lambda: _i(0, 1, 2, dtype=torch.int64),
        "host": lambda: _i(0, 1, 2).cpu(), "every other": lambda: _i(0, 0, 1, 1, 2, 2)[::2], "list": lambda: [0, 1, 2], "four": lambda: _i(0, 1, 2, 3)}
SCALES = {"none": lambda: None, "uint8": lambda: torch.full((9, 2, 16), 120, dtype=torch.uint8, device="cuda"),
          "shape": lambda: _t(9, 2, 8, dtype=torch.uint8), "bfloat16": lambda: _t(9, 2, 16), "host": lambda: _t(9, 2, 16, dtype=torch.uint8).cpu()}
CACHES = {
    "none": lambda: None, "float32": lambda: _t(9, 2, 16, 64, dtype=torch.float32), "float16": lambda: _t(9, 2, 16, 64, dtype=FH),
    "page size": lambda: _t(9, 2, 32, 64), "transposed": lambda: _t(9, 16, 2, 64).transpose(1, 2), "three dimensions": lambda: _t(9, 2, 64),
    "host": lambda: _t(9, 2, 16, 64).cpu(), "heads": lambda: _t(9, 3, 16, 64), "8 bits": lambda: _t(9, 2, 16, 64, dtype=E4),
}
TABLES = {"none": lambda: None, "int64": lambda: _t(3, 3, dtype=torch.int64), "one dimension": lambda: _t(9, dtype=I32),
          "fewer requests": lambda: _t(2, 3, dtype=I32), "every other page": lambda: _t(3, 6, dtype=I32)[:, ::2],
          "host": lambda: _t(3, 3, dtype=I32).cpu(), "no pages": lambda: _t(3, 0, dtype=I32)}
OUTPUTS = {"none": lambda: None, "head size": lambda: _t(3, 4, 32), "float32": lambda: _t(3, 4, 64, dtype=torch.float32),
           "every other head": lambda: _t(3, 8, 64)[:, ::2], "host": lambda: _t(3, 4, 64).cpu(), "float16": lambda: _t(3, 4, 64, dtype=FH),
           "like k and v": lambda: _t(3, 2, 64)}
LSES = {"bfloat16": lambda: _t(3, 4), "shape": lambda: _t(3, 5, dtype=torch.float32), "host": lambda: torch.zeros(3, 4)}
WORKSPACES = {"float32": lambda: _t(1 << 20, dtype=torch.float32), "number": lambda: 4096, "host": lambda: torch.zeros(1 << 22, dtype=torch.uint8),
              "unaligned": lambda: torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")[1:]}
VALUES = {"scale": [0.3, 1, 0.0, -1.0, float("nan"), 3e38, 1e39, "x"], "causal": [False, 0, 1], "max_rows": [1, 0, -1, 40, "x"]}


def _eight_bits(a):
    a.update(k_cache=a["k_cache"].to(E4), v_cache=a["v_cache"].to(E4), k_scale=SCALES["uint8"](), v_scale=SCALES["uint8"]())


def _changes(name):
    """[(words, function that changes the arguments)]"""
    out = [("none", lambda a: None)]

    def single(arg, kinds):
        out.extend((f"{arg}: {w}", lambda a, m=m: a.update({arg: m()})) for w, m in kinds.items())

    def result(arg, kinds):
        out.extend((f"out[{arg}]: {w}", lambda a, m=m: a["out"].update({arg: m()})) for w, m in kinds.items())

    if name != "dspark_kv_read":
        for arg in ("q",) if name == "dspark_paged_attention" else ("k", "v") if name == "dspark_kv_write" else ("q", "k", "v"):
            single(arg, ROWS)
    if name != "dspark_prompt_attention":
        single("k_cache", CACHES)
        single("v_cache", CACHES)
        single("page_table", TABLES)
        single("row_offsets", INTS)
        single("first" if name == "dspark_kv_read" else "cache_len", INTS)
        single("k_scale", SCALES)
        out.extend((f"both caches: {w}", lambda a, m=m: a.update(k_cache=m(), v_cache=m())) for w, m in CACHES.items())
        out.append(("8-bit cache", _eight_bits))
        for arg in ("k_scale", "v_scale"):
            out.extend((f"8-bit cache, {arg}: {w}", lambda a, arg=arg, m=m: (_eight_bits(a), a.update({arg: m()})))
                       for w, m in SCALES.items())
    else:
        single("row_offsets", INTS)
        single("kv_offsets", INTS)
    if name == "dspark_kv_read":
        result("k", OUTPUTS)
        result("v", OUTPUTS)
        out.extend((f"dtype: {d}", lambda a, d=d: a.update(dtype=d)) for d in (None, FH, E4, torch.float32))
        out.extend((f"n_rows: {n}", lambda a, n=n: a.update(n_rows=n)) for n in (2, 4, 0))
    elif name != "dspark_kv_write":
        result("out", OUTPUTS)
        result("lse", LSES)
        result("workspace", WORKSPACES)
        for arg in ("scale", "causal") + (("max_rows",) if name == "dspark_paged_attention" else ()):
            out.extend((f"{arg}: {x}", lambda a, arg=arg, x=x: a.update({arg: x})) for x in VALUES[arg])
    return out


def _outcome(name, change, stream):
    a = CALLS[name]()
    change(a)
    try:
        r = getattr(_ds(), name)(**a, stream=stream)
    except Exception as e:  # noqa: BLE001 -- what is raised is what is compared
        return "refused", type(e), str(e)
    torch.cuda.synchronize()
    tensors = [a[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale") if a.get(n) is not None]
    tensors += [r[n] for n in ("k", "v", "out", "lse") if r is not None and r.get(n) is not None]
    return "done", [t.cpu().contiguous().view(torch.uint8) for t in tensors]


@pytest.mark.parametrize("name", list(CALLS))
def test_both_ways_refuse_and_accept_alike(name):
    done = refused = 0
    for words, change in _changes(name):
        print(f"{name}: {words}", flush=True)
        short = _outcome(name, change, None)
        long = _outcome(name, change, torch.cuda.current_stream())
        assert short[0] == long[0], (words, short, long)
        if short[0] == "refused":
            refused += 1
            assert short[1:] == long[1:], (words, short, long)
        else:
            done += 1
            assert len(short[1]) == len(long[1]) and all(torch.equal(x, y) for x, y in zip(short[1], long[1])), words
    assert done >= 4 and refused >= 20, (done, refused)


@pytest.mark.parametrize("name", list(CALLS))
def test_a_plain_call_takes_the_short_way(name, monkeypatch):
    ds = _ds()
    a = CALLS[name]()

    def long_way(*args):
        raise AssertionError("the call went the long way")

    monkeypatch.setattr(ds, "_call_on", long_way)
    getattr(ds, name)(**a)
    torch.cuda.synchronize()
    with pytest.raises(AssertionError, match="long way"):
        getattr(ds, name)(**a, stream=torch.cuda.current_stream())
