"""The binding's two ways into rotation, cache append, windowed attention and logit
rules accept the same calls, refuse the same calls and give the same results."""
import pytest
import torch

from test_gpu_attention_binding import CACHES, INTS, LSES, OUTPUTS, ROWS, SCALES, TABLES, WORKSPACES, _cache, _ds, _eight_bits, _i, _results, _t

pytestmark = pytest.mark.gpu

BF, FH, E4, I32, F32 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.int32, torch.float32


def _f(n):
    return torch.linspace(0.01, 1.0, n, device="cuda")


def _rotary():
    return dict(q=_t(3, 4, 64), k=_t(3, 2, 64), inv_freq=_f(32), first=_i(0, 5, 16), q_norm=_t(64), k_norm=_t(64, seed=4),
                out={"q": _t(3, 4, 64), "k": _t(3, 2, 64)})


def _append():
    return dict(q=_t(3, 4, 64), k=_t(3, 2, 64), v=_t(3, 2, 64, seed=3), inv_freq=_f(32), cache_len=_i(0, 5, 16),
                out={"q": _t(3, 4, 64)}, **_cache())


def _window():
    q = _t(3, 4, 64)
    return dict(q=q, cache_len=_i(0, 5, 16), window=9, sinks=2,
                out=_results(q, _ds().dspark_window_attention_workspace_size(1, 4, 2, 64)), **_cache())


def _rules():
    return dict(logits=_t(3, 70), history=_t(3, 9, dtype=I32), history_len=_i(9, 0, 5), drafts=_t(3, 2, dtype=I32),
                repetition=_f(3), bias_offsets=_i(0, 1, 2, 2), bias_ids=_i(4, 69), bias_values=_f(2),
                masks=_t(2, 3, dtype=I32), mask_index=_i(1, -1, 0), out=torch.zeros(3, 70, device="cuda"))


CALLS = {"dspark_rotary": _rotary, "dspark_kv_append": _append, "dspark_window_attention": _window, "dspark_logit_rules": _rules}
HEADS = {**ROWS, "as q": lambda: _t(3, 4, 64), "q of float32": lambda: _t(3, 4, 64, dtype=F32), "q's wider rows": lambda: _t(3, 9, 64)[:, 1:5]}
FREQS = {"none": lambda: None, "bfloat16": lambda: _t(32), "sixteen": lambda: _f(16), "odd": lambda: _f(5), "too many": lambda: _f(40),
         "host": lambda: _f(32).cpu(), "two dimensions": lambda: _f(32)[None], "number": lambda: 3.0, "every other": lambda: _f(64)[::2]}
NORMS = {"none": lambda: None, "float32": lambda: _f(64), "float16": lambda: _t(64, dtype=FH), "short": lambda: _t(32), "host": lambda: _t(64).cpu()}
PLANES = {"none": lambda: None, "int64": lambda: _t(3, 9, dtype=torch.int64), "lines": lambda: _t(4, 9, dtype=I32), "flat": lambda: _t(9, dtype=I32),
          "host": lambda: _t(3, 9, dtype=I32).cpu(), "every other": lambda: _t(3, 18, dtype=I32)[:, ::2], "empty": lambda: _t(3, 0, dtype=I32),
          "wide": lambda: _t(3, 40, dtype=I32)}
FLOATS = {"none": lambda: None, "double": lambda: _f(3).double(), "longer": lambda: _f(4), "host": lambda: _f(3).cpu()}
MATRICES = {"none": lambda: None, "float32": lambda: _t(3, 70, dtype=F32), "float16": lambda: _t(3, 70, dtype=FH), "double": lambda: _t(3, 70).double(),
            "rows": lambda: _t(4, 70), "wider rows": lambda: _t(3, 80)[:, :70], "wider float32 rows": lambda: _t(3, 81, dtype=F32)[:, 2:72],
            "transposed": lambda: _t(70, 3).t(), "host": lambda: _t(3, 70).cpu(), "flat": lambda: _t(210), "one": lambda: _t(1, 70)}


def _changes(name):
    out = [("none", lambda a: None)]

    def single(arg, kinds):
        out.extend((f"{arg}: {w}", lambda a, m=m: a.update({arg: m()})) for w, m in kinds.items())

    def result(arg, kinds):
        out.extend((f"out[{arg}]: {w}", lambda a, m=m: a["out"].update({arg: m()})) for w, m in kinds.items())

    if name == "dspark_logit_rules":
        single("logits", MATRICES)
        single("out", MATRICES)
        single("row_offsets", INTS)
        for arg in ("history", "drafts", "masks"):
            single(arg, PLANES)
        for arg in ("history_len", "prompt_len", "mask_index", "bias_offsets", "bias_ids"):
            single(arg, INTS)
        for arg in ("repetition", "frequency", "presence", "bias_values"):
            single(arg, FLOATS)
        return out
    for arg in ("q",) if name == "dspark_window_attention" else ("q", "k") if name == "dspark_rotary" else ("q", "k", "v"):
        single(arg, HEADS)
    if name != "dspark_window_attention":
        single("inv_freq", FREQS)
        single("q_norm", NORMS)
        single("k_norm", NORMS)
        out.append(("both norms in float32", lambda a: a.update(q_norm=_f(64), k_norm=_f(64))))
        out.extend((f"eps: {x}", lambda a, x=x: a.update(eps=x)) for x in (0.0, 1, -1.0, float("nan"), "x"))
        out.extend((f"neighbours: {x}", lambda a, x=x: a.update(neighbours=x)) for x in (True, 1, None))
        result("q", {**OUTPUTS, "wider": lambda: _t(3, 6, 64)[:, :4]})
    if name == "dspark_rotary":
        result("k", {**OUTPUTS, "wider": lambda: _t(3, 6, 64)[:, :2]})
        single("row_offsets", INTS)
        single("first", INTS)
        return out
    single("k_cache", CACHES)
    single("v_cache", CACHES)
    single("page_table", TABLES)
    single("row_offsets", INTS)
    single("cache_len", INTS)
    out.extend((f"both caches: {w}", lambda a, m=m: a.update(k_cache=m(), v_cache=m())) for w, m in CACHES.items())
    out.append(("8-bit cache", _eight_bits))
    for arg in ("k_scale", "v_scale"):
        out.extend((f"8-bit cache, {arg}: {w}", lambda a, arg=arg, m=m: (_eight_bits(a), a.update({arg: m()}))) for w, m in SCALES.items())
    if name == "dspark_window_attention":
        result("out", OUTPUTS)
        result("lse", LSES)
        result("workspace", WORKSPACES)
        for arg, values in (("window", (1, 0, -3, 2.5, True, 1 << 40, None)), ("sinks", (0, -1, 1 << 40, "x")),
                            ("scale", (0.3, 1, 0.0, float("nan"), "x")), ("max_rows", (1, 0, -1, 40, 3000, "x"))):
            out.extend((f"{arg}: {x}", lambda a, arg=arg, x=x: a.update({arg: x})) for x in values)
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
    tensors += [r] if isinstance(r, torch.Tensor) else [r[n] for n in ("q", "k", "out", "lse") if r.get(n) is not None]
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
    assert done >= 8 and refused >= 20, (done, refused)


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
