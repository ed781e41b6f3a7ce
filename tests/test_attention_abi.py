"""Host-side checks of the cache and attention entry points (no GPU needed):
every refusal comes before anything is enqueued, and the binding names what is
wrong with its tensors."""
import ctypes

import pytest
import torch

import draft_sampling_verification_02_amd as ds

P = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10008)  # not 16-byte aligned

ARG, UNSUPPORTED, WORKSPACE = ds.DSPARK_ERR_ARG, ds.DSPARK_ERR_UNSUPPORTED, ds.DSPARK_ERR_WORKSPACE


def _write(**kw):
    a = dict(k=P, v=P, ks=512, vs=512, dtype=0, off=P, n=8, len=P, table=P, B=4, max_pages=10, Hkv=4, D=128, kc=P, vc=P,
             ksc=None, vsc=None, cdt=0, n_pages=50, ps=16)
    a.update(kw)
    return ds.load_library().dspark_kv_write(
        a["k"], a["v"], a["ks"], a["vs"], a["dtype"], a["off"], a["n"], a["len"], a["table"], a["B"], a["max_pages"],
        a["Hkv"], a["D"], a["kc"], a["vc"], a["ksc"], a["vsc"], a["cdt"], a["n_pages"], a["ps"], None)


def _read(**kw):
    a = dict(kc=P, vc=P, ksc=None, vsc=None, cdt=0, n_pages=50, ps=16, off=P, n=8, first=P, table=P, B=4, max_pages=10,
             Hkv=4, D=128, ko=P, vo=P, dtype=0)
    a.update(kw)
    return ds.load_library().dspark_kv_read(
        a["kc"], a["vc"], a["ksc"], a["vsc"], a["cdt"], a["n_pages"], a["ps"], a["off"], a["n"], a["first"], a["table"],
        a["B"], a["max_pages"], a["Hkv"], a["D"], a["ko"], a["vo"], a["dtype"], None)


def _paged(**kw):
    a = dict(q=P, qs=2048, dtype=0, off=P, n=8, max_rows=2, len=P, table=P, B=4, max_pages=10, Hq=16, Hkv=4, D=128, kc=P,
             vc=P, ksc=None, vsc=None, cdt=0, n_pages=50, ps=16, scale=0.1, causal=1, out=P, lse=None, ws=P,
             ws_bytes=1 << 40)
    a.update(kw)
    return ds.load_library().dspark_paged_attention(
        a["q"], a["qs"], a["dtype"], a["off"], a["n"], a["max_rows"], a["len"], a["table"], a["B"], a["max_pages"], a["Hq"],
        a["Hkv"], a["D"], a["kc"], a["vc"], a["ksc"], a["vsc"], a["cdt"], a["n_pages"], a["ps"], a["scale"], a["causal"],
        a["out"], a["lse"], a["ws"], a["ws_bytes"], None)


def _prompt(**kw):
    a = dict(q=P, k=P, v=P, qs=2048, ks=512, vs=512, dtype=0, off=P, n=8, kvoff=P, nkv=9, B=4, Hq=16, Hkv=4, D=128,
             scale=0.1, causal=1, out=P, lse=None, ws=P, ws_bytes=1 << 40)
    a.update(kw)
    return ds.load_library().dspark_prompt_attention(
        a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["dtype"], a["off"], a["n"], a["kvoff"], a["nkv"], a["B"],
        a["Hq"], a["Hkv"], a["D"], a["scale"], a["causal"], a["out"], a["lse"], a["ws"], a["ws_bytes"], None)


CACHE_REFUSALS = [
    (dict(B=0), ARG), (dict(B=65537), ARG), (dict(n=-1), ARG), (dict(n=(1 << 24) + 1), ARG), (dict(off=None), ARG),
    (dict(max_pages=0), ARG), (dict(n_pages=0), ARG), (dict(Hkv=0), ARG), (dict(Hkv=1025), ARG), (dict(D=0), ARG),
    (dict(ps=0), ARG), (dict(max_pages=1 << 27), ARG), (dict(dtype=7), ARG), (dict(cdt=-1), ARG), (dict(dtype=1), UNSUPPORTED),
    (dict(dtype=3), UNSUPPORTED), (dict(cdt=2), UNSUPPORTED), (dict(cdt=1), UNSUPPORTED), (dict(D=96), UNSUPPORTED),
    (dict(D=32), UNSUPPORTED), (dict(ps=8), UNSUPPORTED), (dict(ps=48), UNSUPPORTED), (dict(ps=2048), UNSUPPORTED),
    (dict(table=None), ARG), (dict(kc=None), ARG), (dict(vc=None), ARG), (dict(kc=ODD), ARG), (dict(vc=ODD), ARG),
    (dict(cdt=3), ARG), (dict(cdt=3, ksc=P), ARG), (dict(cdt=3, ksc=P, vsc=ODD), ARG),
]


@pytest.mark.parametrize("change,status", CACHE_REFUSALS)
def test_cache_geometry_is_refused_by_every_entry_point(change, status):
    for call in (_write, _read, _paged):
        kw = dict(change)
        if call is _paged and kw.get("Hkv") == 1025:
            kw["Hq"] = 1025
        assert call(**kw) == status, (call.__name__, change)


@pytest.mark.parametrize("change", [dict(k=None), dict(v=None), dict(len=None), dict(k=ODD), dict(v=ODD), dict(ks=511),
                                    dict(vs=516), dict(ks=508), dict(vs=(1 << 24) + 8), dict(ks=0), dict(ks=-512)])
def test_write_refusals(change):
    assert _write(**change) == ARG


@pytest.mark.parametrize("change", [dict(ko=None), dict(vo=None), dict(ko=ODD), dict(vo=ODD)])
def test_read_refusals(change):
    assert _read(**change) == ARG


@pytest.mark.parametrize("change", [
    dict(q=None), dict(len=None), dict(out=None), dict(q=ODD), dict(out=ODD), dict(qs=2040), dict(qs=2052), dict(Hq=15),
    dict(Hq=0), dict(Hq=1028), dict(max_rows=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(n=1 << 24, Hq=512, qs=512 * 128)])
def test_paged_attention_refusals(change):
    assert _paged(**change) == ARG


@pytest.mark.parametrize("change", [
    dict(q=None), dict(k=None), dict(v=None), dict(off=None), dict(out=None), dict(q=ODD), dict(k=ODD), dict(out=ODD),
    dict(qs=2040), dict(ks=504), dict(vs=516), dict(kvoff=None), dict(n=-1), dict(nkv=-1), dict(nkv=(1 << 24) + 1), dict(B=0),
    dict(B=65537), dict(Hq=6), dict(Hkv=0), dict(D=0), dict(dtype=9), dict(scale=0.0), dict(scale=float("nan"))])
def test_prompt_attention_refusals(change):
    assert _prompt(**change) == ARG
    assert _prompt(D=80) == UNSUPPORTED
    assert _prompt(dtype=1) == UNSUPPORTED and _prompt(dtype=3) == UNSUPPORTED


def test_workspaces():
    need = ds.dspark_paged_attention_workspace_size(2, 16, 4, 128)
    assert need > 0
    assert _paged(ws=None) == WORKSPACE and _paged(ws_bytes=16) == WORKSPACE and _paged(ws=ODD) == WORKSPACE
    assert ds.dspark_prompt_attention_workspace_size(4, 8, 9, 16, 4, 128) > 0
    assert _prompt(ws=None) == WORKSPACE and _prompt(ws_bytes=16) == WORKSPACE and _prompt(ws=ODD) == WORKSPACE
    for bad in [(0, 16, 4, 128), (1, 15, 4, 128), (1, 16, 0, 128), (1, 16, 4, 100), (1, 2048, 4, 128)]:
        assert ds.dspark_paged_attention_workspace_size(*bad) == 0
    for bad in [(0, 8, 8, 16, 4, 128), (1, -1, 8, 16, 4, 128), (1, 8, -1, 16, 4, 128), (1, 8, 8, 15, 4, 128), (1, 8, 8, 16, 4, 60)]:
        assert ds.dspark_prompt_attention_workspace_size(*bad) == 0


def test_no_rows_is_a_call_that_does_nothing():
    assert _write(n=0) == ds.DSPARK_OK and _read(n=0) == ds.DSPARK_OK
    assert _paged(n=0) == ds.DSPARK_OK and _prompt(n=0, nkv=0) == ds.DSPARK_OK


# ---- the binding: CPU tensors stand for wrong ones; nothing reaches a device

BF = torch.bfloat16


def _t(shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def _good():
    return dict(k=_t((4, 2, 64)), kc=_t((6, 2, 16, 64)), vc=_t((6, 2, 16, 64)), ln=_t((4,), torch.int32),
                pt=_t((4, 3), torch.int32), q=_t((4, 4, 64)))


def test_binding_refuses_host_tensors():
    g = _good()
    with pytest.raises(ValueError, match="HIP device"):
        ds.dspark_kv_write(g["k"], g["k"], g["kc"], g["vc"], g["ln"], g["pt"])
    with pytest.raises(ValueError, match="HIP device"):
        ds.dspark_kv_read(g["kc"], g["vc"], g["pt"], 4)
    with pytest.raises(ValueError, match="HIP device"):
        ds.dspark_paged_attention(g["q"], g["kc"], g["vc"], g["ln"], g["pt"])
    with pytest.raises(ValueError, match="HIP device"):
        ds.dspark_prompt_attention(g["q"], g["k"], g["k"], _t((3,), torch.int32))


@pytest.mark.parametrize("change,error,word", [
    (dict(k=_t((4, 2, 64), torch.float32)), (TypeError, ValueError), "v|k"),
    (dict(k=_t((4, 3, 64))), ValueError, "k"),
    (dict(k=_t((4, 2, 128))), ValueError, "k"),
    (dict(k=_t((4, 64, 2)).transpose(1, 2)), ValueError, "dense"),
    (dict(k=None), TypeError, "k"),
    (dict(kc=_t((6, 2, 16, 64), torch.float64)), TypeError, "k_cache"),
    (dict(kc=_t((6, 2, 64))), ValueError, "k_cache"),
    (dict(vc=_t((6, 2, 32, 64))), ValueError, "v_cache"),
    (dict(kc=_t((6, 16, 2, 64)).transpose(1, 2)), ValueError, "contiguous"),
    (dict(ln=_t((5,), torch.int32)), ValueError, "cache_len"),
    (dict(ln=_t((4,), torch.int64)), TypeError, "cache_len"),
    (dict(ln=None), TypeError, "cache_len"),
    (dict(pt=_t((4,), torch.int32)), ValueError, "page_table"),
    (dict(pt=_t((3, 3), torch.int32)), ValueError, "row_offsets"),
])
def test_binding_names_what_is_wrong_with_a_write(change, error, word):
    g = _good()
    g.update(change)
    with pytest.raises(error, match=word):
        ds.dspark_kv_write(g["k"], _t((4, 2, 64)), g["kc"], g["vc"], g["ln"], g["pt"])


def test_binding_checks_scales_outputs_and_offsets():
    g = _good()
    with pytest.raises(ValueError, match="scale"):
        ds.dspark_kv_write(g["k"], g["k"], g["kc"], g["vc"], g["ln"], g["pt"], k_scale=_t((6, 2, 16), torch.uint8))
    e4 = g["kc"].to(torch.float8_e4m3fn)
    with pytest.raises(TypeError, match="k_scale"):
        ds.dspark_kv_write(g["k"], g["k"], e4, e4, g["ln"], g["pt"])
    with pytest.raises(ValueError, match="row_offsets"):
        ds.dspark_paged_attention(g["q"], g["kc"], g["vc"], g["ln"], g["pt"], row_offsets=_t((4,), torch.int32))
    with pytest.raises(ValueError, match="out"):
        ds.dspark_paged_attention(g["q"], g["kc"], g["vc"], g["ln"], g["pt"], out={"out": _t((4, 4, 32))})
    with pytest.raises(TypeError, match="lse"):
        ds.dspark_paged_attention(g["q"], g["kc"], g["vc"], g["ln"], g["pt"], out={"out": _t((4, 4, 64)), "lse": _t((4, 4))})
    with pytest.raises(ValueError, match="kv_offsets"):
        ds.dspark_prompt_attention(g["q"], _t((5, 2, 64)), _t((5, 2, 64)), _t((3,), torch.int32))
    with pytest.raises(ValueError, match="k/v"):
        ds.dspark_prompt_attention(g["q"], _t((4, 2, 64)), _t((4, 2, 128)), _t((3,), torch.int32))
    with pytest.raises(TypeError, match="q"):
        ds.dspark_prompt_attention(_t((4, 4, 64), torch.float32), g["k"], g["k"], _t((3,), torch.int32))


def test_calls_past_one_launch_are_refused():
    # 2^34 pieces of 16 bytes
    assert _write(n=1 << 18, Hkv=1024, D=256, ks=1 << 18, vs=1 << 18) == ARG
    assert _read(n=1 << 18, Hkv=1024, D=256) == ARG
    wide = dict(Hq=256, Hkv=256, D=64, qs=256 * 64, ks=256 * 64, vs=256 * 64)
    assert _prompt(B=65536, n=8, nkv=9, **wide) == ARG
    assert ds.dspark_prompt_attention_workspace_size(65536, 8, 9, 256, 256, 64) == 0
    assert _prompt(B=65534, n=8, nkv=9, ws=None, **wide) == WORKSPACE
    assert ds.dspark_prompt_attention_workspace_size(65534, 8, 9, 256, 256, 64) > 0


def test_binding_names_a_workspace_that_does_not_fit():
    bf, i32 = torch.bfloat16, torch.int32
    q, k = torch.zeros(4, 8, 64, dtype=bf), torch.zeros(4, 2, 64, dtype=bf)
    off = torch.tensor([0, 4], dtype=i32)
    cache, table = torch.zeros(3, 2, 16, 64, dtype=bf), torch.zeros(4, 2, dtype=i32)
    calls = [lambda **kw: ds.dspark_prompt_attention(q, k, k, off, **kw),
             lambda **kw: ds.dspark_paged_attention(q, cache, cache, torch.zeros(4, dtype=i32), table, **kw)]
    for call in calls:
        with pytest.raises(TypeError, match="workspace"):
            call(workspace=torch.zeros(1 << 20, dtype=torch.float32))
        with pytest.raises(TypeError, match="workspace"):
            call(workspace=4096)
        with pytest.raises(ValueError, match="workspace"):
            call(workspace=torch.zeros(1, dtype=torch.uint8).expand(1 << 24))
    with pytest.raises(TypeError, match="row_offsets"):
        ds.dspark_prompt_attention(q, k, k, None)
    with pytest.raises(TypeError, match="page_table"):
        ds.dspark_paged_attention(q, cache, cache, torch.zeros(4, dtype=i32), None)


@pytest.mark.parametrize("scale", [2.31e38, 2.4e38, 3.4e38])
def test_scales_whose_base_2_form_overflows_are_refused(scale):
    # the kernels work in units of scale * log2(e), which would be infinite from 2.36e38 on: 0 * inf where a score is 0
    assert _paged(scale=scale) == ARG and _prompt(scale=scale) == ARG
    assert _paged(scale=2.29e38, ws=None) == WORKSPACE and _prompt(scale=2.29e38, ws=None) == WORKSPACE
