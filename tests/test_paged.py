"""The paged cache's entry points refuse what they cannot take (no GPU needed)."""
import pytest
import torch

import decode_megakernel_06_b200 as mk

PTR = 4096  # never followed: the calls are refused before any launch


def _kv(**kw):
    f = dict(k=PTR, v=PTR, k_scale=None, v_scale=None, page_table=PTR, n_pages=10, page_size=16, max_pages=4,
             n_kv_heads=2, head_dim=64, dtype=mk.MK_BF16)
    f.update(kw)
    return mk.mk_paged_kv(**f)


ST = mk.mk_strides(256, 128, 64)


def _append(kv=None, **kw):
    a = dict(k=PTR, v=PTR, dtype=mk.MK_F32, pos=PTR, B=2, T=3, rope=None, n=0)
    a.update(kw)
    return mk.mk_kv_append(kv or _kv(), a["k"], ST, a["v"], ST, a["dtype"], a["pos"], None, a["B"], a["T"], a["rope"],
                           a["n"], None)


def _gather(kv=None, **kw):
    a = dict(k=PTR, v=PTR, dtype=mk.MK_F32, pos=PTR, B=2, T=3)
    a.update(kw)
    return mk.mk_kv_gather(kv or _kv(), a["pos"], None, a["B"], a["T"], a["k"], ST, a["v"], ST, a["dtype"], None)


def _attention(kv=None, **kw):
    a = dict(q=PTR, dtype=mk.MK_F32, hq=4, pos=PTR, B=2, T=3, scale=0.125, rope=None, n=0, out=PTR, ws=PTR, bytes=1 << 40)
    a.update(kw)
    return mk.mk_paged_attention(kv or _kv(), a["q"], ST, a["dtype"], a["hq"], a["pos"], None, a["B"], a["T"],
                                 a["scale"], a["rope"], a["n"], a["out"], a["ws"], a["bytes"], None)


BAD_KV = [
    (dict(k=None), mk.MK_ERR_ARG), (dict(v=None), mk.MK_ERR_ARG), (dict(page_table=None), mk.MK_ERR_ARG),
    (dict(k=PTR + 8), mk.MK_ERR_ARG), (dict(v=PTR + 2), mk.MK_ERR_ARG), (dict(page_table=PTR + 2), mk.MK_ERR_ARG),
    (dict(dtype=mk.MK_F32), mk.MK_ERR_UNSUPPORTED), (dict(dtype=9), mk.MK_ERR_UNSUPPORTED),
    (dict(dtype=mk.MK_E4M3), mk.MK_ERR_ARG), (dict(dtype=mk.MK_E4M3, k_scale=PTR), mk.MK_ERR_ARG),
    (dict(dtype=mk.MK_E4M3, k_scale=PTR, v_scale=PTR + 2), mk.MK_ERR_ARG),
    (dict(k_scale=PTR), mk.MK_ERR_ARG), (dict(v_scale=PTR), mk.MK_ERR_ARG),
    (dict(n_pages=0), mk.MK_ERR_ARG), (dict(page_size=0), mk.MK_ERR_ARG), (dict(max_pages=0), mk.MK_ERR_ARG),
    (dict(n_kv_heads=0), mk.MK_ERR_ARG), (dict(head_dim=96), mk.MK_ERR_UNSUPPORTED),
    (dict(n_pages=1 << 20, page_size=1 << 10), mk.MK_ERR_UNSUPPORTED),
    (dict(max_pages=1 << 20, page_size=1 << 11), mk.MK_ERR_UNSUPPORTED),
    (dict(page_size=1 << 30, n_kv_heads=2), mk.MK_ERR_UNSUPPORTED)]


@pytest.mark.parametrize("call", [_append, _gather, _attention])
@pytest.mark.parametrize("kw,code", BAD_KV)
def test_cache_refusals(call, kw, code):
    assert call(_kv(**kw)) == code
    assert mk.mk_last_error()


ROWS = [(dict(B=0), mk.MK_ERR_ARG), (dict(T=0), mk.MK_ERR_ARG), (dict(B=-1), mk.MK_ERR_ARG),
        (dict(T=1 << 29), mk.MK_ERR_UNSUPPORTED), (dict(dtype=mk.MK_E4M3), mk.MK_ERR_UNSUPPORTED),
        (dict(dtype=7), mk.MK_ERR_UNSUPPORTED), (dict(pos=None), mk.MK_ERR_ARG)]


@pytest.mark.parametrize("call", [_append, _gather, _attention])
@pytest.mark.parametrize("kw,code", ROWS)
def test_row_refusals(call, kw, code):
    assert call(**kw) == code


@pytest.mark.parametrize("call", [_append, _gather])
@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(k=PTR + 2), dict(v=PTR + 1)])
def test_operand_refusals(call, kw):
    assert call(**kw) == mk.MK_ERR_ARG


@pytest.mark.parametrize("call", [_append, _attention])
@pytest.mark.parametrize("kw", [dict(rope=PTR, n=0), dict(rope=PTR + 4, n=8)])
def test_rope_refusals(call, kw):
    assert call(**kw) == mk.MK_ERR_ARG


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), mk.MK_ERR_ARG), (dict(out=None), mk.MK_ERR_ARG), (dict(out=PTR + 8), mk.MK_ERR_ARG), (dict(hq=3), mk.MK_ERR_ARG),
    (dict(hq=0), mk.MK_ERR_ARG), (dict(scale=float("inf")), mk.MK_ERR_ARG), (dict(scale=float("nan")), mk.MK_ERR_ARG),
    (dict(ws=None), mk.MK_ERR_ARG), (dict(ws=PTR + 4), mk.MK_ERR_ARG),
    (dict(T=1 << 20, hq=1 << 10), mk.MK_ERR_UNSUPPORTED)])
def test_attention_refusals(kw, code):
    assert _attention(**kw) == code


def _tensors(**kw):
    t = dict(k=torch.zeros((4, 2, 8, 64), dtype=torch.bfloat16), v=torch.zeros((4, 2, 8, 64), dtype=torch.bfloat16),
             table=torch.zeros((3, 2), dtype=torch.int32), ks=None, vs=None)
    t.update(kw)
    return mk.PagedKV(t["k"], t["v"], t["table"], t["ks"], t["vs"])


@pytest.mark.parametrize("kw", [
    dict(),  # on the CPU
    dict(k=torch.zeros((4, 2, 8, 64))), dict(k=torch.zeros((4, 2, 64), dtype=torch.bfloat16)),
    dict(k=torch.zeros((4, 2, 8, 128), dtype=torch.bfloat16)[..., :64])])
def test_tensor_refusals(kw):
    with pytest.raises(ValueError):
        _tensors(**kw)


def test_calls_make_their_device_current_and_put_the_other_back(monkeypatch):
    now, seen = [2], []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "set_device", lambda i: now.__setitem__(0, i))

    def call(x):
        seen.append(now[0])
        if x is None:
            raise RuntimeError("within the call")
        return x

    assert mk._call_on(2, call, 5) == 5 and mk._call_on(1, call, 6) == 6 and now == [2]
    with pytest.raises(RuntimeError):
        mk._call_on(0, call, None)
    assert now == [2] and seen == [2, 1, 0]
