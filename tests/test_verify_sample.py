"""Speculative sampling: the definition keeps the target's distribution (CPU), and
the entry point refuses what it cannot take."""
import ctypes

import numpy as np
import pytest

import decode_megakernel_06_b200 as mk
from oracle import verify as overify
from oracle.sample import MASS_SCALE


def _rows(seed, n, V, sigma=1.5):
    return (np.random.default_rng(seed).standard_normal((n, V)) * sigma).astype(np.float32)


@pytest.mark.parametrize("top_p", [1.0, 0.8])
@pytest.mark.parametrize("certain", [False, True])
def test_output_follows_the_target(top_p, certain):
    """Over all drafts (weighted by their probability), all acceptances and all
    draws, the first token's distribution is the target's nucleus."""
    V = 9
    target, draft = _rows(1, 2, V), _rows(2, 1, V)
    a = overify.nucleus_masses(target[0], 1.0, top_p)
    p = a / a.sum()
    d = overify.nucleus_masses(draft[0], 1.0, top_p)
    dx = d / d.sum() if not certain else np.eye(V)[3]
    got = np.zeros(V)
    n = 2000  # midpoints of the draw's uniform: each interval's share to 1 / n
    for x in np.flatnonzero(dx):
        keep = min(1.0, p[x] / dx[x])
        got[x] += dx[x] * keep
        if keep < 1.0:
            u0 = (keep + 1.0) / 2  # any uniform above the border rejects
            for i in range(n):
                b = overify.verify_block(target, None if certain else draft, [0, x], 1.0, top_p, [u0, (i + 0.5) / n])
                assert b.accepted == 1
                got[b.tokens[0]] += dx[x] * (1 - keep) / n
    # each of the V intervals of each residual is off by at most one midpoint
    assert np.abs(got - p).max() <= V / n + V / MASS_SCALE


def test_equal_distributions_accept_everything():
    rows = _rows(3, 4, 50)
    b = overify.verify_block(rows, rows[:3].copy(), [0, 7, 8, 9], 1.0, 1.0, [0.999, 0.5, 0.0, 0.25])
    assert b.accepted == 4 and b.tokens[:3] == [7, 8, 9]


def test_draft_outside_the_vocabulary_ends_the_block():
    rows = _rows(4, 3, 20)
    b = overify.verify_block(rows, rows[:2].copy(), [0, 5, -1], 1.0, 1.0, [0.0, 0.0, 0.5])
    assert b.accepted == 2 and b.tokens[0] == 5 and b.tokens[2] == -1


def test_greedy():
    rows = _rows(5, 3, 20)
    best = [int(r.argmax()) for r in rows]
    b = overify.verify_block(rows, None, [0, best[0], 19 - best[1]], 0.0, 0.5, [0.0] * 3)
    want = 3 if 19 - best[1] == best[1] else 2
    assert b.accepted == want and b.tokens[:2] == best[:2]


PTR = 4096  # never followed: the call is refused before any launch


def _call(**kw):
    a = dict(logits=PTR, draft=None, tokens=PTR + 64, B=2, T=3, V=100, temperature=1.0, top_p=0.9, uniforms=PTR,
             out=PTR, acc=PTR, ws=PTR, n=1 << 20)
    a.update(kw)
    return mk.mk_verify_sample(a["logits"], a["draft"], a["tokens"], a["B"], a["T"], a["V"], a["temperature"],
                               a["top_p"], a["uniforms"], a["out"], a["acc"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), mk.MK_ERR_ARG), (dict(tokens=None), mk.MK_ERR_ARG), (dict(out=None), mk.MK_ERR_ARG),
    (dict(acc=None), mk.MK_ERR_ARG), (dict(uniforms=None), mk.MK_ERR_ARG), (dict(B=0), mk.MK_ERR_ARG),
    (dict(T=0), mk.MK_ERR_ARG), (dict(V=0), mk.MK_ERR_ARG), (dict(V=131073), mk.MK_ERR_UNSUPPORTED),
    (dict(B=1 << 13, T=1 << 12), mk.MK_ERR_UNSUPPORTED), (dict(temperature=float("nan")), mk.MK_ERR_ARG),
    (dict(top_p=float("nan")), mk.MK_ERR_ARG), (dict(ws=None), mk.MK_ERR_ARG), (dict(ws=PTR + 4), mk.MK_ERR_ARG),
    (dict(n=16), mk.MK_ERR_CAPACITY), (dict(tokens=PTR, out=PTR), mk.MK_ERR_ARG)])
def test_refusals(kw, code):
    assert _call(**kw) == code
    assert mk.mk_last_error()


def test_workspace_sizes():
    assert mk.mk_verify_sample_workspace(0, 1) == 0 and mk.mk_verify_sample_workspace(1, 0) == 0
    assert mk.mk_verify_sample_workspace(8, 7) >= 8 * 13 * 8
    with pytest.raises(ValueError):
        mk.verify_sample_workspace(0, 3, 10, "cpu")
    assert ctypes.sizeof(ctypes.c_uint64) == 8


def test_tensor_refusals():
    import torch

    lg = torch.zeros((2, 3, 10))
    tok, acc = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        mk.verify_sample(lg, tok, 1.0, 1.0, None, tok.clone(), acc, torch.zeros(64, dtype=torch.uint8))
    with pytest.raises(ValueError, match="logits"):
        mk.verify_sample(lg[0], tok, 1.0, 1.0, None, tok.clone(), acc, torch.zeros(64, dtype=torch.uint8))
