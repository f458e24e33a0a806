"""Verification of drafts on the GPU against the oracle, token for token.

Both sides decide in the same integers; only the last bit of the fp64
exponential may differ (CUDA's and the host's), which moves a mass by at most
one unit of at least 2^46 in a row's sum.  Blocks whose decisions come within
what that can move are left out, and few may be:
* at an acceptance, the sums A and D by V / 2^46 <= 2^-29 relative and the draft's
  masses by one unit, 2^-21 relative from 2^21 units (a share of 2^-25) on: 2^-20;
* at the draw, V masses by a unit each, and the residual's by one more for the
  factor 2^46 / A (2^46 V / A^2 of each unit, over all masses at most V), twice
  for a and d, and as much again for the point y = u R: 8 V units.
"""
import numpy as np
import pytest
import torch

import decode_megakernel_06_b200 as mk
from oracle import verify as overify
from oracle.sample import masses, nucleus_need

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)


def gpu(logits, draft, tokens, temperature, top_p, u, ws=None, stream=None):
    B, T, V = logits.shape
    up = lambda x, d: None if x is None else torch.tensor(np.ascontiguousarray(x), dtype=d, device=DEV)  # noqa: E731
    out = torch.full((B, T), -7, dtype=torch.int32, device=DEV)
    acc = torch.full((B,), -7, dtype=torch.int32, device=DEV)
    ws = mk.verify_sample_workspace(B, T, V, DEV) if ws is None else ws
    rc = mk.verify_sample(up(logits, torch.float32), up(tokens, torch.int32), temperature, top_p,
                          up(u, torch.float64), out, acc, ws, draft_logits=up(draft, torch.float32), stream=stream)
    assert rc == mk.MK_OK, mk.mk_last_error()
    torch.cuda.synchronize()
    return out.cpu().numpy(), acc.cpu().numpy()


def compare(logits, draft, tokens, temperature, top_p, u):
    out, acc = gpu(logits, draft, tokens, temperature, top_p, u)
    checked = 0
    for b in range(logits.shape[0]):
        ref = overify.verify_block(logits[b], None if draft is None else draft[b], tokens[b], temperature, top_p,
                                   np.zeros(logits.shape[1]) if u is None else u[b])
        if ref.accept_margin < 2.0 ** -20 or ref.draw_margin < 8 * logits.shape[2]:
            continue
        assert acc[b] == ref.accepted and out[b].tolist() == ref.tokens, (b, out[b], ref)
        checked += 1
    return checked


def block(B, T, V, seed, sigma=2.0, noise=0.5, temperature=1.0):
    """Target logits, draft logits near them, drafts drawn from the draft's softmax."""
    rng = np.random.default_rng(seed)
    lg = (rng.standard_normal((B, T, V)) * sigma).astype(np.float32)
    dr = (lg[:, :-1] + rng.standard_normal((B, T - 1, V)) * noise).astype(np.float32)
    tok = np.zeros((B, T), np.int32)
    t = temperature if temperature > 0 else 0.05
    if T > 1:
        tok[:, 1:] = (dr / t + rng.gumbel(size=dr.shape)).argmax(-1)
    return lg, dr, tok, rng.random((B, T))


CASES = [(1, 4, 1024), (3, 2, 1), (2, 3, 7), (8, 7, 4099), (5, 5, 32000), (2, 8, 64000), (1, 2, 131072), (40, 3, 501),
         (2, 1, 1000)]


@pytest.mark.parametrize("B,T,V", CASES)
@pytest.mark.parametrize("certain", [False, True])
def test_against_oracle(B, T, V, certain):
    total = checked = 0
    for i, (temp, top_p) in enumerate([(1.0, 1.0), (0.7, 0.9), (1.5, 0.3), (0.0, 1.0), (1.0, 0.0), (0.3, 1.0)]):
        lg, dr, tok, u = block(B, T, V, 100 * i + V, temperature=temp)
        checked += compare(lg, None if certain else dr, tok, temp, top_p, None if temp == 0 else u)
        total += B
    assert checked >= total - max(1, total // 50), (checked, total)


# Rows enough to take one CTA each, of slices too long for its cache, and two CTAs each.
@pytest.mark.parametrize("B,T,V", [(16, 8, 64000), (11, 8, 40001), (4, 8, 32000)])
def test_many_rows_of_long_vocabularies(B, T, V):
    checked = 0
    for i, (temp, top_p) in enumerate([(0.8, 0.9), (1.2, 0.4)]):
        lg, dr, tok, u = block(B, T, V, 7 * i + V, temperature=temp)
        checked += compare(lg, dr, tok, temp, top_p, u)
    assert checked >= 2 * B - 2, checked


def test_ties_and_signed_zeros():
    B, T, V = 4, 4, 3000
    lg, dr, tok, u = block(B, T, V, 1)
    lg[0], dr[0] = 0.0, 0.0                                            # all tied
    lg[1], dr[1] = np.round(lg[1] * 2) / 2, np.round(dr[1] * 2) / 2     # many ties
    lg[2] = np.where(lg[2] > 0, np.float32(0.0), np.float32(-0.0))
    dr[3] = lg[3, :-1]                                                 # equal: all accepted
    for top_p in (1.0, 0.5, 0.9, 0.001):
        for t in (1.0, 0.25, 40.0):
            for uu in (u, np.zeros_like(u), np.full_like(u, np.nextafter(1.0, 0.0))):
                out, acc = gpu(lg, dr, tok, t, top_p, uu)
                for b in range(B):
                    ref = overify.verify_block(lg[b], dr[b], tok[b], t, top_p, uu[b])
                    if ref.accept_margin < 2.0 ** -20:
                        continue
                    if ref.draw_margin < 8 * V and 0 < uu[b, -1] < 0.9999:
                        continue
                    assert acc[b] == ref.accepted, (b, t, top_p)
                    if ref.draw_margin >= 8 * V or uu[b, -1] == 0:
                        assert out[b].tolist() == ref.tokens, (b, t, top_p, out[b], ref)


def test_wide_row_of_ties():
    """More ties in the threshold's bin than a list holds."""
    V = 120000
    lg = np.zeros((1, 2, V), np.float32)
    lg[0, :, ::3] = 1.0
    dr = np.zeros((1, 1, V), np.float32)
    for top_p in (0.2, 0.7, 0.99):
        for x in (0, 1, 119997, 119999):
            tok = np.array([[0, x]], np.int32)
            for u in (0.05, 0.95):
                uu = np.array([[u, u]])
                out, acc = gpu(lg, dr, tok, 1.0, top_p, uu)
                ref = overify.verify_block(lg[0], dr[0], tok[0], 1.0, top_p, uu[0])
                assert acc[0] == ref.accepted and out[0].tolist() == ref.tokens, (top_p, x, u)


def test_banned_tokens():
    """-inf logits: never drawn, their drafts never kept; a lone token left."""
    lg, dr, tok, u = block(6, 4, 777, 2)
    lg[:, :, 100:700] = -np.inf
    dr[:3, :, 50:650] = -np.inf
    tok[0, 2], tok[1, 1] = 300, 300
    lg[5, 1], lg[5, 1, 33] = -np.inf, 1.0
    for top_p in (1.0, 0.8):
        for t in (1.0, 0.0):
            assert compare(lg, dr, tok, t, top_p, u) >= 5
            assert compare(lg, None, tok, t, top_p, u) >= 5
    out, _ = gpu(lg, dr, tok, 1.0, 1.0, u)
    assert not ((out >= 100) & (out < 700)).any()


def test_rows_that_are_not_finite():
    """Out of contract: some token of the vocabulary, and the other blocks as ever."""
    lg, dr, tok, u = block(8, 3, 900, 12)
    want = gpu(lg, dr, tok, 1.0, 0.9, u)
    bad = lg.copy()
    bad[0, :, 5], bad[1, :], bad[2, :, 7], bad[3, :] = np.nan, np.nan, np.inf, -np.inf
    dbad = dr.copy()
    dbad[4, :, 5], dbad[5, :] = np.nan, -np.inf
    for t, p in ((1.0, 0.9), (1.0, 1.0), (0.0, 1.0)):
        out, acc = gpu(bad, dbad, tok, t, p, u)
        for b in range(8):
            assert 1 <= acc[b] <= 3 and ((out[b, :acc[b]] >= 0) & (out[b, :acc[b]] < 900)).all(), (t, p, b, out[b])
        if (t, p) == (1.0, 0.9):
            assert (out[6:] == want[0][6:]).all() and (acc[6:] == want[1][6:]).all()


def test_drafts_outside_the_vocabulary():
    lg, dr, tok, u = block(4, 5, 600, 3)
    tok[0, 1], tok[1, 3], tok[2, 4], tok[3, 2] = -1, 600, 2 ** 31 - 1, -2 ** 31
    for d in (dr, None):
        assert compare(lg, d, tok, 1.0, 0.9, u) >= 3
        assert compare(lg, d, tok, 0.0, 0.9, None) >= 3


def test_peaked_and_flat_rows():
    for scale in (50.0, 1e-3, 0.0, 1e30):
        lg, dr, tok, u = block(3, 4, 2000, 4)
        lg, dr = (lg * np.float32(scale)).astype(np.float32), (dr * np.float32(scale)).astype(np.float32)
        for top_p in (1.0, 0.9):
            compare(lg, dr, tok, 1.0, top_p, u)
            compare(lg, dr, tok, 1e-30, top_p, u)


def test_equal_distributions_accept_all():
    lg, _, tok, u = block(4, 6, 5000, 5)
    out, acc = gpu(lg, lg[:, :-1], tok, 1.0, 1.0, u)
    assert (acc == 6).all() and (out[:, :5] == tok[:, 1:]).all()


def test_statistics_follow_the_target():
    """20000 blocks of one draft over 6 tokens: the first token's frequencies are the
    target's, within 5 standard deviations."""
    N, V = 20000, 6
    rng = np.random.default_rng(6)
    t, d = rng.standard_normal(V).astype(np.float32), rng.standard_normal(V).astype(np.float32)
    p, q = np.exp(t) / np.exp(t).sum(), np.exp(d) / np.exp(d).sum()
    lg = np.broadcast_to(t, (N, 2, V))
    dr = np.broadcast_to(d, (N, 1, V))
    tok = np.zeros((N, 2), np.int32)
    tok[:, 1] = rng.choice(V, size=N, p=q.astype(np.float64) / q.astype(np.float64).sum())
    for draft in (dr, None):
        out, _ = gpu(lg, draft, tok, 1.0, 1.0, rng.random((N, 2)))
        if draft is None:
            # certain drafts: keep with p(x), else from p without x: p again
            pass
        freq = np.bincount(out[:, 0], minlength=V) / N
        assert (np.abs(freq - p) <= 5 * np.sqrt(p * (1 - p) / N) + 1e-9).all(), (freq, p)


def test_repeatable_on_two_streams_and_in_a_graph():
    lg, dr, tok, u = block(8, 7, 32000, 7, temperature=0.8)
    ref = gpu(lg, dr, tok, 0.8, 0.9, u)
    up = lambda x, d: torch.tensor(np.ascontiguousarray(x), dtype=d, device=DEV)  # noqa: E731
    args = [up(lg, torch.float32), up(tok, torch.int32)]
    d, uu = up(dr, torch.float32), up(u, torch.float64)
    runs = []
    torch.cuda.synchronize()
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        out = torch.empty((8, 7), dtype=torch.int32, device=DEV)
        acc = torch.empty(8, dtype=torch.int32, device=DEV)
        ws = mk.verify_sample_workspace(8, 7, 32000, DEV)
        torch.cuda.synchronize()
        assert mk.verify_sample(*args, 0.8, 0.9, uu, out, acc, ws, draft_logits=d, stream=s) == mk.MK_OK
        runs.append((out, acc, ws))
    torch.cuda.synchronize()
    for out, acc, _ in runs:
        assert (out.cpu().numpy() == ref[0]).all() and (acc.cpu().numpy() == ref[1]).all()
    out, acc, ws = runs[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert mk.verify_sample(*args, 0.8, 0.9, uu, out, acc, ws, draft_logits=d) == mk.MK_OK
    lg2, dr2, tok2, u2 = block(8, 7, 32000, 8, temperature=0.8)
    for new, old in ((lg2, args[0]), (tok2, args[1]), (dr2, d), (u2, uu)):
        old.copy_(torch.from_numpy(np.ascontiguousarray(new)))
    graph.replay()
    torch.cuda.synchronize()
    want = gpu(lg2, dr2, tok2, 0.8, 0.9, u2)
    assert (out.cpu().numpy() == want[0]).all() and (acc.cpu().numpy() == want[1]).all()


def test_odd_row_addresses():
    """Rows that start off 16-byte boundaries."""
    lg, dr, tok, u = block(3, 3, 1003, 9)
    assert compare(lg, dr, tok, 1.0, 0.9, u) >= 2
    flat = torch.zeros(1 + lg.size, device=DEV)
    x = flat[1:].view(lg.shape)
    x.copy_(torch.from_numpy(lg))
    out, acc = torch.empty((3, 3), dtype=torch.int32, device=DEV), torch.empty(3, dtype=torch.int32, device=DEV)
    up = lambda y, d: torch.tensor(y, dtype=d, device=DEV)  # noqa: E731
    ws = mk.verify_sample_workspace(3, 3, 1003, DEV)
    assert mk.verify_sample(x, up(tok, torch.int32), 1.0, 0.9, up(u, torch.float64), out, acc, ws,
                            draft_logits=up(dr, torch.float32)) == mk.MK_OK
    want = gpu(lg, dr, tok, 1.0, 0.9, u)
    assert (out.cpu().numpy() == want[0]).all() and (acc.cpu().numpy() == want[1]).all()


def test_agrees_with_the_sampler_without_drafts():
    """T = 1: the token is mk_sample_top_p's."""
    lg, _, tok, u = block(16, 1, 5000, 10)
    for t, p in ((1.0, 1.0), (0.8, 0.9), (0.0, 1.0)):
        out, acc = gpu(lg, None, tok, t, p, u)
        want = torch.empty(16, dtype=torch.int32, device=DEV)
        assert mk.sample_top_p(torch.tensor(lg[:, 0], device=DEV), t, p, torch.tensor(u[:, 0], device=DEV), want) == mk.MK_OK
        assert (acc == 1).all() and (out[:, 0] == want.cpu().numpy()).all()


def test_tensor_refusals():
    lg, dr, tok, u = (torch.tensor(x, device=DEV) for x in block(2, 3, 50, 11))
    out, acc = torch.empty((2, 3), dtype=torch.int32, device=DEV), torch.empty(2, dtype=torch.int32, device=DEV)
    ws = mk.verify_sample_workspace(2, 3, 50, DEV)
    for f in (lambda: mk.verify_sample(lg, tok, 1.0, 1.0, u.float(), out, acc, ws),
              lambda: mk.verify_sample(lg, tok[:1], 1.0, 1.0, u, out, acc, ws),
              lambda: mk.verify_sample(lg, tok, 1.0, 1.0, u, out, acc, ws, draft_logits=lg),
              lambda: mk.verify_sample(lg, tok, 1.0, 1.0, u, out, acc[:1], ws),
              lambda: mk.verify_sample(lg.double(), tok, 1.0, 1.0, u, out, acc, ws),
              lambda: mk.verify_sample(lg, tok.cpu(), 1.0, 1.0, u, out, acc, ws)):
        with pytest.raises(ValueError):
            f()
    assert mk.verify_sample(lg, tok, 1.0, 1.0, None, out, acc, ws) == mk.MK_ERR_ARG
    assert mk.verify_sample(lg, tok, 1.0, 1.0, u, out, acc, ws[:16]) == mk.MK_ERR_CAPACITY
    assert mk.verify_sample(lg, tok, 1.0, 1.0, u, tok, acc, ws) == mk.MK_ERR_ARG


def flat_row(V, tops, seed):
    """`tops` tokens at one largest logit, the others 26 to 32.6 below it: masses of 0 to 360
    units beside a sum above 2^53, of which fp64 keeps no single units.  The tail's ids, by
    falling logit."""
    rng = np.random.default_rng(seed)
    row = np.full(V, 5.0, np.float32)
    tail = rng.permutation(V)[:V - tops]
    row[tail] = (5.0 - rng.uniform(26.0, 32.6, V - tops)).astype(np.float32)
    return row, tail[np.argsort(-row[tail].astype(np.float64), kind="stable")]


# Blocks few enough for clusters of 8, for clusters of 2 and for single CTAs.
@pytest.mark.parametrize("V,tops,B", [(64000, 60000, 3), (64000, 400, 3), (131072, 131000, 2), (64000, 60000, 20),
                                      (40001, 39000, 3), (9000, 8500, 90)])
@pytest.mark.parametrize("certain", [True, False])
def test_whole_distribution_whose_sum_is_rounded(V, tops, B, certain):
    """top_p = 1 with need = ceil(fp64(Q)) below Q: the least tokens are left out, so the
    nucleus is searched for although the whole distribution was asked for.  u = 0 keeps a
    draft exactly if it belongs to the nucleus; drafts are those on both sides of its end."""
    rows, drafts, left_out = [], [], 0
    seed = 0
    while len(rows) < B:
        row, tail = flat_row(V, tops, seed)
        seed += 1
        a, q = overify.nucleus_masses(row, 1.0, 1.0), masses(row, 1.0).astype(np.int64)
        total, lost = int(q.sum()), int(((q > 0) & (a == 0)).sum())
        if nucleus_need(total, 1.0) >= total or not lost:
            continue
        end = int((a[tail] > 0).sum())  # tail[end - 1] is the last of the nucleus
        at = (end - 1, end, end - 2, end + lost - 1, 0, len(tail) - 1)[len(rows) % 6]
        rows.append(row)
        drafts.append(int(tail[at]))
        left_out += a[tail[at]] == 0
    assert 0 < left_out < B
    lg = np.stack([np.stack([r, rows[i - 1]]) for i, r in enumerate(rows)])
    tok = np.array([[0, x] for x in drafts], np.int32)
    u = np.stack([np.zeros(B), np.random.default_rng(V + B).random(B)], 1)
    dr = None if certain else np.stack([r[None] for r in rows[1:] + rows[:1]])
    out, acc = gpu(lg, dr, tok, 1.0, 1.0, u)
    drawn = 0
    for b in range(B):
        ref = overify.verify_block(lg[b], None if certain else dr[b], tok[b], 1.0, 1.0, u[b])
        assert acc[b] == ref.accepted, b
        if ref.draw_margin >= 8 * V:
            assert out[b].tolist() == ref.tokens, b
            drawn += 1
    assert drawn >= B // 2
    again = gpu(lg, dr, tok, 1.0, 1.0, u)
    assert (again[0] == out).all() and (again[1] == acc).all()


@pytest.mark.parametrize("scale", [50.0, 1e-3, 0.0, 1e30])
@pytest.mark.parametrize("temperature", [1.0, 3.0, 1e-30])
@pytest.mark.parametrize("top_p", [1.0, 0.9])
def test_peaked_and_flat_rows_are_compared(scale, temperature, top_p):
    """Five blocks of six, at least, are clear of their borders, and are compared."""
    lg, dr, tok, u = block(6, 4, 2000, 4)
    lg, dr = (lg * np.float32(scale)).astype(np.float32), (dr * np.float32(scale)).astype(np.float32)
    assert compare(lg, dr, tok, temperature, top_p, u) >= 5
    assert compare(lg, None, tok, temperature, top_p, u) >= 5
