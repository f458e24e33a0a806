"""The decode step over a paged cache (mk_decode_step_paged), and a speculative
round of it: append, attention, logits, verification.

Against the same step over the contiguous cache (the tensor-core sequence in
both): they differ in the attention, whose queries and weights the contiguous one
holds as bf16 pairs (2^-17 of a value, a few of them in each of the tiny model's
layers), and in the order of its sums.  1e-3 of the largest logit leaves room for
that through the layers; a wrong position, head or page is far outside.
"""
import dataclasses

import numpy as np
import pytest
import torch

import decode_megakernel_06_b200 as mk
from oracle import verify as overify
from synthetic import TINY, make_kv_cache, make_tokens, make_uniforms, make_weights

from parity import relerr

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TOL = 1e-3


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)


@pytest.fixture(scope="module")
def weights():
    return make_weights(TINY, 0, DEV)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Pages:
    """The layers' pools for sequences of up to `cap` positions, pages shuffled, and
    the contiguous cache's first lens[b] positions copied into them."""

    def __init__(self, k, v, lens, page, kind, seed=0):
        L, B, H, cap, hd = k.shape
        width = -(-cap // page)
        n = B * width + 2
        order = torch.randperm(n, generator=torch.Generator().manual_seed(seed))[:B * width]
        self.table = order.reshape(B, width).to(torch.int32).to(DEV)
        self.layers = []
        zero = torch.zeros(B, dtype=torch.int32, device=DEV)
        for l in range(L):
            pools = [torch.zeros((n, H, page, hd), dtype=torch.bfloat16, device=DEV).to(kind) for _ in range(2)]
            scales = [torch.zeros((n, H, page), device=DEV) for _ in range(2)] if kind != torch.bfloat16 else [None, None]
            kv = mk.PagedKV(*pools, self.table, *scales)
            assert kv.append(k[l].transpose(1, 2), v[l].transpose(1, 2), zero, counts=i32(lens)) == mk.MK_OK
            self.layers.append(kv)


def setup(weights, B, T, lens, cap=192, page=24, kind=torch.bfloat16, seed=0):
    k, v = make_kv_cache(TINY, B, cap, 3, DEV)
    dec = mk.Decoder(TINY, weights, max_rows=max(2, B * T), max_seqs=B, kv_capacity=cap, variant="tensorcore")
    return dec, k, v, Pages(k, v, lens, page, kind, seed)


def run(dec, tokens, pos, B, T, pages=None, kv=None):
    logits = torch.full((B * T, TINY.vocab), float("nan"), device=DEV)
    am = torch.full((B * T,), -1, dtype=torch.int32, device=DEV)
    if pages is not None:
        rc = dec.step_paged(i32(tokens), i32(pos), B, T, pages.layers, logits, am)
    else:
        rc = dec.step(i32(tokens), i32(pos), B, T, *kv, logits, am)
    assert rc == mk.MK_OK, mk.mk_last_error()
    assert dec.status() == mk.MK_OK, mk.mk_last_error()
    return logits, am


@pytest.mark.parametrize("B,T,page", [(3, 1, 24), (2, 4, 16), (1, 2, 7), (5, 7, 64)])
def test_matches_the_contiguous_step(weights, B, T, page):
    lens = [127 - 9 * b for b in range(B)]
    dec, k, v, pages = setup(weights, B, T, lens, page=page)
    tokens, pos = list(make_tokens(TINY.vocab, B * T, seed=1)), list(lens)
    for step in range(3):
        a, am_a = run(dec, tokens, pos, B, T, pages)
        b, am_b = run(dec, tokens, pos, B, T, kv=(k, v))
        a, b = a.cpu().numpy(), b.cpu().numpy()
        assert relerr(a, b) <= TOL
        top = np.sort(b, -1)
        clear = top[:, -1] - top[:, -2] > 2 * TOL * np.abs(b).max()
        assert (am_a.cpu().numpy() == am_b.cpu().numpy())[clear].all()
        assert (am_a.cpu().numpy() == a.argmax(-1)).all()
        # the rows written: bf16 of values that differ by the layers' error
        out = [torch.zeros((B, T, TINY.n_kv_heads, TINY.head_dim), device=DEV) for _ in range(2)]
        for l in (0, TINY.n_layers - 1):
            assert pages.layers[l].gather(i32(pos), *out) == mk.MK_OK
            for got, cache in zip(out, (k, v)):
                for s in range(B):
                    want = cache[l, s, :, pos[s]:pos[s] + T].transpose(0, 1).float()
                    assert relerr(got[s].cpu(), want.cpu()) <= TOL + 2.0 ** -8
        tokens = [int(x) for x in am_b.cpu().reshape(B, T)[:, -1:].repeat(1, T).reshape(-1)]
        pos = [p + T for p in pos]
    dec.close()


def test_one_row_and_repeats(weights):
    """A single row, twice through the recorded graph: the same logits; and on copies of
    the pools, whose layers are other buffers, too."""
    dec, k, v, pages = setup(weights, 1, 1, [100])
    first, _ = run(dec, [5], [100], 1, 1, pages)
    first = first.clone()
    again, _ = run(dec, [5], [100], 1, 1, pages)
    assert torch.equal(first, again)
    other = Pages(k, v, [100], 24, torch.bfloat16, seed=9)
    third, _ = run(dec, [5], [100], 1, 1, other)
    assert torch.equal(first, third)  # the units of a sequence do not depend on where its pages lie
    dec.close()


def test_eight_bit_cache(weights):
    """Runs, finite, and reads what it wrote: a new row's codes are those of the
    bf16 run's row, to half a step of e4m3 and the layers' error."""
    B, T, lens = 2, 2, [90, 127]
    dec, k, v, pages = setup(weights, B, T, lens, kind=torch.float8_e4m3fn)
    logits, _ = run(dec, [1, 2, 3, 4], lens, B, T, pages)
    assert torch.isfinite(logits).all()
    run(dec, [1, 2, 3, 4], lens, B, T, kv=(k, v))
    out = [torch.zeros((B, T, TINY.n_kv_heads, TINY.head_dim), device=DEV) for _ in range(2)]
    assert pages.layers[0].gather(i32(lens), *out) == mk.MK_OK
    for got, cache in zip(out, (k, v)):
        for s in range(B):
            want = cache[0, s, :, lens[s]:lens[s] + T].transpose(0, 1).float()
            # layer 0 sees no cache before its rows are written: 2^-4 of a value, 2^-10 of the scale
            assert ((got[s] - want).abs() <= (2.0 ** -4 + 2.0 ** -8) * want.abs() + want.abs().amax(-1, keepdim=True) / 448 * 2.0 ** -9).all()
    dec.close()


def test_a_speculative_round(weights):
    """Blocks of 4 rows through the paged step, verified by the target's probabilities:
    the oracle's tokens on the same logits, and the next block continues from them."""
    B, T, lens = 3, 4, [60, 100, 127]
    dec, k, v, pages = setup(weights, B, T, lens)
    ws = mk.verify_sample_workspace(B, T, TINY.vocab, DEV)
    out, acc = torch.empty((B, T), dtype=torch.int32, device=DEV), torch.empty(B, dtype=torch.int32, device=DEV)
    pos, last = list(lens), [3, 4, 5]
    rng = np.random.default_rng(0)
    kept = 0
    for step in range(5):
        block = np.array([[last[b]] + list(rng.integers(0, TINY.vocab, T - 1)) for b in range(B)], np.int32)
        # two passes: the first one's argmax as drafts gives blocks that are partly kept
        logits, am = run(dec, block.reshape(-1), pos, B, T, pages)
        block[:, 1] = am.cpu().numpy().reshape(B, T)[:, 0]
        logits, _ = run(dec, block.reshape(-1), pos, B, T, pages)
        u = np.asarray(make_uniforms(B * T, seed=step)).reshape(B, T)
        temperature = (0.0, 0.05, 1.0)[step % 3]
        rc = mk.verify_sample(logits.view(B, T, -1), torch.tensor(block, device=DEV), temperature, 0.9,
                              torch.tensor(u, dtype=torch.float64, device=DEV), out, acc, ws)
        assert rc == mk.MK_OK, mk.mk_last_error()
        got, n = out.cpu().numpy(), acc.cpu().numpy()
        lg = logits.cpu().numpy().reshape(B, T, -1)
        for b in range(B):
            ref = overify.verify_block(lg[b], None, block[b], temperature, 0.9, u[b])
            if ref.accept_margin >= 2.0 ** -20 and ref.draw_margin >= 8 * TINY.vocab:
                assert got[b].tolist() == ref.tokens and n[b] == ref.accepted
            kept += int(n[b]) - 1
            last[b] = int(got[b, n[b] - 1])
            pos[b] += int(n[b])  # rows behind it are written again before they are read
    assert kept > 0
    dec.close()


def test_status_of_bad_inputs(weights):
    dec, k, v, pages = setup(weights, 1, 1, [50])
    am = torch.empty(1, dtype=torch.int32, device=DEV)
    for tok, pos in ((TINY.vocab, 50), (-1, 50), (0, 192), (0, -1)):
        assert dec.step_paged(i32([tok]), i32([pos]), 1, 1, pages.layers, None, am) == mk.MK_OK
        assert dec.status() == mk.MK_ERR_DEVICE_CHECK
    run(dec, [1], [50], 1, 1, pages)
    dec.close()


def test_refusals(weights):
    dec, k, v, pages = setup(weights, 2, 1, [50, 60])
    am = torch.empty(2, dtype=torch.int32, device=DEV)
    tok, pos = i32([1, 2]), i32([50, 60])
    with pytest.raises(ValueError):
        dec.step_paged(tok, pos, 2, 1, pages.layers[:-1], None, am)
    with pytest.raises(ValueError):
        dec.step_paged(tok, pos, 2, 1, [mk.PagedKV(p.k, p.v, p.page_table[:1].contiguous()) for p in pages.layers],
                       None, am)
    wide = torch.zeros((2, TINY.n_kv_heads + 1, 8, TINY.head_dim), dtype=torch.bfloat16, device=DEV)
    other = [mk.PagedKV(wide, wide.clone(), pages.table)] * TINY.n_layers
    assert dec.step_paged(tok, pos, 2, 1, other, None, am) == mk.MK_ERR_ARG
    assert dec.step_paged(i32([1, 2, 3]), pos, 1, 3, pages.layers, None, i32([0, 0, 0])) == mk.MK_ERR_CAPACITY
    dec.close()
    one = mk.Decoder(TINY, weights, max_rows=1, max_seqs=1, kv_capacity=64)
    assert one.step_paged(tok, pos, 1, 1, pages.layers, None, am) == mk.MK_ERR_UNSUPPORTED
    one.close()


WIDE_HEADS = dataclasses.replace(TINY, name="tiny_128", head_dim=128)


def two_ways(model, weights, kind, B, T, lens, page, cap=192, steps=2):
    """The logits of a few steps over pages of `kind`, and over a contiguous bf16 cache that holds
    the same values: 8-bit pages have powers of two for scales, so that bf16 holds code * scale."""
    L, H, hd = model.n_layers, model.n_kv_heads, model.head_dim
    g = torch.Generator(device=DEV).manual_seed(11)
    width = -(-cap // page)
    n = B * width + 2
    table = torch.randperm(n, generator=torch.Generator().manual_seed(2))[:B * width].reshape(B, width).to(torch.int32).to(DEV)
    dec = mk.Decoder(model, weights, max_rows=max(2, B * T), max_seqs=B, kv_capacity=cap, variant="tensorcore")
    k, v = (torch.zeros((L, B, H, cap, hd), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    layers = []
    for l in range(L):
        pools = [torch.randn((n, H, page, hd), generator=g, device=DEV) for _ in range(2)]
        scales = [None, None]
        if kind == torch.bfloat16:
            pools = [x.to(kind) for x in pools]
        else:
            pools = [(100 * x).clamp(-448, 448).to(kind) for x in pools]
            scales = [torch.exp2(torch.randint(-9, -4, (n, H, page), generator=g, device=DEV).float()) for _ in range(2)]
        kv = mk.PagedKV(*pools, table, *scales)
        views = [x[l][:, :, :max(lens)].transpose(1, 2) for x in (k, v)]
        assert kv.gather(i32([0] * B), *views, counts=i32(lens)) == mk.MK_OK
        layers.append(kv)
    got, pos, tokens = [], list(lens), list(make_tokens(model.vocab, B * T, seed=5))
    for _ in range(steps):
        pair = []
        for paged in (True, False):
            logits = torch.full((B * T, model.vocab), float("nan"), device=DEV)
            am = torch.full((B * T,), -1, dtype=torch.int32, device=DEV)
            rc = (dec.step_paged(i32(tokens), i32(pos), B, T, layers, logits, am) if paged else
                  dec.step(i32(tokens), i32(pos), B, T, k, v, logits, am))
            assert rc == mk.MK_OK and dec.status() == mk.MK_OK, mk.mk_last_error()
            pair.append(logits.cpu().numpy())
        got.append(pair)
        pos = [p + T for p in pos]
    dec.close()
    return got


@pytest.mark.parametrize("model", [TINY, WIDE_HEADS], ids=["64", "128"])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float8_e4m3fn], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("B,T,page", [(3, 2, 24), (9, 1, 16), (2, 7, 64)])
def test_old_positions_count_as_in_the_contiguous_cache(model, kind, B, T, page):
    """Both head sizes and both caches, the whole of the logits.  The key and value projections
    are zero, so that the new rows are zeros, which either cache holds exactly, and the
    steps differ in their attention's arithmetic alone."""
    w = make_weights(model, 0, DEV)
    for lw in w["layers"]:
        lw["wqkv"][model.n_q_heads * model.head_dim:] = 0
    lens = [127 - 11 * b for b in range(B)]
    for paged, flat in two_ways(model, w, kind, B, T, lens, page):
        assert relerr(paged, flat) <= TOL
