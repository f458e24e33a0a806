"""The paged cache on the GPU against the formulas in 64 bits.

Tolerances count roundings (u = 2^-24 is half a step of fp32):
* append: a rotated key is off by 3 u (|a| + |b|) before its own rounding, half
  a step of its type: 2^-8 of the value (bf16), or for a code 2^-4 of the value
  and at least 2^-10 of the row's scale (half of the smallest subnormal);
* gather: one product and one rounding, the same as torch's: exact;
* attention: a score is a sum of hd products, off by at most (hd + 8) u times the sum
  of their sizes; a weight is off by twice the largest such error relative, and
  so is the output, times the largest |v| it averages, twice (numerator and
  denominator); sums of n terms add (n / 8 + 4 sqrt(n) + 32) u: up to 8 terms
  meet in one accumulation step that may truncate, the rest grows as a random
  walk; then half a step of the output's type.
"""
import math

import pytest
import torch

import decode_megakernel_06_b200 as mk

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)


DEV = "cuda:0"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rope_table(n, hd):
    inv = 1e4 ** (-2.0 * torch.arange(hd // 2, dtype=torch.float64) / hd)
    a = torch.arange(n, dtype=torch.float64)[:, None] * inv
    return torch.stack([a.cos(), a.sin()], -1).float()


class Cache:
    """A pool on the CPU with a shuffled page table; `cuda()` gives the PagedKV."""

    def __init__(self, lens, hkv, hd, page, kind, seed=0, extra=3, max_pages=None):
        g = gen(seed)
        need = [max(1, -(-n // page)) for n in lens]
        width = max_pages or max(need)
        self.n_pages = sum(need) + extra
        order = torch.randperm(self.n_pages, generator=g).tolist()
        self.table = torch.full((len(lens), width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.hkv, self.hd, self.page, self.kind = hkv, hd, page, kind
        shape = (self.n_pages, hkv, page, hd)
        x, y = torch.randn(shape, generator=g), torch.randn(shape, generator=g)
        if kind == BF16:
            self.k, self.v, self.ks, self.vs = x.to(BF16), y.to(BF16), None, None
        else:
            self.ks = x.abs().amax(-1) / 448
            self.vs = y.abs().amax(-1) / 448 * torch.exp2(torch.randint(-3, 4, shape[:3], generator=g).float())
            self.k = (x / self.ks[..., None]).to(E4M3)
            self.v = (y / (y.abs().amax(-1) / 448)[..., None]).to(E4M3)

    def cuda(self):
        up = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        self.kv = mk.PagedKV(up(self.k), up(self.v), up(self.table), up(self.ks), up(self.vs))
        return self.kv

    def at(self, b, p):
        """(page, slot) of a position, or None."""
        e = p // self.page
        if p < 0 or e >= self.table.shape[1]:
            return None
        pg = int(self.table[b, e])
        return (pg, p % self.page) if 0 <= pg < self.n_pages else None

    def rows(self, b, n):
        """k, v [n, hkv, hd] in 64 bits and which of the first n positions are held."""
        k, v = torch.zeros((n, self.hkv, self.hd), dtype=torch.float64), torch.zeros((n, self.hkv, self.hd), dtype=torch.float64)
        held = torch.zeros(n, dtype=torch.bool)
        for e in range(-(-n // self.page)):
            where = self.at(b, e * self.page)
            if where is None:
                continue
            lo, hi = e * self.page, min(n, (e + 1) * self.page)
            held[lo:hi] = True
            for out, pool, sc in ((k, self.k, self.ks), (v, self.v, self.vs)):
                x = pool[where[0]].double()
                if sc is not None:
                    x = x * sc[where[0]].double()[..., None]
                out[lo:hi] = x.transpose(0, 1)[:hi - lo]
        return k, v, held


def again(c):
    """A Cache of the same pages, to be uploaded anew."""
    d = object.__new__(Cache)
    d.__dict__.update({k: v for k, v in c.__dict__.items() if k != "kv"})
    return d


def turned(x, rope, p):
    """Rotate-half of x [..., hd] in 64 bits by the table's entry for p."""
    half = x.shape[-1] // 2
    c, s = rope[p, :, 0].double(), rope[p, :, 1].double()
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def check_attention(c, q, positions, counts=None, scale=None, rope=None, out=None, ws=None, stream=None, qgpu=None):
    """Runs the operator and compares every row with the formula."""
    B, T, hq, hd = q.shape
    qg = q.to(DEV) if qgpu is None else qgpu
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV) if out is None else out
    ws = mk.paged_attention_workspace(torch.device(DEV)) if ws is None else ws
    up = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    pos = torch.tensor(positions, dtype=torch.int32)
    cnt = None if counts is None else torch.tensor(counts, dtype=torch.int32)
    kv = getattr(c, "kv", None) or c.cuda()
    rc = kv.attention(qg, up(pos), out, ws, counts=up(cnt), scale=scale, rope=up(rope), stream=stream)
    assert rc == mk.MK_OK, mk.mk_last_error()
    torch.cuda.synchronize()
    got = out.cpu()
    compare_attention(c, q, positions, counts, scale, rope, got)
    return out


def compare_attention(c, q, positions, counts, scale, rope, got):
    B, T, hq, hd = q.shape
    sc = hd ** -0.5 if scale is None else scale
    sc = torch.tensor(sc, dtype=F32).double()
    G = hq // c.hkv
    eps = torch.finfo(q.dtype).eps / 2
    for b in range(B):
        n_rows = T if counts is None else max(0, min(T, counts[b]))
        assert (got[b, n_rows:] == 7.0).all(), "rows behind the sequence are left alone"
        top = min(positions[b] + n_rows, c.table.shape[1] * c.page)
        k, v, held = c.rows(b, max(top, 0))
        for t in range(n_rows):
            p = positions[b] + t
            n = max(0, min(p + 1, top))
            on = held[:n].nonzero()[:, 0]
            for h in range(c.hkv):
                qs = q[b, t, h * G:(h + 1) * G].double()
                g = got[b, t, h * G:(h + 1) * G].double()
                if len(on) == 0 or (rope is not None and p >= rope.shape[0]):
                    assert (g == 0).all(), (b, t, h)
                    continue
                rot = qs if rope is None else turned(qs, rope, p)
                kk, vv = k[on, h], v[on, h]
                s = rot @ kk.T * sc
                o = torch.softmax(s, -1) @ vv
                if not torch.isfinite(o).all():
                    assert torch.isnan(g).all(-1).equal(torch.isnan(o).all(-1)), (b, t, h)
                    fine = torch.isfinite(o).all(-1)
                    o, g, rot, s = o[fine], g[fine], rot[fine], s[fine]
                    if not len(o):
                        continue
                if rope is not None:  # three roundings of a rotated value
                    half = hd // 2
                    size = (qs.abs() + torch.cat([qs[:, half:], qs[:, :half]], -1).abs())
                    size = size[:len(o)] if len(size) != len(o) else size
                else:
                    size = rot.abs()
                ds = (hd + 12) * U * float((size @ kk.abs().T * sc.abs()).max())
                m = len(on)
                tol = (2 * (2 * ds) + (m / 8 + 4 * math.sqrt(m) + 32) * U) * float(vv.abs().max())
                bad = (g - o).abs() > tol + eps * o.abs()
                assert not bad.any(), (b, t, h, float((g - o).abs().max()), tol)


HEADS = [(4, 2, 64), (16, 4, 128), (8, 8, 64), (12, 2, 128), (9, 3, 64), (5, 1, 128), (16, 2, 128), (20, 2, 64)]


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("act", [F32, BF16], ids=["f32", "abf16"])
def test_attention_heads(heads, kind, act):
    hq, hkv, hd = heads
    T = 3
    lens = [T, T + 1, 130, 515]
    c = Cache(lens, hkv, hd, 24, kind, seed=hq)
    q = torch.randn((4, T, hq, hd), generator=gen(1)).to(act)
    check_attention(c, q, [n - T for n in lens], rope=rope_table(600, hd))


@pytest.mark.parametrize("page", [1, 7, 8, 16, 100, 128, 256])
@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_attention_pages_and_lengths(page, kind):
    lens = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 700]
    c = Cache(lens, 2, 128, page, kind, seed=page)
    q = torch.randn((len(lens), 1, 8, 128), generator=gen(2))
    check_attention(c, q, [n - 1 for n in lens])


@pytest.mark.parametrize("T", [2, 7, 8, 33, 70])
@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_attention_blocks(T, kind):
    lens = [T, T + 5, 300]
    c = Cache(lens, 2, 64, 16, kind, seed=T)
    q = torch.randn((3, T, 10, 64), generator=gen(3))
    check_attention(c, q, [n - T for n in lens], counts=[T, max(1, T // 2), 0])


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_attention_long_split(kind):
    """Long caches beside short ones: the work is split over blocks and joined."""
    lens = [9000, 1, 4097, 12345]
    c = Cache(lens, 1, 128, 64, kind, seed=5)
    q = torch.randn((4, 1, 4, 128), generator=gen(4))
    first = check_attention(c, q, [n - 1 for n in lens])
    again = check_attention(c, q, [n - 1 for n in lens])
    assert torch.equal(first, again)


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_attention_long_sums_do_not_drift(kind):
    """100k positions in fp32: each term's error is its own, so the output's is that of a
    term, not of the sum: 8 u for a weight (score, exponential, pieces), 8 u for the
    sums' own roundings and the truncation within a unit."""
    n, page, hd, hq, hkv = 100_000, 64, 128, 16, 4
    g = torch.Generator(device=DEV).manual_seed(31)
    pages = -(-n // page)
    k, v = (torch.randn((pages, hkv, page, hd), generator=g, device=DEV) for _ in range(2))
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    if kind == BF16:
        kv = mk.PagedKV(k.to(BF16), v.to(BF16), table)
        kk, vv = kv.k.double(), kv.v.double()
    else:
        sk, sv = k.abs().amax(-1) / 448, v.abs().amax(-1) / 448
        kv = mk.PagedKV((k / sk[..., None]).to(E4M3), (v / sv[..., None]).to(E4M3), table, sk, sv)
        kk, vv = kv.k.double() * sk.double()[..., None], kv.v.double() * sv.double()[..., None]
    q = torch.randn((1, 1, hq, hd), generator=g, device=DEV)
    out = torch.empty_like(q)
    assert kv.attention(q, torch.tensor([n - 1], dtype=torch.int32, device=DEV), out, mk.paged_attention_workspace(q.device)) == mk.MK_OK
    for h in range(hkv):
        a, b = kk[:, h].reshape(-1, hd)[:n], vv[:, h].reshape(-1, hd)[:n]
        ref = torch.softmax(q[0, 0, 4 * h:4 * h + 4].double() @ a.T * hd ** -0.5, -1) @ b
        assert float((out[0, 0, 4 * h:4 * h + 4].double() - ref).norm() / ref.norm()) <= 16 * U


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("act", [F32, BF16], ids=["f32", "abf16"])
def test_long_sums_keep_no_bias(kind, act):
    """A million positions (64 pages, again and again: the softmax is that over one round of them),
    with as many items as blocks, so that one warp adds 16384 units.  An error that always
    points towards zero grows with their number; errors of single roundings do not.  The
    mean relative error over N outputs in [1, 2): the outputs' own rounding, uniform
    within half a step h of at most 2^-8 (bf16), has a standard deviation of h / sqrt(3 N),
    of which 8 are allowed; and 64 u for the roundings of weights and sums."""
    B, hkv, hq, hd, page, pages, rounds = 60, 8, 32, 64, 64, 64, 256
    n = pages * page * rounds
    g = torch.Generator(device=DEV).manual_seed(41)
    k = torch.randn((pages, hkv, page, hd), generator=g, device=DEV)
    v = 1 + torch.rand((pages, hkv, page, hd), generator=g, device=DEV)
    table = torch.arange(pages, dtype=torch.int32, device=DEV).repeat(rounds).expand(B, -1).contiguous()
    if kind == BF16:
        kv = mk.PagedKV(k.to(BF16), v.to(BF16), table)
        kk, vv = kv.k.double(), kv.v.double()
    else:
        sk, sv = k.abs().amax(-1) / 448, v.abs().amax(-1) / 448
        kv = mk.PagedKV((k / sk[..., None]).to(E4M3), (v / sv[..., None]).to(E4M3), table, sk, sv)
        kk, vv = kv.k.double() * sk.double()[..., None], kv.v.double() * sv.double()[..., None]
    q = (2 * torch.randn((B, 1, hq, hd), generator=g, device=DEV)).to(act)
    out = torch.empty_like(q)
    pos = torch.full((B,), n - 1, dtype=torch.int32, device=DEV)
    assert kv.attention(q, pos, out, mk.paged_attention_workspace(q.device)) == mk.MK_OK
    kk, vv = (x.transpose(0, 1).reshape(hkv, pages * page, hd) for x in (kk, vv))
    qq = q[:, 0].double().reshape(B, hkv, hq // hkv, hd)
    ref = torch.softmax(qq @ kk.transpose(-1, -2) * hd ** -0.5, -1) @ vv
    err = (out[:, 0].double().reshape(ref.shape) - ref) / ref
    h = torch.finfo(act).eps / 2
    assert abs(float(err.mean())) <= 8 * h / math.sqrt(3 * err.numel()) + 64 * U


def test_attention_many_sequences():
    lens = [1 + (37 * i) % 90 for i in range(700)]
    c = Cache(lens, 2, 64, 16, BF16, seed=6)
    q = torch.randn((700, 1, 4, 64), generator=gen(5)).to(BF16)
    check_attention(c, q, [n - 1 for n in lens])


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("lo,hi", [(700, 2600), (1500, 1500)])
def test_attention_equal_parts_of_many_sequences(kind, lo, hi):
    """More than 32 sequences, each long enough to be cut into several parts of one size."""
    lens = [lo + (hi - lo) * ((29 * i) % 37) // 36 for i in range(37)]
    c = Cache(lens, 1, 64, 48, kind, seed=39)
    q = torch.randn((37, 2, 3, 64), generator=gen(40))
    check_attention(c, q, [n - 2 for n in lens], counts=[2 - (i % 5 == 4) for i in range(37)])


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_attention_rows_that_see_nothing(kind):
    lens = [40, 40, 40, 40, 40]
    c = Cache(lens, 2, 64, 16, kind, seed=7)
    c.table[1] = -1                      # nothing mapped
    c.table[2, 1] = 10 ** 6              # a page outside the pool
    c.table[3, 0] = -5                   # a hole at the start
    q = torch.randn((5, 4, 4, 64), generator=gen(6))
    # sequence 0 starts before its cache: rows 0 and 1 see nothing
    check_attention(c, q, [-2, 36, 36, 14, 36], counts=[4, 4, 4, 4, -3])
    check_attention(c, q, [-9, 36, 36, 100, 36])  # past the table's end: what is mapped
    check_attention(c, q, [0, 36, 36, 36, 36], rope=rope_table(38, 64))  # rows past rope


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attention_ignores_what_is_masked(kind, bad):
    T = 5
    lens = [T, 60, 131]
    c = Cache(lens, 2, 64, 16, kind, seed=8)
    used = {int(p) for row in c.table for p in row if p >= 0}
    for pg in range(c.n_pages):
        if pg not in used:
            c.k[pg], c.v[pg] = float("nan"), float("nan")
            if kind == E4M3:
                c.ks[pg], c.vs[pg] = bad, bad
    for b, n in enumerate(lens):  # slots behind each sequence's last position
        pg, slot = c.at(b, n - 1)
        for pool in (c.k, c.v):
            pool[pg, :, slot + 1:] = float("nan") if kind == E4M3 else bad
        if kind == E4M3:
            c.ks[pg, :, slot + 1:] = c.vs[pg, :, slot + 1:] = bad
    # a block's own newest position is bad: only the rows that see it may show it
    pg, slot = c.at(2, lens[2] - 1)
    c.v[pg, 0, slot, 3] = float("nan")
    c.k[pg, 1, slot, 5] = float("nan")
    pg, slot = c.at(1, lens[1] - 2)
    if kind == E4M3:
        c.vs[pg, :, slot] = bad
    else:
        c.v[pg, :, slot] = bad
    q = torch.randn((3, T, 4, 64), generator=gen(9))
    ws = mk.paged_attention_workspace(torch.device(DEV))
    out = torch.full(q.shape, 7.0, device=DEV)
    c.cuda()
    pos = [n - T for n in lens]
    rc = c.kv.attention(q.to(DEV), torch.tensor(pos, dtype=torch.int32, device=DEV), out, ws)
    assert rc == mk.MK_OK
    got = out.cpu()
    # rows before the bad positions are finite and right; later ones follow the formula
    compare_attention(c, q[:, :3], pos, None, None, None, got[:, :3])
    assert torch.isfinite(got[0]).all() and torch.isfinite(got[2, :4]).all()
    assert not torch.isfinite(got[1, 3:]).any()
    assert torch.isnan(got[2, 4, :2, 3]).all() and torch.isfinite(got[2, 4, :2, :3]).all()  # v: its dimension alone
    assert torch.isnan(got[2, 4, 2:]).all()  # k: the whole row


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("act", [F32, BF16], ids=["f32", "abf16"])
@pytest.mark.parametrize("at", [3, 61, 130])
def test_attention_scores_of_minus_infinity(kind, act, at):
    """A key (or its scale) that is not finite and scores -inf: the rows that see it are
    not finite, wherever it stands; rows before it and the other head are right."""
    T, n = 5, 133
    c = Cache([n, n], 2, 64, 16, kind, seed=34)
    pg, slot = c.at(0, at)
    if kind == BF16:
        c.k[pg, 0, slot, 9] = -float("inf")
    else:
        c.k[pg, 0, slot] = (-c.k[pg, 0, slot].float().abs() - 1).to(E4M3)
        c.ks[pg, 0, slot] = float("inf")
    q = (torch.rand((2, T, 4, 64), generator=gen(35)) + 0.5).to(act)
    out = torch.full(q.shape, 7.0, dtype=act, device=DEV)
    c.cuda()
    pos = [n - T, n - T]
    ws = mk.paged_attention_workspace(torch.device(DEV))
    assert c.kv.attention(q.to(DEV), torch.tensor(pos, dtype=torch.int32, device=DEV), out, ws) == mk.MK_OK
    got = out.cpu().float()
    sees = torch.arange(n - T, n) >= at
    assert not torch.isfinite(got[0, sees, :2]).any() and torch.isfinite(got[0, ~sees, :2]).all()
    assert torch.isfinite(got[0, :, 2:]).all() and torch.isfinite(got[1]).all()
    if kind == BF16:
        c.k[pg, 0, slot, 9] = 0
    else:
        c.ks[pg, 0, slot] = 1.0
    good = check_attention(again(c), q, pos).cpu()
    got = out.cpu()
    got[0, sees, :2] = good[0, sees, :2]
    compare_attention(c, q, pos, None, None, None, got)


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_attention_scores_beyond_fp32(kind):
    """Rows whose every score is -inf see positions all the same: NaN, not the zeros of a row
    that sees none."""
    c = Cache([70], 1, 64, 16, kind, seed=36)
    c.k = c.k.float().abs().clamp_min(0.25).to(kind)
    q = torch.ones((1, 2, 4, 64))
    q[0, :, 1, 3] = -float("inf")
    q[0, :, 2] = -1e38
    out = torch.full(q.shape, 7.0, device=DEV)
    ws = mk.paged_attention_workspace(torch.device(DEV))
    pos = torch.tensor([68], dtype=torch.int32, device=DEV)
    assert c.cuda().attention(q.to(DEV), pos, out, ws, scale=100.0) == mk.MK_OK
    got = out.cpu()
    assert torch.isnan(got[0, :, 1:3]).all() and torch.isfinite(got[0, :, ::3]).all()


@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_attention_extreme_scores(kind):
    lens = [200, 200]
    c = Cache(lens, 2, 64, 16, kind, seed=10)
    q = torch.randn((2, 2, 4, 64), generator=gen(10))
    check_attention(c, q * 200, [198, 198])            # one weight carries a row
    check_attention(c, q, [198, 198], scale=0.0)       # the mean
    check_attention(c, q, [198, 198], scale=-0.3)
    check_attention(c, torch.zeros_like(q), [198, 198])
    check_attention(c, q * 1e-30, [198, 198])
    q[0, 1, 2, 7] = float("nan")
    q[1, 0, 0, 0] = float("inf")
    check_attention(c, q, [198, 198])                  # those rows alone are NaN


def test_attention_values_of_very_different_size():
    """Scales from 2^-60 to 2^40: a huge value with no weight must not cost the others."""
    lens = [300]
    c = Cache(lens, 1, 64, 16, E4M3, seed=11)
    pg, slot = c.at(0, 7)
    c.vs[pg, 0, slot] = 2.0 ** 40
    c.k[pg, 0, slot] = (-c.k[pg, 0, slot].float().abs()).to(E4M3)
    c.ks[pg, 0, slot] = 40.0                           # far below every other score
    for p in range(100, 200):
        pg, slot = c.at(0, p)
        c.vs[pg, 0, slot] = 2.0 ** -60
    q = torch.rand((1, 1, 4, 64), generator=gen(11)) + 0.5
    out = check_attention(c, q, [299])
    k, v, _ = c.rows(0, 300)
    p = torch.softmax(q[0, 0].double() @ k[:, 0].T / 8, -1)
    ref = p @ v[:, 0]
    assert float(p[:, 7].max()) < 2.0 ** -100
    # the same bound with the values that carry weight: the huge one is out of it
    others = torch.arange(300) != 7
    rest = float(v[others, 0].abs().max())
    ds = 76 * U * float((q[0, 0].double() @ k[others, 0].abs().T / 8).max())
    assert float((out[0, 0].cpu().double() - ref).abs().max()) <= (4 * ds + 150 * U) * rest


@pytest.mark.parametrize("exp", [-70, -84, -100, -113, -126])
@pytest.mark.parametrize("act", [F32, BF16], ids=["f32", "abf16"])
def test_attention_tiny_value_scales(exp, act):
    """Value scales down to 2^-126, the least that an append gives, to the same relative bound;
    beside far smaller ones, rows of zeros, and a large one that only the last row sees."""
    T = 4
    lens = [33, 150, 90, 64]
    c = Cache(lens, 2, 64, 16, E4M3, seed=37)
    c.vs = torch.exp2(torch.full_like(c.vs, exp))
    for p in range(0, 90, 3):
        pg, slot = c.at(2, p)
        c.vs[pg, :, slot] = 2.0 ** max(exp - 20, -126)
        pg, slot = c.at(2, p + 1)
        c.v[pg, :, slot], c.vs[pg, :, slot] = 0, 2.0 ** -126
    pg, slot = c.at(3, 63)
    c.vs[pg, :, slot] = 1.0
    q = torch.randn((4, T, 10, 64), generator=gen(38)).to(act)
    check_attention(c, q, [n - T for n in lens], rope=rope_table(160, 64))


def test_attention_operand_layouts():
    """q as a slice of a fused row, then at an odd offset (no 16-byte loads)."""
    lens = [70, 90]
    c = Cache(lens, 2, 64, 16, E4M3, seed=12)
    c.cuda()
    for off, width in ((0, 8 * 64), (1, 8 * 64 + 3)):
        fused = torch.randn((2, 2, width), generator=gen(12)).to(DEV)
        q = fused[:, :, off:off + 4 * 64].unflatten(-1, (4, 64))
        check_attention(c, q.cpu(), [68, 88], qgpu=q)


def test_attention_large_pool():
    """A pool whose element offsets pass 32 bits, used at its end."""
    n_pages, page, hd = 66000, 256, 128
    k = torch.empty((n_pages, 1, page, hd), dtype=E4M3, device=DEV)
    v = torch.empty((n_pages, 1, page, hd), dtype=E4M3, device=DEV)
    ks, vs = torch.ones((n_pages, 1, page), device=DEV), torch.ones((n_pages, 1, page), device=DEV)
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32, device=DEV)
    kv = mk.PagedKV(k, v, table, ks, vs)
    x = torch.randn((1, 300, 1, hd), generator=gen(13)).to(DEV)
    y = torch.randn((1, 300, 1, hd), generator=gen(14)).to(DEV)
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert kv.append(x, y, zero) == mk.MK_OK
    c = Cache([300], 1, hd, page, E4M3, extra=0)
    c.table = torch.tensor([[1, 0]], dtype=torch.int32)
    c.k, c.v, c.ks, c.vs = k[-2:].cpu(), v[-2:].cpu(), ks[-2:].cpu(), vs[-2:].cpu()
    c.n_pages = 2
    back = [torch.zeros((1, 300, 1, hd), device=DEV) for _ in range(2)]
    assert kv.gather(zero, *back) == mk.MK_OK
    rk, rv, held = c.rows(0, 300)
    assert held.all()
    assert torch.equal(back[0][0].cpu(), rk.float()) and torch.equal(back[1][0].cpu(), rv.float())
    assert float((back[0] - x).abs().max()) <= 2.0 ** -4 * float(x.abs().max())
    q = torch.randn((1, 1, 4, hd), generator=gen(15))
    c.kv = kv
    check_attention(c, q, [299])


def test_attention_streams_and_graphs():
    """Two streams at once with a workspace each; a captured call replayed on new
    positions, queries and table."""
    lens = [600, 200]
    c = Cache(lens, 2, 128, 16, BF16, seed=16)
    c.cuda()
    q = [torch.randn((2, 1, 8, 128), generator=gen(17 + i)) for i in range(4)]
    ws = [mk.paged_attention_workspace(torch.device(DEV)) for _ in range(2)]
    outs = [torch.full(q[0].shape, 7.0, device=DEV) for _ in range(4)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    qg = [x.to(DEV) for x in q]
    pos = [torch.tensor([n - 1 - i for n in lens], dtype=torch.int32, device=DEV) for i in range(4)]
    torch.cuda.synchronize()
    for i in range(4):
        assert c.kv.attention(qg[i], pos[i], outs[i], ws[i % 2], stream=streams[i % 2]) == mk.MK_OK
    torch.cuda.synchronize()
    for i in range(4):
        compare_attention(c, q[i], [n - 1 - i for n in lens], None, None, None, outs[i].cpu())
    graph = torch.cuda.CUDAGraph()
    p, x, out = pos[0].clone(), qg[0].clone(), torch.full(q[0].shape, 7.0, device=DEV)
    with torch.cuda.graph(graph):
        assert c.kv.attention(x, p, out, ws[0]) == mk.MK_OK
    for i, at in ((1, [3, 150]), (2, [599, 0]), (3, [64, 199])):
        p.copy_(torch.tensor(at, dtype=torch.int32))
        x.copy_(q[i])
        graph.replay()
        torch.cuda.synchronize()
        compare_attention(c, q[i], at, None, None, None, out.cpu())


# ---- append and gather --------------------------------------------------------

def expected_codes(x):
    """The e4m3 rows of fp32 x: codes (as torch rounds them) and scales."""
    fin = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
    s = (fin.amax(-1) / 448).clamp_min(2.0 ** -126)
    y = x / s[..., None]
    y = torch.where(torch.isinf(y), torch.copysign(torch.full_like(y, 448.0), y), y)
    return y.to(E4M3), s


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("act", [F32, BF16], ids=["f32", "abf16"])
@pytest.mark.parametrize("page", [1, 16, 100])
@pytest.mark.parametrize("with_rope", [False, True])
def test_append(hd, kind, act, page, with_rope):
    B, T, hkv = 4, 37, 3
    starts, counts = [0, 5, 90, 40], [37, 0, 20, 37]
    c = Cache([s + T for s in starts], hkv, hd, page, kind, seed=20)
    c.table[3, 50 // page] = -1  # a hole: those rows are dropped
    k = torch.randn((B, T, hkv, hd), generator=gen(21)).to(act)
    v = (torch.randn((B, T, hkv, hd), generator=gen(22)) * 30).to(act)
    v[0, 3, 1] = 0.0
    rope = rope_table(200, hd) if with_rope else None
    c.cuda()
    before = [t.cpu().clone() if t is not None else None for t in (c.kv.k, c.kv.v, c.kv.k_scale, c.kv.v_scale)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    rc = c.kv.append(k.to(DEV), v.to(DEV), i32(starts), counts=i32(counts), rope=None if rope is None else rope.to(DEV))
    assert rc == mk.MK_OK, mk.mk_last_error()
    torch.cuda.synchronize()
    for name, x, pool, old, sc, old_sc in (("k", k, c.kv.k, before[0], c.kv.k_scale, before[2]),
                                           ("v", v, c.kv.v, before[1], c.kv.v_scale, before[3])):
        got, sgot = pool.cpu(), None if sc is None else sc.cpu()
        for b in range(B):
            for t in range(counts[b]):
                where = c.at(b, starts[b] + t)
                if where is None:
                    continue
                row, g = x[b, t].float(), got[where[0], :, where[1]]
                old[where[0], :, where[1]] = g  # what is left of `old` must be untouched
                if rope is not None and name == "k":
                    exact = turned(row.double(), rope, starts[b] + t)
                    half = hd // 2
                    off = 4 * U * (row.abs() + torch.cat([row[:, half:], row[:, :half]], -1).abs()).double()
                    if kind == BF16:
                        assert ((g.double() - exact).abs() <= 2.0 ** -8 * exact.abs() + off * 1.01).all()
                    else:
                        s = sgot[where[0], :, where[1]].double()
                        old_sc[where[0], :, where[1]] = s.float()
                        es = exact.abs().amax(-1) / 448
                        assert ((s - es).abs() <= 2 * U * es + off.amax(-1) / 448).all()
                        err = (g.double() * s[:, None] - exact).abs()
                        assert (err <= 2.0 ** -4 * exact.abs() + 2.0 ** -10 * s[:, None] + 2 * off).all()
                elif kind == BF16:
                    assert torch.equal(g, row.to(BF16))
                else:
                    codes, s = expected_codes(row)
                    old_sc[where[0], :, where[1]] = s
                    assert torch.equal(g.view(torch.uint8), codes.view(torch.uint8))
                    assert torch.equal(sgot[where[0], :, where[1]], s)
        assert torch.equal(got.view(torch.uint8), old.view(torch.uint8)), "other slots are left alone"
        if sgot is not None:
            assert torch.equal(sgot, old_sc)


def test_append_special_values():
    hd = 64
    c = Cache([8], 1, hd, 8, E4M3, seed=23)
    c.cuda()
    x = torch.randn((1, 8, 1, hd), generator=gen(24))
    x[0, 0, 0, 5] = float("inf")
    x[0, 1, 0, 6] = float("-inf")
    x[0, 2, 0, 7] = float("nan")
    x[0, 3] = 0.0
    x[0, 4] = 1e-42                                   # below the smallest scale
    x[0, 5] = float("inf")                            # nothing finite
    x[0, 6, 0, 0] = 3e38
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert c.kv.append(x.to(DEV), x.to(DEV), zero) == mk.MK_OK
    pg, _ = c.at(0, 0)
    codes, s = expected_codes(x[0, :, 0])
    got = c.kv.k.cpu()[pg, 0]
    nan = torch.isnan(x[0, :, 0])
    assert torch.equal(got.view(torch.uint8)[~nan], codes.view(torch.uint8)[~nan])
    assert torch.isnan(got.float()[nan]).all()
    assert torch.equal(c.kv.k_scale.cpu()[pg, 0], s) and torch.equal(c.kv.v_scale.cpu()[pg, 0], s)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("act", [F32, BF16], ids=["f32", "abf16"])
def test_append_midpoints_at_every_scale(hd, act):
    """Values at and next to the midpoints between codes, with scales from 2^-126 to 2^110
    of random mantissas: exactly the codes of the fp32 quotients x / scale (compared as the
    values they stand for: a zero may have either sign)."""
    g = gen(32)
    T, B = 237 * 4, 3
    e = (torch.arange(T) // 4 - 126).double()
    s = torch.exp2(e) * (1 + torch.rand((B, T), generator=g, dtype=torch.float64))
    amax = (448 * s).float().to(act).float()
    s = (amax / 448).clamp_min(2.0 ** -126).double()
    mid = torch.cat([(torch.arange(16, 32) + 0.5) / 16 * 2.0 ** i for i in range(-6, 8)])
    mid = torch.cat([mid, (torch.arange(16) + 0.5) * 2.0 ** -9])
    mid = mid[mid < 440]
    pick = mid[torch.randint(len(mid), (B, T, hd), generator=g)] * torch.where(torch.rand((B, T, hd), generator=g) < 0.5, -1, 1)
    x = (pick * s[..., None]).float()
    step = torch.randint(-2, 3, x.shape, generator=g)
    for _ in range(2):
        x = torch.where(step > 0, torch.nextafter(x, torch.full_like(x, 1e38)), x)
        x = torch.where(step < 0, torch.nextafter(x, torch.full_like(x, -1e38)), x)
        step = step - step.sign()
    x = x.to(act).float()
    x[..., 5] = amax
    codes, scales = expected_codes(x)
    c = Cache([T] * B, 1, hd, 64, E4M3, seed=33)
    c.cuda()
    xg = x[:, :, None].to(act).to(DEV)
    assert c.kv.append(xg, -xg, torch.zeros(B, dtype=torch.int32, device=DEV)) == mk.MK_OK
    minus = expected_codes(-x)[0]
    got_k, got_v, got_s = c.kv.k.cpu().float(), c.kv.v.cpu().float(), c.kv.k_scale.cpu()
    for b in range(B):
        where = [c.at(b, t) for t in range(T)]
        pg, slot = (torch.tensor([w[i] for w in where]) for i in (0, 1))
        assert torch.equal(got_s[pg, 0, slot], scales[b])
        assert torch.equal(got_k[pg, 0, slot], codes[b].float())
        assert torch.equal(got_v[pg, 0, slot], minus[b].float())


def test_append_outside_the_cache():
    """Negative positions, rows past the table and past rope are dropped."""
    c = Cache([16, 16, 16], 2, 64, 8, BF16, seed=25)
    c.cuda()
    k = torch.randn((3, 6, 2, 64), generator=gen(26)).to(DEV)
    old = c.kv.k.cpu().clone()
    pos = torch.tensor([-3, 13, 9], dtype=torch.int32, device=DEV)
    rope = torch.zeros((12, 32, 2), device=DEV)
    rope[..., 0] = 1.0  # turns nothing
    assert c.kv.append(k, k, pos, rope=rope) == mk.MK_OK
    got = c.kv.k.cpu()
    for b, t, p in [(0, 3, 0), (0, 4, 1), (0, 5, 2), (2, 0, 9), (2, 1, 10), (2, 2, 11)]:
        pg, slot = c.at(b, p)
        old[pg, :, slot] = k[b, t].cpu().to(BF16)
    assert torch.equal(got, old)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("kind", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("act", [F32, BF16], ids=["f32", "abf16"])
@pytest.mark.parametrize("layout", ["rows", "cache", "odd"])
def test_gather(hd, kind, act, layout):
    B, T, hkv, page = 3, 50, 3, 24
    starts, counts = [0, 17, 70], [50, 0, 33]
    c = Cache([s + T for s in starts], hkv, hd, page, kind, seed=27)
    c.table[2, 80 // page] = -1
    c.cuda()
    outs = []
    for _ in range(2):
        if layout == "rows":
            outs.append(torch.full((B, T, hkv, hd), 7.0, dtype=act, device=DEV))
        elif layout == "cache":  # [B, heads, capacity, hd]
            outs.append(torch.full((B, hkv, T + 6, hd), 7.0, dtype=act, device=DEV)[:, :, :T].transpose(1, 2))
        else:
            outs.append(torch.full((B, T, hkv * hd + 1), 7.0, dtype=act, device=DEV)[..., 1:].unflatten(-1, (hkv, hd)))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    assert c.kv.gather(i32(starts), *outs, counts=i32(counts)) == mk.MK_OK, mk.mk_last_error()
    torch.cuda.synchronize()
    for b in range(B):
        k, v, _ = c.rows(b, starts[b] + T)
        for x, out in ((k, outs[0].cpu()), (v, outs[1].cpu())):
            n = counts[b]
            assert torch.equal(out[b, :n], x[starts[b]:starts[b] + n].float().to(act))
            assert (out[b, n:] == 7.0).all()


def test_round_trip_into_the_contiguous_cache():
    """Append, gather into [B, heads, capacity, hd], append again: the same pages."""
    c = Cache([40, 40], 2, 64, 16, BF16, seed=28)
    c.cuda()
    zero = torch.zeros(2, dtype=torch.int32, device=DEV)
    cache = [torch.zeros((2, 2, 64, 64), dtype=BF16, device=DEV) for _ in range(2)]
    views = [x[:, :, :40].transpose(1, 2) for x in cache]
    assert c.kv.gather(zero, *views) == mk.MK_OK
    other = Cache([40, 40], 2, 64, 8, BF16, seed=29)
    other.cuda()
    assert other.kv.append(*views, zero) == mk.MK_OK
    back = [torch.zeros_like(v) for v in views]
    assert other.kv.gather(zero, *back) == mk.MK_OK
    assert all(torch.equal(a, b) for a, b in zip(views, back))


def test_tensor_refusals():
    c = Cache([40, 40], 2, 64, 16, E4M3, seed=30)
    kv = c.cuda()
    z = torch.zeros(2, dtype=torch.int32, device=DEV)
    row = torch.zeros((2, 3, 2, 64), device=DEV)
    ws = mk.paged_attention_workspace(torch.device(DEV))
    bad = [
        lambda: mk.PagedKV(kv.k, kv.v, kv.page_table),
        lambda: mk.PagedKV(kv.k, kv.v[:-1], kv.page_table, kv.k_scale, kv.v_scale),
        lambda: mk.PagedKV(kv.k, kv.v, kv.page_table.long(), kv.k_scale, kv.v_scale),
        lambda: mk.PagedKV(kv.k, kv.v, kv.page_table, kv.k_scale[:, :1], kv.v_scale),
        lambda: kv.append(row.half(), row.half(), z), lambda: kv.append(row, row.bfloat16(), z),
        lambda: kv.append(row[:1], row[:1], z), lambda: kv.append(row[..., :32], row[..., :32], z),
        lambda: kv.append(row, row, z[:1]), lambda: kv.append(row, row, z.long()),
        lambda: kv.append(row.cpu(), row.cpu(), z), lambda: kv.append(row, row, z, counts=z[:1]),
        lambda: kv.append(row, row, z, rope=torch.zeros((9, 16, 2), device=DEV)),
        lambda: kv.gather(z, row[:, :1].expand(2, 3, 2, 64), row),
        lambda: kv.attention(row, z, row[:, :, :1].contiguous(), ws),
        lambda: kv.attention(row, z, row.bfloat16(), ws), lambda: kv.attention(row, z, row, ws.int())]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    out = torch.zeros((2, 3, 3, 64), device=DEV)
    assert kv.attention(out, z, out.clone(), ws) == mk.MK_ERR_ARG  # 3 heads over 2
    assert kv.attention(row, z, row.clone(), ws[:64]) == mk.MK_ERR_CAPACITY
