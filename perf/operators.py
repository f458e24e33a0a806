"""Cases, plain forms and framework calls of the serving operators: the paged
key/value cache (written, read back, attended to) and the verification of
drafted tokens.

A case is a dict with its operator under ``"op"``:

* ``append``: new keys and values rotated, rounded or quantised, and written
  into the pages of a cache;
* ``gather``: positions of a paged cache read back into contiguous rows;
* ``attention``: attention of the newest tokens of each sequence over its pages;
* ``verify``: acceptance of drafted tokens by the target's probabilities, and
  the token drawn after them.

Head layouts, contexts, vocabularies and batch sizes are those of the decoders
in ``synthetic`` (4/2 heads of 64, 16/4 and 32/8 of 128; contexts of 127 to
4095 tokens; blocks of 1 and 7 rows; vocabularies of 1024, 32000 and 64000) and
of longer caches.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY_SCALE = 2.0 ** -126  # smallest scale a row of an 8-bit cache is given
MASS = 2.0 ** 46          # fixed-point unit of the sampler's masses


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # One token of the tiny decoder: latency alone.
        _attention("attention_tiny_bs1", 1, 1, 4, 2, 64, 16, 128, 128, "bf16", "f32", False),
        # The large decoder's batch of 8 single tokens at a context of 4096.
        _attention("attention_large_bs8", 8, 1, 32, 8, 128, 64, 4096, 4096, "bf16", "f32", True),
        # Small-batch serving: contexts of 512 to 2048, 8-bit cache, odd page size.
        _attention("attention_ragged_bs32", 32, 1, 16, 4, 128, 24, 512, 2048, "e4m3", "bf16", False),
        # The verify block of 7 rows for 8 sequences at a context of 2048.
        _attention("attention_verify56", 8, 7, 16, 4, 128, 32, 2048, 2055, "e4m3", "f32", True),
        # Long-document serving: four caches of 128k tokens.
        _attention("attention_long_bs4", 4, 1, 32, 8, 128, 64, 131071, 131072, "bf16", "bf16", False),
        # One decode step's rows, 8 sequences.
        _append("append_decode_bs8", 8, 1, 8, 128, 64, 4096, 4096, "e4m3", "f32", True, False),
        # Prompts of up to 4096 tokens written into an 8-bit cache, ragged.
        _append("append_prompt_bs8", 8, 4096, 8, 128, 64, 0, 0, "e4m3", "bf16", True, True),
        # A few pages read back for one sequence.
        _gather("gather_bs1", 1, 200, 4, 128, 16, 17, 17, "e4m3", "bf16", False),
        # Whole sequences of an 8-bit cache expanded to bf16.
        _gather("gather_bs16", 16, 4096, 8, 128, 32, 0, 0, "e4m3", "bf16", True),
        # One sequence with three drafts from a prompt's n-grams (no draft logits).
        _verify("verify_tiny_bs1", 1, 4, 1024, 1.0, 1.0, 0),
        # The 56-row verify block on the small decoder's vocabulary, nucleus 0.9.
        _verify("verify_small_56", 8, 7, 32000, 0.8, 0.9, 1),
        # The same block size on the large vocabulary, whole distribution.
        _verify("verify_large_64", 8, 8, 64000, 1.0, 1.0, 1),
    ]


def _attention(name, batch, tokens, q_heads, kv_heads, head_dim, page, lo, hi, cache, act, rope):
    return dict(name=name, op="attention", batch=batch, tokens=tokens, q_heads=q_heads, kv_heads=kv_heads,
                head_dim=head_dim, page=page, lo=lo, hi=hi, cache=cache, act=act, rope=rope)


def _append(name, batch, tokens, kv_heads, head_dim, page, lo, hi, cache, act, rope, ragged):
    return dict(name=name, op="append", batch=batch, tokens=tokens, kv_heads=kv_heads, head_dim=head_dim, page=page,
                lo=lo, hi=hi, cache=cache, act=act, rope=rope, ragged=ragged)


def _gather(name, batch, tokens, kv_heads, head_dim, page, lo, hi, cache, act, ragged):
    return dict(name=name, op="gather", batch=batch, tokens=tokens, kv_heads=kv_heads, head_dim=head_dim, page=page,
                lo=lo, hi=hi, cache=cache, act=act, ragged=ragged)


def _verify(name, batch, tokens, vocab, temperature, top_p, drafts):
    return dict(name=name, op="verify", batch=batch, tokens=tokens, vocab=vocab, temperature=temperature,
                top_p=top_p, drafts=drafts)


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "gather", "verify", "verify"])
    heads, head_dim = rng.choice([((4, 2), 64), ((16, 4), 128), ((32, 8), 128), ((8, 8), 64), ((12, 2), 128),
                                  ((16, 2), 128), ((9, 3), 64), ((5, 1), 128)])
    page = rng.choice([8, 16, 24, 32, 64, 100, 128, 256])
    cache, act = rng.choice(["bf16", "e4m3"]), rng.choice(["f32", "bf16"])
    if op == "attention":
        batch, tokens = _log_int(rng, 1, 48), rng.choice([1, 1, 1, 2, 3, 5, 7, 8])
        # at most half of the longest listed case's cache
        most = max(64, int(4 * 131072 * 8 * 128 / 2 / (batch * heads[1] * head_dim)))
        hi = _log_int(rng, 32, min(131072, most))
        lo = max(tokens, int(hi * rng.uniform(0.2, 1.0)))
        return _attention("", batch, tokens, heads[0], heads[1], head_dim, page, min(lo, hi), hi, cache, act,
                          rng.random() < 0.5) | {"name": "drawn"}
    if op == "append":
        tokens = rng.choice([1, 1, 2, 7, _log_int(rng, 9, 3000)])
        batch = _log_int(rng, 1, max(1, min(64, 16000 // tokens)))
        lo = rng.randrange(0, 3000)
        return _append("drawn", batch, tokens, heads[1], head_dim, page, lo, lo + rng.randrange(0, 1000), cache, act,
                       rng.random() < 0.5, rng.random() < 0.5)
    if op == "gather":
        tokens = _log_int(rng, 1, 4096)
        batch = _log_int(rng, 1, max(1, min(48, 40000 // tokens)))
        lo = rng.randrange(0, 500)
        return _gather("drawn", batch, tokens, heads[1], head_dim, page, lo, lo + rng.randrange(0, 200), cache, act,
                       rng.random() < 0.5)
    batch, tokens = _log_int(rng, 1, 16), rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    return _verify("drawn", batch, tokens, _log_int(rng, 500, 64000), rng.choice([0.0, 0.5, 0.7, 0.8, 1.0, 1.25]),
                   rng.choice([0.5, 0.8, 0.9, 0.95, 1.0, 1.0]), rng.choice([0, 1, 1, 1]))


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spread."""
    return [lo + (hi - lo) * i // (n - 1) if n > 1 else hi for i in range(n)]


def _counts(case):
    """Rows of each sequence: all of them, or from a third of them up to all."""
    b, t = case["batch"], case["tokens"]
    return _spread(max(1, t // 3), t, b) if case["ragged"] else [t] * b


# ---- inputs -----------------------------------------------------------------

def _dtype(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[name]


def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed(1009 * seed + salt)


def _quantise(x):
    """fp32 rows to e4m3 codes and one scale a row: amax / 448 (at least 2^-126)."""
    scale = (x.abs().amax(-1) / E4M3_MAX).clamp_min(TINY_SCALE)
    return (x / scale.unsqueeze(-1)).to(torch.float8_e4m3fn), scale


def _pool(case, seed, salt, n_pages):
    """A cache pool of N(0, 1) rows: the pages and, for 8 bits, their scales."""
    shape = (n_pages, case["kv_heads"], case["page"], case["head_dim"])
    if case["cache"] == "bf16":
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=_gen(seed, salt)), None
    codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(shape[:3], dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
    g = _gen(seed, salt)
    for i in range(0, n_pages, step):
        x = torch.randn((min(step, n_pages - i),) + shape[1:], generator=g, device="cuda")
        codes[i:i + step], scales[i:i + step] = _quantise(x)
    return codes, scales


def _pages(case, seed, lens):
    """A page table [batch, pages of the longest]: pages in shuffled order, -1
    behind each sequence's last, and the pool's size (a few pages are free)."""
    need = [-(-n // case["page"]) for n in lens]
    g = torch.Generator().manual_seed(7 * seed + 3)
    order = torch.randperm(sum(need) + 3, generator=g).tolist()
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (max(need) - n))
        at += n
    return torch.tensor(table, dtype=torch.int32, device="cuda").reshape(len(lens), max(need)), len(order)


def _rope_table(length, head_dim):
    inv = 1e4 ** (-2.0 * torch.arange(head_dim // 2, dtype=torch.float64, device="cuda") / head_dim)
    a = torch.arange(length, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.stack([a.cos(), a.sin()], -1).float()


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    st = {"case": dict(case)}
    if case["op"] == "verify":
        return _prepare_verify(case, seed, st)
    b, t, hkv, hd = case["batch"], case["tokens"], case["kv_heads"], case["head_dim"]
    if case["op"] == "attention":
        lens = _spread(case["lo"], case["hi"], b)
        st["positions"] = _ints([n - t for n in lens])
        st["q"] = torch.randn((b, t, case["q_heads"], hd), generator=_gen(seed, 1), device="cuda").to(_dtype(case["act"]))
        st["out"] = torch.empty_like(st["q"])
    else:
        starts, counts = _spread(case["lo"], case["hi"], b), _counts(case)
        lens = [s + c for s, c in zip(starts, counts)]
        st["positions"], st["counts"] = _ints(starts), _ints(counts)
        shape, dt = (b, t, hkv, hd), _dtype(case["act"])
        if case["op"] == "append":
            st["k_new"] = torch.randn(shape, generator=_gen(seed, 1), device="cuda").to(dt)
            st["v_new"] = torch.randn(shape, generator=_gen(seed, 2), device="cuda").to(dt)
        else:  # rows of a contiguous cache [batch, heads, tokens, head_dim], seen token by token
            st["out_k"] = torch.full((b, hkv, t, hd), 0.5, dtype=dt, device="cuda").transpose(1, 2)
            st["out_v"] = torch.full((b, hkv, t, hd), -0.5, dtype=dt, device="cuda").transpose(1, 2)
    st["table"], n_pages = _pages(case, seed, lens)
    st["longest"] = max(lens)
    st["k"], st["k_scale"] = _pool(case, seed, 11, n_pages)
    st["v"], st["v_scale"] = _pool(case, seed, 12, n_pages)
    st["rope"] = _rope_table(max(lens), hd) if case.get("rope") else None
    if own:
        import decode_megakernel_06_b200 as mk

        st["cache"] = mk.PagedKV(st["k"], st["v"], st["table"], st["k_scale"], st["v_scale"])
        if case["op"] == "attention":
            st["workspace"] = mk.paged_attention_workspace(st["q"].device)
    return st


def _prepare_verify(case, seed, st):
    """Target logits N(0, 2), draft logits near them (N(0, 0.5) off), drafts
    drawn from the draft's own distribution (or from the target's, without draft
    logits), uniforms in [0, 1)."""
    b, t, v = case["batch"], case["tokens"], case["vocab"]
    st["logits"] = 2.0 * torch.randn((b, t, v), generator=_gen(seed, 1), device="cuda")
    near = st["logits"][:, :t - 1] + 0.5 * torch.randn((b, t - 1, v), generator=_gen(seed, 2), device="cuda")
    noise = torch.rand((b, t - 1, v), generator=_gen(seed, 3), device="cuda").clamp(1e-9, 1 - 1e-7)
    temperature = case["temperature"] if case["temperature"] > 0 else 0.05
    gumbel = -torch.log(-torch.log(noise))
    st["tokens"] = torch.zeros((b, t), dtype=torch.int32, device="cuda")
    if t > 1:
        st["tokens"][:, 1:] = (near / temperature + gumbel).argmax(-1)
    st["draft_logits"] = near if case["drafts"] else None
    st["uniforms"] = torch.rand((b, t), generator=_gen(seed, 4), device="cuda", dtype=torch.float64)
    st["out_tokens"] = torch.empty((b, t), dtype=torch.int32, device="cuda")
    st["out_accepted"] = torch.empty((b,), dtype=torch.int32, device="cuda")
    if own:
        import decode_megakernel_06_b200 as mk

        st["workspace"] = mk.verify_sample_workspace(b, t, v, st["logits"].device)
    return st


# ---- one pass ---------------------------------------------------------------

def run(st):
    case = st["case"]
    if own:
        return _RUN_OWN[case["op"]](st)
    return _RUN_PLAIN[case["op"]](st)


def _checked(code):
    if code != 0:
        import decode_megakernel_06_b200 as mk

        raise RuntimeError(mk.mk_last_error())


def _own_append(st):
    _checked(st["cache"].append(st["k_new"], st["v_new"], st["positions"], counts=st["counts"], rope=st["rope"]))
    return _pools(st)


def _own_gather(st):
    _checked(st["cache"].gather(st["positions"], st["out_k"], st["out_v"], counts=st["counts"]))
    return {"k": st["out_k"], "v": st["out_v"]}


def _own_attention(st):
    _checked(st["cache"].attention(st["q"], st["positions"], st["out"], st["workspace"], rope=st["rope"]))
    return st["out"]


def _own_verify(st):
    import decode_megakernel_06_b200 as mk

    case = st["case"]
    _checked(mk.verify_sample(st["logits"], st["tokens"], case["temperature"], case["top_p"], st["uniforms"],
                              st["out_tokens"], st["out_accepted"], st["workspace"], draft_logits=st["draft_logits"]))
    return {"tokens": st["out_tokens"], "accepted": st["out_accepted"]}


def _pools(st):
    out = {"k": st["k"], "v": st["v"]}
    if st["k_scale"] is not None:
        out |= {"k_scale": st["k_scale"], "v_scale": st["v_scale"]}
    return out


def _rotate(x, rope, at):
    """Rotate-half of x [B, T, H, hd] at positions `at` [B, T], in fp32."""
    half = x.shape[-1] // 2
    cs = rope[at].unsqueeze(2)
    c, s = cs[..., 0], cs[..., 1]
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _where(st, steps):
    """For `steps` positions from each sequence's start: positions, pages, slots
    and whether each is within its count (all [B, steps])."""
    case = st["case"]
    t = torch.arange(steps, device="cuda")
    at = st["positions"].long()[:, None] + t
    inside = t < st["counts"][:, None]
    entry = (at // case["page"]).clamp_max(st["table"].shape[1] - 1)
    return at, st["table"].long().gather(1, entry), at % case["page"], inside


def _plain_append(st):
    case = st["case"]
    at, page, slot, inside = _where(st, case["tokens"])
    k, v = st["k_new"].float(), st["v_new"].float()
    if st["rope"] is not None:
        k = _rotate(k, st["rope"], at.clamp_max(st["rope"].shape[0] - 1))
    page, slot = page[inside], slot[inside]
    for new, pool, scales in ((k, st["k"], st["k_scale"]), (v, st["v"], st["v_scale"])):
        rows = new[inside]
        if scales is None:
            pool[page, :, slot] = rows.to(pool.dtype)
        else:
            codes, scale = _quantise(rows)
            pool.view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
            scales[page, :, slot] = scale
    return _pools(st)


def _values(pool, scales, index):
    x = pool.view(torch.uint8)[index].view(pool.dtype).float() if scales is not None else pool[index].float()
    return x if scales is None else x * scales[index].unsqueeze(-1)


def _plain_gather(st):
    case = st["case"]
    _, page, slot, inside = _where(st, case["tokens"])
    page = page.clamp_min(0)
    out = {}
    for name, old in (("k", st["out_k"]), ("v", st["out_v"])):
        heads = torch.arange(case["kv_heads"], device="cuda")
        index = (page[:, :, None], heads[None, None], slot[:, :, None])
        x = _values(st[name], st[name + "_scale"], index).to(old.dtype)
        out[name] = torch.where(inside[:, :, None, None], x, old)
    return out


def _plain_attention(st):
    case = st["case"]
    b, t, hq, hd = st["q"].shape
    hkv, n = case["kv_heads"], st["longest"]
    q = st["q"].float()
    at = st["positions"].long()[:, None] + torch.arange(t, device="cuda")
    if st["rope"] is not None:
        q = _rotate(q, st["rope"], at)
    g = hq // hkv
    q = q.reshape(b, t, hkv, g, hd).permute(0, 2, 1, 3, 4).reshape(b, hkv, t * g, hd)
    table = st["table"].long().clamp_min(0)

    def dense(pool, scales):  # [B, Hkv, pages * page_size, hd] -> the first n positions
        x = _values(pool, scales, table).transpose(1, 2)
        return x.reshape(b, hkv, -1, hd)[:, :, :n]

    scores = q @ dense(st["k"], st["k_scale"]).transpose(-1, -2) / math.sqrt(hd)
    seen = torch.arange(n, device="cuda") <= at[:, :, None]
    seen = seen[:, None, :, None].expand(b, 1, t, g, n).reshape(b, 1, t * g, n)
    scores = scores.masked_fill(~seen, -math.inf)
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    o = p @ dense(st["v"], st["v_scale"]) / p.sum(-1, keepdim=True)
    return o.reshape(b, hkv, t, g, hd).permute(0, 2, 1, 3, 4).reshape(b, t, hq, hd).to(st["q"].dtype)


def _single(x):
    """A float as the fp32 number that the call takes."""
    return torch.tensor(x, dtype=torch.float32).item()


def _masses(logits, temperature, top_p):
    """Fixed-point masses of each row's nucleus, in id order, and their sum."""
    l = logits.double()
    q = torch.round(torch.exp((l - l.amax(-1, keepdim=True)) * (1.0 / _single(temperature))) * MASS).long()
    total = q.sum(-1, keepdim=True)
    need = torch.ceil(_single(top_p) * total.double()).clamp_min(1.0).minimum(total.double()).long()
    order = torch.sort(logits, dim=-1, descending=True, stable=True).indices
    ranked = q.gather(-1, order)
    before = ranked.cumsum(-1) - ranked
    kept = torch.where(before < need, ranked, 0)
    a = torch.zeros_like(q).scatter(-1, order, kept)
    return a, a.sum(-1)


def _plain_verify(st):
    case = st["case"]
    b, t, v = st["logits"].shape
    drafts = st["tokens"].long()[:, 1:]
    u = st["uniforms"]
    ids = torch.arange(v, device="cuda")
    if not case["temperature"] > 0:
        top = st["logits"].amax(-1, keepdim=True)
        best = torch.where(st["logits"] == top, ids, v).amin(-1)
        kept = (drafts == best[:, :-1]).long().cumprod(-1).sum(-1)
        last = best.gather(1, kept[:, None])[:, 0]
        return _block(st, kept, last)
    a, a_sum = _masses(st["logits"], case["temperature"], case["top_p"])
    a_x = a[:, :-1].gather(-1, drafts[..., None])[..., 0].double()
    if st["draft_logits"] is not None and t > 1:
        d, d_sum = _masses(st["draft_logits"], case["temperature"], case["top_p"])
        d_x = d.gather(-1, drafts[..., None])[..., 0].double()
        ok = u[:, :-1] * (d_x * a_sum[:, :-1].double()) < a_x * d_sum.double()
    else:
        d = None
        ok = u[:, :-1] * a_sum[:, :-1].double() < a_x
    kept = ok.long().cumprod(-1).sum(-1)
    row = torch.arange(b, device="cuda")
    p, p_sum = a[row, kept], a_sum[row, kept]
    if t > 1:
        at = kept.clamp_max(t - 2)
        if d is None:
            rest = torch.where(ids == drafts[row, at][:, None], 0, p)
        else:
            share = torch.round(p.double() * (MASS / p_sum.double())[:, None]).long()
            other = torch.round(d[row, at].double() * (MASS / d_sum[row, at].double())[:, None]).long()
            rest = (share - other).clamp_min(0)
        use = (kept < t - 1) & (rest.sum(-1) > 0)
        p = torch.where(use[:, None], rest, p)
        p_sum = p.sum(-1)
    y = torch.minimum(torch.floor(u[:, -1] * p_sum.double()).long(), p_sum - 1)
    last = (p.cumsum(-1) <= y[:, None]).sum(-1)
    return _block(st, kept, last)


def _block(st, kept, last):
    """Accepted drafts, the drawn token, -1 behind it; and how many there are."""
    t = st["tokens"].shape[1]
    i = torch.arange(t, device="cuda")
    moved = torch.cat([st["tokens"][:, 1:], st["tokens"][:, :1]], 1)
    out = torch.where(i < kept[:, None], moved, -1)
    out = torch.where(i == kept[:, None], last[:, None].to(torch.int32), out)
    return {"tokens": out, "accepted": (kept + 1).to(torch.int32)}


_RUN_OWN = {"append": _own_append, "gather": _own_gather, "attention": _own_attention, "verify": _own_verify}
_RUN_PLAIN = {"append": _plain_append, "gather": _plain_gather, "attention": _plain_attention, "verify": _plain_verify}


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    b, t = case["batch"], case["tokens"]
    if case["op"] == "verify":
        rows = b * t + (b * (t - 1) if case["drafts"] and case["temperature"] > 0 else 0)
        return {"bytes": 4 * rows * case["vocab"] + 8 * b * t + 8 * b * t + 4 * b, "flops": rows * case["vocab"]}
    hkv, hd = case["kv_heads"], case["head_dim"]
    row = 2 * hkv * (2 * hd if case["cache"] == "bf16" else hd + 4)  # a position's keys and values
    act = 4 if case["act"] == "f32" else 2
    if case["op"] == "attention":
        lens = _spread(case["lo"], case["hi"], b)
        seen = sum(n - t + 1 + i for n in lens for i in range(t))
        io = 2 * b * t * case["q_heads"] * hd * act
        return {"bytes": sum(lens) * row + io, "flops": 4 * hd * case["q_heads"] * seen}
    n = sum(_counts(case))
    return {"bytes": n * (row + 2 * hkv * hd * act), "flops": n * 2 * hkv * hd * (3 if case.get("rope") else 1)}


# ---- the definitions in 64 bits ----------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return _EXACT[case["op"]](case, st)


def _places(case, st, b, first, count):
    """(page, slot) of `count` positions of sequence b."""
    p = torch.arange(first, first + count, device="cuda")
    return st["table"][b].long()[p // case["page"]], p % case["page"]


def _rows64(st, name, page, slot):
    """[count, Hkv, hd] in 64 bits."""
    pool, scales = st[name], st[name + "_scale"]
    if scales is None:
        return pool[page, :, slot].double()
    return pool.view(torch.uint8)[page, :, slot].view(pool.dtype).double() * scales[page, :, slot].double()[..., None]


def _turned64(x, rope, positions):
    """Each pair (i, i + hd/2) as a complex number, turned by its table entry."""
    half = x.shape[-1] // 2
    z = torch.complex(x[..., :half], x[..., half:])
    w = rope[positions].double()
    z = z * torch.complex(w[..., 0], w[..., 1])[:, None]
    return torch.cat([z.real, z.imag], -1)


def _exact_attention(case, st):
    b, t, hq, hd = st["q"].shape
    g = hq // case["kv_heads"]
    out = torch.zeros((b, t, hq, hd), dtype=torch.float64, device="cuda")
    for i in range(b):
        p0 = int(st["positions"][i])
        page, slot = _places(case, st, i, 0, p0 + t)
        k, v = _rows64(st, "k", page, slot), _rows64(st, "v", page, slot)
        q = st["q"][i].double()
        if st["rope"] is not None:
            q = _turned64(q, st["rope"], torch.arange(p0, p0 + t, device="cuda"))
        for j in range(t):
            n = p0 + j + 1
            for h in range(case["kv_heads"]):
                s = (k[:n, h] @ q[j, h * g:(h + 1) * g].T) * hd ** -0.5
                out[i, j, h * g:(h + 1) * g] = torch.softmax(s, 0).T @ v[:n, h]
    return out


def _exact_append(case, st):
    out = {"k": st["k"].double(), "v": st["v"].double()}
    if st["k_scale"] is not None:
        out |= {"k_scale": st["k_scale"].double(), "v_scale": st["v_scale"].double()}
    for i in range(case["batch"]):
        first, n = int(st["positions"][i]), int(st["counts"][i])
        page, slot = _places(case, st, i, first, n)
        k, v = st["k_new"][i, :n].double(), st["v_new"][i, :n].double()
        if st["rope"] is not None:
            k = _turned64(k, st["rope"], torch.arange(first, first + n, device="cuda"))
        for name, x in (("k", k), ("v", v)):
            if st[name + "_scale"] is not None:
                s = x.abs().amax(-1) / E4M3_MAX
                out[name + "_scale"][page, :, slot] = s
                x = x / s[..., None]
            out[name][page, :, slot] = x
    return out


def _exact_gather(case, st):
    out = {"k": st["out_k"].double(), "v": st["out_v"].double()}
    for i in range(case["batch"]):
        n = int(st["counts"][i])
        page, slot = _places(case, st, i, int(st["positions"][i]), n)
        for name in out:
            out[name][i, :n] = _rows64(st, name, page, slot)
    return out


def _nucleus64(row, temperature, top_p):
    """The nucleus masses of one row, by walking down its sorted tokens."""
    z = [(x - max(row)) / temperature for x in row]
    q = [round(math.exp(x) * 2 ** 46) if x > -40 else 0 for x in z]
    total = sum(q)
    need = max(1, min(total, math.ceil(top_p * float(total))))
    mass, got = [0] * len(row), 0
    for i in sorted(range(len(row)), key=lambda j: (-row[j], j)):
        if got >= need:
            break
        mass[i] = q[i]
        got += q[i]
    return mass, got


def _exact_verify(case, st):
    b, t, v = st["logits"].shape
    temperature, top_p = _single(case["temperature"]), _single(case["top_p"])
    if b * t * v > 1 << 21:  # rows of this many logits are walked in about 20 seconds
        return None
    tokens, counts = [], []
    drafts = st["tokens"].tolist()
    u = st["uniforms"].tolist()
    for i in range(b):
        got = []
        while len(got) < t:
            j = len(got)
            row = st["logits"][i, j].tolist()
            x = drafts[i][j + 1] if j + 1 < t else None
            if not temperature > 0:
                got.append(row.index(max(row)))
                if got[-1] != x:
                    break
                continue
            p, p_sum = _nucleus64(row, temperature, top_p)
            if x is not None:
                if st["draft_logits"] is None:
                    accept = u[i][j] * float(p_sum) < float(p[x])
                    rest = p[:x] + [0] + p[x + 1:]
                else:
                    d, d_sum = _nucleus64(st["draft_logits"][i, j].tolist(), temperature, top_p)
                    accept = u[i][j] * (float(d[x]) * float(p_sum)) < float(p[x]) * float(d_sum)
                    ps, ds = 2 ** 46 / float(p_sum), 2 ** 46 / float(d_sum)
                    rest = [max(0, round(m * ps) - round(n * ds)) for m, n in zip(p, d)]
                if accept:
                    got.append(x)
                    continue
                if sum(rest) > 0:
                    p, p_sum = rest, sum(rest)
            y = min(p_sum - 1, math.floor(u[i][t - 1] * float(p_sum)))
            run_sum = 0
            for token, m in enumerate(p):
                run_sum += m
                if run_sum > y:
                    got.append(token)
                    break
            break
        counts.append(len(got))
        tokens.append(got + [-1] * (t - len(got)))
    return {"tokens": _ints(tokens), "accepted": _ints(counts)}


_EXACT = {"append": _exact_append, "gather": _exact_gather, "attention": _exact_attention, "verify": _exact_verify}
