"""Cases of what long contexts need of the paged cache beyond its 16-bit and e4m3 forms: their inputs, their plain form in
elementary torch operations, the framework's calls, and their value in 64 bits.

Three operators:
  append  new tokens into the cache (16-bit, e4m3 or 4-bit) with the position rotation applied on the way, and their queries
          rotated beside them
  paged4  attention of each sequence's new tokens (one, a few, or a chunk) over a cache held in 4 bits
  select  the bounds of the keys of the pages that the new tokens came into, and attention of each token over the few pages
          that a score from those bounds selects for it

Token tensors are [tokens, heads, d]. Sequence s owns tokens cu[s] .. cu[s+1] - 1. A cache is
[pages, kv heads, page size, d]; position t of sequence s is slot t % page of page table[s, t // page]. Token i of
sequence s's new tokens has position length[s] - new[s] + i, and sees the positions up to its own.

4 bits: 32 neighbouring features of a vector share a scale, the largest of their magnitudes over 7 rounded to 4 significant
bits; a value is its nearest whole multiple, -7 to 7. A byte holds multiple + 8 of two neighbouring features, the first in its
low bits; a scale (1 + m / 8) 2^(e - 15) is the byte 8 e + m.

Rotation: features j and j + r/2 (or 2 j and 2 j + 1, interleaved) of the first r turn by the angle whose cosine and sine stand
in columns j and r/2 + j of the token's row of a table.

Bounds: largest and smallest key of a page for each feature, as whole multiples (8 bits) of the smallest power of two under
which all lie within 127; queries likewise, one power for each vector. A page's score is the largest over the query heads of
a group of the sum over features of max(query * largest, query * smallest): whole numbers times powers of two, so that the
choice is the same in any order of summation. A token's own page is always chosen, the others by score, the first of equal ones.
"""
import random

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
BLOCK = 1024  # query tokens that the plain form and the 64-bit form hold scores for at a time


def listed():
    return [
        # one step of a running batch: a token for each sequence is rotated into a 16-bit cache
        {"name": "append_step_f16", "op": "append", "dtype": "f16", "cache": "same", "d": 128, "hq": 32, "hkv": 8, "seqs": 24,
         "new": 24, "before": 6000, "page": 16, "rot": 128, "inter": False, "mix": 1},
        # a prefill batch of a small model into the 8-bit cache, half of the features rotated, neighbouring ones paired
        {"name": "append_prompt_e4m3", "op": "append", "dtype": "f16", "cache": "e4m3", "d": 64, "hq": 8, "hkv": 2, "seqs": 24,
         "new": 16384, "before": 5000, "page": 64, "rot": 32, "inter": True, "mix": 2},
        # a prefill batch of the large head dimension into the 4-bit cache
        {"name": "append_prompt_4bit", "op": "append", "dtype": "bf16", "cache": "4bit", "d": 128, "hq": 32, "hkv": 8, "seqs": 24,
         "new": 16384, "before": 5000, "page": 16, "rot": 128, "inter": False, "mix": 3},
        # one user, one token over a short cache: the latency of a step
        {"name": "paged4_one_f16", "op": "paged4", "dtype": "f16", "cache": "4bit", "d": 128, "hq": 32, "hkv": 8, "seqs": 1,
         "new": 1, "before": 4001, "page": 16, "mix": 4},
        # a full decoding batch of ragged contexts, as many sequences as fit a cache of a quarter of the size
        {"name": "paged4_batch_bf16", "op": "paged4", "dtype": "bf16", "cache": "4bit", "d": 128, "hq": 32, "hkv": 8, "seqs": 128,
         "new": 128, "before": 1000000, "page": 32, "mix": 5},
        # a step that checks a few drafted tokens of each sequence
        {"name": "paged4_few_f16_d64", "op": "paged4", "dtype": "f16", "cache": "4bit", "d": 64, "hq": 8, "hkv": 2, "seqs": 40,
         "new": 160, "before": 400000, "page": 64, "mix": 6},
        # chunked prefill: a chunk of a long prompt over what is already in the cache
        {"name": "paged4_chunk_bf16", "op": "paged4", "dtype": "bf16", "cache": "4bit", "d": 128, "hq": 32, "hkv": 8, "seqs": 1,
         "new": 2048, "before": 32000, "page": 16, "mix": 7},
        # a mixed step: some chunks, the other sequences a few tokens each
        {"name": "paged4_mixed_f16_d64", "op": "paged4", "dtype": "f16", "cache": "4bit", "d": 64, "hq": 8, "hkv": 2, "seqs": 12,
         "new": 3000, "before": 60000, "page": 64, "mix": 8},
        # one user, one token over a long document
        {"name": "select_one_f16", "op": "select", "dtype": "f16", "cache": "same", "d": 128, "hq": 32, "hkv": 8, "seqs": 1,
         "new": 1, "before": 131072, "page": 64, "pages": 32, "mix": 9},
        # a decoding batch over long documents in 4 bits
        {"name": "select_batch_4bit", "op": "select", "dtype": "bf16", "cache": "4bit", "d": 128, "hq": 32, "hkv": 8, "seqs": 48,
         "new": 48, "before": 1000000, "page": 32, "pages": 64, "mix": 10},
        # drafted tokens over the 8-bit cache of a small model, small pages
        {"name": "select_few_e4m3_d64", "op": "select", "dtype": "bf16", "cache": "e4m3", "d": 64, "hq": 8, "hkv": 2, "seqs": 20,
         "new": 60, "before": 400000, "page": 16, "pages": 100, "mix": 11},
        # the end of a long prompt: each of its tokens chooses for itself
        {"name": "select_chunk_bf16", "op": "select", "dtype": "bf16", "cache": "same", "d": 128, "hq": 32, "hkv": 8, "seqs": 1,
         "new": 200, "before": 65536, "page": 64, "pages": 16, "mix": 12},
    ]


def draw(rng):
    def over(low, high):
        return int(round(low * (high / low) ** rng.random()))

    op = rng.choice(["append", "paged4", "paged4", "paged4", "select", "select"])
    d = rng.choice([64, 128])
    hq, hkv = rng.choice([(8, 8), (8, 2), (32, 8), (16, 2), (6, 2), (5, 1), (12, 4), (28, 4), (1, 1), (16, 1)])
    case = {"op": op, "dtype": rng.choice(["f16", "bf16"]), "d": d, "hq": hq, "hkv": hkv, "page": rng.choice([16, 32, 64, 128]),
            "mix": rng.randrange(1, 10 ** 6)}
    seqs = over(1, 100)
    if op == "append":
        return case | {"cache": rng.choice(["same", "e4m3", "4bit"]), "seqs": seqs, "new": max(seqs, over(1, 16384)),
                       "before": over(200, 6000), "rot": rng.choice([d, d, d // 2, d // 4]), "inter": rng.random() < 0.4}
    if op == "paged4":
        kind = rng.choice(["token", "token", "few", "chunk"])
        new = seqs if kind == "token" else seqs * rng.randrange(2, 7) if kind == "few" else over(64, 2048)
        before = over(300, 400000 if kind != "chunk" else 16000)
        return case | {"cache": "4bit", "seqs": min(seqs, new), "new": new, "before": before}
    seqs = over(1, 40)
    return case | {"cache": rng.choice(["same", "e4m3", "4bit"]), "seqs": seqs, "new": seqs * rng.choice([1, 1, 1, 2, 3]),
                   "before": over(2000, 400000), "pages": min(over(2, 200), 4096 // case["page"])}


def _spread(total, n, mix, even=False):
    """n lengths, some of them short and now and then one of zero, that sum to total."""
    rng = random.Random(mix)
    share = [0.0 if n > 4 and rng.random() < 0.05 else rng.expovariate(1.0) + 0.05 for _ in range(n)]
    if even or not sum(share):
        share = [1.0] * n
    ends = np.floor(np.cumsum(share) / sum(share) * total + 1e-9).astype(np.int64)
    ends[-1] = total
    return np.diff(np.concatenate([[0], ends]))


def _lengths(case):
    """The new tokens of each sequence, and its length with them."""
    few = case["new"] % case["seqs"] == 0 and case["new"] // case["seqs"] < 16
    new = _spread(case["new"], case["seqs"], case["mix"], even=few)
    return new, new + _spread(case["before"], case["seqs"], case["mix"] + 1)


def _starts(lengths):
    return np.concatenate([[0], np.cumsum(lengths)])


# ---- what the cache's bytes stand for

def _to_e4m3(x):
    """Bytes under one power of two for each vector, the smallest under which its largest value is at most 448."""
    m, e = torch.frexp(x.abs().amax(-1, keepdim=True))
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-126, 127)
    e = torch.where(m == 0, torch.full_like(e, -126), e)
    return torch.ldexp(x, -e).to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)[..., 0]


def _to_4bit(x):
    g = x.unflatten(-1, (-1, 32))
    top = g.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(top / torch.full_like(top, 7))  # (a quotient; by a plain 7 it would be a product with the rounded 1 / 7)
    scale = torch.ldexp(torch.round(m * 16) / 16, e).clamp(2.0 ** -14, 61440.0)
    code = (torch.round(g / scale).clamp(-7, 7) + 8).to(torch.uint8).flatten(-2)
    m, e = torch.frexp(scale[..., 0])
    return code[..., 0::2] | (code[..., 1::2] << 4), (8 * (e + 14) + (2 * m - 1) * 8).to(torch.uint8)


def _quantise(kind, x):
    return _to_e4m3(x.float()) if kind == "e4m3" else _to_4bit(x.float())


def _stands_for(kind, byte, scale):
    """The values of a cache's bytes in 32 bits (16-bit caches: byte is the value, and scale None)."""
    if kind == "same":
        return byte.float()
    if kind == "e4m3":
        return torch.ldexp(byte.view(torch.float8_e4m3fn).float(), scale[..., None].int() - 127)
    whole = torch.stack([byte & 15, byte >> 4], -1).flatten(-2).float() - 8
    s = torch.ldexp(1 + (scale & 7).float() / 8, (scale >> 3).int() - 15)
    return (whole.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def _bounds(x):
    """x [..., slots, d] as whole multiples of its largest and smallest values, [..., 2, d], and the power's byte."""
    both = torch.stack([x.amax(-2), x.amin(-2)], -2)
    m, e = torch.frexp(both.abs().amax((-1, -2)))
    e = torch.where(m <= 127 / 128, e - 7, e - 6).clamp(-126, 121)
    e = torch.where(m == 0, torch.full_like(e, -126), e)
    return torch.round(torch.ldexp(both, -e[..., None, None])).to(torch.int8), (e + 127).to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + case["mix"])
    dt, d, hkv, page, kind = DTYPES[case["dtype"]], case["d"], case["hkv"], case["page"], case["cache"]

    def normal(*shape, times=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * times).to(dt)

    new, length = _lengths(case)
    start, total = _starts(new), int(sum(new))
    per_seq = -(-length // page)
    pages, most = int(sum(per_seq)) + 3, int(max(per_seq))
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    at = torch.tensor(_starts(per_seq)[:-1], device="cuda")[:, None] + torch.arange(most, device="cuda")[None, :]
    table = torch.where(torch.arange(most, device="cuda")[None, :] < torch.tensor(per_seq, device="cuda")[:, None],
                        order[at.clamp(max=pages - 1)], torch.zeros((), dtype=torch.int32, device="cuda"))
    kc, vc = normal(pages, hkv, page, d, times=1.5), normal(pages, hkv, page, d)
    if case["op"] == "select":  # neighbouring keys are alike
        kc += normal(pages, hkv, 1, d)
    kc += normal(1, hkv, 1, d, times=0.5)  # keys have features that are never near zero
    state = {"case": case, "start": start.tolist(), "length": length.tolist(), "table": table.contiguous(),
             "cu": torch.tensor(start, dtype=torch.int32, device="cuda"),
             "lengths": torch.tensor(length, dtype=torch.int32, device="cuda"), "ks": None, "vs": None,
             "most_new": int(max(new)), "most": int(max(length)), "q": normal(total, case["hq"], d)}
    if kind != "same":
        kc, state["ks"] = _by_pages(lambda x: _quantise(kind, x), kc)
        vc, state["vs"] = _by_pages(lambda x: _quantise(kind, x), vc)
    state |= {"kc": kc, "vc": vc}
    if case["op"] == "append":
        angle = torch.arange(int(max(length)), device="cuda", dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64) * 2 / case["rot"])
        state |= {"k": normal(total, hkv, d, times=1.5), "v": normal(total, hkv, d),
                  "turn": torch.cat([torch.cos(angle), torch.sin(angle)], -1).float().contiguous()}
    if case["op"] == "select":
        state["bounds"], state["bound_exp"] = _by_pages(lambda c, s=None: _bounds(_stands_for(kind, c, s)), kc, state["ks"])
    return state


def _by_pages(f, *x):
    """f of a cache, some pages at a time."""
    x = [t for t in x if t is not None]
    n = max(1, 2 ** 27 // x[0][0].numel())
    got = [f(*(t[i:i + n] for t in x)) for i in range(0, x[0].shape[0], n)]
    return tuple(torch.cat(t) for t in zip(*got))


# ---- append

def _slots(state):
    """Position, page and slot of every new token."""
    cu, page = state["cu"].long(), state["case"]["page"]
    token = torch.arange(state["start"][-1], device="cuda")
    s = torch.searchsorted(cu, token, right=True) - 1
    position = state["lengths"].long()[s] - (cu[s + 1] - token)
    return position, state["table"][s, position // page].long(), position % page


def _turned(x, turn, case):
    """x [tokens, heads, d] in 32 bits, each pair of its first `rot` features turned."""
    half, x = case["rot"] // 2, x.float()
    c, s = turn[:, None, :half], turn[:, None, half:]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if case["inter"] else (x[..., :half], x[..., half:2 * half])
    pair = torch.stack([a * c - b * s, b * c + a * s], -1 if case["inter"] else -2).flatten(-2)
    return torch.cat([pair, x[..., 2 * half:]], -1)


def _append(state):
    case = state["case"]
    position, page, slot = _slots(state)
    turn = state["turn"][position]
    q, k = _turned(state["q"], turn, case).to(state["q"].dtype), _turned(state["k"], turn, case)
    if state["ks"] is None:
        for c, x in ((state["kc"], k), (state["vc"], state["v"])):
            c[page, :, slot] = x.to(c.dtype)
        return q, state["kc"], state["vc"]
    got = [q]
    for c, scale, x in ((state["kc"], state["ks"], k), (state["vc"], state["vs"], state["v"])):
        c[page, :, slot], scale[page, :, slot] = _quantise(case["cache"], x)
        got.append(_stands_for(case["cache"], c[page, :, slot], scale[page, :, slot]).to(q.dtype))
    return tuple(got)


# ---- attention over the cache

def _blocks(state, block):
    """(sequence, first new token, tokens, position of the first) for at most `block` new tokens of a sequence at a time."""
    start, length = state["start"], state["length"]
    return [(s, start[s] + i, min(block, start[s + 1] - start[s] - i), length[s] - (start[s + 1] - start[s]) + i)
            for s in range(len(length)) for i in range(0, start[s + 1] - start[s], block)]


def _keys(state, s):
    """Keys and values of sequence s in 32 bits, [kv heads, length, d]."""
    n = state["length"][s]
    at = state["table"][s, : -(-n // state["case"]["page"])].long()
    found = []
    for c, scale in ((state["kc"], state["ks"]), (state["vc"], state["vs"])):
        x = _stands_for(state["case"]["cache"], c[at], None if scale is None else scale[at])
        found.append(x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])[:, :n])
    return found


def _heads_last(x):
    """[kv heads, group, tokens, d] as [tokens, heads, d]."""
    return x.permute(2, 0, 1, 3).reshape(x.shape[2], -1, x.shape[3])


def _attend_paged(state):
    q, hkv = state["q"], state["case"]["hkv"]
    out = torch.zeros_like(q)
    lse = torch.zeros(q.shape[1], q.shape[0], device="cuda")
    now, k, v = None, None, None
    for s, at, n, first in _blocks(state, BLOCK):
        if s != now:
            now, (k, v) = s, _keys(state, s)
        seen = min(k.shape[1], first + n)
        grouped = q[at:at + n].float().reshape(n, hkv, -1, q.shape[2]).permute(1, 2, 0, 3)
        x = (grouped * q.shape[2] ** -0.5) @ k[:, None, :seen].transpose(-1, -2)
        ahead = torch.arange(seen, device="cuda")[None, :] > first + torch.arange(n, device="cuda")[:, None]
        x = x.masked_fill(ahead, float("-inf"))
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - top)
        total = p.sum(-1, keepdim=True)
        out[at:at + n] = _heads_last((p @ v[:, None, :seen]) / total).to(q.dtype)
        lse[:, at:at + n] = (top + torch.log(total))[..., 0].reshape(-1, n)
    return out, lse


# ---- attention over selected pages

def _update_bounds(state):
    """The bounds of the pages that hold new tokens, from their filled slots."""
    case, page = state["case"], state["case"]["page"]
    position, at, _ = _slots(state)
    cu = state["cu"].long()
    s = torch.searchsorted(cu, torch.arange(len(at), device="cuda"), right=True) - 1
    filled = (state["lengths"].long()[s] - position // page * page).clamp(max=page)  # of the token's page
    x = _stands_for(case["cache"], state["kc"][at], None if state["ks"] is None else state["ks"][at])
    hidden = torch.arange(page, device="cuda")[None, :] >= filled[:, None]
    x = torch.where(hidden[:, None, :, None], x[:, :, :1], x)  # (slot 0 is filled, and counts once more)
    state["bounds"][at], state["bound_exp"][at] = _bounds(x)


def _choose(state, s, q, first):
    """The pages of sequence s that tokens q [n, heads, d] at positions first.. attend to: [n, kv heads, pages], ascending, -1
    behind them."""
    case, n = state["case"], q.shape[0]
    own_page = (first + torch.arange(n, device="cuda")) // case["page"]
    most = int((first + n - 1) // case["page"])  # pages before the last token's
    at = state["table"][s, :most].long()
    m, e = torch.frexp(q.float().abs().amax(-1, keepdim=True))
    e = torch.where(m <= 127 / 128, e - 7, e - 6).clamp(-126, 121)
    code = torch.round(torch.ldexp(q.float(), -e)).reshape(n, case["hkv"], -1, case["d"]).transpose(0, 1)
    e = e.reshape(n, case["hkv"], -1, 1).transpose(0, 1)
    b = state["bounds"][at].float().permute(1, 2, 3, 0)  # [kv heads, 2, d, pages]
    x = code.clamp(min=0) @ b[:, None, 0] + code.clamp(max=0) @ b[:, None, 1]
    x = torch.ldexp(x, e - e.amax(2, keepdim=True)).amax(2)
    x = torch.ldexp(x, state["bound_exp"][at].int().T[:, None] - 127)  # [kv heads, n, pages]
    x = x.masked_fill(torch.arange(most, device="cuda")[None, :] >= own_page[:, None], float("-inf"))
    value, order = torch.sort(x, dim=-1, descending=True, stable=True)
    take = min(case["pages"] - 1, most)
    order = torch.where(value[..., :take] == float("-inf"), torch.full_like(order[..., :take], 1 << 40), order[..., :take])
    order = torch.cat([order, own_page[None, :, None].expand(case["hkv"], -1, 1)], -1).sort(-1)[0]
    pages = torch.full((n, case["hkv"], case["pages"]), -1, dtype=torch.int32, device="cuda")
    pages[..., :take + 1] = torch.where(order == 1 << 40, torch.full_like(order, -1), order).transpose(0, 1).to(torch.int32)
    return pages


def _attend_selected(state):
    case, q = state["case"], state["q"]
    hkv, d, page = case["hkv"], case["d"], case["page"]
    out = torch.zeros_like(q)
    lse = torch.zeros(q.shape[1], q.shape[0], device="cuda")
    chosen = torch.full((q.shape[0], hkv, case["pages"]), -1, dtype=torch.int32, device="cuda")
    head = torch.arange(hkv, device="cuda")[None, :, None]
    for s, at, n, first in _blocks(state, max(1, 2 ** 28 // (case["pages"] * page * d * hkv))):
        mine = slice(at, at + n)
        chosen[mine] = _choose(state, s, q[mine], first)
        phys = state["table"][s][chosen[mine].clamp(min=0).long()].long()
        k, v = (_stands_for(case["cache"], c[phys, head], None if z is None else z[phys, head]).flatten(2, 3)
                for c, z in ((state["kc"], state["ks"]), (state["vc"], state["vs"])))  # [n, kv heads, slots, d]
        x = (q[mine].float().reshape(n, hkv, -1, d) * d ** -0.5) @ k.transpose(-1, -2)
        position = (chosen[mine].long()[..., None] * page + torch.arange(page, device="cuda")).flatten(2)
        hidden = (position < 0) | (position > first + torch.arange(n, device="cuda")[:, None, None])
        x = x.masked_fill(hidden[:, :, None], float("-inf"))
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - top)
        total = p.sum(-1, keepdim=True)
        out[mine] = ((p @ v) / total).reshape(n, -1, d).to(q.dtype)
        lse[:, mine] = (top + torch.log(total))[..., 0].reshape(n, -1).T
    return out, lse, chosen


def run(state):
    case = state["case"]
    if own:
        import exact_long_context_tcgen05_gb300 as cq
        paged = (state["kc"], state["vc"], state["table"], state["cu"], state["lengths"])
        scales = {"k_scale": state["ks"], "v_scale": state["vs"]}
        if case["op"] == "append":
            q = cq.kv_cache_append(state["q"], state["k"], state["v"], state["turn"], *paged, interleaved=case["inter"], **scales)
            if state["ks"] is None:
                return q, state["kc"], state["vc"]
            return q, *cq.kv_cache_read(*paged, q.shape[0], q.dtype, **scales)
        if case["op"] == "paged4":
            return cq.attention_paged(state["q"], *paged, state["most_new"], state["most"], return_lse=True, **scales)
        cq.kv_page_bounds(state["kc"], state["table"], state["cu"], state["lengths"], state["bounds"], state["bound_exp"],
                          state["most_new"], k_scale=state["ks"])
        out, lse, pages = cq.attention_selected(state["q"], *paged, state["bounds"], state["bound_exp"], case["pages"], state["most"],
                                                return_lse=True, return_pages=True, **scales)
        return out, lse, pages, state["bounds"]
    if case["op"] == "append":
        return _append(state)
    if case["op"] == "paged4":
        return _attend_paged(state)
    _update_bounds(state)
    return *_attend_selected(state), state["bounds"]


def work(case):
    new, length = (x.astype(np.float64) for x in _lengths(case))
    d, hkv, hq, page, total = case["d"], case["hkv"], case["hq"], case["page"], float(sum(new))
    vector = {"same": 2 * d, "e4m3": d + 1, "4bit": d // 2 + d // 32}[case["cache"]]  # bytes of a cached vector
    if case["op"] == "append":
        moved = total * (hq * 4 * d + hkv * 4 * d + 2 * hkv * vector + case["rot"] * 4)
        if case["cache"] != "same":
            moved += total * hkv * 2 * (2 * d + vector)
        return {"bytes": moved, "flops": total * (hq + hkv) * case["rot"] * 3}
    tokens = total * 2 * hq * d * 2 + total * hq * 4
    if case["op"] == "paged4":
        pairs = float(sum(new * length - new * (new - 1) / 2))
        return {"bytes": tokens + float(sum(length)) * hkv * 2 * vector, "flops": 4 * pairs * hq * d}
    own_pages = float(sum(np.ceil(new / page) + (new > 0)))  # that new tokens came into
    bounds = float(sum(np.where(new > 0, np.ceil(length / page), 0))) * hkv * (2 * d + 1)  # read once for all of a sequence's tokens
    slots = float(sum(np.where(new > 0, np.minimum(length, new * case["pages"] * page), 0)))  # at least, if tokens choose alike: once each
    pairs = float(sum(new * np.minimum(length, case["pages"] * page)))
    scored = float(sum(new * np.ceil(length / page)))
    return {"bytes": tokens + bounds + own_pages * hkv * (page * vector + 2 * d) + slots * hkv * 2 * vector + total * hkv * case["pages"] * 4,
            "flops": 4 * pairs * hq * d + 4 * scored * hq * d}


# ---- the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "paged4": _exact_paged, "select": _exact_select}[case["op"]](case, st, *_lengths(case))


def _value64(case, byte, scale):
    """What bytes of a cache stand for."""
    if case["cache"] == "same":
        return byte.double()
    if case["cache"] == "e4m3":
        return byte.view(torch.float8_e4m3fn).double() * torch.exp2(scale.double() - 127)[..., None]
    x = torch.empty(*byte.shape[:-1], 2 * byte.shape[-1], dtype=torch.float64, device=byte.device)
    x[..., 0::2], x[..., 1::2] = (byte % 16).double() - 8, (byte // 16).double() - 8
    unit = torch.tensor([(8 + i % 8) * 2.0 ** (i // 8 - 18) for i in range(256)], dtype=torch.float64, device=byte.device)
    return x * unit[scale.long()].repeat_interleave(32, -1)


def _nearest64(case, x):
    """x as the nearest values of the cache's grid."""
    if case["cache"] == "same":
        return x
    if case["cache"] == "e4m3":
        unit = torch.exp2(torch.ceil(torch.log2(x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -117) / 448)).clamp(min=-126))
        y = x / unit
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        return torch.round(y / step) * step * unit
    got = torch.empty_like(x)
    grid = torch.tensor([(8 + m) * 2.0 ** (e - 18) for e in range(1, 31) for m in range(8)], dtype=torch.float64, device=x.device)
    for i in range(0, x.shape[-1], 32):
        part = x[..., i:i + 32]
        want = part.abs().amax(-1, keepdim=True) / 7
        above = torch.searchsorted(grid, want).clamp(1, len(grid) - 1)
        low, high = grid[above - 1], grid[above]
        up = (high - want < want - low) | ((high - want == want - low) & (above % 2 == 0))
        unit = torch.where(up, high, low)
        got[..., i:i + 32] = torch.clamp(torch.round(part / unit), -7, 7) * unit
    return got


def _exact_append(case, st, new, length):
    r, place = case["rot"], []
    for s in range(len(new)):
        t = torch.arange(int(length[s] - new[s]), int(length[s]), device="cuda")
        place.append(torch.stack([t, st["table"][s].long()[t // case["page"]], t % case["page"]]))
    position, page, slot = torch.cat(place, 1)
    c, z = st["turn"][position, :r // 2].double(), st["turn"][position, r // 2:].double()
    turned = []
    for x in (st["q"].double(), st["k"].double()):
        y = x.clone()
        for j in range(r // 2):
            a, b = (2 * j, 2 * j + 1) if case["inter"] else (j, j + r // 2)
            y[..., a] = x[..., a] * c[:, j:j + 1] - x[..., b] * z[:, j:j + 1]
            y[..., b] = x[..., a] * z[:, j:j + 1] + x[..., b] * c[:, j:j + 1]
        turned.append(y)
    q, k = turned
    if case["cache"] != "same":
        return q, _nearest64(case, k), _nearest64(case, st["v"].double())
    caches = st["kc"].double(), st["vc"].double()
    for cache, x in zip(caches, (k, st["v"].double())):
        cache[page, :, slot] = x
    return q, *caches


def _exact_paged(case, st, new, length):
    """One query head at a time."""
    q = st["q"].double()
    out, lse = torch.zeros_like(q), torch.zeros(case["hq"], q.shape[0], dtype=torch.float64, device="cuda")
    start = _starts(new)
    for s in range(len(new)):
        a, n, m = int(start[s]), int(new[s]), int(length[s])
        if not n:
            continue
        t = torch.arange(m, device="cuda")
        pg, sl = st["table"][s].long()[t // case["page"]], t % case["page"]
        k, v = (_value64(case, x[pg, :, sl], z[pg, :, sl]) for x, z in ((st["kc"], st["ks"]), (st["vc"], st["vs"])))
        for h in range(case["hq"]):
            g = h // (case["hq"] // case["hkv"])
            for i in range(0, n, 2 * BLOCK):
                j = min(n, i + 2 * BLOCK)
                seen = m - n + j
                x = q[a + i:a + j, h] @ k[:seen, g].T / case["d"] ** 0.5
                x += torch.full_like(x, float("-inf")).triu(m - n + i + 1)
                z = torch.logsumexp(x, -1, keepdim=True)
                out[a + i:a + j, h], lse[h, a + i:a + j] = torch.exp(x - z) @ v[:seen, g], z[:, 0]
    return out, lse


def _whole64(x):
    """Vectors x [..., d] (or pairs of them, [..., 2, d], under one power) as whole numbers and their powers of two."""
    top = x.abs().amax((-1, -2), keepdim=True)
    unit = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0 ** -110) / 127)).clamp(min=-126))
    return torch.round(x / unit), unit


def _exact_select(case, st, new, length):
    """One token and key head at a time."""
    q, page, group = st["q"].double(), case["page"], case["hq"] // case["hkv"]
    out, lse = torch.zeros_like(q), torch.zeros(case["hq"], q.shape[0], dtype=torch.float64, device="cuda")
    start = _starts(new)
    for s in range(len(new)):
        a, n, m = int(start[s]), int(new[s]), int(length[s])
        if not n:
            continue
        row = st["table"][s].long()
        old = int(m - n) // page  # pages without new tokens keep the bounds that they came with
        bound = st["bounds"][row[:-(-m // page)]].double() * torch.exp2(st["bound_exp"][row[:-(-m // page)]].double() - 127)[..., None, None]
        for p in range(old, -(-m // page)):
            pg, filled = row[p], min(page, m - p * page)
            x = _value64(case, st["kc"][pg], None if st["ks"] is None else st["ks"][pg])[:, :filled]
            w, unit = _whole64(torch.stack([x.max(1)[0], x.min(1)[0]], 1))
            bound[p] = w * unit
        for i in range(n):
            position = m - n + i
            here = position // page
            for g in range(case["hkv"]):
                heads = q[a + i, g * group:(g + 1) * group]
                w, unit = _whole64(heads[:, None])
                w = (w * unit)[:, 0]
                x = torch.maximum(w[:, None] * bound[None, :here, g, 0], w[:, None] * bound[None, :here, g, 1]).sum(-1).amax(0)
                best = torch.argsort(-x, dim=-1, stable=True)[:case["pages"] - 1]
                at = torch.cat([best.sort()[0], torch.tensor([here], device="cuda")])
                t = (at[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)
                t = t[t <= position]
                pg, sl = row[t // page], t % page
                k, v = (_value64(case, c[pg, g, sl], None if z is None else z[pg, g, sl])
                        for c, z in ((st["kc"], st["ks"]), (st["vc"], st["vs"])))
                x = heads @ k.T / case["d"] ** 0.5
                z = torch.logsumexp(x, -1, keepdim=True)
                out[a + i, g * group:(g + 1) * group] = torch.exp(x - z) @ v
                lse[g * group:(g + 1) * group, a + i] = z[:, 0]
    return out, lse, None, None
