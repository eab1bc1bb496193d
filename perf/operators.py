"""Cases of the sequence operators (packed prompts, a paged key/value cache and the attention over it): their
inputs, their plain form in elementary torch operations, the framework's calls, and their value in 64 bits.

Four operators:
  prompt  attention of whole prompts packed end to end, with grouped heads, causal or not
  grad    its gradients (dq, dk, dv) from the forward's output and log-sum-exp
  cache   writing new tokens into a paged cache (16-bit, or e4m3 with a power-of-two scale per token and
          head) and reading them back
  paged   attention of each sequence's new tokens (one, a few, or a chunk) over its pages

Token tensors are [tokens, heads, d]. Sequence s owns tokens cu[s] .. cu[s+1] - 1. A cache is
[pages, kv heads, page size, d]; position t of sequence s is slot t % page of page table[s, t // page]. Token i of
sequence s's new tokens has position length[s] - new[s] + i, and sees the positions up to its own.
"""
import random

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
BLOCK = 1024  # query tokens that the plain form and the 64-bit form hold scores for at a time


def listed():
    return [
        # a burst of short prompts: what a chat server gets between two steps
        {"name": "prompt_short_f16_d64", "op": "prompt", "dtype": "f16", "d": 64, "hq": 8, "hkv": 2, "seqs": 24,
         "tokens": 1000, "causal": True, "mix": 1},
        # a prefill batch of ragged prompts at the framework's large head dimension
        {"name": "prompt_ragged_bf16_d128", "op": "prompt", "dtype": "bf16", "d": 128, "hq": 32, "hkv": 8, "seqs": 24,
         "tokens": 16384, "causal": True, "mix": 2},
        # one long prompt: the benchmark's length and heads, the heads grouped
        {"name": "prompt_long_f16_d64", "op": "prompt", "dtype": "f16", "d": 64, "hq": 8, "hkv": 2, "seqs": 1,
         "tokens": 32768, "causal": True, "mix": 3},
        # a small training step's packed row of documents
        {"name": "grad_f16_d64", "op": "grad", "dtype": "f16", "d": 64, "hq": 8, "hkv": 2, "seqs": 9, "tokens": 4099,
         "causal": True, "mix": 4},
        # a training step's packed batch at the large head dimension
        {"name": "grad_bf16_d128", "op": "grad", "dtype": "bf16", "d": 128, "hq": 32, "hkv": 8, "seqs": 8,
         "tokens": 16384, "causal": True, "mix": 5},
        # one step of a running batch: a token for each sequence goes into the cache
        {"name": "cache_step_f16", "op": "cache", "dtype": "f16", "cache": "same", "d": 128, "hkv": 8, "seqs": 24,
         "new": 24, "before": 6000, "page": 16, "mix": 6},
        # a prefill batch's keys and values, quantised on the way in and read back
        {"name": "cache_prompt_e4m3", "op": "cache", "dtype": "bf16", "cache": "e4m3", "d": 128, "hkv": 8, "seqs": 24,
         "new": 16384, "before": 5000, "page": 16, "mix": 7},
        # one user, one token: the latency of a step
        {"name": "token_one_f16", "op": "paged", "dtype": "f16", "cache": "same", "d": 128, "hq": 32, "hkv": 8,
         "seqs": 1, "new": 1, "before": 3001, "page": 16, "causal": True, "mix": 8},
        # a full decoding batch of ragged contexts
        {"name": "token_batch_bf16", "op": "paged", "dtype": "bf16", "cache": "same", "d": 128, "hq": 32, "hkv": 8,
         "seqs": 64, "new": 64, "before": 300000, "page": 16, "causal": True, "mix": 9},
        # the same over a quantised cache, where twice the sequences fit
        {"name": "token_batch_e4m3", "op": "paged", "dtype": "bf16", "cache": "e4m3", "d": 128, "hq": 32, "hkv": 8,
         "seqs": 128, "new": 128, "before": 500000, "page": 32, "causal": True, "mix": 10},
        # chunked prefill: a chunk of a long prompt over what is already in the cache
        {"name": "chunk_bf16_d128", "op": "paged", "dtype": "bf16", "cache": "same", "d": 128, "hq": 32, "hkv": 8,
         "seqs": 1, "new": 2048, "before": 32000, "page": 16, "causal": True, "mix": 11},
        # a mixed step over a quantised cache: some chunks, the other sequences a few tokens each
        {"name": "chunk_mixed_e4m3", "op": "paged", "dtype": "f16", "cache": "e4m3", "d": 64, "hq": 8, "hkv": 2,
         "seqs": 12, "new": 3000, "before": 60000, "page": 64, "causal": True, "mix": 12},
    ]


def draw(rng):
    def over(low, high):
        return int(round(low * (high / low) ** rng.random()))

    op = rng.choice(["prompt", "prompt", "grad", "cache", "paged", "paged", "paged"])
    case = {"op": op, "dtype": rng.choice(["f16", "bf16"]), "d": rng.choice([64, 128]), "mix": rng.randrange(1, 10 ** 6)}
    hq, hkv = rng.choice([(8, 8), (8, 2), (32, 8), (16, 2), (6, 2), (5, 1), (12, 4), (28, 4), (1, 1), (16, 1)])
    if op in ("prompt", "grad"):
        most = {"prompt": 32768, "grad": 16384}[op] * 64 * 8 // (case["d"] * max(hq, 8))
        tokens = over(70, max(512, most))
        case |= {"hq": hq, "hkv": hkv, "seqs": min(over(1, 64), tokens), "tokens": tokens, "causal": rng.random() < 0.8}
        return case
    case |= {"hkv": hkv, "cache": rng.choice(["same", "e4m3"]), "page": rng.choice([16, 32, 64, 128])}
    seqs = over(1, 100)
    if op == "cache":
        return case | {"seqs": seqs, "new": max(seqs, over(1, 16384)), "before": over(200, 6000)}
    kind = rng.choice(["token", "few", "chunk"])
    new = seqs if kind == "token" else seqs * rng.randrange(2, 7) if kind == "few" else over(64, 2048)
    before = over(300, 200000 if kind != "chunk" else 16000)
    return case | {"hq": hq, "seqs": min(seqs, new), "new": new, "before": before, "causal": kind == "token" or rng.random() < 0.9}


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
    if case["op"] in ("prompt", "grad"):
        new = _spread(case["tokens"], case["seqs"], case["mix"])
        return new, new
    few = case["new"] % case["seqs"] == 0 and case["new"] // case["seqs"] < 16
    new = _spread(case["new"], case["seqs"], case["mix"], even=few)
    return new, new + _spread(case["before"], case["seqs"], case["mix"] + 1)


def _starts(lengths):
    return np.concatenate([[0], np.cumsum(lengths)])


def _quantise(x):
    """x as e4m3 bytes with one power of two for each vector, the smallest under which its largest value is at most 448."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1, keepdim=True))
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-126, 127)
    e = torch.where(m == 0, torch.full_like(e, -126), e)
    return torch.ldexp(x, -e).to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)[..., 0]


def _stands_for(byte, scale):
    return torch.ldexp(byte.view(torch.float8_e4m3fn).float(), scale[..., None].int() - 127)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + case["mix"])
    dt, d, hkv = DTYPES[case["dtype"]], case["d"], case["hkv"]

    def normal(*shape, times=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * times).to(dt)

    new, length = _lengths(case)
    start, total = _starts(new), int(sum(new))
    state = {"case": case, "start": start.tolist(), "length": length.tolist(),
             "cu": torch.tensor(start, dtype=torch.int32, device="cuda")}
    if case["op"] in ("prompt", "grad"):
        state |= {"q": normal(total, case["hq"], d), "k": normal(total, hkv, d, times=1.5), "v": normal(total, hkv, d)}
        if case["op"] == "grad":
            out, lse = _attend_packed(state)
            state |= {"out": out, "lse": lse, "dout": normal(total, case["hq"], d)}
        return state
    page = case["page"]
    per_seq = -(-length // page)
    pages, most = int(sum(per_seq)) + 3, int(max(per_seq))
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    at = torch.tensor(_starts(per_seq)[:-1], device="cuda")[:, None] + torch.arange(most, device="cuda")[None, :]
    table = torch.where(torch.arange(most, device="cuda")[None, :] < torch.tensor(per_seq, device="cuda")[:, None],
                        order[at.clamp(max=pages - 1)], torch.zeros((), dtype=torch.int32, device="cuda"))
    kc, vc = normal(pages, hkv, page, d, times=1.5), normal(pages, hkv, page, d)
    state |= {"table": table.contiguous(), "lengths": torch.tensor(length, dtype=torch.int32, device="cuda"),
              "ks": None, "vs": None, "most_new": int(max(new)), "most": int(max(length))}
    if case["cache"] == "e4m3":
        kc, state["ks"] = _quantise(kc)
        vc, state["vs"] = _quantise(vc)
    state |= {"kc": kc, "vc": vc}
    if case["op"] == "cache":
        state |= {"k": normal(total, hkv, d, times=1.5), "v": normal(total, hkv, d)}
    else:
        state["q"] = normal(total, case["hq"], d)
    return state


def _blocks(state):
    """(sequence, first new token, tokens, position of the first) for at most BLOCK new tokens of a sequence at a time."""
    start, length = state["start"], state["length"]
    return [(s, start[s] + i, min(BLOCK, start[s + 1] - start[s] - i), length[s] - (start[s + 1] - start[s]) + i)
            for s in range(len(length)) for i in range(0, start[s + 1] - start[s], BLOCK)]


def _keys(state, s):
    """Keys and values of sequence s in 32 bits, [kv heads, length, d]."""
    n = state["length"][s]
    if "k" in state:
        a, b = state["start"][s], state["start"][s + 1]
        return state["k"][a:b].float().transpose(0, 1), state["v"][a:b].float().transpose(0, 1)
    at = state["table"][s, : -(-n // state["case"]["page"])].long()
    found = []
    for c, scale in ((state["kc"], state["ks"]), (state["vc"], state["vs"])):
        x = c[at].float() if scale is None else _stands_for(c[at], scale[at])
        found.append(x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])[:, :n])
    return found


def _scores(state, q, k, first):
    """Scaled scores [kv heads, group, tokens, keys] of q [tokens, heads, d], the first at position `first`."""
    t, hq, d = q.shape
    grouped = q.float().reshape(t, k.shape[0], hq // k.shape[0], d).permute(1, 2, 0, 3)
    seen = k.shape[1] if not state["case"]["causal"] else min(k.shape[1], first + t)
    x = (grouped * d ** -0.5) @ k[:, None, :seen].transpose(-1, -2)
    if state["case"]["causal"]:
        ahead = torch.arange(seen, device="cuda")[None, :] > first + torch.arange(t, device="cuda")[:, None]
        x = x.masked_fill(ahead, float("-inf"))
    return x, grouped


def _heads_last(x):
    """[kv heads, group, tokens, d] as [tokens, heads, d]."""
    return x.permute(2, 0, 1, 3).reshape(x.shape[2], -1, x.shape[3])


def _attend_packed(state):
    q = state["q"]
    out = torch.zeros_like(q)
    lse = torch.zeros(q.shape[1], q.shape[0], device="cuda")
    now, k, v = None, None, None
    for s, at, n, first in _blocks(state):
        if s != now:
            now, (k, v) = s, _keys(state, s)
        x, _ = _scores(state, q[at:at + n], k, first)
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - top)
        total = p.sum(-1, keepdim=True)
        out[at:at + n] = _heads_last((p @ v[:, None, :x.shape[3]]) / total).to(q.dtype)
        lse[:, at:at + n] = (top + torch.log(total))[..., 0].reshape(-1, n)
    return out, lse


def _gradients(state):
    q, k16, scale = state["q"], state["k"], state["case"]["d"] ** -0.5
    dq = torch.zeros_like(q)
    dk, dv = (torch.zeros(k16.shape[1], k16.shape[0], k16.shape[2], device="cuda") for _ in range(2))
    now, k, v = None, None, None
    for s, at, n, first in _blocks(state):
        if s != now:
            now, (k, v) = s, _keys(state, s)
        x, grouped = _scores(state, q[at:at + n], k, first)
        seen, own_rows = x.shape[3], slice(state["start"][s], state["start"][s] + x.shape[3])
        p = torch.exp(x - state["lse"][:, at:at + n].reshape(x.shape[0], x.shape[1], n, 1))
        do = state["dout"][at:at + n].float().reshape(n, x.shape[0], x.shape[1], -1).permute(1, 2, 0, 3)
        o = state["out"][at:at + n].float().reshape(n, x.shape[0], x.shape[1], -1).permute(1, 2, 0, 3)
        ds = p * (do @ v[:, None, :seen].transpose(-1, -2) - (do * o).sum(-1, keepdim=True))
        dq[at:at + n] = _heads_last(ds @ k[:, None, :seen] * scale).to(q.dtype)
        dk[:, own_rows] += (ds.transpose(-1, -2) @ grouped).sum(1) * scale
        dv[:, own_rows] += (p.transpose(-1, -2) @ do).sum(1)
    return dq, dk.transpose(0, 1).to(q.dtype).contiguous(), dv.transpose(0, 1).to(q.dtype).contiguous()


def _slots(state):
    """Page and slot of every new token."""
    cu, page = state["cu"].long(), state["case"]["page"]
    token = torch.arange(state["start"][-1], device="cuda")
    s = torch.searchsorted(cu, token, right=True) - 1
    position = state["lengths"].long()[s] - (cu[s + 1] - token)
    return state["table"][s, position // page].long(), position % page


def _write_and_read(state):
    page, slot = _slots(state)
    if state["ks"] is None:
        for c, x in ((state["kc"], state["k"]), (state["vc"], state["v"])):
            c[page, :, slot] = x
        return state["kc"], state["vc"]
    got = []
    for c, scale, x in ((state["kc"], state["ks"], state["k"]), (state["vc"], state["vs"], state["v"])):
        c[page, :, slot], scale[page, :, slot] = _quantise(x)
        got.append(_stands_for(c[page, :, slot], scale[page, :, slot]).to(x.dtype))
    return tuple(got)


def run(state):
    case = state["case"]
    if own:
        import exact_long_context_tcgen05_gb300 as cq
        if case["op"] == "prompt":
            return cq.attention_packed(state["q"], state["k"], state["v"], state["cu"], causal=case["causal"], return_lse=True)
        if case["op"] == "grad":
            return cq.attention_packed_backward(state["q"], state["k"], state["v"], state["out"], state["dout"], state["lse"],
                                                state["cu"], causal=case["causal"])
        paged = (state["kc"], state["vc"], state["table"], state["cu"], state["lengths"])
        if case["op"] == "paged":
            return cq.attention_paged(state["q"], *paged, state["most_new"], state["most"], causal=case["causal"],
                                      k_scale=state["ks"], v_scale=state["vs"], return_lse=True)
        cq.kv_cache_write(state["k"], state["v"], *paged, k_scale=state["ks"], v_scale=state["vs"])
        if state["ks"] is None:
            return state["kc"], state["vc"]
        return cq.kv_cache_read(*paged, state["k"].shape[0], state["k"].dtype, k_scale=state["ks"], v_scale=state["vs"])
    if case["op"] == "grad":
        return _gradients(state)
    if case["op"] == "cache":
        return _write_and_read(state)
    return _attend_packed(state)


def work(case):
    new, length = (x.astype(np.float64) for x in _lengths(case))
    d, hkv, total = case["d"], case["hkv"], float(sum(new))
    vector = 2 * d if case.get("cache", "same") == "same" else d + 1  # bytes of a cached vector
    if case["op"] == "cache":
        moved = total * hkv * 2 * (2 * d + vector)
        return {"bytes": moved if case["cache"] == "same" else 2 * moved, "flops": 0.0}
    hq = case["hq"]
    pairs = float(sum(new * length - new * (new - 1) / 2)) if case["causal"] else float(sum(new * length))
    if case["op"] == "prompt":
        return {"bytes": total * (2 * hq + 2 * hkv) * d * 2 + total * hq * 4, "flops": 4 * pairs * hq * d}
    if case["op"] == "grad":
        return {"bytes": total * (4 * hq + 4 * hkv) * d * 2 + total * hq * 4, "flops": 10 * pairs * hq * d}
    return {"bytes": total * 2 * hq * d * 2 + total * hq * 4 + float(sum(length)) * hkv * 2 * vector, "flops": 4 * pairs * hq * d}


def exact(case, seed):
    """The operators' definitions, one query head at a time, in 64 bits."""
    st = prepare(case, seed)
    new, length = _lengths(case)
    start = _starts(new)
    if case["op"] == "cache":
        return _exact_cache(case, st, new, length)
    q = st["q"].double()
    group = case["hq"] // case["hkv"]
    out, lse = torch.zeros_like(q), torch.zeros(case["hq"], q.shape[0], dtype=torch.float64, device="cuda")
    grads = [torch.zeros_like(q)] + [torch.zeros(q.shape[0], case["hkv"], case["d"], dtype=torch.float64, device="cuda") for _ in range(2)]
    for s in range(len(new)):
        a, n, m = int(start[s]), int(new[s]), int(length[s])
        if not n:
            continue
        if "k" in st:
            k, v = st["k"][a:a + n].double(), st["v"][a:a + n].double()
        else:
            t = torch.arange(m, device="cuda")
            pg, sl = st["table"][s].long()[t // case["page"]], t % case["page"]
            k, v = st["kc"][pg, :, sl], st["vc"][pg, :, sl]
            if st["ks"] is not None:
                k, v = (x.view(torch.float8_e4m3fn).double() * torch.exp2(z[pg, :, sl].double() - 127)[..., None]
                        for x, z in ((k, st["ks"]), (v, st["vs"])))
            k, v = k.double(), v.double()
        for h in range(case["hq"]):
            g = h // group
            for i in range(0, n, 4 * BLOCK):
                j = min(n, i + 4 * BLOCK)
                seen = m - n + j if case["causal"] else m
                x = q[a + i:a + j, h] @ k[:seen, g].T / case["d"] ** 0.5
                if case["causal"]:
                    x += torch.full_like(x, float("-inf")).triu(m - n + i + 1)
                z = torch.logsumexp(x, -1, keepdim=True)
                p = torch.exp(x - z)
                o = p @ v[:seen, g]
                out[a + i:a + j, h], lse[h, a + i:a + j] = o, z[:, 0]
                if case["op"] == "grad":
                    do = st["dout"][a + i:a + j, h].double()
                    ds = p * (do @ v[:seen, g].T - (do * o).sum(-1, keepdim=True)) / case["d"] ** 0.5
                    grads[0][a + i:a + j, h] = ds @ k[:seen, g]
                    grads[1][a:a + seen, g] += ds.T @ q[a + i:a + j, h]
                    grads[2][a:a + seen, g] += p.T @ do
    return tuple(grads) if case["op"] == "grad" else (out, lse)


def _exact_cache(case, st, new, length):
    """Each new vector as the nearest values of its grid: 4 exponent and 3 fraction bits under the vector's power of two."""
    got, a = [], 0
    pages, slots = [], []
    for s in range(len(new)):
        t = torch.arange(int(length[s] - new[s]), int(length[s]), device="cuda")
        pages.append(st["table"][s].long()[t // case["page"]])
        slots.append(t % case["page"])
    pages, slots = torch.cat(pages), torch.cat(slots)
    for c, x in ((st["kc"], st["k"].double()), (st["vc"], st["v"].double())):
        if st["ks"] is None:
            c = c.double()
            c[pages, :, slots] = x
            got.append(c)
            continue
        unit = torch.exp2(torch.ceil(torch.log2(x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -117) / 448)).clamp(min=-126))
        y = x / unit
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        got.append(torch.round(y / step) * step * unit)
    return tuple(got)
