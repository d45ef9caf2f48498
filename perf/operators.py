"""The operators of the 4-bit key-value cache: what is measured, and their plain forms.

A cache is a pool of pages of `page` tokens.  A page holds, for each kv head, first the keys and
then the values of its tokens: the 4-bit levels of every token, then one (scale, low) pair of
bfloat16 for each token and group of 32 channels.  A value stands for low + scale * level.

    append  writes the last tokens of each sequence into its pages
    read    gives the last tokens of each sequence back
    attend  is causal attention of the last tokens of each sequence over all of its tokens, or
            over the listed blocks of them

A batch is described by the lengths of its sequences (the new tokens counted), the running sum of
the number of new tokens (sequence b has the rows cu[b] to cu[b + 1] of k, v, q and the output) and
a table of page numbers.  `own` chooses the framework's kernels; without it `run` computes the same
from elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

GROUP = 32
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
DEVICE = "cuda"
#: The plain attention takes as many kv heads at a time as keep its scores under this many values.
SCORES = 2 ** 31


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one generated token of one request goes into the cache: latency alone
        dict(name="append_step", op="append", seqs=1, shortest=1311, longest=1311, new_least=1, new_most=1,
             hkv=8, d=128, page=64, dtype="bf16", token_major=True, stored=False, spare=0),
        # a 128k prompt, as the projections leave it (token after token), for one layer of 8 kv heads
        dict(name="append_prompt", op="append", seqs=1, shortest=131072, longest=131072, new_least=131072,
             new_most=131072, hkv=8, d=128, page=64, dtype="bf16", token_major=True, stored=False, spare=0),
        # ragged prompts in fp32 behind what is already cached, and what was stored for the prompt's own attention
        dict(name="append_ragged", op="append", seqs=7, shortest=333, longest=9001, new_least=97, new_most=2999,
             hkv=4, d=64, page=16, dtype="fp32", token_major=False, stored=True, spare=5),
        # the cached context of one request back as K and V, to be pooled or prefilled over again
        dict(name="read_context", op="read", seqs=1, shortest=32768, longest=32768, new_least=32768, new_most=32768,
             hkv=8, d=128, page=64, dtype="bf16", token_major=False, stored=False, spare=0),
        # the ends of a few sequences in fp32
        dict(name="read_ends", op="read", seqs=5, shortest=129, longest=4173, new_least=1, new_most=515,
             hkv=2, d=64, page=32, dtype="fp32", token_major=False, stored=False, spare=3),
        # one token over a short context in fp32: latency alone
        dict(name="attend_short", op="attend", seqs=1, shortest=77, longest=77, new_least=1, new_most=1, hq=4, hkv=2,
             d=64, page=16, dtype="fp32", token_major=True, blocks=0, block=0, spare=0),
        # a decoding batch of mixed lengths
        dict(name="attend_batch", op="attend", seqs=48, shortest=211, longest=16411, new_least=1, new_most=1, hq=32,
             hkv=8, d=128, page=64, dtype="bf16", token_major=True, blocks=0, block=0, spare=0),
        # one token over half a million, 64 query heads
        dict(name="attend_long", op="attend", seqs=1, shortest=524288, longest=524288, new_least=1, new_most=1, hq=64,
             hkv=8, d=128, page=128, dtype="bf16", token_major=True, blocks=0, block=0, spare=0),
        # 33 blocks of 128 tokens a kv head of each 128k context: block-sparse decoding
        dict(name="attend_listed", op="attend", seqs=8, shortest=131072, longest=131072, new_least=1, new_most=1,
             hq=64, hkv=8, d=128, page=64, dtype="bf16", token_major=True, blocks=33, block=128, spare=0),
        # drafted tokens of a few requests checked at once
        dict(name="attend_draft", op="attend", seqs=12, shortest=907, longest=20011, new_least=3, new_most=6, hq=32,
             hkv=8, d=128, page=32, dtype="bf16", token_major=True, blocks=0, block=0, spare=2),
        # ends of prompts of mixed lengths in one call, smaller heads
        dict(name="attend_chunks", op="attend", seqs=3, shortest=701, longest=6007, new_least=333, new_most=1025,
             hq=8, hkv=2, d=64, page=64, dtype="bf16", token_major=True, blocks=0, block=0, spare=9),
        # a chunk of a long prompt over what is cached of it
        dict(name="attend_prompt", op="attend", seqs=1, shortest=32768, longest=32768, new_least=4096, new_most=4096,
             hq=32, hkv=8, d=128, page=64, dtype="bf16", token_major=True, blocks=0, block=0, spare=0),
    ]


def _between(rng, low, high):
    """A whole number from low to high, spread over the logarithm, most of them odd."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "attend"])
    d = rng.choice([64, 128, 128])
    case = dict(op=op, d=d, page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "bf16", "fp32"]),
                token_major=rng.random() < 0.7, spare=rng.choice([0, 0, 1, 7]))
    if op != "attend":
        case |= dict(hkv=rng.choice([1, 2, 4, 8]), seqs=_between(rng, 1, 32), stored=op == "append" and rng.random() < 0.5)
        longest = _between(rng, 1, (32768 if case["stored"] or case["dtype"] == "fp32" else 131072) // case["seqs"])
        shortest = _between(rng, max(1, longest // 9), longest)
        most = 1 if op == "append" and rng.random() < 0.3 else _between(rng, 1, longest)
        return case | dict(longest=longest, shortest=shortest, new_most=most, new_least=_between(rng, 1, most))
    kind = rng.choice(["step", "step", "listed", "draft", "chunk"])
    hkv = rng.choice([1, 2, 4, 8])
    case |= dict(hkv=hkv, hq=hkv * rng.choice([1, 2, 4, 5, 8]), blocks=0, block=0)
    if kind == "chunk":
        case["dtype"] = "bf16"
        seqs = rng.choice([1, 1, 2, 4])
        most = _between(rng, 65, 4096 // seqs)
        longest = most + _between(rng, 1, 24576 * 32 // max(32, case["hq"]) // seqs)
        return case | dict(seqs=seqs, new_most=most, new_least=_between(rng, max(1, most // 4), most), longest=longest,
                           shortest=_between(rng, max(most, longest // 6), longest))
    seqs = _between(rng, 1, 64)
    longest = _between(rng, 16, 262144 // seqs)
    shortest = _between(rng, max(8, longest // 50), longest)
    case |= dict(seqs=seqs, longest=longest, shortest=shortest, new_least=1, new_most=1)
    if kind == "draft":
        case["new_most"] = rng.choice([2, 3, 5, 8])
    if kind == "listed":
        case["block"] = rng.choice([64, 128]) if case["page"] <= 64 else 128
        case["blocks"] = _between(rng, 1, 40)
    return case


def _spread(low, high, n):
    """n whole numbers from high down to low, evenly in the logarithm."""
    return [max(1, round(high * (low / high) ** (i / max(1, n - 1)))) for i in range(n)]


def _lengths(case):
    """The sequences' lengths, and how many of their tokens are new."""
    lens = _spread(case["shortest"], case["longest"], case["seqs"])
    new = _spread(case["new_least"], case["new_most"], case["seqs"])
    new = new[1::2] + new[::2]
    return lens, [min(a, b) for a, b in zip(new, lens)]


def work(case):
    lens, new = _lengths(case)
    size = 4 if case["dtype"] == "fp32" else 2
    token = 2 * case["hkv"] * (case["d"] // 2 + case["d"] // 8)           # one token's levels, scales and lows
    rows = 2 * case["hkv"] * case["d"] * size * sum(new)                   # the new tokens' keys and values
    if case["op"] == "append":
        return {"bytes": rows * (2 if case["stored"] else 1) + token * sum(new), "flops": 4 * rows // size}
    if case["op"] == "read":
        return {"bytes": rows + token * sum(new), "flops": 2 * rows // size}
    pairs, seen = 0, 0
    for n, m in zip(lens, new):
        if case["blocks"]:
            nb = -(-n // case["block"])
            n = min(case["blocks"], nb) * case["block"] - (nb * case["block"] - n)    # the newest block is listed
        seen += n
        pairs += m * n - m * (m - 1) // 2
    return {"bytes": token * seen + 2 * case["hq"] * case["d"] * size * sum(new), "flops": 4 * case["d"] * case["hq"] * pairs}


# ------------------------------------------------------------------------------------- plain forms

def _levels(packed, off, values):
    """The 4-bit levels [..., d] of packed rows [..., d / 2].  Channel c of a key is 32 g + 8 q + i and
    lies in byte q d/8 + 4 g + i/2 of its row; channel c of a value is 32 g + 4 r + i and lies in byte
    r d/16 + 2 g + i/2; the even i lies in the low half of the byte.  With 128 channels the
    two halves of a value's row change places in the tokens of a page whose number has bit 1 set."""
    half = packed.shape[-1]
    ng = 2 * half // GROUP
    lead = packed.shape[:-1]
    if values and ng == 4:
        turned = packed.unflatten(-1, (2, half // 2)).flip(-2).flatten(-2)
        packed = torch.where(((off >> 1) & 1).bool().unsqueeze(-1), turned, packed)
    both = torch.stack((packed & 15, packed >> 4), dim=-1)
    split = both.view(*lead, 8, ng, 2, 2) if values else both.view(*lead, 4, ng, 4, 2)
    return split.transpose(-4, -3).reshape(*lead, 2 * half)


def _packed(levels, off, values):
    """The rows [..., d / 2] of levels [..., d]: the other way round."""
    d = levels.shape[-1]
    ng, lead = d // GROUP, levels.shape[:-1]
    split = levels.view(*lead, ng, 8, 2, 2) if values else levels.view(*lead, ng, 4, 4, 2)
    both = split.transpose(-4, -3).reshape(*lead, d // 2, 2)
    packed = both[..., 0] | (both[..., 1] << 4)
    if values and ng == 4:
        turned = packed.unflatten(-1, (2, d // 4)).flip(-2).flatten(-2)
        packed = torch.where(((off >> 1) & 1).bool().unsqueeze(-1), turned, packed)
    return packed


def _quantised(x):
    """Levels [..., d] (uint8), scale and low [..., d / 32] (fp32 that are bf16 values) of x [..., d].
    low is the least value rounded down to bf16, scale the range times fp32's 1/15 rounded up to bf16 (so that 15
    steps reach the largest value), the level the nearest step.  A range under 2^-100 is stored as a
    constant; a group with a NaN or an infinity, or a range that overflows, stands for NaN."""
    x = x.float().unflatten(-1, (-1, GROUP))
    low = x.amin(-1) + 0.0
    bits = low.view(torch.int32)
    down = torch.where(bits < 0, bits + 0xFFFF, bits) & -65536
    low = down.view(torch.float32)
    span = x.amax(-1) - low
    scale = span * (1.0 / 15.0)
    up = ((scale.view(torch.int32) + 0xFFFF) & -65536).view(torch.float32)
    scale = torch.where(span < 2.0 ** -100, torch.zeros_like(up), up)
    bad = ~(torch.isfinite(span) & torch.isfinite(scale) & torch.isfinite(x).all(-1))
    inv = torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))
    levels = torch.clamp(torch.round((x - low.unsqueeze(-1)) * inv.unsqueeze(-1)), 0.0, 15.0)
    levels = torch.where(bad.unsqueeze(-1), torch.zeros_like(levels), levels)
    nan = torch.full_like(low, math.nan)
    return levels.to(torch.uint8).flatten(-2), torch.where(bad, nan, scale), torch.where(bad, nan, low)


def _pairs(scale, low):
    """Scale and low as the bytes [..., d / 8] of their bf16 pairs (NaN as 0x7fc0)."""
    both = torch.stack((scale, low), dim=-1)
    bits = (both.view(torch.int32) >> 16) & 0xFFFF
    bits = torch.where(torch.isnan(both), torch.full_like(bits, 0x7FC0), bits)
    return torch.stack((bits & 0xFF, bits >> 8), dim=-1).to(torch.uint8).flatten(-3)


def _views(data, d):
    """The levels [pages, Hkv, 2, page, d / 2] and the pairs [pages, Hkv, 2, page, d / 8] of the cache, as views."""
    n, hkv, two, page, row = data.shape
    flat = data.view(n, hkv, two, page * row)
    cut = page * d // 2
    return flat[..., :cut].unflatten(-1, (page, d // 2)), flat[..., cut:].unflatten(-1, (page, d // 8))


def _stands_for(data, d, number, head, off, values):
    """fp32 [..., d] of the rows (page number, kv head, token of the page) of the cache."""
    levels, pairs = _views(data, d)
    lev = _levels(levels[number, head, values, off], off, values).float().unflatten(-1, (-1, GROUP))
    bits = pairs[number, head, values, off].unflatten(-1, (-1, 2, 2)).int()
    pair = ((bits[..., 0] << 16) | (bits[..., 1] << 24)).view(torch.float32)
    return (lev * pair[..., 0:1] + pair[..., 1:2]).flatten(-2)


def _places(s):
    """Of each new token (the rows behind the last sequence left out): its sequence, position, page number and token of the page."""
    at = torch.arange(s["total"], device=s["lens"].device)
    seq = torch.searchsorted(s["cu"].long(), at, right=True) - 1
    pos = s["lens"].long()[seq] - s["cu"].long()[seq + 1] + at
    return seq, pos, s["table"].long()[seq, pos // s["page"]], pos % s["page"]


def _append(s):
    _, _, number, off = _places(s)
    levels, pairs = _views(s["data"], s["d"])
    for values, x, stored in ((0, s["k"], s["k_stored"]), (1, s["v"], s["v_stored"])):
        lev, scale, low = _quantised(x[:, :s["total"]])
        levels[number, :, values, off] = _packed(lev, off, values).transpose(0, 1)
        pairs[number, :, values, off] = _pairs(scale, low).transpose(0, 1)
        if stored is not None:
            means = lev.float().unflatten(-1, (-1, GROUP)) * scale.unsqueeze(-1) + low.unsqueeze(-1)
            stored[:, :s["total"]] = means.flatten(-2)


def _read(s):
    _, _, number, off = _places(s)
    head = torch.arange(s["data"].shape[1], device=number.device).unsqueeze(1)
    s["k_out"][:, :s["total"]] = _stands_for(s["data"], s["d"], number, head, off, 0)
    s["v_out"][:, :s["total"]] = _stands_for(s["data"], s["d"], number, head, off, 1)


def _attend(s):
    d, page, hkv, hq, block = s["d"], s["page"], s["data"].shape[1], s["q"].shape[0], s["block"]
    lens, cu, dev = s["lens"].long(), s["cu"].long(), s["lens"].device
    seqs, group, most = lens.numel(), hq // hkv, s["max_new"]
    if block:      # the positions of the listed blocks [B, Hkv, listed tokens]
        pos = (s["idx"].long().unsqueeze(-1) * block + torch.arange(block, device=dev)).flatten(-2)
        pos = torch.where((s["idx"] >= 0).repeat_interleave(block, dim=-1), pos, torch.full_like(pos, 2 ** 40))
    else:
        pos = torch.arange(s["longest"], device=dev).expand(seqs, hkv, -1)
    there = pos < lens.view(-1, 1, 1)
    pos = torch.where(there, pos, torch.zeros_like(pos))
    seq, new_pos, _, _ = _places(s)
    row = torch.arange(s["total"], device=dev) - cu[seq]
    q = torch.zeros(seqs, most, hq, d, device=dev)
    q[seq, row] = s["q"][:, :s["total"]].transpose(0, 1).float()
    q = q.view(seqs, most, hkv, group, d).permute(2, 0, 3, 1, 4)                   # [Hkv, B, G, new, d]
    q_pos = torch.full((seqs, most), -1, device=dev)
    q_pos[seq, row] = new_pos
    o = torch.empty_like(q)
    step = max(1, min(hkv, SCORES // max(1, q[0].numel() // d * pos.shape[-1])))
    for h in range(0, hkv, step):
        at = pos[:, h:h + step].transpose(0, 1)                                     # [heads, B, tokens]
        ok = there[:, h:h + step].transpose(0, 1)
        number = s["table"].long()[torch.arange(seqs, device=dev).unsqueeze(-1), at // page]
        head = torch.arange(h, h + at.shape[0], device=dev).view(-1, 1, 1)
        k = _stands_for(s["data"], d, number, head, at % page, 0)
        v = _stands_for(s["data"], d, number, head, at % page, 1)
        score = torch.matmul(q[h:h + step].flatten(2, 3), k.transpose(-1, -2)).unflatten(2, (group, most)) / math.sqrt(d)
        seen = ok.unsqueeze(2) & (at.unsqueeze(2) <= q_pos.view(1, seqs, most, 1))           # [heads, B, new, tokens]
        score = torch.where(seen.unsqueeze(2), score, torch.full((), -math.inf, device=dev))
        top = score.amax(-1, keepdim=True)
        score = torch.exp(score - torch.where(torch.isinf(top), torch.zeros_like(top), top))
        total = score.sum(-1, keepdim=True)
        score = score / torch.where(total > 0, total, torch.ones_like(total))
        o[h:h + step] = torch.matmul(score.flatten(2, 3), v).unflatten(2, (group, most))
    o = o.permute(1, 3, 0, 2, 4).reshape(seqs, most, hq, d)
    s["out"][:, :s["total"]] = o[seq, row].transpose(0, 1)


# ---------------------------------------------------------------------------------- inputs, one pass

def _rows(g, heads, tokens, d, dtype, token_major, scale=1.0, shift=None):
    """Random rows [heads, tokens, d]; token-major ones are a view of [tokens, heads, d]."""
    x = torch.randn(tokens, heads, d, generator=g, device=DEVICE) * scale
    if shift is not None:
        x += shift
    x = x.to(dtype).transpose(0, 1)
    return x if token_major else x.contiguous()


def _fill(data, d, g):
    """A used cache: keys with a few channels far from zero, values around zero."""
    levels, pairs = _views(data, d)
    n, hkv, _, page, _ = data.shape
    off = torch.arange(page, device=data.device)
    shift = torch.randn(hkv, 1, d, generator=g, device=data.device)
    shift = torch.where(shift.abs() > 1.8, shift * 4.0, shift * 0.5)
    step = max(1, 2 ** 27 // (hkv * page * d))
    for at in range(0, n, step):
        m = min(step, n - at)
        for values in (0, 1):
            x = torch.randn(m, hkv, page, d, generator=g, device=data.device)
            lev, scale, low = _quantised((x if values else x + shift).to(torch.bfloat16))
            levels[at:at + m, :, values] = _packed(lev, off.expand(m, hkv, page), values)
            pairs[at:at + m, :, values] = _pairs(scale, low)
    return shift


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    rng = np.random.RandomState(seed % 2 ** 32)
    lens, new = _lengths(case)
    page, d, hkv, dt = case["page"], case["d"], case["hkv"], DTYPES[case["dtype"]]
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    order = rng.permutation(pages).astype(np.int32)
    table = np.zeros((len(lens), max(need)), np.int32)       # places behind a sequence's last page are not read
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    total = sum(new)
    rows = total + case["spare"]
    s = dict(op=case["op"], d=d, page=page, total=total, max_new=max(new), longest=max(lens), block=case.get("block", 0),
             lens=torch.tensor(lens, dtype=torch.int32, device=DEVICE), table=torch.from_numpy(table).to(DEVICE),
             cu=torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device=DEVICE))
    shape = (pages, hkv, 2, page, 5 * d // 8)
    if case["op"] == "append":
        s["data"] = torch.randint(0, 256, shape, generator=g, device=DEVICE, dtype=torch.uint8)
        shift = torch.randn(hkv, d, generator=g, device=DEVICE)
        shift = torch.where(shift.abs() > 1.8, shift * 4.0, shift * 0.5)
        s["k"] = _rows(g, hkv, rows, d, dt, case["token_major"], 1.0, shift)
        s["v"] = _rows(g, hkv, rows, d, dt, case["token_major"])
        s["k_stored"] = torch.zeros(hkv, rows, d, dtype=dt, device=DEVICE) if case["stored"] else None
        s["v_stored"] = torch.zeros(hkv, rows, d, dtype=dt, device=DEVICE) if case["stored"] else None
        return s
    s["data"] = torch.empty(shape, device=DEVICE, dtype=torch.uint8)
    shift = _fill(s["data"], d, g)
    if case["op"] == "read":
        s["k_out"] = torch.zeros(hkv, rows, d, dtype=dt, device=DEVICE)
        s["v_out"] = torch.zeros(hkv, rows, d, dtype=dt, device=DEVICE)
        return s
    lean = shift[:, 0].repeat_interleave(case["hq"] // hkv, dim=0) * 0.05
    s["q"] = _rows(g, case["hq"], rows, d, dt, case["token_major"], 1.5, lean)
    s["out"] = torch.zeros(rows, case["hq"], d, dtype=dt, device=DEVICE).transpose(0, 1)
    s["idx"] = s["cnt"] = None
    if case["blocks"]:
        # each kv head's list: the newest block and others drawn from those before it, ascending, then -1
        idx = np.full((len(lens), hkv, case["blocks"]), -1, np.int32)
        cnt = np.zeros((len(lens), hkv), np.int32)
        for b, n in enumerate(lens):
            nb = -(-n // case["block"])
            c = min(case["blocks"], nb)
            for h in range(hkv):
                idx[b, h, :c] = sorted(rng.choice(nb - 1, c - 1, replace=False).tolist() + [nb - 1])
                cnt[b, h] = c
        s["idx"], s["cnt"] = torch.from_numpy(idx).to(DEVICE), torch.from_numpy(cnt).to(DEVICE)
    return s


def run(state):
    s = state
    if own:
        from block_sparse_attention_sbsa_b200 import kv4
        if s["op"] == "append":
            kv4.append(s["data"], s["k"], s["v"], s["table"], s["lens"], s["cu"], k_stored=s["k_stored"], v_stored=s["v_stored"])
        elif s["op"] == "read":
            kv4.read(s["data"], s["table"], s["lens"], s["cu"], k_out=s["k_out"], v_out=s["v_out"])
        else:
            kv4.attend(s["data"], s["q"], s["table"], s["lens"], s["cu"], s["max_new"], idx=s["idx"], cnt=s["cnt"],
                       block_size=s["block"], out=s["out"])
    else:
        {"append": _append, "read": _read, "attend": _attend}[s["op"]](s)
    if s["op"] == "append":
        return {"data": s["data"]} | ({"k": s["k_stored"], "v": s["v_stored"]} if s["k_stored"] is not None else {})
    return {"k": s["k_out"], "v": s["v_out"]} if s["op"] == "read" else {"o": s["out"]}


# --------------------------------------------------------------------------------------- in 64 bits

def _decoded(data, d):
    """float64 [pages, page, Hkv, d] of the whole cache's keys and of its values, channel by channel."""
    n, hkv, _, page, _ = data.shape
    raw = data.reshape(n, hkv, 2, -1)
    out = []
    for values in (0, 1):
        levels = raw[:, :, values, :page * d // 2].reshape(n, hkv, page, d // 2)
        words = raw[:, :, values, page * d // 2:].contiguous().view(torch.bfloat16).reshape(n, hkv, page, d // GROUP, 2).double()
        c = torch.arange(d, device=data.device)
        i = c % (4 if values else 8)
        lane = c % GROUP // (4 if values else 8)
        t = torch.arange(page, device=data.device).unsqueeze(1)
        if values:
            turn = ((t >> 1) & 1) * 4 if d == 128 else t * 0
            byte = (lane ^ turn) * (d // 16) + (c // GROUP) * 2 + i // 2
        else:
            byte = (lane * (d // 8) + (c // GROUP) * 4 + i // 2).expand(page, d)
        picked = torch.gather(levels, 3, byte.expand(n, hkv, page, d))
        level = (picked >> ((i % 2) * 4).to(torch.uint8)) & 15
        full = words[..., 0].repeat_interleave(GROUP, -1) * level + words[..., 1].repeat_interleave(GROUP, -1)
        out.append(full.transpose(1, 2))
    return out


def exact(case, seed):
    """What the cache's levels, scales and lows stand for, and attention over it, in 64 bits.  What append writes
    into the cache are whole numbers and has no such value; what it gives back as stored goes by the format's own
    scale, low and level of each group, which are defined on fp32 values."""
    s = prepare(case, seed)
    lens, new = _lengths(case)
    d, page = s["d"], s["page"]
    if case["op"] == "append":
        if not case["stored"]:
            return None
        out = {"data": None}
        for name in ("k", "v"):
            x = s[name].float().cpu().numpy()[:, :s["total"]].reshape(-1, GROUP)
            low = x.min(1).astype(np.float64)
            grid = (x.min(1).view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32).astype(np.float64)     # towards zero
            nxt = ((x.min(1).view(np.uint32) & np.uint32(0xFFFF0000)) + np.uint32(0x10000)).view(np.float32).astype(np.float64)
            low = np.where(grid > low, nxt, grid)
            span = (x.max(1).astype(np.float64) - low).astype(np.float32)
            sc = (span.astype(np.float64) * np.float64(np.float32(1 / 15))).astype(np.float32)
            cut = (sc.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
            sc = np.where(cut < sc, ((sc.view(np.uint32) & np.uint32(0xFFFF0000)) + np.uint32(0x10000)).view(np.float32), cut)
            inv = np.where(sc > 0, np.float32(1) / np.where(sc > 0, sc, np.float32(1)), np.float32(0)).astype(np.float32)
            lev = np.clip(np.rint((x - low[:, None].astype(np.float32)) * inv[:, None]), 0, 15).astype(np.float64)
            full = np.zeros(s[name].shape, np.float64)
            full[:, :s["total"]] = (low[:, None] + sc.astype(np.float64)[:, None] * lev).reshape(s[name].shape[0], -1, d)
            out[name] = torch.from_numpy(full)
        return out
    if sum(m * n for n, m in zip(lens, new)) * case.get("hq", 0) * d > 3e12:
        return None
    k, v = _decoded(s["data"], d)
    table, at = s["table"].long(), 0
    parts = []
    for b, (n, m) in enumerate(zip(lens, new)):
        kb = k[table[b, :-(-n // page)]].flatten(0, 1)[:n]                          # [n, Hkv, d]
        vb = v[table[b, :-(-n // page)]].flatten(0, 1)[:n]
        if case["op"] == "read":
            parts.append((kb[n - m:].transpose(0, 1), vb[n - m:].transpose(0, 1)))
            continue
        heads = []
        for h in range(case["hq"]):
            g = h // (case["hq"] // case["hkv"])
            score = s["q"][h, at:at + m].double() @ kb[:, g].T / math.sqrt(d)
            hidden = torch.arange(n, device=k.device) > torch.arange(n - m, n, device=k.device).unsqueeze(1)
            if case["blocks"]:
                kept = s["idx"][b, g, :int(s["cnt"][b, g])].long()
                hidden |= ~torch.isin(torch.arange(n, device=k.device) // case["block"], kept)
            heads.append(torch.softmax(score.masked_fill_(hidden, -math.inf), -1) @ vb[:, g])
        parts.append(torch.stack(heads))
        at += m
    spare = case["spare"]
    if case["op"] == "read":
        return {name: torch.nn.functional.pad(torch.cat([p[i] for p in parts], 1), (0, 0, 0, spare)) for i, name in enumerate("kv")}
    return {"o": torch.nn.functional.pad(torch.cat(parts, 1), (0, 0, 0, spare))}
