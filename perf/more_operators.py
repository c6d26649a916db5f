"""Cases, plain forms and reference results of the 8-bit cache and of shared prefixes.

Four operators around a paged key-value cache:

* ``kv_append_q8``: the new tokens' keys (rotated by their positions) and values go
  into a cache of 8-bit codes, e4m3 or int8, with one scale for each token and head;
* ``kv_read_q8``: cached tokens come back packed, as 16-bit values;
* ``attn_decode_q8``: attention of one new token per sequence over that cache;
* ``attn_decode_shared``: attention of one new token per sequence over a prefix that
  the whole batch shares and the sequence's own tokens behind it (16-bit cache).

The scale of a row x of d channels is ``max(max|x| / top, 2^-126)`` with top 448 (e4m3)
or 127 (int8), in 32 bits, and its codes are ``x * (1 / scale)`` rounded to nearest even.

A case is a dict of plain values.  Sequence lengths are drawn from the case's own
``mix`` between ``low`` and ``high`` (the first sequence has ``high``).
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
_CODES = {"e4m3": (torch.float8_e4m3fn, 448.0), "int8": (torch.int8, 127.0)}


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one new token of one stream: what a single-user loop pays at every step
        {"name": "append_one_token", "op": "append", "type": "fp16", "codes": "e4m3", "seqs": 1,
         "low": 1, "high": 1, "past_low": 700, "past_high": 700, "mix": 1, "heads": 12,
         "kv_heads": 12, "dim": 64, "page": 16, "axes": 1, "rotary": 64, "paired": False},
        # prompt chunks of a server, behind what the cache holds already
        {"name": "append_prompts", "op": "append", "type": "bf16", "codes": "e4m3", "seqs": 11,
         "low": 290, "high": 4999, "past_low": 1, "past_high": 2900, "mix": 2, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 16, "axes": 1, "rotary": 128, "paired": False},
        # one new token of each of many streams in int8, their own short tails read back
        {"name": "chunk_token_batch", "op": "chunk", "type": "bf16", "codes": "int8", "seqs": 150,
         "low": 1, "high": 1, "past_low": 0, "past_high": 130, "mix": 3, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 16, "axes": 1, "rotary": 64, "paired": True},
        # frames of 512x384 cut into 16-pixel patches (32x24 = 768 tokens), rotated by row and
        # column, added to a memory of earlier frames that is then read whole
        {"name": "chunk_frames", "op": "chunk", "type": "fp16", "codes": "int8", "seqs": 12,
         "low": 768, "high": 768, "past_low": 0, "past_high": 2304, "mix": 4, "heads": 12,
         "kv_heads": 12, "dim": 64, "page": 64, "axes": 2, "rotary": 64, "paired": False},
        # the cached part of one short conversation, for a prompt that continues it
        {"name": "read_one", "op": "read", "type": "fp16", "codes": "int8", "seqs": 1, "low": 333,
         "high": 333, "mix": 5, "heads": 8, "kv_heads": 8, "dim": 72, "page": 24},
        # the cached parts of many, in one packed call
        {"name": "read_batch", "op": "read", "type": "bf16", "codes": "e4m3", "seqs": 24,
         "low": 100, "high": 9001, "mix": 6, "heads": 32, "kv_heads": 8, "dim": 128, "page": 16},
        # one stream's next token over a short cache: latency
        {"name": "decode_one", "op": "decode", "type": "fp16", "codes": "e4m3", "seqs": 1,
         "low": 805, "high": 805, "mix": 7, "heads": 16, "kv_heads": 16, "dim": 64, "page": 16,
         "lse": False},
        # a server's step over streams of very different lengths
        {"name": "decode_batch", "op": "decode", "type": "bf16", "codes": "e4m3", "seqs": 90,
         "low": 50, "high": 9000, "mix": 8, "heads": 32, "kv_heads": 8, "dim": 128, "page": 16,
         "lse": False},
        # few streams with very long caches
        {"name": "decode_far", "op": "decode", "type": "bf16", "codes": "int8", "seqs": 4,
         "low": 80001, "high": 131000, "mix": 9, "heads": 32, "kv_heads": 4, "dim": 128,
         "page": 64, "lse": True},
        # a few answers drawn from one short question
        {"name": "shared_few", "op": "shared", "type": "fp16", "seqs": 6, "low": 1, "high": 150,
         "prefix": 1300, "mix": 10, "heads": 16, "kv_heads": 16, "dim": 64, "page": 16,
         "lse": False},
        # a server's step: streams behind one system prompt
        {"name": "shared_batch", "op": "shared", "type": "bf16", "seqs": 32, "low": 10,
         "high": 1500, "prefix": 9001, "mix": 11, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 16, "lse": False},
        # many questions to one long document; the log-sums are kept to join with another part
        {"name": "shared_document", "op": "shared", "type": "bf16", "seqs": 144, "low": 5,
         "high": 700, "prefix": 30011, "mix": 12, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "lse": True},
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["append", "chunk", "read", "decode", "decode", "shared", "shared"])
    case = {"op": op, "type": rng.choice(["bf16", "fp16"]), "mix": rng.randrange(1 << 20),
            "kv_heads": rng.choice([1, 2, 3, 4, 8, 16]),
            "dim": rng.choice([32, 40, 64, 64, 72, 80, 96, 112, 128, 128]),
            "page": rng.choice([1, 8, 16, 16, 24, 32, 64, 100, 128])}
    case["heads"] = case["kv_heads"] * rng.choice([1, 1, 2, 3, 4, 5, 7, 8])
    if case["heads"] * case["dim"] > 4096:
        case["heads"] = case["kv_heads"]
    width, kv_width = case["heads"] * case["dim"], case["kv_heads"] * case["dim"]
    if op != "shared":
        case["codes"] = "e4m3" if op == "append" else rng.choice(["e4m3", "int8"])
    if op in ("append", "chunk"):
        tokens = min(_log_int(rng, 1, 40000000 // width), 16000)    # in all sequences
        case["seqs"] = _log_int(rng, 1, min(tokens, 256))
        case["high"] = max(1, tokens // case["seqs"])
        case["low"] = rng.randint(1, case["high"])
        past = 4000 if op == "append" else max(1, 16000 // case["seqs"])
        case["past_high"] = _log_int(rng, 1, past)
        case["past_low"] = rng.randint(0, case["past_high"])
        case["axes"] = rng.choice([1, 1, 2])
        case["rotary"] = rng.choice([case["dim"], case["dim"] // 16 * 8])
        case["rotary"] -= case["rotary"] % (2 * case["axes"])
        case["paired"] = rng.random() < 0.4
        return case
    if op == "read":
        case["seqs"] = _log_int(rng, 1, 100)
        case["high"] = _log_int(rng, 1, max(2, 50000000 // (kv_width * case["seqs"])))
    elif op == "decode":
        case["seqs"] = _log_int(rng, 1, 200)
        case["high"] = _log_int(rng, 1, max(2, 180000000 // (kv_width * case["seqs"])))
        case["lse"] = rng.random() < 0.3
    else:
        case["seqs"] = _log_int(rng, 2, 256)
        # pairs of a stream and a prefix token, bounded by the longest listed case's
        case["prefix"] = _log_int(rng, 16, max(17, min(40000, 17000000000 // (width * case["seqs"]))))
        case["high"] = _log_int(rng, 1, max(2, min(3000, 90000000 // (kv_width * case["seqs"]))))
        case["lse"] = rng.random() < 0.3
    case["low"] = rng.randint(1, case["high"])
    return case


def _lengths(case):
    """New (or cached) tokens and earlier tokens of each sequence."""
    rng = random.Random(case["mix"])
    new = [case["high"]] + [_log_int(rng, case["low"], case["high"])
                            for _ in range(case["seqs"] - 1)]
    past = [0] * case["seqs"]
    if case.get("past_high"):
        past = [case["past_high"]] + [rng.randint(case["past_low"], case["past_high"])
                                      for _ in range(case["seqs"] - 1)]
    return new, past


def _starts(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return at


def work(case):
    new, past = _lengths(case)
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    tokens, seqs = sum(new), case["seqs"]

    def pages(lengths):
        return sum(-(-n // case["page"]) for n in lengths)

    coded = 2 * hk * (d + 4)                # a token's codes and scales, keys and values
    if case["op"] in ("append", "chunk"):
        totals = [n + p for n, p in zip(new, past)]
        # q, k, v read, q written; the codes and scales written
        moved = tokens * ((2 * hq + 2 * hk) * d * 2 + coded)
        moved += tokens * 8 if case["axes"] == 2 else 0
        moved += 8 * seqs + case["rotary"] // (2 * case["axes"]) * 8
        flops = tokens * (3 * (hq + hk) * case["rotary"] + 3 * 2 * hk * d)
        if case["op"] == "append":
            moved += 4 * (pages(totals) - sum(p // case["page"] for p in past))
        else:                               # all that is cached: read, and written packed
            moved += sum(totals) * (coded + 2 * hk * d * 2) + 4 * pages(totals) + 4 * seqs
            flops += sum(totals) * 2 * hk * d
        return {"bytes": moved, "flops": flops}
    if case["op"] == "read":
        return {"bytes": tokens * (coded + 2 * hk * d * 2) + 4 * pages(new) + 4 * seqs,
                "flops": tokens * 2 * hk * d}
    moved = 2 * seqs * hq * d * 2 + 4 * pages(new) + 4 * seqs
    moved += 4 * seqs * hq if case["lse"] else 0
    if case["op"] == "decode":
        return {"bytes": moved + tokens * coded, "flops": 4 * d * hq * tokens}
    moved += (tokens + case["prefix"]) * 2 * hk * d * 2 + 4 * pages([case["prefix"]])
    return {"bytes": moved, "flops": 4 * d * hq * (tokens + seqs * case["prefix"])}


# ------------------------------------------------------------------ the inputs
def _table(totals, page, gen):
    """Pages of a cache dealt to sequences in a random order: table, number of pages."""
    need = [-(-n // page) for n in totals]
    count = sum(need) + 3                               # a few pages belong to nobody
    deal = torch.randperm(count, generator=gen, device="cuda").to(torch.int32)
    width = max(need)
    at = torch.tensor(_starts(need)[:-1], device="cuda")[:, None]
    number = torch.arange(width, device="cuda")[None, :]
    live = number < torch.tensor(need, device="cuda")[:, None]
    return torch.where(live, deal[(at + number).clamp_(max=count - 1)], 0), count


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    kind = _TYPES[case["type"]]
    hq, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    new, past = _lengths(case)
    totals = [n + p for n, p in zip(new, past)]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=kind)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    state = {"case": case}
    table, pages = _table(totals + ([case["prefix"]] if case["op"] == "shared" else []), page, gen)
    state["k_cache"], state["v_cache"] = normal(pages, page, hk, d), normal(pages, page, hk, d)
    state["table"] = table
    if case["op"] in ("decode", "shared"):
        # Scores of a trained layer are uneven: a direction that a sequence's first key and,
        # more weakly, every query shares draws much of the weight.
        lean = torch.randn(hk, d, generator=gen, device="cuda").to(kind)
        state["q"] = normal(case["seqs"], hq, d) + 0.4 * lean.repeat_interleave(hq // hk, 0)
        state["k_cache"][table[:, 0].long(), 0] += lean
        state["lens"] = ints(new)
    if case["op"] == "shared":
        state["prefix_pages"] = table[-1, :-(-case["prefix"] // page)].clone()
        state["table"] = table[:-1, :-(-max(new) // page)].contiguous()
        state["prefix_len"] = ints([case["prefix"]])
        return state
    # values of heads and tokens differ in size as a layer's do
    for name in ("k_cache", "v_cache"):
        state[name] *= torch.exp(0.5 * torch.randn(pages, page, hk, 1, generator=gen,
                                                   device="cuda")).to(kind)
    codes, scales = zip(*(_quantise(state[name], case["codes"]) for name in ("k_cache", "v_cache")))
    state["k_cache"], state["v_cache"] = codes
    # [pages, heads, rows, (key, value)]
    state["scales"] = torch.stack(scales, -1).transpose(1, 2).contiguous()
    state["totals"] = sum(totals)
    state["cu_all"] = ints(_starts(totals))
    if case["op"] in ("append", "chunk"):
        # one projection's output holds queries, keys and values of a token side by side
        rows = normal(sum(new), hq + 2 * hk, d)
        pairs = case["rotary"] // (2 * case["axes"])
        state.update(q=rows[:, :hq], k=rows[:, hq:hq + hk], v=rows[:, hq + hk:], start=ints(past),
                     cu=ints(_starts(new)), positions=None,
                     inv_freq=10000.0 ** (-torch.arange(pairs, device="cuda", dtype=torch.float64)
                                          / pairs))
        if case["axes"] == 2:                           # patch rows of 32 columns
            at = torch.cat([torch.arange(n, device="cuda", dtype=torch.int32) for n in new])
            state["positions"] = torch.stack([at // 32, at % 32], 1).contiguous()
    return state


# -------------------------------------------------------------- the plain forms
def _quantise(x, codes):
    """Codes and scales of rows of channels."""
    kind, top = _CODES[codes]
    x = x.float()
    scale = (x.abs().amax(-1) / top).clamp_min(2.0 ** -126)
    x = x * (1.0 / scale)[..., None]
    return (x.to(kind) if kind.is_floating_point else x.round().to(kind)), scale


def _rotate(x, cos, sin, axes, paired):
    """x [T, H, d] float, cos and sin [T, axes, pairs]."""
    pairs = cos.shape[2]
    head, rest = x[..., :2 * pairs * axes], x[..., 2 * pairs * axes:]
    # [T, H, axes, pairs] of the first and the second channel of each pair
    if paired:
        one, two = head.unflatten(-1, (axes, pairs, 2)).unbind(-1)
    else:
        one, two = head.unflatten(-1, (axes, 2, pairs)).unbind(-2)
    c, s = cos[:, None], sin[:, None]
    turned = torch.stack([one * c - two * s, two * c + one * s], -1 if paired else -2)
    return torch.cat([turned.flatten(2), rest], -1)


def _places(cu, start, count):
    """Sequence and number in it of each packed token."""
    token = torch.arange(count, device="cuda")
    seq = torch.searchsorted(cu[1:].long(), token, right=True)
    return seq, token - cu[seq].long() + (0 if start is None else start[seq].long())


def _plain_append(s):
    case, kind = s["case"], s["q"].dtype
    seq, place = _places(s["cu"], s["start"], s["q"].shape[0])
    where = s["positions"] if s["positions"] is not None else place[:, None]
    # far positions lose their angle in 32 bits
    angle = where.double()[:, :, None] * s["inv_freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _rotate(s["q"].float(), cos, sin, case["axes"], case["paired"]).to(kind)
    k = _rotate(s["k"].float(), cos, sin, case["axes"], case["paired"])
    page, row = s["table"][seq, place // case["page"]].long(), place % case["page"]
    k_codes, k_scale = _quantise(k, case["codes"])
    v_codes, v_scale = _quantise(s["v"], case["codes"])
    s["k_cache"].view(torch.uint8)[page, row] = k_codes.view(torch.uint8)
    s["v_cache"].view(torch.uint8)[page, row] = v_codes.view(torch.uint8)
    s["scales"].transpose(1, 2)[page, row] = torch.stack([k_scale, v_scale], -1)
    return q


def _decoded(s, name, which, page, row):
    """Cached rows as the 32-bit values they stand for."""
    cache = s[name]
    codes = cache.view(torch.uint8)[page, row].view(cache.dtype).float()
    return codes * s["scales"].transpose(1, 2)[page, row][..., which, None]


def _plain_read(s):
    case, kind = s["case"], _TYPES[s["case"]["type"]]
    seq, place = _places(s["cu_all"], None, s["totals"])
    page, row = s["table"][seq, place // case["page"]].long(), place % case["page"]
    return (_decoded(s, "k_cache", 0, page, row).to(kind),
            _decoded(s, "v_cache", 1, page, row).to(kind))


def _softmax_rows(score):
    """Unnormalised weights, totals and log-sums along the last axis."""
    top = score.amax(-1, keepdim=True)
    weight = (score - top).exp()
    total = weight.sum(-1, keepdim=True)
    return weight, total, (top + total.log()).squeeze(-1)


def _padded(s):
    """Pages and rows of every sequence's tokens up to the longest one's, and which exist."""
    case = s["case"]
    at = torch.arange(case["high"], device="cuda")
    page = s["table"][:, at // case["page"]].long()
    return page, (at % case["page"]).expand_as(page), at < s["lens"][:, None]


def _plain_decode(s):
    case = s["case"]
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    page, row, there = _padded(s)
    query = s["q"].float().view(-1, hk, hq // hk, d)
    key = _decoded(s, "k_cache", 0, page, row)                         # [seqs, keys, heads, d]
    score = (query @ key.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(d))   # [seqs, heads, group, keys]
    del key
    score.masked_fill_(~there[:, None, None, :], -math.inf)
    weight, total, lse = _softmax_rows(score)
    value = _decoded(s, "v_cache", 1, page, row)
    out = ((weight @ value.transpose(1, 2)) / total).reshape(-1, hq, d).to(s["q"].dtype)
    return (out, lse.reshape(-1, hq)) if case["lse"] else out


def _plain_shared(s):
    case = s["case"]
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    seqs, group, prefix = case["seqs"], hq // hk, case["prefix"]
    query = s["q"].float().view(seqs, hk, group, d) * (1.0 / math.sqrt(d))
    # the prefix once for all sequences' queries of a head
    first = s["prefix_pages"].long()
    key = s["k_cache"][first].flatten(0, 1)[:prefix].float()           # [prefix, heads, d]
    value = s["v_cache"][first].flatten(0, 1)[:prefix].float()
    ahead = query.transpose(0, 1).reshape(hk, seqs * group, d) @ key.permute(1, 2, 0)
    ahead = ahead.view(hk, seqs, group, prefix)
    page, row, there = _padded(s)
    tail = query @ s["k_cache"][page, row].float().permute(0, 2, 3, 1)
    tail = tail.masked_fill_(~there[:, None, None, :], -math.inf).transpose(0, 1)
    weight, total, lse = _softmax_rows(torch.cat([ahead, tail], -1))   # [heads, seqs, group, keys]
    del ahead, tail
    out = (weight[..., :prefix].reshape(hk, seqs * group, prefix) @ value.transpose(0, 1))
    out = out.view(hk, seqs, group, d).transpose(0, 1)
    out = out + weight[..., prefix:].transpose(0, 1) @ s["v_cache"][page, row].float().transpose(1, 2)
    out = (out / total.transpose(0, 1)).reshape(seqs, hq, d).to(s["q"].dtype)
    return (out, lse.transpose(0, 1).reshape(seqs, hq)) if case["lse"] else out


# ------------------------------------------------------------ the measured calls
def _cached(s, q):
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"], "scales": s["scales"]}


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        if op == "append":
            return _cached(s, _plain_append(s))
        if op == "chunk":
            q = _plain_append(s)
            k, v = _plain_read(s)
            return {"q": q, "k": k, "v": v}
        if op == "read":
            k, v = _plain_read(s)
            return {"k": k, "v": v}
        return _plain_decode(s) if op == "decode" else _plain_shared(s)
    import reciprocal_nearest_neighbour_b200 as rnn

    q = None
    if op in ("append", "chunk"):
        q, _ = rnn.kv_append_q8(s["k"], s["v"], s["k_cache"], s["v_cache"], s["scales"], s["table"],
                                s["start"], s["cu"], q=s["q"], inv_freq=s["inv_freq"],
                                positions=s["positions"], paired=case["paired"])
        if op == "append":
            return _cached(s, q)
    if op in ("chunk", "read"):
        k, v = rnn.kv_read_q8(s["k_cache"], s["v_cache"], s["scales"], s["table"], s["cu_all"],
                              s["totals"], _TYPES[case["type"]])
        return {"k": k, "v": v} if q is None else {"q": q, "k": k, "v": v}
    if op == "decode":
        return rnn.attn_decode_q8(s["q"], s["k_cache"], s["v_cache"], s["scales"], s["table"],
                                  s["lens"], with_lse=case["lse"])
    return rnn.attn_decode_shared(s["q"], s["k_cache"], s["v_cache"], s["prefix_pages"],
                                  s["prefix_len"], s["table"], s["lens"], with_lse=case["lse"])


# ---------------------------------------------------------- the 64-bit reference
def _exact_turn(x, places, inv_freq, axes, paired):
    """Rotation as a product of complex numbers, in 64 bits."""
    pairs = inv_freq.numel()
    y = x.double().clone()
    for a in range(axes):
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           places[:, a, None].double() * inv_freq)[:, None, :]
        first = torch.arange(pairs, device="cuda")
        first = 2 * pairs * a + (2 * first if paired else first)
        second = first + (1 if paired else pairs)
        z = torch.complex(x[..., first].double(), x[..., second].double()) * turn
        y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_codes(x, codes, rounded):
    """Codes (`rounded`, or as they are before the rounding) and scales in 64 bits."""
    kind, top = _CODES[codes]
    scale = torch.clamp(torch.linalg.vector_norm(x, math.inf, -1) / top, min=2.0 ** -126)
    ratio = torch.clamp(x / scale[..., None], -top, top)
    if rounded:
        step = torch.exp2(torch.floor(torch.log2(ratio.abs().clamp(min=2.0 ** -6))) - 3) \
            if codes == "e4m3" else torch.ones((), dtype=torch.float64, device="cuda")
        ratio = torch.round(ratio / step) * step
    return ratio, scale


def _exact_rows(s, totals):
    """Page and row of every cached token of every sequence, packed."""
    size = s["case"]["page"]
    pages, rows = [], []
    for b, n in enumerate(totals):
        at = torch.arange(n, device="cuda")
        pages.append(s["table"][b].long()[torch.div(at, size, rounding_mode="floor")])
        rows.append(at.remainder(size))
    return torch.cat(pages), torch.cat(rows)


def _exact_attend(query, key, value, scale):
    """Softmax of one head in 64 bits: outputs and log-sums."""
    logit = torch.einsum("rc,kc->rk", query, key) * scale
    lse = torch.logsumexp(logit, 1)
    return torch.einsum("rk,kc->rc", torch.exp(logit - lse[:, None]), value), lse


def exact(case, seed):
    s = prepare(case, seed)
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    group, op = hq // hk, case["op"]
    new, past = _lengths(case)
    totals = [n + p for n, p in zip(new, past)]
    result = {}
    if op != "shared":
        k_codes, v_codes = s["k_cache"].double(), s["v_cache"].double()
        scales = s["scales"].double()
    if op in ("append", "chunk"):
        places, pages, rows = [], [], []
        for b, (n, p) in enumerate(zip(new, past)):
            at = torch.arange(p, p + n, device="cuda")
            places.append(at)
            pages.append(s["table"][b].long()[torch.div(at, case["page"], rounding_mode="floor")])
            rows.append(at.remainder(case["page"]))
        places, pages, rows = torch.cat(places), torch.cat(pages), torch.cat(rows)
        where = places[:, None] if s["positions"] is None else s["positions"]
        result["q"] = _exact_turn(s["q"], where, s["inv_freq"], case["axes"], case["paired"])
        k = _exact_turn(s["k"], where, s["inv_freq"], case["axes"], case["paired"])
        for which, (cache, x) in enumerate(((k_codes, k), (v_codes, s["v"].double()))):
            cache[pages, rows], scale = _exact_codes(x, case["codes"], op == "chunk")
            for h in range(hk):
                scales[pages, h, rows, which] = scale[:, h]
        if op == "append":
            result.update(k_cache=k_codes, v_cache=v_codes, scales=scales)
            return result
    if op in ("chunk", "read"):
        pages, rows = _exact_rows(s, totals)
        for which, (name, cache) in enumerate((("k", k_codes), ("v", v_codes))):
            scale = torch.stack([scales[pages, h, rows, which] for h in range(hk)], 1)
            result[name] = cache[pages, rows] * scale[..., None]
        return result
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    scale = float(d) ** -0.5
    at = torch.arange(case.get("prefix", 0), device="cuda")
    if op == "shared":
        first = s["prefix_pages"].long()[torch.div(at, case["page"], rounding_mode="floor")]
        ahead = [(s["k_cache"][first, at.remainder(case["page"]), h].double(),
                  s["v_cache"][first, at.remainder(case["page"]), h].double()) for h in range(hk)]
        # the prefix's part of all sequences at once; it is joined by the log-sums below
        front = [_exact_attend(s["q"][:, h * group:(h + 1) * group].double().flatten(0, 1),
                               *ahead[h], scale) for h in range(hk)]
    for b, n in enumerate(new):
        at = torch.arange(n, device="cuda")
        page = s["table"][b].long()[torch.div(at, case["page"], rounding_mode="floor")]
        row = at.remainder(case["page"])
        for h in range(hk):
            heads = slice(h * group, (h + 1) * group)
            query = s["q"][b, heads].double()
            if op == "decode":
                key = k_codes[page, row, h] * scales[page, h, row, 0, None]
                value = v_codes[page, row, h] * scales[page, h, row, 1, None]
                out[b, heads], lse[b, heads] = _exact_attend(query, key, value, scale)
                continue
            mine, its = _exact_attend(query, s["k_cache"][page, row, h].double(),
                                      s["v_cache"][page, row, h].double(), scale)
            other, theirs = (x[b * group:(b + 1) * group] for x in front[h])
            both = torch.logaddexp(its, theirs)
            lse[b, heads] = both
            out[b, heads] = mine * torch.exp(its - both)[:, None] + \
                other * torch.exp(theirs - both)[:, None]
    return (out, lse) if case["lse"] else out
