"""Cases, plain forms and reference results of the attention operators.

Three operators that a program runs over a model's tokens before its descriptor
maps are matched:

* ``kv_append``: the new tokens' keys and values go into a paged cache, keys
  (and queries) rotated by their positions on the way;
* ``attn_prompt``: attention of packed sequences of different lengths, causal or
  full, with grouped heads;
* ``attn_decode``: attention of one new token per sequence over the paged cache.

A case is a dict of plain values.  Sequence lengths are drawn from the case's
own ``mix`` between ``low`` and ``high`` (the first sequence has ``high``).
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one new token of one stream: what a single-user loop pays at every step
        {"name": "append_one_token", "op": "append", "type": "fp16", "seqs": 1, "low": 1, "high": 1,
         "past_low": 600, "past_high": 600, "mix": 1, "heads": 12, "kv_heads": 12, "dim": 64,
         "page": 16, "axes": 1, "rotary": 64, "paired": False, "keys_out": False},
        # one new token of each of many streams, as a batched server's step has them
        {"name": "append_token_batch", "op": "append", "type": "bf16", "seqs": 200, "low": 1,
         "high": 1, "past_low": 90, "past_high": 6000, "mix": 2, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "axes": 1, "rotary": 128, "paired": False, "keys_out": False},
        # frames of 512x384 cut into 16-pixel patches (32x24 = 768 tokens), rotated by row and column
        {"name": "append_frames", "op": "append", "type": "fp16", "seqs": 24, "low": 768,
         "high": 768, "past_low": 0, "past_high": 0, "mix": 3, "heads": 12, "kv_heads": 12,
         "dim": 64, "page": 64, "axes": 2, "rotary": 64, "paired": False, "keys_out": True},
        # chunks of long prompts behind what the cache holds already, half of each head rotated
        {"name": "append_prompts", "op": "append", "type": "bf16", "seqs": 14, "low": 310,
         "high": 5003, "past_low": 1, "past_high": 3100, "mix": 4, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 48, "axes": 1, "rotary": 64, "paired": True, "keys_out": True},
        # a few short prompts: latency only
        {"name": "prompt_short", "op": "prompt", "type": "fp16", "seqs": 3, "low": 1, "high": 45,
         "past_low": 0, "past_high": 0, "mix": 5, "heads": 8, "kv_heads": 8, "dim": 64,
         "causal": True, "lse": False},
        # an encoder's full attention within each 512x384 frame of a batch
        {"name": "prompt_frames", "op": "prompt", "type": "fp16", "seqs": 24, "low": 768,
         "high": 768, "past_low": 0, "past_high": 0, "mix": 6, "heads": 16, "kv_heads": 16,
         "dim": 64, "causal": False, "lse": False},
        # ordinary prompts of very different lengths in one packed call
        {"name": "prompt_mixed", "op": "prompt", "type": "bf16", "seqs": 20, "low": 17,
         "high": 4001, "past_low": 0, "past_high": 0, "mix": 7, "heads": 32, "kv_heads": 8,
         "dim": 128, "causal": True, "lse": False},
        # new frames' tokens looking at all that was kept of earlier ones; the log-sums are kept to
        # join the result with another part
        {"name": "prompt_memory", "op": "prompt", "type": "bf16", "seqs": 9, "low": 301,
         "high": 1207, "past_low": 700, "past_high": 9000, "mix": 8, "heads": 12, "kv_heads": 4,
         "dim": 96, "causal": False, "lse": True},
        # one long document
        {"name": "prompt_long", "op": "prompt", "type": "bf16", "seqs": 1, "low": 16384,
         "high": 16384, "past_low": 0, "past_high": 0, "mix": 9, "heads": 32, "kv_heads": 8,
         "dim": 128, "causal": True, "lse": False},
        # one stream's next token over a short cache: latency
        {"name": "decode_one", "op": "decode", "type": "fp16", "seqs": 1, "low": 901, "high": 901,
         "mix": 10, "heads": 16, "kv_heads": 16, "dim": 64, "page": 16, "lse": False},
        # a server's step over streams of very different lengths
        {"name": "decode_batch", "op": "decode", "type": "bf16", "seqs": 96, "low": 50,
         "high": 8000, "mix": 11, "heads": 32, "kv_heads": 8, "dim": 128, "page": 16,
         "lse": False},
        # few streams with very long caches
        {"name": "decode_far", "op": "decode", "type": "bf16", "seqs": 4, "low": 90001,
         "high": 131000, "mix": 12, "heads": 32, "kv_heads": 4, "dim": 128, "page": 64,
         "lse": True},
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["append", "prompt", "prompt", "decode", "decode"])
    case = {"op": op, "type": rng.choice(["bf16", "fp16"]), "mix": rng.randrange(1 << 20),
            "kv_heads": rng.choice([1, 2, 3, 4, 8, 16]),
            "dim": rng.choice([32, 40, 64, 64, 72, 80, 96, 112, 128, 128])}
    case["heads"] = case["kv_heads"] * rng.choice([1, 1, 2, 3, 4, 5, 7, 8])
    if case["heads"] * case["dim"] > 4096:
        case["heads"] = case["kv_heads"]
    width = case["heads"] * case["dim"]
    if op == "append":
        tokens = _log_int(rng, 1, 40000000 // width)  # in all sequences
        tokens = min(tokens, 18000)
        case["seqs"] = _log_int(rng, 1, min(tokens, 256))
        case["high"] = max(1, tokens // case["seqs"])
        case["low"] = rng.randint(1, case["high"])
        case["past_high"] = _log_int(rng, 1, 4000)
        case["past_low"] = rng.randint(0, case["past_high"])
        case["page"] = rng.choice([1, 8, 16, 24, 32, 64, 100, 128])
        case["axes"] = rng.choice([1, 1, 2])
        case["rotary"] = rng.choice([case["dim"], case["dim"] // 16 * 8])
        case["rotary"] -= case["rotary"] % (2 * case["axes"])
        case["paired"] = rng.random() < 0.4
        case["keys_out"] = rng.random() < 0.5
    elif op == "prompt":
        case["seqs"] = _log_int(rng, 1, 48)
        # pairs of a query and a key in a sequence, bounded by the longest listed prompt's
        top = int(math.sqrt(1.2e11 / (width * case["seqs"])))
        case["high"] = _log_int(rng, 1, max(2, min(top, 9000)))
        case["low"] = rng.randint(1, case["high"])
        past = rng.random() < 0.4
        case["past_high"] = _log_int(rng, 1, max(1, min(top, 4 * case["high"]))) if past else 0
        case["past_low"] = rng.randint(0, case["past_high"])
        case["causal"] = rng.random() < 0.65
        case["lse"] = rng.random() < 0.3
    else:
        kv_width = case["kv_heads"] * case["dim"]
        case["seqs"] = _log_int(rng, 1, 200)
        case["high"] = _log_int(rng, 1, max(2, 180000000 // (kv_width * case["seqs"])))
        case["low"] = rng.randint(1, case["high"])
        case["page"] = rng.choice([1, 8, 16, 16, 24, 32, 64, 100, 128, 256])
        case["lse"] = rng.random() < 0.3
    return case


def _lengths(case):
    """New tokens and earlier tokens of each sequence."""
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


def _visible(case):
    """Pairs of a query and a key that it sees, over all sequences of a prompt case."""
    new, past = _lengths(case)
    if not case["causal"]:
        return sum(n * (n + p) for n, p in zip(new, past))
    return sum(n * p + n * (n + 1) // 2 for n, p in zip(new, past))


def work(case):
    new, past = _lengths(case)
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    tokens = sum(new)
    if case["op"] == "append":
        pages = sum(-(-(n + p) // case["page"]) - p // case["page"] for n, p in zip(new, past))
        moved = tokens * (2 * hq + 4 * hk) * d * 2      # q, k, v read; q, the cache's k, v written
        moved += tokens * hk * d * 2 if case["keys_out"] else 0
        moved += tokens * 8 if case["axes"] == 2 else 0
        moved += 4 * pages + 8 * case["seqs"] + case["rotary"] // (2 * case["axes"]) * 8
        return {"bytes": moved, "flops": 3 * tokens * (hq + hk) * case["rotary"]}
    if case["op"] == "prompt":
        keys = tokens + sum(past)
        moved = 2 * tokens * hq * d * 2 + 2 * keys * hk * d * 2 + 8 * (case["seqs"] + 1)
        moved += 4 * tokens * hq if case["lse"] else 0
        return {"bytes": moved, "flops": 4 * d * hq * _visible(case)}
    pages = sum(-(-n // case["page"]) for n in new)
    moved = 2 * tokens * hk * d * 2 + 2 * case["seqs"] * hq * d * 2 + 4 * pages + 4 * case["seqs"]
    moved += 4 * case["seqs"] * hq if case["lse"] else 0
    return {"bytes": moved, "flops": 4 * d * hq * tokens}


# ------------------------------------------------------------------ the inputs
def _table(totals, page, gen):
    """Pages of a cache dealt to sequences in a random order: table, number of pages."""
    need = [-(-n // page) for n in totals]
    count = sum(need) + 3                               # a few pages belong to nobody
    deal = torch.randperm(count, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(len(totals), max(need), dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = deal[at:at + n]
        at += n
    return table, count


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    kind = _TYPES[case["type"]]
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    new, past = _lengths(case)
    totals = [n + p for n, p in zip(new, past)]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=kind)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    state = {"case": case, "new": new, "past": past}
    if case["op"] == "append":
        table, pages = _table(totals, case["page"], gen)
        # one projection's output holds queries, keys and values of a token side by side
        rows = normal(sum(new), hq + 2 * hk, d)
        pairs = case["rotary"] // (2 * case["axes"])
        state.update(q=rows[:, :hq], k=rows[:, hq:hq + hk], v=rows[:, hq + hk:],
                     k_cache=normal(pages, case["page"], hk, d),
                     v_cache=normal(pages, case["page"], hk, d),
                     table=table, start=ints(past), cu=ints(_starts(new)), positions=None,
                     inv_freq=10000.0 ** (-torch.arange(pairs, device="cuda", dtype=torch.float64)
                                          / pairs))
        if case["axes"] == 2:                           # patch rows of 32 columns
            at = torch.cat([torch.arange(n, device="cuda", dtype=torch.int32) for n in new])
            state["positions"] = torch.stack([at // 32, at % 32], 1).contiguous()
        return state
    # Scores of a trained layer are uneven: a direction that a sequence's first key and, more
    # weakly, every query shares draws much of the weight.
    lean = torch.randn(hk, d, generator=gen, device="cuda").to(kind)
    tilt = lean.repeat_interleave(hq // hk, 0)
    if case["op"] == "prompt":
        state.update(q=normal(sum(new), hq, d) + 0.4 * tilt, k=normal(sum(totals), hk, d),
                     v=normal(sum(totals), hk, d), cu_q=ints(_starts(new)),
                     cu_k=ints(_starts(totals)))
        state["k"][state["cu_k"][:-1].long()] += lean
        return state
    table, pages = _table(new, case["page"], gen)
    state.update(q=normal(case["seqs"], hq, d) + 0.4 * tilt,
                 k_cache=normal(pages, case["page"], hk, d),
                 v_cache=normal(pages, case["page"], hk, d), table=table, lens=ints(new))
    state["k_cache"][table[:, 0].long(), 0] += lean
    return state


# -------------------------------------------------------------- the plain forms
def _rotate(x, cos, sin, axes, paired):
    """x [T, H, d] float, cos and sin [T, axes, pairs]."""
    pairs = cos.shape[2]
    out = x.clone()
    for a in range(axes):
        block = x[..., 2 * pairs * a:2 * pairs * (a + 1)]
        c, s = cos[:, None, a], sin[:, None, a]
        if paired:
            one, two = block[..., 0::2], block[..., 1::2]
            turned = torch.stack([one * c - two * s, two * c + one * s], -1).flatten(-2)
        else:
            one, two = block[..., :pairs], block[..., pairs:]
            turned = torch.cat([one * c - two * s, two * c + one * s], -1)
        out[..., 2 * pairs * a:2 * pairs * (a + 1)] = turned
    return out


def _plain_append(s):
    case, kind = s["case"], s["q"].dtype
    token = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(s["cu"][1:].long(), token, right=True)
    place = s["start"][seq].long() + token - s["cu"][seq].long()
    where = s["positions"] if s["positions"] is not None else place[:, None]
    # far positions lose their angle in 32 bits
    angle = where.double()[:, :, None] * s["inv_freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _rotate(s["q"].float(), cos, sin, case["axes"], case["paired"]).to(kind)
    k = _rotate(s["k"].float(), cos, sin, case["axes"], case["paired"]).to(kind)
    page = s["table"][seq, place // case["page"]].long()
    s["k_cache"][page, place % case["page"]] = k
    s["v_cache"][page, place % case["page"]] = s["v"]
    return {"q": q, "k": k if case["keys_out"] else None, "k_cache": s["k_cache"],
            "v_cache": s["v_cache"]}


def _plain_prompt(s):
    case = s["case"]
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    group = hq // hk
    scale = 1.0 / math.sqrt(d)
    out = torch.empty_like(s["q"])
    lse = torch.empty(s["q"].shape[:2], device="cuda") if case["lse"] else None
    at_q, at_k = 0, 0
    for n, p in zip(s["new"], s["past"]):
        m = n + p
        for h in range(hk):
            key = s["k"][at_k:at_k + m, h].float()
            value = s["v"][at_k:at_k + m, h].float()
            rows = max(1, 200000000 // (m * group))
            for r in range(0, n, rows):
                e = min(n, r + rows)
                query = s["q"][at_q + r:at_q + e, h * group:(h + 1) * group].float()
                score = (query @ key.t()) * scale                      # [rows, group, keys]
                if case["causal"]:
                    last = torch.arange(r, e, device="cuda") + p
                    hidden = torch.arange(m, device="cuda")[None, :] > last[:, None]
                    score.masked_fill_(hidden[:, None, :], -math.inf)
                top = score.amax(-1, keepdim=True)
                weight = score.sub_(top).exp_()
                total = weight.sum(-1, keepdim=True)
                out[at_q + r:at_q + e, h * group:(h + 1) * group] = (weight @ value) / total
                if lse is not None:
                    lse[at_q + r:at_q + e, h * group:(h + 1) * group] = \
                        (top + total.log()).squeeze(-1)
        at_q, at_k = at_q + n, at_k + m
    return (out, lse) if case["lse"] else out


def _plain_decode(s):
    case = s["case"]
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    scale = 1.0 / math.sqrt(d)
    out = torch.empty_like(s["q"])
    lse = torch.empty(s["q"].shape[:2], device="cuda") if case["lse"] else None
    for b, n in enumerate(s["new"]):
        pages = s["table"][b, :-(-n // case["page"])].long()
        key = s["k_cache"][pages].flatten(0, 1)[:n].float()            # [keys, heads, d]
        value = s["v_cache"][pages].flatten(0, 1)[:n].float()
        query = s["q"][b].float().view(hk, hq // hk, d)
        score = (query @ key.permute(1, 2, 0)) * scale                 # [heads, group, keys]
        top = score.amax(-1, keepdim=True)
        weight = (score - top).exp()
        total = weight.sum(-1, keepdim=True)
        out[b] = ((weight @ value.transpose(0, 1)) / total).reshape(hq, d)
        if lse is not None:
            lse[b] = (top + total.log()).reshape(hq)
    return (out, lse) if case["lse"] else out


# ------------------------------------------------------------ the measured calls
def run(state):
    op = state["case"]["op"]
    if not own:
        return {"append": _plain_append, "prompt": _plain_prompt, "decode": _plain_decode}[op](state)
    import reciprocal_nearest_neighbour_b200 as rnn

    s, case = state, state["case"]
    if op == "append":
        q, k = rnn.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["start"],
                             s["cu"], q=s["q"], inv_freq=s["inv_freq"], positions=s["positions"],
                             paired=case["paired"], with_k=case["keys_out"])
        return {"q": q, "k": k, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "prompt":
        return rnn.attn_prompt(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=case["causal"],
                               with_lse=case["lse"])
    return rnn.attn_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                           with_lse=case["lse"])


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


def _exact_softmax(query, key, value, scale, first_hidden=None):
    """Softmax of one head in 64 bits: outputs and log-sums; row i sees keys [0, first_hidden[i])."""
    logit = torch.einsum("rc,kc->rk", query, key) * scale
    if first_hidden is not None:
        at = torch.arange(key.shape[0], device="cuda")
        logit = torch.where(at[None] < first_hidden[:, None], logit,
                            torch.full((), -math.inf, dtype=torch.float64, device="cuda"))
    lse = torch.logsumexp(logit, 1)
    return torch.einsum("rk,kc->rc", torch.exp(logit - lse[:, None]), value), lse


def exact(case, seed):
    s = prepare(case, seed)
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    group = hq // hk
    if case["op"] == "append":
        places, pages, rows = [], [], []
        for b, (n, p) in enumerate(zip(s["new"], s["past"])):
            at = torch.arange(p, p + n, device="cuda")
            places.append(at)
            pages.append(s["table"][b].long()[torch.div(at, case["page"], rounding_mode="floor")])
            rows.append(at.remainder(case["page"]))
        places, pages, rows = torch.cat(places), torch.cat(pages), torch.cat(rows)
        where = places[:, None] if s["positions"] is None else s["positions"]
        q = _exact_turn(s["q"], where, s["inv_freq"], case["axes"], case["paired"])
        k = _exact_turn(s["k"], where, s["inv_freq"], case["axes"], case["paired"])
        k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
        k_cache[pages, rows], v_cache[pages, rows] = k, s["v"].double()
        return {"q": q, "k": k if case["keys_out"] else None, "k_cache": k_cache,
                "v_cache": v_cache}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    scale = float(d) ** -0.5
    if case["op"] == "decode":
        for b, n in enumerate(s["new"]):
            at = torch.arange(n, device="cuda")
            page = s["table"][b].long()[torch.div(at, case["page"], rounding_mode="floor")]
            for h in range(hk):
                key = s["k_cache"][page, at.remainder(case["page"]), h].double()
                value = s["v_cache"][page, at.remainder(case["page"]), h].double()
                heads = slice(h * group, (h + 1) * group)
                out[b, heads], lse[b, heads] = _exact_softmax(s["q"][b, heads].double(), key,
                                                              value, scale)
        return (out, lse) if case["lse"] else out
    starts_q, starts_k = _starts(s["new"]), _starts([n + p for n, p in zip(s["new"], s["past"])])
    for b, n in enumerate(s["new"]):
        m = starts_k[b + 1] - starts_k[b]
        step = max(1, 150000000 // m)
        for h in range(hq):
            key = s["k"][starts_k[b]:starts_k[b + 1], h // group].double()
            value = s["v"][starts_k[b]:starts_k[b + 1], h // group].double()
            for r in range(0, n, step):
                e = min(n, r + step)
                seen = torch.arange(r, e, device="cuda") + (m - n + 1) if case["causal"] else None
                rows = slice(starts_q[b] + r, starts_q[b] + e)
                # under the causal mask no row of this block sees a key at or behind `far`
                far = m - n + e if case["causal"] else m
                out[rows, h], lse[rows, h] = _exact_softmax(s["q"][rows, h].double(), key[:far],
                                                            value[:far], scale, seen)
    return (out, lse) if case["lse"] else out
