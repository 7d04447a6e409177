"""What surrounds a paged cache's decoding step, as it is measured: rotary
positions, attention over whole prompts and its gradients, and the maps that
bring new tokens to their slots and sequences to their pages.

Rows of q, k and v are fp16 [T, heads, D], tokens of all sequences one after
another; they lie in the output of one projection, q | k | v, so they are
strided.  cu int32 [B + 1] holds the sequences' borders.

  turn    token at position p, pair i: the angle p * freq[i], the pair turned by
          it (backwards for gradients) and multiplied by an amplitude.  Pairs are
          (i, i + rot / 2), or (2 i, 2 i + 1) when interleaved; channels from rot
          on stay.
  attend  out_i = sum_j p_ij v_j, p_i = softmax_j(scale q_i . k_j) over the keys
          j <= i + nk - nq of the sequence (causal; all of them otherwise), of
          those the last `window` if it is not 0; a row without keys gives zeros,
          lse -inf.  lse_i = log sum_j exp(scale q_i . k_j).
  learn   the gradients of q, k and v, from dout, out and lse.
  map     token t of sequence b: its row b, slot lens[b] + t - cu[b] and position
          first[b] + t - cu[b]; -1 behind the last token.
  pages   sequence b needs ceil(want / page) pages.  Those it lacks come off the
          head of a ring of free pages, sequence after sequence, as long as they
          last; those past its need go to the ring's tail, entries become -1.
"""
from __future__ import annotations

import math

import torch

own = False

TURN, ATTEND, LEARN, MAP, PAGES = "turn", "attend", "learn", "map", "pages"
PLAIN, LINEAR, BASE, RAMP = "plain", "linear", "base", "ramp"  # ways of scaling frequencies


# ------------------------------------------------------------------ cases
def listed():
    return [
        # A decoding step of one sequence: q and k of its token (launch latency).
        dict(name="turn 1 token", op=TURN, T=1, q_heads=32, heads=8, D=128, rot=128, interleaved=False, inverse=False,
             scaling=PLAIN, far=5000),
        # Long prompts of a model whose context was extended: far positions.
        dict(name="turn 32768 tokens, far", op=TURN, T=32768, q_heads=32, heads=8, D=128, rot=128, interleaved=False,
             inverse=False, scaling=RAMP, far=131072),
        # One short question (latency).
        dict(name="attend 77 tokens", op=ATTEND, B=1, len_min=77, len_max=77, extra=0, q_heads=32, heads=8, D=128,
             causal=True, window=0, lse=False),
        # A batch of ragged prompts, with what training needs of it.
        dict(name="attend 16 prompts", op=ATTEND, B=16, len_min=3, len_max=4001, extra=0, q_heads=32, heads=8, D=128,
             causal=True, window=0, lse=True),
        # One long document.
        dict(name="attend 16384 tokens", op=ATTEND, B=1, len_min=16384, len_max=16384, extra=0, q_heads=32, heads=8,
             D=128, causal=True, window=0, lse=False),
        # A chunk of a long prompt behind what came before it: few rows, a long axis, wide heads.
        dict(name="attend chunk 500 of 15500", op=ATTEND, B=1, len_min=500, len_max=500, extra=15000, q_heads=16,
             heads=4, D=256, causal=True, window=0, lse=False),
        # A training step on sequences of one length.
        dict(name="learn 4 x 2048", op=LEARN, B=4, len_min=2048, len_max=2048, extra=0, q_heads=32, heads=8, D=128,
             causal=True, window=0),
        # A training step on packed texts: narrow heads in groups of five, a sliding window.
        dict(name="learn 12 texts, window", op=LEARN, B=12, len_min=60, len_max=3001, extra=0, q_heads=40, heads=8,
             D=64, causal=True, window=1000),
        # A decoding step: one token for each of a batch.
        dict(name="map 48 tokens", op=MAP, B=48, new_min=1, new_max=1, held=1000, pad=0),
        # Prompts of a serving batch, the arrays padded to a fixed size for a graph.
        dict(name="map 64 prompts", op=MAP, B=64, new_min=0, new_max=2049, held=0, pad=4000),
        # A decoding step: some sequences cross into a new page.
        dict(name="pages of 48 sequences", op=PAGES, B=48, len_min=100, len_max=1000, new_max=1, ended=0.0, page=64,
             max_pages=16),
        # A batch turns over: some requests have ended, long prompts enter, the pool runs short.
        dict(name="pages of 256 sequences", op=PAGES, B=256, len_min=0, len_max=4000, new_max=2000, ended=0.4, page=16,
             max_pages=512),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice([TURN, ATTEND, ATTEND, LEARN, LEARN, MAP, PAGES])
    if op == MAP:
        top = _spread(rng, 1, 2049)
        return dict(op=op, B=_spread(rng, 1, 300 if top < 400 else 60), new_min=rng.randint(0, top), new_max=top,
                    held=rng.randint(0, 5000), pad=rng.choice([0, _spread(rng, 1, 4000)]))
    if op == PAGES:
        page = rng.choice([16, 32, 64, 128])
        top = _spread(rng, 1, 4000)
        return dict(op=op, B=_spread(rng, 1, 256), len_min=rng.randint(0, top), len_max=top,
                    new_max=_spread(rng, 1, 2000), ended=rng.choice([0.0, 0.3, 0.6]), page=page,
                    max_pages=rng.randint(1, 8192 // page))
    D = rng.choice([64, 128, 128, 256])
    heads = rng.choice([1, 2, 4, 5, 8])
    q_heads = heads * rng.choice([1, 2, 4, 5, 7, 8])
    if op == TURN:
        most = max(2, 32768 * 40 * 128 // ((q_heads + heads) * D))
        return dict(op=op, T=_spread(rng, 1, min(32768, most)), q_heads=q_heads, heads=heads, D=D,
                    rot=rng.choice([D, D, D // 2, D // 4]), interleaved=rng.random() < 0.4,
                    inverse=rng.random() < 0.4, scaling=rng.choice([PLAIN, LINEAR, BASE, RAMP]),
                    far=_spread(rng, 100, 1 << 20))
    # Visible pairs, query heads and channels together stay below those of the listed cases.
    B = _spread(rng, 1, 24)
    most = 1.5e10 / (1 if op == ATTEND else 4) / (B * q_heads * D)
    top = _spread(rng, 1, max(16, min(8192, int(math.sqrt(most)))))
    low = rng.randint(1, top)
    causal = rng.random() < 0.8
    return dict(op=op, B=B, len_min=low, len_max=top, extra=rng.choice([0, 0, 0, _spread(rng, 1, top), -(low // 2)]),
                q_heads=q_heads, heads=heads, D=D, causal=causal,
                window=_spread(rng, 1, top) if causal and rng.random() < 0.4 else 0,
                **({"lse": rng.random() < 0.5} if op == ATTEND else {}))


def _even(lo, hi, n):
    """n whole numbers spread evenly from lo to hi (hi alone for n == 1)."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lens(case):
    """Queries and keys of every sequence, the longest neither first nor last."""
    lens = _even(case["len_min"], case["len_max"], case["B"])
    lens = lens[0::2] + lens[1::2][::-1]
    return lens, [max(0, n + case["extra"]) for n in lens]


# ------------------------------------------------------------------ inputs
def _borders(lens):
    return torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()


SCALES = {PLAIN: (1.0, 0), LINEAR: (4.0, 0), BASE: (8.0, 0), RAMP: (16.0, 8192)}  # factor, length before


def _frequencies(rot, scaling, base=10000.0, fast=32.0, slow=1.0):
    """Radians per position of every pair, float64, and the amplitude.  linear:
    all divided by the factor; base: the base raised so that the slowest pair is;
    ramp: pairs that turn more than `fast` times within the length before stay,
    those below `slow` times are divided, linearly in the pair in between."""
    factor, before = SCALES[scaling]
    pair = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == BASE:
        base *= factor ** (rot / (rot - 2))
    freq = base ** (-2.0 * pair / rot)
    if scaling == LINEAR:
        freq = freq / factor
    if scaling != RAMP:
        return freq, 1.0
    lo, hi = (rot * math.log(before / (2.0 * math.pi * turns)) / (2.0 * math.log(base)) for turns in (fast, slow))
    lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
    part = ((pair - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
    return freq * (1.0 - part) + freq / factor * part, 0.1 * math.log(factor) + 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=dict(case))
    return {TURN: _prepare_turn, ATTEND: _prepare_attend, LEARN: _prepare_attend, MAP: _prepare_map,
            PAGES: _prepare_pages}[case["op"]](s, case, gen)


def _rows(s, case, gen, Tq, Tk):
    """q, k and v as slices of a projection's output; keys with an outlier channel, as such models have."""
    q_heads, heads, D = case["q_heads"], case["heads"], case["D"]
    if Tq == Tk:
        qkv = torch.randn((Tq, q_heads + 2 * heads, D), generator=gen, device="cuda", dtype=torch.float16)
        s["q"], s["k"], s["v"] = qkv.split([q_heads, heads, heads], 1)
    else:
        s["q"] = torch.randn((Tq, q_heads, D), generator=gen, device="cuda", dtype=torch.float16)
        kv = torch.randn((Tk, 2 * heads, D), generator=gen, device="cuda", dtype=torch.float16)
        s["k"], s["v"] = kv.split([heads, heads], 1)
    s["k"][..., 5] += 4.0


def _prepare_turn(s, case, gen):
    _rows(s, case, gen, case["T"], case["T"])
    s["freq"], s["amplitude"] = _frequencies(case["rot"], case["scaling"])
    s["freq"] = s["freq"].cuda()
    # Prompts one after another: positions run on, and begin somewhere.
    at = torch.arange(case["T"], device="cuda") + torch.randint(0, case["far"], (1,), generator=gen, device="cuda")
    s["position"] = (at % case["far"]).to(torch.int32)
    if own:
        # The program has its frequencies from the framework.
        from outlier_aware_bit_amd import qlin
        factor, before = SCALES[case["scaling"]]
        s["freq"], s["amplitude"] = qlin.qlin_rope_freqs(case["rot"], scaling=case["scaling"], factor=factor,
                                                         original_len=before)
    return s


def _prepare_attend(s, case, gen):
    nq, nk = _lens(case)
    s["cu_q"], s["cu_k"] = _borders(nq), _borders(nk)
    s["lens"] = list(zip(nq, nk))  # the host knows them, as it made up the batch
    _rows(s, case, gen, sum(nq), sum(nk))
    s["scale"] = case["D"] ** -0.5
    if case["op"] == LEARN:
        out, lse = _attention(s)
        s["out"], s["lse"] = out.half(), lse
        s["dout"] = torch.randn(s["q"].shape, generator=gen, device="cuda", dtype=torch.float16) * 0.02
    return s


def _prepare_map(s, case, gen):
    B = case["B"]
    add = torch.tensor(_even(case["new_min"], case["new_max"], B), dtype=torch.int32, device="cuda")
    s["add"] = add[torch.randperm(B, generator=gen, device="cuda")].contiguous()
    s["lens"] = torch.randint(0, case["held"] + 1, (B,), generator=gen, device="cuda").to(torch.int32)
    # Evictions have left fewer slots than positions in some sequences.
    s["first"] = s["lens"] + torch.randint(0, 500, (B,), generator=gen, device="cuda").to(torch.int32)
    s["T"] = sum(_even(case["new_min"], case["new_max"], B)) + case["pad"]
    return s


def _prepare_pages(s, case, gen):
    B, page, most = case["B"], case["page"], case["max_pages"]
    lens = torch.randint(case["len_min"], case["len_max"] + 1, (B,), generator=gen, device="cuda")
    lens = lens.clamp(max=most * page)
    held = (lens + page - 1) // page
    new = torch.randint(0, case["new_max"] + 1, (B,), generator=gen, device="cuda")
    ended = torch.rand((B,), generator=gen, device="cuda") < case["ended"]
    s["want"] = torch.where(ended, 0, lens + new).to(torch.int32)
    total = int(held.sum())
    pages = B * (1 + min(most, -(-case["len_max"] // page))) + 1
    free = min(pages - total, (total + B) // 4 + 1)  # other tables hold the rest
    ids = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    at = torch.arange(most, device="cuda")
    mine = at < held[:, None]
    s["table"] = torch.where(mine, ids[((held.cumsum(0) - held)[:, None] + at).clamp(max=pages - 1)], -1)
    s["table"] = s["table"].to(torch.int32).contiguous()
    s["held"] = held.to(torch.int32)
    # The ring of free pages begins anywhere.
    head = int(torch.randint(0, pages, (1,), generator=gen, device="cuda"))
    s["ring"] = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    s["ring"][(torch.arange(free, device="cuda") + head) % pages] = ids[total:total + free]
    s["state"] = torch.tensor([head, free], dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return {TURN: _own_turn, ATTEND: _own_attend, LEARN: _own_learn, MAP: _own_map, PAGES: _own_pages}[op](s)
    return {TURN: _plain_turn, ATTEND: _plain_attend, LEARN: _plain_learn, MAP: _plain_map, PAGES: _plain_pages}[op](s)


def _own_turn(s):
    from outlier_aware_bit_amd import qlin
    q, k = qlin.qlin_rope(s["q"], s["k"], s["position"], s["freq"], interleaved=s["case"]["interleaved"],
                          inverse=s["case"]["inverse"], amplitude=s["amplitude"])
    return {"q": q, "k": k}


def _own_attend(s):
    from outlier_aware_bit_amd import qlin
    case = s["case"]
    out, lse = qlin.qlin_attn_prompt(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], scale=s["scale"],
                                     causal=case["causal"], window=case["window"], want_lse=case["lse"])
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def _own_learn(s):
    from outlier_aware_bit_amd import qlin
    case = s["case"]
    dq, dk, dv = qlin.qlin_attn_prompt_backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["cu_q"],
                                                s["cu_k"], scale=s["scale"], causal=case["causal"],
                                                window=case["window"])
    return {"dq": dq, "dk": dk, "dv": dv}


def _own_map(s):
    from outlier_aware_bit_amd import qlin
    cu, row, slot, position, lens = qlin.qlin_kv_slots(s["lens"], s["add"], s["T"], first=s["first"])
    return {"cu": cu, "row": row, "slot": slot, "position": position, "lens": lens}


def _own_pages(s):
    from outlier_aware_bit_amd import qlin
    out = {n + "_out": torch.empty_like(s[n]) for n in ("table", "held", "state")}
    table, held, state, missing = qlin.qlin_kv_pages(s["want"], s["case"]["page"], s["table"], s["held"], s["ring"],
                                                     s["state"], **out)
    return {"table": table, "held": held, "ring": s["ring"], "state": state, "missing": missing}


def _plain_turn(s):
    case = s["case"]
    rot, sign = case["rot"], -1.0 if case["inverse"] else 1.0
    angle = s["position"].double()[:, None] * s["freq"]
    c = (torch.cos(angle) * s["amplitude"]).float()[:, None]
    n = (torch.sin(angle) * (s["amplitude"] * sign)).float()[:, None]
    got = {}
    for name in ("q", "k"):
        x = s[name].float()
        t = x[..., :rot]
        if case["interleaved"]:
            a, b = t[..., 0::2], t[..., 1::2]
            t = torch.stack([a * c - b * n, a * n + b * c], -1).flatten(-2)
        else:
            a, b = t[..., :rot // 2], t[..., rot // 2:]
            t = torch.cat([a * c - b * n, a * n + b * c], -1)
        got[name] = torch.cat([t, x[..., rot:]], -1).half()
    return got


ROWS = 2048  # queries at a time: their scores are held in full


def _chunks(s):
    """(first query, one past, first key, one past, mask or None) of up to ROWS
    queries of one sequence and the keys that any of them can see."""
    case, at_q, at_k = s["case"], 0, 0
    for nq, nk in s["lens"]:
        for i in range(0, nq, ROWS):
            j = min(nq, i + ROWS)
            low, high, seen = 0, nk, None
            if case["causal"]:
                high = min(nk, max(0, j + nk - nq))
                low = min(high, max(0, i + nk - nq + 1 - case["window"])) if case["window"] else 0
                last = torch.arange(i + nk - nq, j + nk - nq, device="cuda")[:, None]
                key = torch.arange(low, high, device="cuda")
                seen = key <= last
                if case["window"]:
                    seen &= key > last - case["window"]
            yield at_q + i, at_q + j, at_k + low, at_k + high, seen
        at_q, at_k = at_q + nq, at_k + nk


def _grouped(x, heads):
    """fp32 rows [T, heads * group, D] by kv head: [heads, group * T, D]."""
    T, n, D = x.shape
    return x.float().reshape(T, heads, n // heads, D).permute(1, 2, 0, 3).reshape(heads, -1, D)


def _ungrouped(x, T):
    heads, n, D = x.shape
    return x.reshape(heads, n // T, T, D).permute(2, 0, 1, 3).reshape(T, -1, D)


def _scores(s, i, j, low, high, seen):
    """scale q . k of a chunk, -inf where not seen: [heads, group * queries, keys]."""
    heads = s["case"]["heads"]
    t = torch.bmm(_grouped(s["q"][i:j], heads), _grouped(s["k"][low:high], heads).transpose(1, 2).contiguous())
    t *= s["scale"]
    if seen is not None:
        t.view(heads, -1, j - i, high - low).masked_fill_(~seen, -math.inf)
    return t


def _attention(s):
    """out and lse in fp32."""
    heads = s["case"]["heads"]
    out = torch.zeros(s["q"].shape, device="cuda")
    lse = torch.full((s["q"].shape[1], s["q"].shape[0]), -math.inf, device="cuda")
    for i, j, low, high, seen in _chunks(s):
        if high == low:
            continue
        t = _scores(s, i, j, low, high, seen)
        top = t.amax(-1, keepdim=True)
        t = t.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
        total = t.sum(-1, keepdim=True)
        o = torch.bmm(t, _grouped(s["v"][low:high], heads)) / torch.where(total == 0.0, 1.0, total)
        out[i:j] = _ungrouped(o, j - i)
        lse[:, i:j] = (top + total.log()).reshape(-1, j - i)
    return out, lse


def _plain_attend(s):
    out, lse = _attention(s)
    return {"out": out.half(), "lse": lse} if s["case"]["lse"] else {"out": out.half()}


def _plain_learn(s):
    heads = s["case"]["heads"]
    dq = torch.zeros(s["q"].shape, device="cuda")
    dk, dv = (torch.zeros(s["k"].shape, device="cuda") for _ in range(2))
    delta = (s["dout"].float() * s["out"].float()).sum(-1).t()  # [query heads, T]
    for i, j, low, high, seen in _chunks(s):
        if high == low:
            continue
        lse = s["lse"][:, i:j].reshape(heads, -1, 1)
        p = _scores(s, i, j, low, high, seen).sub_(torch.where(lse == -math.inf, 0.0, lse)).exp_()
        do = _grouped(s["dout"][i:j], heads)
        dv[low:high] += _ungrouped(torch.bmm(p.transpose(1, 2).contiguous(), do), high - low)
        ds = torch.bmm(do, _grouped(s["v"][low:high], heads).transpose(1, 2).contiguous())
        ds = ds.sub_(delta[:, i:j].reshape(heads, -1, 1)).mul_(p).mul_(s["scale"])
        dq[i:j] = _ungrouped(torch.bmm(ds, _grouped(s["k"][low:high], heads)), j - i)
        dk[low:high] += _ungrouped(torch.bmm(ds.transpose(1, 2).contiguous(), _grouped(s["q"][i:j], heads)), high - low)
    return {"dq": dq.half(), "dk": dk.half(), "dv": dv.half()}


def _plain_map(s):
    T, end = s["T"], s["add"].cumsum(0)
    cu = torch.cat([end.new_zeros(1), end])
    at = torch.arange(T, device="cuda")
    b = (at[:, None] >= end).sum(1)  # sequences that end before token t
    here = b < s["case"]["B"]
    b = b.clamp(max=s["case"]["B"] - 1)
    off = at - cu[b]
    return {"cu": cu.to(torch.int32), "row": torch.where(here, b, -1).to(torch.int32),
            "slot": torch.where(here, s["lens"][b] + off, -1).to(torch.int32),
            "position": torch.where(here, s["first"][b] + off, -1).to(torch.int32), "lens": s["lens"] + s["add"]}


def _plain_pages(s):
    page, most, size = s["case"]["page"], s["case"]["max_pages"], s["ring"].numel()
    head, count = s["state"][0].long(), s["state"][1].long()
    held = s["held"].long()
    need = (s["want"].long().clamp(min=0) + page - 1) // page
    fits = need <= most
    grow = torch.where(fits, need - held, 0).clamp(min=0)
    served = fits & ((grow == 0) | (grow.cumsum(0) <= count))
    left = torch.where(served, need, held)
    missing = torch.where(served, 0, need - held).sum()
    at = torch.arange(most, device="cuda")
    taken = (at >= held[:, None]) & (at < left[:, None])
    given = (at < held[:, None]) & (at >= left[:, None])
    rank = taken.flatten().cumsum(0).reshape(taken.shape) - 1
    table = torch.where(taken, s["ring"][(head + rank) % size], s["table"])
    table = torch.where(given, -1, table)
    rank = given.flatten().cumsum(0).reshape(given.shape) - 1
    s["ring"][(head + count + rank[given]) % size] = s["table"][given]
    out, back = taken.sum(), given.sum()
    state = torch.stack([(head + out) % size, count - out + back])
    return {"table": table, "held": left.to(torch.int32), "ring": s["ring"], "state": state.to(torch.int32),
            "missing": missing.to(torch.int32).reshape(1)}


# ------------------------------------------------------------------ what a pass cannot do without
def _pairs(case):
    """Visible (query, key) pairs of all sequences."""
    n = 0
    for nq, nk in zip(*_lens(case)):
        if not case["causal"]:
            n += nq * nk
            continue
        first, last = nk - nq + 1, nk  # keys up to the first and the last query's own
        up = lambda x: max(0, x) * (max(0, x) + 1) // 2  # noqa: E731
        n += up(last) - up(first - 1)
        if case["window"]:
            w = case["window"]
            n -= up(last - w) - up(first - 1 - w)
    return n


def work(case):
    op = case["op"]
    if op == MAP:
        total = sum(_even(case["new_min"], case["new_max"], case["B"]))
        return {"bytes": 12 * (total + case["pad"]) + 20 * case["B"], "flops": total}
    if op == PAGES:
        # Every entry of the table is written; held, want, one move of a page for each that changes hands.
        moved = case["B"] * ((1 - case["ended"]) * case["new_max"] / 2
                             + case["ended"] * (case["len_min"] + case["len_max"]) / 2) / case["page"]
        return {"bytes": int(4 * case["B"] * (2 * case["max_pages"] + 3) + 8 * moved), "flops": case["B"]}
    q_heads, heads, D = case["q_heads"], case["heads"], case["D"]
    if op == TURN:
        T = case["T"]
        return {"bytes": 4 * T * (q_heads + heads) * D + 4 * T + 4 * case["rot"],
                "flops": 3 * T * (q_heads + heads) * case["rot"]}
    nq, nk = (sum(n) for n in _lens(case))
    pairs = _pairs(case) * q_heads * D
    if op == ATTEND:
        return {"bytes": 4 * D * (nq * q_heads + nk * heads) + (4 * nq * q_heads if case["lse"] else 0),
                "flops": 4 * pairs}
    return {"bytes": 8 * D * (nq * q_heads + nk * heads) + 4 * nq * q_heads, "flops": 10 * pairs}


# ------------------------------------------------------------------ the definition, in 64 bits
def _exact_turn(s):
    case, rot = s["case"], s["case"]["rot"]
    freq, amplitude = _frequencies(rot, case["scaling"])
    unit = torch.polar(torch.full((1,), amplitude, dtype=torch.float64, device="cuda"),
                       s["position"].double()[:, None] * freq.cuda())
    unit = (unit.conj() if case["inverse"] else unit)[:, None]
    got = {}
    for name in ("q", "k"):
        x = s[name].double()
        pairs = x[..., :rot].unflatten(-1, (-1, 2)) if case["interleaved"] else x[..., :rot].unflatten(-1, (2, -1)).mT
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit)
        x[..., :rot] = (z if case["interleaved"] else z.mT).flatten(-2)
        got[name] = x
    return got


def _exact_head(q, k, v, case, scale):
    """One head's attention in float64: [nq, D] by [nk, D]; (out, lse)."""
    nq, nk = q.shape[0], k.shape[0]
    logits = q @ k.t() * scale
    if case["causal"]:
        ago = torch.arange(nq, device="cuda")[:, None] + (nk - nq) - torch.arange(nk, device="cuda")
        hidden = ago < 0
        if case["window"]:
            hidden |= ago >= case["window"]
        logits = logits.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(logits, 1)
    p = torch.exp(logits - torch.where(lse == -math.inf, 0.0, lse)[:, None])
    return p @ v, lse


def _exact_attend(s):
    case, group = s["case"], s["case"]["q_heads"] // s["case"]["heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((case["q_heads"], out.shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    at_q = at_k = 0
    for nq, nk in s["lens"]:
        i, j = slice(at_q, at_q + nq), slice(at_k, at_k + nk)
        for h in range(case["q_heads"] if nk else 0):
            out[i, h], lse[h, i] = _exact_head(s["q"][i, h].double(), s["k"][j, h // group].double(),
                                               s["v"][j, h // group].double(), case, s["scale"])
        at_q, at_k = at_q + nq, at_k + nk
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def _exact_learn(s):
    """The definition's gradients by differentiation of _exact_head."""
    case, group = s["case"], s["case"]["q_heads"] // s["case"]["heads"]
    dq = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    dk, dv = (torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
    at_q = at_k = 0
    for nq, nk in s["lens"]:
        i, j = slice(at_q, at_q + nq), slice(at_k, at_k + nk)
        i = slice(max(at_q, at_q + nq - nk), at_q + nq) if case["causal"] else i  # rows before see no key
        for h in range(case["q_heads"] if nk else 0):
            g = h // group
            leaves = [t.double().requires_grad_() for t in (s["q"][i, h], s["k"][j, g], s["v"][j, g])]
            with torch.enable_grad():
                o, _ = _exact_head(*leaves, case, s["scale"])
            grads = torch.autograd.grad(o, leaves, s["dout"][i, h].double())
            dq[i, h] = grads[0]
            dk[j, g] += grads[1]
            dv[j, g] += grads[2]
        at_q, at_k = at_q + nq, at_k + nk
    return {"dq": dq, "dk": dk, "dv": dv}


def exact(case, seed):
    if case["op"] in (MAP, PAGES):
        return None  # whole numbers
    s = prepare(case, seed)
    return {TURN: _exact_turn, ATTEND: _exact_attend, LEARN: _exact_learn}[case["op"]](s)
