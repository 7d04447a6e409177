"""The paged key/value cache of a decoding model, as it is measured: appending
rows, attention of one new token, and eviction by accumulated attention weight.

The cache is a pool of pages.  Page p holds `page` slots of every kv head:
  k, v          fp16 [pages, heads, page, D], or uint8 codes
                [pages, heads, page, D * bits / 8] (int4: low nibble = even d)
  kmeta, vmeta  fp16 [pages, heads, page, 2]: (step, lo) of every row of codes;
                the row stands for lo + step * code
  table         int32 [B, max_pages]: slot i of sequence b is line i % page of
                page table[b, i // page]; unused entries are -1
  mass, pos     fp32 / int32 [B, heads, ld]: accumulated attention weight and
                token position of every slot
With `signs` (D = 128) the stored K rows are (k * d) H_128, H the natural-order
Sylvester matrix, evaluated as a butterfly of spans 1, 2, .., 64 in fp32.

Codes decide on whole numbers, so their rule is stated to the operation: in
IEEE fp32, one rounding each, t the fp32 row, qmax = 2^bits - 1,
  lo = fp16(min t), step = fp16(fp32(max t - lo) / qmax), inv = 1 / step
  (0 if step == 0), code = clamp(rint(fp32((t - lo)) * inv), 0, qmax).
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

APPEND, ATTEND, EVICT = "append", "attend", "evict"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # Decoding one sequence: its token's rows enter an fp16 cache (launch latency).
        dict(name="append 1 token, fp16", op=APPEND, B=1, first=700, new_min=1, new_max=1, heads=8, D=128, page=16,
             bits=16, rotate=False, track=False),
        # Decoding a batch: one token each, tracked for eviction.
        dict(name="append 48 tokens, int8", op=APPEND, B=48, first=1000, new_min=1, new_max=1, heads=8, D=64, page=64,
             bits=8, rotate=False, track=True),
        # A batch of prompts into the 4-bit cache, K through the Hadamard.
        dict(name="append 8 prompts, int4", op=APPEND, B=8, first=0, new_min=500, new_max=4096, heads=8, D=128,
             page=64, bits=4, rotate=True, track=True),
        # Prompts of a model with wide heads.
        dict(name="append 16 prompts, int8 D=256", op=APPEND, B=16, first=0, new_min=300, new_max=2049, heads=4, D=256,
             page=128, bits=8, rotate=False, track=False),
        # A short chat turn, every query head with its own kv head.
        dict(name="attend 100 slots, fp16", op=ATTEND, B=1, len_min=100, len_max=100, empty=0, q_heads=32, heads=32,
             D=128, page=16, bits=16, rotate=False, window=0, track=False),
        # One long document: the cache's length is the only thing to split.
        dict(name="attend 65537 slots, int4", op=ATTEND, B=1, len_min=65537, len_max=65537, empty=0, q_heads=32,
             heads=8, D=128, page=64, bits=4, rotate=True, window=0, track=False),
        # A ragged batch with an idle row, narrow heads in groups of five, a sliding window, tracked.
        dict(name="attend ragged 16, int8 D=64", op=ATTEND, B=16, len_min=1, len_max=3001, empty=1, q_heads=40,
             heads=8, D=64, page=32, bits=8, rotate=False, window=1024, track=True),
        # A batch without grouped heads on an fp16 cache.
        dict(name="attend batch 32, fp16", op=ATTEND, B=32, len_min=500, len_max=4000, empty=0, q_heads=32, heads=32,
             D=128, page=16, bits=16, rotate=False, window=0, track=False),
        # A full serving batch on the 4-bit cache, tracked for eviction.
        dict(name="attend batch 64, int4", op=ATTEND, B=64, len_min=1500, len_max=12000, empty=0, q_heads=32, heads=8,
             D=128, page=64, bits=4, rotate=True, window=0, track=True),
        # The step after a full cache took one token: one slot of each head goes.
        dict(name="evict 1 of 1025, int4", op=EVICT, B=16, len_min=1025, len_max=1025, budget=1024, recent=256,
             heads=8, D=128, page=16, bits=4, scrambled=True),
        # After long prompts: most slots go.
        dict(name="evict 16k to 2k, fp16", op=EVICT, B=4, len_min=9001, len_max=16384, budget=2048, recent=512,
             heads=8, D=128, page=64, bits=16, scrambled=False),
        # A large batch back under its budget, some rows within it already.
        dict(name="evict batch 32, int8", op=EVICT, B=32, len_min=3000, len_max=9000, budget=4096, recent=1000,
             heads=8, D=128, page=64, bits=8, scrambled=False),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice([APPEND, ATTEND, EVICT])
    bits = rng.choice([16, 8, 4])
    D = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    heads = rng.choice([1, 2, 4, 5, 8])
    rotate = bits < 16 and D == 128 and rng.random() < 0.5
    if op == APPEND:
        decode = rng.random() < 0.5
        B = _spread(rng, 1, 64 if decode else 8)
        top = 1 if decode else _spread(rng, 2, 2048)
        return dict(op=op, B=B, first=_spread(rng, 1, 2000) if decode else 0, new_min=1 if decode else (top + 1) // 2,
                    new_max=top, heads=heads, D=D, page=page, bits=bits, rotate=rotate, track=rng.random() < 0.5)
    if op == ATTEND:
        group = rng.choice([1, 2, 4, 5, 7, 8, 16, 20])
        B = _spread(rng, 1, 48)
        top = _spread(rng, 1, max(64, 131072 // B // heads))
        return dict(op=op, B=B, len_min=(top + 2) // 3, len_max=top, empty=int(B > 2 and rng.random() < 0.3),
                    q_heads=heads * group, heads=heads, D=D, page=page, bits=bits, rotate=rotate,
                    window=_spread(rng, 1, top) if rng.random() < 0.3 else 0, track=rng.random() < 0.5)
    B = _spread(rng, 1, 32)
    top = _spread(rng, 16, max(64, 131072 // B // heads))
    budget = _spread(rng, 1, top)
    return dict(op=op, B=B, len_min=max(1, top // 2), len_max=top, budget=budget, recent=rng.randint(0, budget),
                heads=heads, D=D, page=page, bits=bits, scrambled=rng.random() < 0.5)


def _even(lo, hi, n):
    """n whole numbers spread evenly from lo to hi (hi alone for n == 1)."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lens(case):
    if case["op"] == APPEND:
        return _even(case["new_min"], case["new_max"], case["B"])
    lens = _even(case["len_min"], case["len_max"], case["B"])
    e = case.get("empty", 0)
    return [0] * e + lens[e:]


# ------------------------------------------------------------------ inputs
def _quantize(t, bits):
    """Codes (uint8, one each) and (step, lo) fp16 of fp32 rows."""
    qmax = float(2 ** bits - 1)
    lo = t.amin(-1, keepdim=True).half()
    step = ((t.amax(-1, keepdim=True) - lo.float()) / qmax).half()
    inv = torch.where(step == 0, torch.zeros_like(step, dtype=torch.float32), 1.0 / step.float())
    codes = torch.round((t - lo.float()) * inv).clamp(0.0, qmax).to(torch.uint8)
    return codes, torch.cat([step, lo], -1)


def _rotate(x, signs):
    """(x * signs) H_128 of fp32 rows: a butterfly of spans 1, 2, .., 64."""
    u = x * signs.float()
    shape = u.shape
    h = 1
    while h < 128:
        w = u.reshape(*shape[:-1], 128 // (2 * h), 2, h)
        u = torch.stack([w[..., 0, :] + w[..., 1, :], w[..., 0, :] - w[..., 1, :]], -2).reshape(shape)
        h *= 2
    return u


def _encode(x, bits, signs=None):
    """fp16 rows as they are stored: (rows or packed codes, meta or None)."""
    if bits == 16:
        return x, None
    codes, meta = _quantize(x.float() if signs is None else _rotate(x.float(), signs), bits)
    if bits == 4:
        codes = codes[..., 0::2] | (codes[..., 1::2] << 4)
    return codes, meta


def _decode(rows, meta, bits):
    """The fp32 values of stored rows."""
    if bits == 16:
        return rows.float()
    if bits == 4:
        rows = torch.stack([rows & 15, rows >> 4], -1).flatten(-2)
    return meta[..., 1:].float() + meta[..., :1].float() * rows.float()


def _rows(gen, shape, outliers):
    """fp16 rows N(0, 1); with `outliers`, three channels hold a large constant
    offset, as the keys of such models do."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16)
    if outliers:
        x[..., 5::max(8, shape[-1] // 3)] += 6.0
    return x


def _pool(state, case, gen, pages, filled):
    """The pool's tensors: drawn rows in every slot, or zeros."""
    shape = (pages, case["heads"], case["page"], case["D"])
    bits = case["bits"]
    width = case["D"] if bits == 16 else case["D"] * bits // 8
    dtype = torch.float16 if bits == 16 else torch.uint8
    for n in ("k", "v"):
        state[n] = torch.zeros(shape[:3] + (width,), dtype=dtype, device="cuda")
        state[n + "meta"] = None if bits == 16 else torch.zeros(shape[:3] + (2,), dtype=torch.float16, device="cuda")
        some = max(1, (1 << 26) // (shape[1] * shape[2] * shape[3]))
        for at in range(0, pages if filled else 0, some):
            x = _rows(gen, (min(some, pages - at),) + shape[1:], n == "k")
            rows, meta = _encode(x, bits, state["signs"] if n == "k" else None)
            state[n][at:at + some] = rows
            if meta is not None:
                state[n + "meta"][at:at + some] = meta


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, page, heads, D = case["B"], case["page"], case["heads"], case["D"]
    order = torch.randperm(B, generator=gen, device="cuda")
    lens = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")[order]
    s = dict(case=dict(case), signs=None)
    if case.get("rotate"):
        s["signs"] = (torch.randint(0, 2, (128,), generator=gen, device="cuda") * 2 - 1).to(torch.int8)
        s["signs"][0] = 1
    first = case.get("first", 0)
    need = (lens + first + page - 1) // page
    max_pages = max(1, int(need.max()))
    pages = int(need.sum()) + 3
    ids = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    at = torch.arange(max_pages, device="cuda")
    s["table"] = torch.where(at < need[:, None], ids[((need.cumsum(0) - need)[:, None] + at).clamp(max=pages - 1)], -1)
    s["table"] = s["table"].to(torch.int32).contiguous()
    _pool(s, case, gen, pages, case["op"] != APPEND)
    ld = max_pages * page
    if case["op"] == APPEND:
        T = int(lens.sum())
        # The new rows lie in the output of one projection, q | k | v, so that k and v are strided.
        qkv = _rows(gen, (T, 4, heads, D), True)
        s["k_new"], s["v_new"] = qkv[:, 2], qkv[:, 3]
        s["row"] = torch.repeat_interleave(torch.arange(B, device="cuda"), lens.long()).to(torch.int32)
        start = (lens.cumsum(0) - lens).long()
        s["slot"] = (first + torch.arange(T, device="cuda") - start[s["row"].long()]).to(torch.int32)
        s["position"] = s["slot"] + 7
        if case["track"]:
            s["mass"] = torch.rand((B, heads, ld), generator=gen, device="cuda")
            s["pos"] = torch.randint(0, 1 << 20, (B, heads, ld), generator=gen, device="cuda").to(torch.int32)
    else:
        s["lens"] = lens
        s["max_len"] = max(1, max(_lens(case)))
        if case["op"] == ATTEND:
            s["q"] = torch.randn((B, case["q_heads"], D), generator=gen, device="cuda", dtype=torch.float16)
            s["scale"] = D ** -0.5
            if case["track"]:
                s["mass"] = torch.rand((B, heads, ld), generator=gen, device="cuda") * 4
                s["mass_out"] = torch.zeros_like(s["mass"])
        else:
            # Accumulated weights are heavy-tailed, and slots that were hardly looked at tie at nothing.
            m = torch.exp(2.0 * torch.randn((B, heads, ld), generator=gen, device="cuda"))
            s["mass"] = torch.where(m < 0.3, torch.zeros_like(m), m)
            slot = torch.arange(ld, device="cuda")
            if case["scrambled"]:
                # Earlier evictions left the first `budget` slots in any order.
                front = min(case["budget"], ld)
                key = torch.rand((B, heads, ld), generator=gen, device="cuda")
                key[..., front:] = 2.0
                slot = torch.sort(key, stable=True).indices
            s["pos"] = (slot + 11).to(torch.int32).expand(B, heads, ld).contiguous()
            s["mass_out"], s["pos_out"] = torch.zeros_like(s["mass"]), torch.zeros_like(s["pos"])
            s["lens_out"] = torch.zeros_like(lens)
            s["kept"] = torch.full((B, heads, case["budget"]), -1, dtype=torch.int32, device="cuda")
    if own:
        # The handle that a program keeps beside its pool: the same tensors, checked once.
        from outlier_aware_bit_amd import qlin
        s["cache"] = qlin.KVCache(s["k"], s["v"], head_dim=D, bits=case["bits"], kmeta=s["kmeta"], vmeta=s["vmeta"],
                                  signs=s["signs"])
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if own:
        return {APPEND: _own_append, ATTEND: _own_attend, EVICT: _own_evict}[case["op"]](s)
    return {APPEND: _plain_append, ATTEND: _plain_attend, EVICT: _plain_evict}[case["op"]](s)


def _pool_out(s):
    return {n: s[n] for n in ("k", "v", "kmeta", "vmeta") if s[n] is not None}


def _own_append(s):
    from outlier_aware_bit_amd import qlin
    qlin.qlin_kv_append(s["cache"], s["k_new"], s["v_new"], s["table"], s["slot"], row=s["row"],
                        position=s["position"] if s["case"]["track"] else None, mass=s.get("mass"), pos=s.get("pos"))
    return {**_pool_out(s), **{n: s[n] for n in ("mass", "pos") if n in s}}


def _own_attend(s):
    from outlier_aware_bit_amd import qlin
    out, mass = qlin.qlin_attn_decode(s["cache"], s["q"], s["table"], s["lens"], s["max_len"], scale=s["scale"],
                                      window=s["case"]["window"], mass=s.get("mass"), mass_out=s.get("mass_out"))
    return {"out": out} if mass is None else {"out": out, "mass": mass}


def _own_evict(s):
    from outlier_aware_bit_amd import qlin
    qlin.qlin_kv_evict(s["cache"], s["table"], s["lens"], s["max_len"], s["case"]["budget"], s["case"]["recent"],
                       s["mass"], s["pos"], mass_out=s["mass_out"], pos_out=s["pos_out"], lens_out=s["lens_out"],
                       kept=s["kept"])
    return _evict_out(s)


def _evict_out(s):
    return {**_pool_out(s), **{n: s[n] for n in ("mass_out", "pos_out", "lens_out", "kept")}}


def _plain_append(s):
    case, row, slot = s["case"], s["row"].long(), s["slot"].long()
    page = s["table"][row, slot // case["page"]].long()
    line = slot % case["page"]
    for n in ("k", "v"):
        rows, meta = _encode(s[n + "_new"], case["bits"], s["signs"] if n == "k" else None)
        s[n][page, :, line] = rows
        if meta is not None:
            s[n + "meta"][page, :, line] = meta
    if case["track"]:
        s["mass"][row, :, slot] = 0.0
        s["pos"][row, :, slot] = s["position"][:, None].expand(-1, case["heads"])
    return {**_pool_out(s), **{n: s[n] for n in ("mass", "pos") if n in s}}


def _gathered(s, n, length):
    """The fp32 rows of slots 0..length-1 of every sequence: [B, heads, length, D]."""
    case = s["case"]
    count = -(-length // case["page"])
    ids = s["table"][:, :count].long().clamp(min=0)
    x = _decode(s[n][ids], None if s[n + "meta"] is None else s[n + "meta"][ids], case["bits"])
    return x.transpose(1, 2).reshape(case["B"], case["heads"], count * case["page"], case["D"])[:, :, :length]


def _plain_attend(s):
    case, n = s["case"], s["max_len"]
    B, heads, D = case["B"], case["heads"], case["D"]
    group = case["q_heads"] // heads
    q = s["q"].float()
    if s["signs"] is not None:
        q = _rotate(q, s["signs"]) / 128.0
    at = torch.arange(n, device="cuda")
    low = (s["lens"] - case["window"]).clamp(min=0) if case["window"] else torch.zeros_like(s["lens"])
    seen = ((at >= low[:, None]) & (at < s["lens"][:, None]))[:, None, :, None]
    qt = q.reshape(B * heads, group, D).transpose(1, 2).contiguous()
    scores = torch.bmm(_gathered(s, "k", n).reshape(B * heads, n, D), qt).reshape(B, heads, n, group) * s["scale"]
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(2, keepdim=True)
    e = torch.where(seen, torch.exp(scores - torch.where(seen.any(2, keepdim=True), top, 0.0)), 0.0)
    total = e.sum(2, keepdim=True)
    p = e / torch.where(total == 0.0, 1.0, total)
    v = torch.where(seen, _gathered(s, "v", n), 0.0)
    o = torch.bmm(p.transpose(2, 3).reshape(B * heads, group, n).contiguous(), v.reshape(B * heads, n, D))
    out = {"out": o.reshape(B, case["q_heads"], D).half()}
    if case["track"]:
        s["mass_out"][..., :n] = torch.where(seen[..., 0] | (at < s["lens"][:, None])[:, None],
                                             s["mass"][..., :n] + p.sum(3), s["mass_out"][..., :n])
        out["mass"] = s["mass_out"]
    return out


def _plain_evict(s):
    case, n = s["case"], s["max_len"]
    B, heads, budget = case["B"], case["heads"], case["budget"]
    at = torch.arange(n, device="cuda")
    here = (at < s["lens"][:, None])[:, None].expand(B, heads, n)
    left = s["lens"].clamp(max=budget)
    mass, pos = s["mass"][..., :n], s["pos"][..., :n].long()
    newest = torch.where(here, pos, -1).amax(2, keepdim=True)
    kept_anyway = here & (pos > newest - case["recent"])
    # Order of keeping: the newest, then by mass, then by slot; slots past the length last.
    by_mass = torch.sort(torch.where(here, mass, -math.inf), dim=2, descending=True, stable=True).indices
    again = torch.sort((~kept_anyway).to(torch.int32).gather(2, by_mass), dim=2, stable=True).indices
    rank = torch.empty_like(by_mass).scatter_(2, by_mass.gather(2, again), at.expand(B, heads, n))
    keep = here & (rank < left[:, None, None])
    # The j-th kept slot past the new length goes to the j-th freed slot before it.
    m = left[:, None, None].long()
    free, moved = ~keep & (at < m), keep & (at >= m)
    src = at.expand(B, heads, n).clone()
    # Both sides in ascending order within each (sequence, head), and equally many of each.
    b, h, to = free.nonzero(as_tuple=True)
    frm = moved.nonzero(as_tuple=True)[2]
    src[b, h, to] = frm
    page = case["page"]
    p_to, p_frm = s["table"][b, to // page].long(), s["table"][b, frm // page].long()
    for t in ("k", "v", "kmeta", "vmeta"):
        if s[t] is not None:
            s[t][p_to, h, to % page] = s[t][p_frm, h, frm % page]
    c = min(budget, n)
    fresh = (at[:c] < m).expand(B, heads, c)
    s["kept"][..., :c] = torch.where(fresh, src[..., :c], -1).to(torch.int32)
    for t in ("mass", "pos"):
        s[t + "_out"][..., :c] = torch.where(fresh, s[t].gather(2, src[..., :c]), s[t + "_out"][..., :c])
    s["lens_out"].copy_(left)
    return _evict_out(s)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    lens, heads, D, bits = _lens(case), case["heads"], case["D"], case["bits"]
    row = 2 * (D * bits // 8 + (0 if bits == 16 else 4))  # k and v of one slot and head, as stored
    if case["op"] == APPEND:
        T = sum(lens)
        flops = 2 * T * heads * D * (0 if bits == 16 else 4) + (T * heads * D * 8 if case["rotate"] else 0)
        return {"bytes": T * heads * (4 * D + row + (8 if case["track"] else 0)) + 16 * T, "flops": flops}
    if case["op"] == ATTEND:
        seen = sum(min(n, case["window"]) if case["window"] else n for n in lens)
        return {"bytes": seen * heads * row + (8 * heads * sum(lens) if case["track"] else 0)
                + 4 * case["B"] * case["q_heads"] * D,
                "flops": 4 * seen * case["q_heads"] * D}
    moved = kept = 0
    for n in lens:
        left = min(n, case["budget"])
        over, newest = n - left, min(case["recent"], left)
        late = min(over, newest)  # of the newest, those past the budget
        kept += left
        # The others are kept by mass, wherever they lie.
        moved += late + (left - newest) * (over - late) / max(1, n - newest)
    return {"bytes": int(heads * (8 * sum(lens) + 12 * kept + 2 * moved * row)), "flops": heads * sum(lens)}


# ------------------------------------------------------------------ the definition, in 64 bits
def _table_rows(s, name, b, n):
    """float64 rows of the first n slots of sequence b: [heads, n, D]."""
    case = s["case"]
    slot = torch.arange(n, device="cuda")
    ids = s["table"][b].long()[slot // case["page"]]
    raw = s[name][ids, :, slot % case["page"]].transpose(0, 1)
    if case["bits"] == 16:
        return raw.double()
    if case["bits"] == 4:
        full = torch.empty(raw.shape[:2] + (case["D"],), dtype=torch.float64, device="cuda")
        full[..., 0::2], full[..., 1::2] = (raw % 16).double(), torch.div(raw, 16, rounding_mode="floor").double()
        raw = full
    meta = s[name + "meta"][ids, :, slot % case["page"]].transpose(0, 1).double()
    return raw.double() * meta[..., 0, None] + meta[..., 1, None]


def _hadamard():
    i = np.arange(128)
    bits = np.array([bin(v).count("1") for v in range(128)])
    return 1.0 - 2.0 * (bits[i[:, None] & i[None, :]] % 2)


def _exact_attend(s):
    case = s["case"]
    group = case["q_heads"] // case["heads"]
    out = torch.zeros((case["B"], case["q_heads"], case["D"]), dtype=torch.float64, device="cuda")
    mass = s["mass_out"].double().clone() if case["track"] else None
    for b, n in enumerate(s["lens"].tolist()):
        low = max(0, n - case["window"]) if case["window"] else 0
        if n == 0:
            continue
        q = s["q"][b].double().reshape(case["heads"], group, case["D"])
        if s["signs"] is not None:
            q = (q * s["signs"].double()) @ torch.from_numpy(_hadamard()).cuda() / 128.0
        logits = (_table_rows(s, "k", b, n)[:, low:] @ q.transpose(1, 2).contiguous()) * s["scale"]
        p = torch.softmax(logits, 1)
        out[b] = (p.transpose(1, 2).contiguous() @ _table_rows(s, "v", b, n)[:, low:]).reshape(case["q_heads"], -1)
        if mass is not None:
            mass[b, :, :n] = s["mass"][b, :, :n].double()
            mass[b, :, low:n] += p.sum(2)
    return {"out": out} if mass is None else {"out": out, "mass": mass}


def _exact_append(s):
    """Rows and (step, lo) from float64 arithmetic, rounded where the definition
    stores fp16; the codes follow fp32 decisions, so they have no 64-bit value."""
    case = s["case"]
    row, slot = s["row"].long().tolist(), s["slot"].long().tolist()
    table = s["table"].tolist()
    page = torch.tensor([table[r][i // case["page"]] for r, i in zip(row, slot)], device="cuda")
    line = torch.tensor([i % case["page"] for i in slot], device="cuda")
    got = {}
    for n in ("k", "v"):
        x = s[n + "_new"].double()
        if case["bits"] == 16:
            got[n] = s[n].double().clone()
            got[n][page, :, line] = x
            continue
        if n == "k" and s["signs"] is not None:
            x = (x * s["signs"].double()) @ torch.from_numpy(_hadamard()).cuda()
        low = x.amin(-1).half().double()
        step = ((x.amax(-1) - low) / (2.0 ** case["bits"] - 1.0)).half().double()
        got[n], got[n + "meta"] = None, s[n + "meta"].double().clone()
        got[n + "meta"][page, :, line] = torch.stack([step, low], -1)
    if case["track"]:
        got["mass"], got["pos"] = s["mass"].double().clone(), None
        got["mass"][s["row"].long(), :, s["slot"].long()] = 0.0
    return got


def _exact_evict(s):
    """The masses of the kept slots, by Python's own sort; the moved rows' (step, lo) and fp16 rows."""
    case, budget = s["case"], s["case"]["budget"]
    got = {n: s[n].double().clone() if s[n].is_floating_point() else None for n in _pool_out(s)}
    got["mass_out"] = s["mass_out"].double().clone()
    got["pos_out"] = got["lens_out"] = got["kept"] = None
    mass, pos, table = s["mass"].cpu().numpy().astype(np.float64), s["pos"].cpu().numpy(), s["table"].cpu().numpy()
    lens = s["lens"].tolist()
    for b in range(case["B"]):
        n, left = lens[b], min(lens[b], budget)
        for h in range(case["heads"]):
            m, p = mass[b, h, :n], pos[b, h, :n]
            late = p > p.max(initial=-1) - case["recent"]
            order = np.lexsort((np.arange(n), -m, ~late))[:left]
            stay = np.sort(order)
            frm = stay[stay >= left]
            to = np.setdiff1d(np.arange(left), stay)
            at = np.arange(left)
            at[to] = frm
            got["mass_out"][b, h, :left] = torch.from_numpy(m[at]).cuda()
            pf, pt = (torch.from_numpy(table[b, i // case["page"]].astype(np.int64)).cuda() for i in (frm, to))
            lf, lt = (torch.from_numpy(i % case["page"]).cuda() for i in (frm, to))
            for t in ("k", "v", "kmeta", "vmeta"):
                if got.get(t) is not None:
                    got[t][pt, h, lt] = got[t][pf, h, lf]
    return got


def exact(case, seed):
    s = prepare(case, seed)
    return {APPEND: _exact_append, ATTEND: _exact_attend, EVICT: _exact_evict}[case["op"]](s)
