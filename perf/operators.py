"""Cases, plain forms and exact values of the per-head key-value cache operators: appending tokens to a paged cache,
attention of one new token per sequence over it (with or without each slot's accumulated attention weight), and
eviction of the slots that gathered the least weight."""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _attend(name, B, H, Hkv, d, lo, hi, page, *, dtype="bf16", window=0, sink=False, weigh=False, shared=False, head_major=False):
    c = {"op": "attend", "B": B, "H": H, "Hkv": Hkv, "d": d, "lo": lo, "hi": hi, "page": page, "dtype": dtype, "window": window,
         "sink": sink, "weigh": weigh, "shared": shared, "head_major": head_major}
    return dict(c, name=name) if name else c


def _evict(name, B, Hkv, d, n, budget, recent, first, page, *, dtype="bf16", settled=True):
    c = {"op": "evict", "B": B, "Hkv": Hkv, "d": d, "n": n, "budget": budget, "recent": recent, "first": first, "page": page, "dtype": dtype,
         "settled": settled}
    return dict(c, name=name) if name else c


def _append(name, B, Hkv, d, lo, hi, new_lo, new_hi, page, *, dtype="bf16", track=False):
    c = {"op": "append", "B": B, "Hkv": Hkv, "d": d, "lo": lo, "hi": hi, "new_lo": new_lo, "new_hi": new_hi, "page": page, "dtype": dtype,
         "track": track}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a single user's first token after a short prompt: one sequence, little to read, all latency
        _attend("attend_one_short", 1, 32, 8, 128, 200, 200, 16),
        # a serving batch in which some sequences have just begun and others have run for long; learned sinks
        _attend("attend_ragged_batch", 48, 64, 8, 128, 1, 6000, 64, sink=True),
        # the eight-KV-head baseline at 128K tokens of context
        _attend("attend_long_context", 8, 64, 8, 128, 131072, 131072, 64),
        # every query head with a KV head of its own, an odd head width, fp16, contiguous storage
        _attend("attend_own_heads_fp16", 24, 20, 20, 96, 700, 3500, 0, dtype="fp16"),
        # a small batch that tracks which slots its attention uses
        _attend("weigh_small_batch", 4, 32, 8, 128, 900, 1500, 16, weigh=True),
        # a serving batch near the length at which it evicts
        _attend("weigh_serving_batch", 32, 64, 8, 128, 2049, 8192, 64, weigh=True),
        # heavily compressed entries of 1M tokens (8192 of them, one shared key-value head) tracked for eviction
        _attend("weigh_shared_entries", 8, 64, 1, 128, 8192, 8192, 64, weigh=True, shared=True),
        # a decode step at the budget: one slot out per step, in every head of every sequence
        _evict("evict_one_slot", 64, 8, 128, 2049, 2048, 512, 4, 64),
        # eviction every 256 steps
        _evict("evict_chunk", 32, 8, 128, 2304, 2048, 512, 4, 64),
        # a long prompt cut to a budget before decoding begins
        _evict("evict_prompt", 2, 8, 128, 65536, 4096, 1024, 4, 64, settled=False),
        # a decode step's new token of every sequence
        _append("append_step", 64, 8, 128, 100, 4000, 1, 1, 64, track=True),
        # prompts, or pieces of prompts, packed end to end
        _append("append_prompts", 8, 8, 128, 0, 2000, 500, 4000, 64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    d = rng.choice([64, 64, 72, 96, 128, 128, 128, 192, 256])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    page = rng.choice([0, 1, 5, 16, 32, 64, 64, 100, 256])
    kind = rng.choice(["attend", "attend", "weigh", "weigh", "evict", "append"])
    if kind in ("attend", "weigh"):
        Hkv = rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
        H = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 17, 32, 64] if Hkv == 1 else [1, 2, 3, 4, 5, 8, 16])
        hi = _log(rng, 1, 100000)
        B = min(_log(rng, 1, 200), max(1, 1000000000 // (hi * Hkv * d * 2)), max(1, 400000000 // (hi * H)))
        lo = rng.choice([0, 1, hi // 2, hi])
        window = rng.choice([0, 0, 0, 1, 128, 1000]) if kind == "attend" else 0
        return _attend(None, B, H, Hkv, d, min(lo, hi), hi, page, dtype=dtype, window=window, sink=rng.random() < 0.4, weigh=kind == "weigh",
                       shared=rng.random() < 0.15, head_major=rng.random() < 0.3)
    Hkv = rng.choice([1, 2, 5, 8])
    if kind == "evict":
        budget = _log(rng, 2, 8000)
        n = budget + rng.choice([0, 1, 17, _log(rng, 1, 30000)])
        recent = rng.randint(1, max(1, budget // 2))
        first = min(rng.choice([0, 1, 4]), budget - recent)
        B = min(_log(rng, 1, 128), max(1, 400000000 // (n * Hkv * d * 2)))
        return _evict(None, B, Hkv, d, n, budget, recent, first, page, dtype=dtype, settled=rng.random() < 0.6)
    hi = _log(rng, 1, 10000)
    new_hi = rng.choice([1, 1, _log(rng, 1, 3000)])
    new_lo = 1 if new_hi == 1 else rng.choice([0, 1, new_hi // 2])
    B = min(_log(rng, 1, 256), max(1, 400000000 // ((hi + new_hi) * Hkv * d * 2)))
    return _append(None, B, Hkv, d, rng.choice([0, hi // 2]), hi, new_lo, new_hi, page, dtype=dtype, track=rng.random() < 0.5)


def _spread(lo, hi, B, phase=0.0):
    """B lengths over [lo, hi], fixed by the case: multiples of the golden ratio, modulo one."""
    return [lo + int((hi - lo + 1) * ((phase + 0.61803398875 * (b + 1)) % 1.0)) if hi > lo else hi for b in range(B)]


def _evict_lens(c):
    """One sequence in four is a little shorter than the rest: a batch is not in step."""
    return [c["n"] if b % 4 != 3 else c["n"] - c["n"] // 64 for b in range(c["B"])]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _pool(g, B, cap, page, Hkv, d, dtype, head_major=False, shared=False):
    """A key and a value cache of B sequences of up to `cap` slots: [pages, page_size, Hkv, d], in a shuffled order of the pages behind a page
    table, or (page = 0) one run of `cap` slots per sequence. Keys and values have an offset of each channel, as trained ones have."""
    if page:
        per = -(-cap // page)
        n = B * per + 3
        table = torch.randperm(n, generator=g, device=DEV)[:B * per].to(torch.int32).reshape(B, per)
    else:
        n, page, table = B, cap, None
    shape = (n, Hkv, page, d) if head_major else (n, page, Hkv, d)

    def one():
        t = torch.randn(shape, generator=g, device=DEV, dtype=dtype)
        off = 0.5 * torch.randn((Hkv, 1, d) if head_major else (Hkv, d), generator=g, device=DEV, dtype=dtype)
        t.add_(off)
        return t.transpose(1, 2) if head_major else t

    k = one()
    return k, (k if shared else one()), table


def prepare(case, seed):
    c, B, Hkv, d = case, case["B"], case["Hkv"], case["d"]
    g = torch.Generator(device=DEV).manual_seed(1000003 * seed + 17)
    dt = DTYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] == "attend":
        cap = max(1, c["hi"])
        s["k"], s["v"], s["table"] = _pool(g, B, cap, c["page"], Hkv, d, dt, c["head_major"], c["shared"])
        s["lens"] = torch.tensor(_spread(c["lo"], c["hi"], B), dtype=torch.int32, device=DEV)
        s["q"] = (2.0 * torch.randn(B, c["H"], d, generator=g, device=DEV)).to(dt)   # some heads look sharply at a few slots
        s["scale"] = 1.0 / math.sqrt(d)
        s["sink"] = torch.randn(c["H"], generator=g, device=DEV) if c["sink"] else None
        s["max_len"] = cap
        if c["weigh"]:
            live = torch.arange(cap, device=DEV)[None, None, :] < s["lens"][:, None, None]
            s["weights"] = torch.rand(B, Hkv, cap, generator=g, device=DEV).square_().mul_(live)
            s["weights_out"] = torch.zeros_like(s["weights"])
    elif c["op"] == "evict":
        n, budget = c["n"], c["budget"]
        s["k"], s["v"], s["table"] = _pool(g, B, n, c["page"], Hkv, d, dt)
        s["lens"] = torch.tensor(_evict_lens(c), dtype=torch.int32, device=DEV)
        live = torch.arange(n, device=DEV)[None, None, :] < s["lens"][:, None, None]
        # attention mass per slot: heavy-tailed, and nothing at all on some slots
        w = torch.rand(B, Hkv, n, generator=g, device=DEV).pow_(6).mul_(8)
        w[w < 1e-6] = 0
        s["weights"] = w.mul_(live)
        at = torch.arange(n, device=DEV, dtype=torch.int32)
        pos = at.expand(B, Hkv, n).clone()
        if c["settled"]:   # earlier evictions have put the older tokens into slots in an order of each head's own
            old = min(budget, n) - min(c["recent"], budget - 1)
            order = torch.rand(B, Hkv, old, generator=g, device=DEV).argsort(-1)
            pos[..., :old] = at[:old][order]
        s["slot_pos"] = pos.mul_(live)
        s["pos"] = s["lens"] - 1
        s["weights_out"], s["slot_pos_out"], s["lens_out"] = torch.empty_like(w), torch.empty_like(pos), torch.empty_like(s["lens"])
    else:
        lens = _spread(c["lo"], c["hi"], B)
        new = _spread(c["new_lo"], c["new_hi"], B, 0.3)
        cap = max(a + b for a, b in zip(lens, new))
        cap = max(1, cap)
        s["k"], s["v"], s["table"] = _pool(g, B, cap, c["page"], Hkv, d, dt)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        start = [0]
        for x in new:
            start.append(start[-1] + x)
        T = start[-1]
        s["start"] = None if c["new_hi"] == 1 and c["new_lo"] == 1 else torch.tensor(start, dtype=torch.int32, device=DEV)
        # keys and values as two thirds of one projection's output
        kv = torch.randn(T, 2 * Hkv, d, generator=g, device=DEV, dtype=dt)
        s["k_new"], s["v_new"] = kv[:, :Hkv], kv[:, Hkv:]
        s["lens_out"] = torch.empty_like(s["lens"])
        s["weights"] = s["slot_pos"] = s["pos"] = None
        if c["track"]:
            s["weights"] = torch.rand(B, Hkv, cap, generator=g, device=DEV)
            s["slot_pos"] = torch.randint(0, cap, (B, Hkv, cap), generator=g, device=DEV, dtype=torch.int32)
            s["pos"] = s["lens"] * 2 + 5   # some of the sequence's tokens have been evicted
    if own:
        import compressed_sparse_kv_03_b200 as csa
        s["cache"] = csa.KVCache(s["k"], s["v"], s["table"])
        s["ws"] = csa.Workspace(DEV)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    s, c = state, state["case"]
    if own:
        import compressed_sparse_kv_03_b200 as csa
        if c["op"] == "attend":
            if c["weigh"]:
                out, lse = csa.kv_attn_decode(s["q"], s["cache"], s["lens"], s["scale"], max_len=s["max_len"], window=c["window"], sink=s["sink"],
                                              weights=s["weights"], weights_out=s["weights_out"], return_lse=True, ws=s["ws"])
                return out, lse, s["weights_out"]
            return csa.kv_attn_decode(s["q"], s["cache"], s["lens"], s["scale"], max_len=s["max_len"], window=c["window"], sink=s["sink"],
                                      return_lse=True, ws=s["ws"])
        if c["op"] == "evict":
            csa.kv_evict(s["cache"], s["lens"], s["weights"], s["slot_pos"], s["pos"], c["budget"], c["recent"], keep_first=c["first"],
                         max_len=c["n"], lens_out=s["lens_out"], weights_out=s["weights_out"], slot_pos_out=s["slot_pos_out"], ws=s["ws"])
            return s["k"], s["v"], s["weights_out"], s["slot_pos_out"], s["lens_out"]
        csa.kv_append(s["k_new"], s["v_new"], s["cache"], s["lens"], token_start=s["start"], pos=s["pos"], weights=s["weights"],
                      slot_pos=s["slot_pos"], lens_out=s["lens_out"], ws=s["ws"])
        return [x for x in (s["k"], s["v"], s["lens_out"], s["weights"], s["slot_pos"]) if x is not None]
    return {"attend": _plain_attend, "evict": _plain_evict, "append": _plain_append}[c["op"]](s, c)


def _place(s, c, seq, slot):
    """(page, row in the page) of slots of sequences."""
    if s["table"] is None:
        return seq.expand_as(slot), slot
    return s["table"][seq, slot // c["page"]].long(), slot % c["page"]


def _plain_attend(s, c):
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    n = s["max_len"]
    seq, slot = torch.arange(B, device=DEV)[:, None], torch.arange(n, device=DEV)[None, :].expand(B, n)
    page, row = _place(s, c, seq, slot)
    keys = s["k"][page, row].float().permute(0, 2, 3, 1)                       # [B, Hkv, d, n]
    q = s["q"].float().reshape(B, Hkv, H // Hkv, d)
    z = (q @ keys) * s["scale"]
    seen = slot < s["lens"][:, None]
    if c["window"]:
        seen = seen & (slot >= s["lens"][:, None] - c["window"])
    z = z.masked_fill(~seen[:, None, None, :], -math.inf)
    top = z.amax(-1, keepdim=True)
    if s["sink"] is not None:
        sink = s["sink"].reshape(1, Hkv, H // Hkv, 1)
        top = torch.maximum(top, sink)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(z - top)
    den = p.sum(-1, keepdim=True)
    if s["sink"] is not None:
        den = den + torch.exp(sink - top)
    lse = (top + torch.log(den)).reshape(B, H)
    p = p / torch.where(den == 0, torch.ones_like(den), den)
    values = s["v"][page, row].float().permute(0, 2, 1, 3)                     # [B, Hkv, n, d]
    out = (p @ values.masked_fill(~seen[:, None, :, None], 0.0)).reshape(B, H, d).to(s["q"].dtype)
    if c["weigh"]:
        torch.add(s["weights"], p.sum(2), out=s["weights_out"])
        return out, lse, s["weights_out"]
    return out, lse


def _plain_evict(s, c):
    n, budget, recent, first = c["n"], c["budget"], c["recent"], c["first"]
    slot = torch.arange(n, device=DEV)
    live = slot < s["lens"][:, None, None]
    held = (s["slot_pos"] > (s["pos"] - recent)[:, None, None]) | (s["slot_pos"] < first)
    rank = s["weights"].masked_fill(held, math.inf).masked_fill(~live, -math.inf)
    order = rank.sort(dim=-1, descending=True, stable=True).indices[..., :budget]     # ties: the lower slot first
    kept = torch.zeros_like(live.expand_as(rank)).scatter_(-1, order, True) & live
    low = slot < budget
    hole, mover = ~kept & low & live, kept & ~low
    # the j-th hole takes the j-th mover
    b, h, dst = hole.nonzero(as_tuple=True)
    count = mover.sum(-1)
    nth = hole.cumsum(-1)[b, h, dst]
    b, h, dst = (x[nth <= count[b, h]] for x in (b, h, dst))
    src = mover.nonzero(as_tuple=True)[2]
    w, pos = s["weights_out"], s["slot_pos_out"]
    w.copy_(s["weights"].masked_fill(~(low & live), 0.0))
    pos.copy_(s["slot_pos"].masked_fill(~(low & live), 0))
    w[b, h, dst] = s["weights"][b, h, src]
    pos[b, h, dst] = s["slot_pos"][b, h, src]
    (pd, rd), (ps, rs) = _place(s, c, b, dst), _place(s, c, b, src)
    for t in (s["k"], s["v"]):
        t[pd, rd, h] = t[ps, rs, h]
    s["lens_out"].copy_(s["lens"].clamp(max=budget))
    return s["k"], s["v"], w, pos, s["lens_out"]


def _plain_append(s, c):
    B, T = c["B"], s["k_new"].shape[0]
    if s["start"] is None:
        seq, i, count = torch.arange(B, device=DEV), torch.zeros(B, dtype=torch.long, device=DEV), 1
    else:
        t = torch.arange(T, device=DEV)
        seq = torch.searchsorted(s["start"][1:].long(), t, right=True)
        i, count = t - s["start"][seq], s["start"][1:] - s["start"][:-1]
    slot = s["lens"][seq] + i
    page, row = _place(s, c, seq, slot)
    s["k"][page, row] = s["k_new"]
    s["v"][page, row] = s["v_new"]
    torch.add(s["lens"], count, out=s["lens_out"])
    if c["track"]:
        s["weights"][seq, :, slot] = 0.0
        s["slot_pos"][seq, :, slot] = (s["pos"][seq] + i).to(torch.int32)[:, None].expand(-1, c["Hkv"])
    return [x for x in (s["k"], s["v"], s["lens_out"], s["weights"], s["slot_pos"]) if x is not None]


# ---------------------------------------------------------------------------
# what one pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c, row = case, case["Hkv"] * case["d"] * 2
    if c["op"] == "attend":
        seen = [min(n, c["window"]) if c["window"] else n for n in _spread(c["lo"], c["hi"], c["B"])]
        n = sum(seen)
        small = c["B"] * c["H"] * (4 * c["d"] + 4)
        if c["weigh"]:   # read and written over the whole array's live part
            small += 8 * c["Hkv"] * n
        return {"bytes": n * row * (1 if c["shared"] else 2) + small, "flops": 4.0 * n * c["H"] * c["d"]}
    if c["op"] == "evict":
        total = 0.0
        for n in _evict_lens(c):
            out, free = max(0, n - c["budget"]), max(1, n - c["recent"] - c["first"])
            # slots below the budget that lose their row and take one from above it: the share `out / free` of those not held
            holes = max(0, min(n - c["recent"], c["budget"]) - c["first"]) * min(1.0, out / free)
            total += c["Hkv"] * 8 * (n + min(n, c["budget"])) + min(holes, out) * row * 4
        return {"bytes": total, "flops": 1.0 * c["B"] * c["Hkv"] * c["n"]}
    T = sum(_spread(c["new_lo"], c["new_hi"], c["B"], 0.3))
    return {"bytes": T * row * 4 + (8 * T * c["Hkv"] if c["track"] else 0) + 8 * c["B"], "flops": 1.0 * T}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    held = own
    globals()["own"] = False
    try:
        s = prepare(case, seed)
    finally:
        globals()["own"] = held
    return {"attend": _exact_attend, "evict": _exact_evict, "append": _exact_append}[case["op"]](s, case)


def _rows(s, c, t, b, lo, hi):
    """Rows lo .. hi-1 of sequence b, [hi - lo, Hkv, d] in 64 bits."""
    if s["table"] is None:
        return t[b, lo:hi].double()
    first, last = lo // c["page"], -(-hi // c["page"])
    whole = t[s["table"][b, first:last].long()].flatten(0, 1)
    return whole[lo - first * c["page"]:hi - first * c["page"]].double()


def _exact_attend(s, c):
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    G = H // Hkv
    out = torch.zeros(B, H, d, dtype=torch.float64, device=DEV)
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device=DEV)
    weights = s["weights"].double() if c["weigh"] else None
    sink = s["sink"].double() if s["sink"] is not None else None
    for b, n in enumerate(s["lens"].tolist()):
        lo = max(0, n - c["window"]) if c["window"] else 0
        if n == lo:
            if sink is not None:
                lse[b] = sink
            continue
        k, v = _rows(s, c, s["k"], b, lo, n), _rows(s, c, s["v"], b, lo, n)
        for h in range(Hkv):
            q = s["q"][b, h * G:(h + 1) * G].double()
            z = torch.einsum("nd,gd->gn", k[:, h], q) * s["scale"]
            if sink is not None:
                z = torch.cat([z, sink[h * G:(h + 1) * G, None]], 1)
            total = torch.logsumexp(z, 1)
            p = torch.exp(z[:, :n - lo] - total[:, None])
            out[b, h * G:(h + 1) * G] = torch.einsum("gn,nd->gd", p, v[:, h])
            lse[b, h * G:(h + 1) * G] = total
            if weights is not None:
                weights[b, h, lo:n] += p.sum(0)
    return (out, lse) if weights is None else (out, lse, weights)


def _exact_evict(s, c):
    budget, recent, first = c["budget"], c["recent"], c["first"]
    lens, pos = s["lens"].cpu().tolist(), s["pos"].cpu().tolist()
    w, sp = s["weights"].double().cpu().numpy(), s["slot_pos"].cpu().numpy()
    wo, po = w * 0, sp * 0
    take = []
    for b, n in enumerate(lens):
        for h in range(c["Hkv"]):
            key = [(0 if sp[b, h, j] > pos[b] - recent or sp[b, h, j] < first else 1, -w[b, h, j], j) for j in range(n)]
            keep = sorted(j for _, _, j in sorted(key)[:budget])
            have = set(keep)
            movers = [j for j in keep if j >= budget]
            holes = [j for j in range(min(n, budget)) if j not in have]
            m = min(n, budget)
            wo[b, h, :m], po[b, h, :m] = w[b, h, :m], sp[b, h, :m]
            for to, j in zip(holes, movers):
                wo[b, h, to], po[b, h, to] = w[b, h, j], sp[b, h, j]
                take.append((b, h, to, j))
    k, v = s["k"].double(), s["v"].double()
    if take:
        b, h, to, j = torch.tensor(take, device=DEV).T
        if s["table"] is None:
            at, came = (b, to), (b, j)
        else:
            t = s["table"].long()
            at, came = (t[b, to // c["page"]], to % c["page"]), (t[b, j // c["page"]], j % c["page"])
        for x in (k, v):
            x[at[0], at[1], h] = x[came[0], came[1], h]
    return k, v, torch.from_numpy(wo), torch.from_numpy(po), torch.tensor([min(n, budget) for n in lens], dtype=torch.int32)


def _exact_append(s, c):
    k, v = s["k"].double(), s["v"].double()
    lens = s["lens"].cpu().tolist()
    start = list(range(c["B"] + 1)) if s["start"] is None else s["start"].cpu().tolist()
    w, sp = (s["weights"].double(), s["slot_pos"].clone()) if c["track"] else (None, None)
    end = []
    for b, n in enumerate(lens):
        new = start[b + 1] - start[b]
        end.append(n + new)
        if not new:
            continue
        slots = list(range(n, n + new))
        if s["table"] is None:
            page, row = torch.full((new,), b, device=DEV), torch.tensor(slots, device=DEV)
        else:
            page = s["table"][b].long()[torch.tensor([x // c["page"] for x in slots], device=DEV)]
            row = torch.tensor([x % c["page"] for x in slots], device=DEV)
        k[page, row], v[page, row] = s["k_new"][start[b]:start[b + 1]].double(), s["v_new"][start[b]:start[b + 1]].double()
        if w is not None:
            w[b, :, n:n + new] = 0
            sp[b, :, n:n + new] = int(s["pos"][b]) + torch.arange(new, device=DEV, dtype=torch.int32)
    return [x for x in (k, v, torch.tensor(end, dtype=torch.int32), w, sp) if x is not None]
