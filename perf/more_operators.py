"""Generation for many sequences at once: cases to measure.

Four operators of a generated token's layer step, for sequences of different lengths:

  push    keys and values of new tokens enter a memory held in pages
  step    the same for 1..16 new tokens a sequence, and their relative attention over the pages; in some
          cases the attention weight that every position receives is added up
  evict   the memory is cut to a number of positions a sequence: the newest and the most attended stay
  linear  products of few rows with 4-bit weights (groups along k share a bf16 step and minimum)

Each pass exists in a plain form (elementary torch operations) and as calls of the package (`own`).
"""
import math

import torch

own = False


# ------------------------------------------------------------------------------------ cases
def listed():
    """Shapes of the package's workloads: generation (B8 H16 D64 over 4096 positions, clamped at 1000),
    the base shape (d_model 410, H10 d_head 41), the stream shape (H16 d_head 128), the tiny fp32 one."""
    return [
        # one generated token of eight sequences enters their pages: launch latency
        dict(name="push token", op="push", B=8, H=16, D=64, T=1, length=700, ragged=True, idle=0, page=64, dtype="bf16"),
        # prompts of different lengths enter together (padded batch), pages of 16
        dict(name="push prompts", op="push", B=8, H=16, D=64, T=1600, length=0, ragged=False, idle=3, page=16,
             dtype="bf16"),
        # the smallest call, fp32
        dict(name="step tiny f32", op="step", B=1, H=2, D=8, T=1, length=8, ragged=False, idle=0, page=16, C=16,
             gaps=False, weights=False, dtype="f32"),
        # generation: one token a sequence over long memories, distances clamped at 1000
        dict(name="step token", op="step", B=8, H=16, D=64, T=1, length=4096, ragged=False, idle=0, page=64, C=1000,
             gaps=False, weights=False, dtype="bf16"),
        # a serving batch: lengths between a few and 4096, some sequences idle, memories that positions were
        # evicted from, and the attention weights added up for the next eviction
        dict(name="step serving weights", op="step", B=32, H=16, D=64, T=1, length=4096, ragged=True, idle=5, page=64,
             C=1000, gaps=True, weights=True, dtype="bf16"),
        # one sequence with a very long memory, a position table longer than the memory
        dict(name="step long", op="step", B=1, H=16, D=64, T=1, length=65536, ragged=False, idle=0, page=128, C=70000,
             gaps=False, weights=False, dtype="bf16"),
        # a few drafted tokens a sequence, d_head 128, pages of 16
        dict(name="step draft", op="step", B=4, H=16, D=128, T=5, length=2048, ragged=True, idle=0, page=16, C=1000,
             gaps=False, weights=True, dtype="bf16"),
        # a bounded memory's regular eviction: 64 of 1088 positions leave each of eight sequences
        dict(name="evict regular", op="evict", B=8, H=16, D=64, length=1088, ragged=False, keep=1024, recent=256,
             page=64, dtype="bf16"),
        # long prompts cut to a quarter
        dict(name="evict prompts", op="evict", B=4, H=16, D=64, length=16384, ragged=True, keep=4096, recent=512,
             page=128, dtype="bf16"),
        # the base shape's q|k|v projection of a token of five sequences: odd k and n
        dict(name="linear base", op="linear", m=5, k=410, n=1230, group=64, dtype="bf16"),
        # a token's output projection at d_model 1024
        dict(name="linear token", op="linear", m=1, k=1024, n=1024, group=64, dtype="bf16"),
        # eight tokens against a large matrix
        dict(name="linear eight", op="linear", m=8, k=8192, n=8192, group=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["push", "step", "step", "step", "evict", "linear", "linear"])
    if op == "linear":
        m = _log(rng, 1, 16)
        k = _log(rng, 100, 8192)
        n = _log(rng, 100, max(100, min(8192, 8192 * 8192 * 8 // (k * m))))
        if rng.random() < 0.5:
            k, n = (k + 63) // 64 * 64, (n + 63) // 64 * 64
        return dict(op=op, m=m, k=k, n=n, group=rng.choice([32, 64, 64, 128]), dtype="bf16")
    D = rng.choice([8, 24, 41, 64, 64, 64, 80, 96, 128, 128])
    H = rng.randint(1, 16)
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    e = 4 if dtype == "f32" else 2
    c = dict(op=op, H=H, D=D, page=rng.choice([16, 32, 48, 64, 64, 128]), ragged=rng.random() < 0.5, dtype=dtype)
    c["B"] = _log(rng, 1, 32)
    room = c["B"] * H * max(D, 32) * e // 2                 # positions' cost against the listed cases'
    if op == "push":
        c["T"] = _log(rng, 1, max(1, min(4096, 8 * 16 * 64 * 1600 // room)))
        c["length"] = rng.choice([0, rng.randint(0, 500)])
        c["idle"] = rng.choice([0, 0, 3])
    elif op == "step":
        c["T"] = rng.choice([1, 1, 1, 1, 2, 3, 4, 5, 7, 8, 11, 16])
        cost = 1 if dtype != "f32" else 2 + c["T"]
        c["length"] = _log(rng, 1, max(64, min(40000, 32 * 16 * 64 * 2000 // (room * cost * (2 if c["T"] > 4 else 1)))))
        c["idle"] = rng.choice([0, 0, 3])
        c["C"] = rng.choice([200, 1000, 1000, 2 * c["length"] + 16])
        c["gaps"] = rng.random() < 0.4
        c["weights"] = rng.random() < 0.4
    else:
        c["length"] = _log(rng, 64, max(64, min(20000, 4 * 16 * 64 * 16384 // room)))
        c["keep"] = rng.randint(max(1, c["length"] // 4), c["length"])
        c["recent"] = rng.randint(0, c["keep"])
    return c


def _lengths(c):
    """Positions that every sequence holds before the call."""
    n, B = c["length"], c["B"]
    return [1 + (n - 1) * ((b * 7) % B + 1) // B if c["ragged"] and n else n for b in range(B)]


def _counts(c):
    """New tokens of every sequence: T, fewer in a push of prompts, none for an idle sequence."""
    T, idle = c["T"], c["idle"]
    if c["op"] == "push" and idle:
        return [T - (T * (b % idle)) // (idle + 1) for b in range(c["B"])]
    return [0 if idle and b % idle == idle - 1 else T for b in range(c["B"])]


def work(c):
    if c["op"] == "linear":
        m, k, n = c["m"], c["k"], c["n"]
        return {"bytes": (k * n + 1) // 2 + 4 * ((k + c["group"] - 1) // c["group"]) * n + 2 * m * (k + n),
                "flops": 2 * m * k * n}
    B, H, D = c["B"], c["H"], c["D"]
    e = 4 if c["dtype"] == "f32" else 2
    held = _lengths(c)
    if c["op"] == "push":                                   # k, v read and written; a position and a weight each
        n = sum(_counts(c))
        return {"bytes": n * (4 * H * D * e + 8), "flops": n * H * D}
    if c["op"] == "evict":                                  # weights and positions read; at most the evicted slots filled
        cut = [max(0, n - c["keep"]) for n in held]
        moved = sum(min(x, c["keep"]) * c["keep"] // (c["keep"] + x) for x in cut)
        return {"bytes": 8 * sum(held) + moved * (4 * H * D * e + 8), "flops": sum(held)}
    counts = _counts(c)
    n_rows = _n_rows(c)
    keys = sum(held[b] + t for b, t in enumerate(counts) if t)
    pairs = sum(t * held[b] + t * (t + 1) // 2 for b, t in enumerate(counts))
    return {"bytes": keys * (2 * H * D * e + 4 + 8 * c["weights"]) + n_rows * H * D * e + 5 * sum(counts) * H * D * e,
            "flops": 6 * H * D * pairs}


# ------------------------------------------------------------------------------------ inputs
def _dtype(c):
    return torch.float32 if c["dtype"] == "f32" else torch.bfloat16


def _first_new(c):
    """The position of a sequence's first new token; beyond its length where positions were evicted."""
    return [n + n // 2 if c.get("gaps") else n for n in _lengths(c)]


def _n_rows(c):
    return min(max(_first_new(c)) + c["T"], c["C"] + 1)


def _normal(gen, dtype, *shape):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for part in out.split(max(1, 2 ** 24 // max(1, out[0].numel()))):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda"))
    return out


def _memory(c, seed):
    """A memory in pages, drawn from the seed: every sequence has the same number of pages, anywhere in the
    pool, its first slots hold positions (in order, or any positions in any order where some were evicted)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, H, D, page = c["B"], c["H"], c["D"], c["page"]
    held, T = _lengths(c), c.get("T", 0)
    per = (max(held) + T + page - 1) // page
    pool = B * per + 3
    x = {"k_pool": _normal(gen, _dtype(c), pool, H, page, D), "v_pool": _normal(gen, _dtype(c), pool, H, page, D)}
    if c["op"] != "push":
        # heads differ in how sharply they attend
        x["k_pool"] *= (0.3 + torch.rand(H, 1, 1, generator=gen, device="cuda") * 1.7).to(_dtype(c))
    x["table"] = torch.randperm(pool, generator=gen, device="cuda")[: B * per].view(B, per).int()
    x["length"] = torch.tensor(held, dtype=torch.int32, device="cuda")
    x["next"] = torch.tensor(_first_new(c), dtype=torch.int32, device="cuda")
    pos = torch.zeros(B, per * page, dtype=torch.int32, device="cuda")
    for b, n in enumerate(held):
        seen = _first_new(c)[b]
        pick = torch.randperm(seen, generator=gen, device="cuda")[:n] if c.get("gaps") else torch.arange(n, device="cuda")
        if c["op"] == "evict":                              # the first third of the slots was refilled before
            pick[: n // 3] = pick[torch.randperm(n // 3, generator=gen, device="cuda")]
        pos[b, :n] = pick.int()
    x["pos"] = torch.zeros(pool, page, dtype=torch.int32, device="cuda")
    x["pos"][x["table"].long()] = pos.view(B, per, page)
    # accumulated weights: a few positions received most, many next to nothing, some nothing at all
    w = torch.rand(pool, page, generator=gen, device="cuda") ** 8 * 20
    x["weight"] = torch.where(torch.rand(pool, page, generator=gen, device="cuda") < 0.05, 0.0, w)
    return x, gen


def _inputs(c, seed):
    if c["op"] == "linear":
        gen = torch.Generator(device="cuda").manual_seed(seed)
        gain = 0.5 + torch.rand(c["n"], generator=gen, device="cuda")
        W = torch.randn(c["k"], c["n"], generator=gen, device="cuda") * gain * c["k"] ** -0.5
        return {"W": W.bfloat16(), "x": _normal(gen, _dtype(c), c["m"], c["k"])}
    x, gen = _memory(c, seed)
    B, H, D = c["B"], c["H"], c["D"]
    if c["op"] == "evict":
        return x
    T = c["T"]
    x["k"], x["v"] = _normal(gen, _dtype(c), B, T, H, D), _normal(gen, _dtype(c), B, T, H, D)
    x["counts"] = torch.tensor(_counts(c), dtype=torch.int32, device="cuda")
    if c["op"] == "step":
        x["q"] = _normal(gen, _dtype(c), B, T, H, D)
        x["u"] = 0.02 * torch.randn(H, D, generator=gen, device="cuda")
        x["vb"] = 0.02 * torch.randn(H, D, generator=gen, device="cuda")
        # r = R W_R for distances 0 .. n_rows-1, R the interleaved sinusoid
        n_rows, dm = _n_rows(c), 128
        ang = torch.arange(n_rows, dtype=torch.float64, device="cuda")[:, None] * torch.pow(
            10000.0, -2.0 * torch.arange(dm // 2, dtype=torch.float64, device="cuda") / dm)
        R = torch.stack((ang.sin(), ang.cos()), -1).reshape(n_rows, dm).float()
        W = torch.randn(dm, H * D, generator=gen, device="cuda") * dm ** -0.5
        r = torch.zeros(n_rows, H, (D + 7) // 8 * 8, dtype=_dtype(c), device="cuda")
        r[..., :D] = (R @ W).view(n_rows, H, D)
        x["r"] = r
    return x


def prepare(case, seed):
    c, x = case, _inputs(case, seed)
    s = dict(c=c, x=x)
    if c["op"] == "linear":
        if own:
            import transformer_xl_relative_gb300 as txl
            s["txl"] = txl
            s["w"] = txl.QuantWeight.quantise(x.pop("W"), group=c["group"])
            s["y"] = torch.empty(c["m"], c["n"], dtype=_dtype(c), device="cuda")
        else:
            s["w"] = _quantise(x.pop("W"), c["group"])
        return s
    # what a pass changes besides the pages lies in one piece, so that one copy brings it back
    now = torch.cat([x[n].view(torch.int32).flatten() for n in ("length", "next", "pos", "weight")])
    s["then"], s["now"] = now, now.clone()
    at = 0
    for n in ("length", "next", "pos", "weight"):
        size = x[n].numel()
        x[n] = s["now"][at:at + size].view(x[n].dtype).view(x[n].shape)
        at += size
    if c["op"] == "step":
        s["out"] = torch.zeros_like(x["q"])
    if own:
        import transformer_xl_relative_gb300 as txl
        s["txl"] = txl
        s["mem"] = txl.PagedMemory(*_padded(x.pop("k_pool"), x.pop("v_pool")), x["pos"], x["weight"], x["table"],
                                   x["length"], x["next"])
        if c["op"] == "step":
            need = txl.rel_attn_paged_workspace_size(x["q"], s["mem"], _n_rows(c), accumulate=c["weights"])
            s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        elif c["op"] == "evict":
            s["ws"] = torch.empty(max(txl.paged_evict_workspace_size(s["mem"]), 16), dtype=torch.uint8, device="cuda")
    return s


def _padded(k, v):
    """The pools with rows of a multiple of 16 bytes, as the package keeps them."""
    D, unit = k.shape[-1], 16 // k.element_size()
    if D % unit == 0:
        return k, v
    pad = (D + unit - 1) // unit * unit - D
    return tuple(torch.nn.functional.pad(t, (0, pad))[..., :D] for t in (k, v))


# ------------------------------------------------------------------------------------ plain form
def _bf16_toward(x, up):
    """x (fp32) rounded to bf16 toward +inf (up) or -inf."""
    bits = x.view(torch.int32)
    cut = bits & -65536
    t = cut.view(torch.float32)
    away = (t < x) if up else (t > x)
    return torch.where(away, (cut + 65536).view(torch.float32), t).bfloat16()


def _quantise(W, group):
    """W [k, n] bf16 -> codes uint8 [groups, group, n], step and lo bf16 [groups, n]: lo the largest bf16 not
    above the group's least, step the smallest not below (most - lo) / 15, codes the nearest integers."""
    k, n = W.shape
    G = (k + group - 1) // group
    x = torch.nn.functional.pad(W.float(), (0, 0, 0, G * group - k), value=math.nan).view(G, group, n)
    pad = torch.isnan(x)
    lo = _bf16_toward(torch.where(pad, math.inf, x).amin(1), up=False)
    span = torch.where(pad, -math.inf, x).amax(1).double() - lo.double()
    step = _bf16_toward((span / 15).float(), up=True)
    # the quotient was rounded: one bf16 up or down where that crossed the exact value
    step = torch.where(step.double() * 15 < span, (step.view(torch.int16) + 1).view(torch.bfloat16), step)
    less = (step.view(torch.int16) - 1).clamp(min=0).view(torch.bfloat16)
    step = torch.where(less.double() * 15 >= span, less, step)
    code = torch.empty(G, group, n, dtype=torch.uint8, device=W.device)
    for g in range(G):
        d = (x[g].double() - lo[g].double()) / step[g].double()
        code[g] = torch.where(pad[g] | (step[g] == 0), 0.0, torch.round(d)).to(torch.uint8)
    return code, step, lo


def _slots(x, n):
    """Pool rows (page, row in the page) of the first n slots of every sequence."""
    s, page = torch.arange(n, device="cuda"), x["pos"].shape[1]
    return x["table"][:, s // page].long(), (s % page)


def _push_plain(c, x):
    """The new tokens' keys, values and positions into their slots; rows past a sequence's count write the
    pool's last page, which no sequence has, back to itself."""
    T, page = c["T"], c["page"]
    t = torch.arange(T, device="cuda")
    slot = x["length"].long()[:, None] + t
    live = t < x["counts"][:, None]
    free = _free_page(x)
    row = torch.where(live, slot % page, 0)
    pg = torch.where(live, torch.gather(x["table"].long(), 1, (slot // page).clamp(max=x["table"].shape[1] - 1)), free)
    heads = torch.arange(c["H"], device="cuda")
    at = (pg[:, :, None], heads, row[:, :, None])
    for n in "kv":
        x[n + "_pool"][at] = torch.where(live[:, :, None, None], x[n], x[n + "_pool"][free, :, 0])
    x["pos"][pg, row] = torch.where(live, x["next"][:, None] + t.int(), x["pos"][free, 0])
    x["weight"][pg, row] = torch.where(live, 0.0, x["weight"][free, 0])
    x["length"] += x["counts"]
    x["next"] += x["counts"]


def _free_page(x):
    """A page that no sequence has (the pool has three of them)."""
    used = torch.zeros(x["pos"].shape[0], dtype=torch.int32, device="cuda")
    used[x["table"].flatten().long()] = 1
    return torch.argmin(used)


def _step_plain(state, c, x):
    H, D, T, C = c["H"], c["D"], c["T"], c["C"]
    _push_plain(c, x)
    cap = max(_lengths(c)) + T
    pg, row = _slots(x, cap)
    out = state["out"]
    i = torch.arange(T, device="cuda")
    # sequences in pieces, so that long memories fit
    most = max(1, 2 ** 28 // (H * cap * D))
    for b in range(0, c["B"], most):
        s = slice(b, b + most)
        k, v = (x[n][pg[s], :, row].float().transpose(1, 2) for n in ("k_pool", "v_pool"))   # [b, H, cap, D]
        q = x["q"][s].float().transpose(1, 2)
        at = (x["next"][s] - x["counts"][s])[:, None].long() + i                               # the queries' positions
        delta = at[:, :, None] - x["pos"][pg[s], row].long()[:, None]
        seen = (delta >= 0) & (torch.arange(cap, device="cuda") < x["length"][s, None])[:, None]
        seen = seen & (i < x["counts"][s, None])[:, :, None]
        bd = (q + x["vb"][:, None]) @ x["r"][..., :D].float().permute(1, 2, 0)
        near = delta.clamp(0, min(C, x["r"].shape[0] - 1))
        a = (q + x["u"][:, None]) @ k.transpose(-1, -2)
        a = (a + bd.gather(-1, near[:, None].expand(a.shape))) / math.sqrt(D)
        a = torch.where(seen[:, None], a, -math.inf)
        most_a = a.amax(-1, keepdim=True)
        p = torch.exp(a - torch.where(most_a == -math.inf, 0.0, most_a))
        total = p.sum(-1, keepdim=True)
        p = p / torch.where(total == 0, 1.0, total)
        y = (p @ torch.where(seen.any(1)[:, None, :, None], v, 0.0)).transpose(1, 2).to(_dtype(c))
        live = (i < x["counts"][s, None])[:, :, None, None]
        out[s] = torch.where(live, y, out[s])
        if c["weights"]:
            x["weight"][pg[s], row] = x["weight"][pg[s], row] + p.sum((1, 2))
    return out


def _evict_plain(c, x):
    keep, H = c["keep"], c["H"]
    n = max(_lengths(c))
    if n > keep:
        pg, row = _slots(x, n)
        w, p = x["weight"][pg, row], x["pos"][pg, row]
        slot = torch.arange(n, device="cuda").expand(w.shape)
        held = slot < x["length"][:, None]
        may = held & (p < (x["next"] - c["recent"])[:, None])
        # the least weight leaves first, of equal ones the oldest
        by_age = torch.argsort(p, dim=1, stable=True)
        w = torch.where(may, w, math.inf).gather(1, by_age)
        order = by_age.gather(1, torch.argsort(w, dim=1, stable=True))
        rank = torch.empty_like(order)
        rank.scatter_(1, order, slot.contiguous())
        out = may & (rank < (x["length"] - keep).clamp(min=0)[:, None])
        # the k-th survivor behind the first `keep` slots fills the k-th hole among them
        hole, mover = out & (slot < keep), held & ~out & (slot >= keep)
        movers = torch.argsort(torch.where(mover, slot, n + slot), dim=1)[:, :keep]
        kth = (hole.long().cumsum(1) - 1).clamp(0, movers.shape[1] - 1)
        source = torch.where(hole, movers.gather(1, kth), slot)[:, :keep]
        spg = pg.gather(1, source)
        srow = row[source]
        for t in ("pos", "weight"):
            x[t][pg[:, :keep], row[:keep]] = x[t][spg, srow]
        for b in range(c["B"]):
            for t in ("k_pool", "v_pool"):
                x[t][pg[b, :keep], :, row[:keep]] = x[t][spg[b], :, srow[b]]
        x["length"].clamp_(max=keep)


def run(state):
    c, x = state["c"], state["x"]
    if c["op"] == "linear":
        if own:
            return state["txl"].linear_q4(x["x"], state["w"], state["y"])
        code, step, lo = state["w"]
        W = (lo.float()[:, None] + step.float()[:, None] * code.float()).view(-1, c["n"])[: c["k"]]
        return (x["x"].float() @ W).to(_dtype(c))
    state["now"].copy_(state["then"])                       # every pass starts from the same memory
    if own:
        txl, mem = state["txl"], state["mem"]
        if c["op"] == "push":
            txl.paged_push(mem, x["k"], x["v"], counts=x["counts"])
        elif c["op"] == "evict":
            txl.paged_evict(mem, c["keep"], c["recent"], workspace=state["ws"])
        else:
            txl.rel_attn_paged(x["q"], mem, x["k"], x["v"], x["u"], x["vb"], x["r"], x["r"].shape[0], c["C"],
                               state["out"], counts=x["counts"], accumulate=c["weights"], workspace=state["ws"])
        pools = mem.k, mem.v
    else:
        {"push": lambda: _push_plain(c, x), "evict": lambda: _evict_plain(c, x),
         "step": lambda: _step_plain(state, c, x)}[c["op"]]()
        pools = x["k_pool"], x["v_pool"]
    return [*([state["out"]] if c["op"] == "step" else []), *pools, x["length"], x["next"], x["pos"], x["weight"]]


# ------------------------------------------------------------------------------------ 64 bits
def _grid8(x, up):
    """x >= 0 to 8 significant bits, up or down (bf16's subnormals apart); fp64."""
    m, e = torch.frexp(x)
    unit = ((e.long() - 8 + 1023) << 52).view(torch.float64)      # 2^(e-8), exactly
    return (torch.ceil(m * 256.0) if up else torch.floor(m * 256.0)) * unit


def exact(case, seed):
    c, x = case, _inputs(case, seed)
    if c["op"] == "linear":
        y = torch.zeros(c["m"], c["n"], dtype=torch.float64, device="cuda")
        for at in range(0, c["k"], c["group"]):
            w = x["W"][at:at + c["group"]].double()
            least, most = torch.aminmax(w, dim=0)
            lo = torch.where(least < 0, -_grid8(-least, up=True), _grid8(least, up=False))
            # (division by a tensor: by a number the device multiplies with its rounded reciprocal)
            step = _grid8((most - lo) / torch.full_like(lo, 15), up=True)
            w = lo + torch.where(step > 0, ((w - lo) / step).round(), 0.0) * step
            y += x["x"][:, at:at + c["group"]].double() @ w
        return y
    B, H, D, page = c["B"], c["H"], c["D"], c["page"]
    held, new, tables = _lengths(c), _first_new(c), x["table"].long()
    if c["op"] == "evict":
        for b, n in enumerate(held):
            cut = n - c["keep"]
            if cut <= 0:
                continue
            s = torch.arange(n, device="cuda")
            pg, row = tables[b, s // page], s % page
            w, p = x["weight"][pg, row].tolist(), x["pos"][pg, row].tolist()
            gone = sorted((w[i], p[i], i) for i in range(n) if p[i] < new[b] - c["recent"])[:cut]
            gone = {i for _, _, i in gone}
            holes = [i for i in range(c["keep"]) if i in gone]
            stay = [i for i in range(c["keep"], n) if i not in gone]
            to, fr = (torch.tensor(t, dtype=torch.long, device="cuda") for t in (holes, stay))
            for t in ("k_pool", "v_pool"):
                x[t][pg[to], :, row[to]] = x[t][pg[fr], :, row[fr]]
            for t in ("pos", "weight"):
                x[t][pg[to], row[to]] = x[t][pg[fr], row[fr]]
            x["length"][b] = c["keep"]
        return [x["k_pool"], x["v_pool"], x["length"], x["next"], x["pos"], x["weight"]]
    counts = _counts(c)
    out = torch.zeros(B, c["T"], H, D, dtype=torch.float64, device="cuda")
    weight = x["weight"].double()
    for b, (n, t) in enumerate(zip(held, counts)):
        s = torch.arange(n, n + t, device="cuda")
        pg, row = tables[b, s // page], s % page
        x["k_pool"][pg, :, row], x["v_pool"][pg, :, row] = x["k"][b, :t], x["v"][b, :t]
        x["pos"][pg, row] = torch.arange(new[b], new[b] + t, device="cuda").int()
        weight[pg, row] = 0.0
        if c["op"] == "push" or not t:
            continue
        s = torch.arange(n + t, device="cuda")
        pg, row = tables[b, s // page], s % page
        age = torch.arange(new[b], new[b] + t, device="cuda")[:, None] - x["pos"][pg, row].long()
        reach = age.clamp(0, min(c["C"], x["r"].shape[0] - 1))
        for h in range(H):
            k, v = x["k_pool"][pg, h, row].double(), x["v_pool"][pg, h, row].double()
            q = x["q"][b, :t, h].double()
            content = torch.einsum("id,jd->ij", q + x["u"][h].double(), k)
            position = torch.einsum("id,nd->in", q + x["vb"][h].double(), x["r"][:, h, :D].double())
            a = (content + torch.gather(position, 1, reach)) * D ** -0.5
            p = torch.softmax(a.masked_fill(age < 0, -math.inf), -1)
            out[b, :t, h] = p @ v
            if c["weights"]:
                weight[pg, row] += p.sum(0)
    length, nxt = (x[n] + x["counts"] for n in ("length", "next"))
    return [*([out] if c["op"] == "step" else []), x["k_pool"], x["v_pool"], length, nxt, x["pos"], weight]
