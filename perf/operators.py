"""The quantised key/value memory and the relative attention that reads it: cases to measure.

Four kinds of pass, over a ring memory of M positions whose keys and values are held as 4- or 8-bit
codes (groups of 32 channels, each with a bf16 step and minimum):

  push     a segment of L positions is quantised into the ring, and those positions are read back
  read     n positions of the memory are read back in logical order
  decode   relative attention of 1..16 queries over [memory ++ segment] (generation)
  segment  the same for longer segments (evaluation, prompts)

Each pass exists in a plain form (elementary torch operations) and as calls of the package (`own`).
"""
import math

import torch

own = False

GROUP = 32


# ------------------------------------------------------------------------------------ cases
def listed():
    """Shapes of the package's workloads: generation (B8 H16 D64 over 4096 positions), the base
    shape (d_head 41, heads 48 apart), large, long memory, stream, and the tiny fp32 one."""
    return [
        # one generated token enters a long memory: launch latency
        dict(name="push token 4b", op="push", B=8, H=16, D=64, L=1, M=4096, valid=4096, wp=1001, bits=4, dtype="bf16",
             hs=64),
        # a training-length segment enters the memory
        dict(name="push large 4b", op="push", B=16, H=16, D=64, L=384, M=384, valid=384, wp=0, bits=4, dtype="bf16",
             hs=64),
        # the base shape's memory read back: odd d_head, padded heads, a wrapped ring
        dict(name="read base 8b", op="read", B=32, H=10, D=41, L=150, M=150, valid=150, wp=77, bits=8, dtype="bf16",
             hs=48),
        # a long d_head-128 memory read back
        dict(name="read stream 4b", op="read", B=4, H=16, D=128, L=2048, M=2048, valid=2048, wp=512, bits=4,
             dtype="bf16", hs=128),
        # the smallest call, in fp32
        dict(name="decode tiny f32 8b", op="decode", B=1, H=2, D=8, L=8, M=8, valid=8, wp=3, C=16, bits=8, dtype="f32",
             hs=8),
        # generation: one token per sequence, a long memory, distances clamped at 1000
        dict(name="decode token 4b", op="decode", B=8, H=16, D=64, L=1, M=4096, valid=4096, wp=1001, C=1000, bits=4,
             dtype="bf16", hs=64),
        dict(name="decode token 8b", op="decode", B=8, H=16, D=64, L=1, M=4096, valid=4096, wp=1001, C=1000, bits=8,
             dtype="bf16", hs=64),
        # one sequence with a very long memory, the position table as long as the memory
        dict(name="decode long 4b", op="decode", B=1, H=16, D=64, L=1, M=65536, valid=65536, wp=0, C=70000, bits=4,
             dtype="bf16", hs=64),
        # a few drafted tokens over the stream shape's memory, partly filled
        dict(name="decode draft 4b", op="decode", B=4, H=16, D=128, L=4, M=2048, valid=1900, wp=300, C=1000, bits=4,
             dtype="bf16", hs=128),
        # the most queries of a decode call, over the long-memory shape, distances not clamped
        dict(name="decode sixteen 8b", op="decode", B=8, H=16, D=64, L=16, M=1600, valid=1600, wp=37, C=2000, bits=8,
             dtype="bf16", hs=64),
        # a segment of the large shape over its memory
        dict(name="segment large 4b", op="segment", B=16, H=16, D=64, L=384, M=384, valid=384, wp=100, C=1000, bits=4,
             dtype="bf16", hs=64),
        # a segment of the long-memory shape
        dict(name="segment longmem 8b", op="segment", B=8, H=16, D=64, L=128, M=1600, valid=1600, wp=0, C=1000, bits=8,
             dtype="bf16", hs=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["push", "read", "decode", "decode", "decode", "segment"])
    D = rng.choice([8, 24, 32, 41, 64, 64, 64, 80, 96, 128, 128])
    hs = (D + 7) // 8 * 8 if rng.random() < 0.7 else D
    H = rng.randint(1, 16)
    bits = rng.choice([4, 4, 8])
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    c = dict(op=op, H=H, D=D, bits=bits, dtype=dtype, hs=hs)
    if op in ("push", "read"):
        c["B"] = _log(rng, 1, 32)
        room = max(1, 16 * 16 * 64 * 384 // (c["B"] * H * (256 if dtype == "f32" else 128)))
        c["L"] = _log(rng, 1, room)
        c["M"] = c["L"] + (rng.randint(0, 300) if rng.random() < 0.5 else 0)
        c["valid"] = c["M"] if op == "push" else rng.randint(c["L"], c["M"])
    elif op == "decode":
        c["L"] = rng.choice([1, 1, 1, 2, 3, 4, 5, 7, 8, 11, 16])
        c["B"] = _log(rng, 1, 16)
        room = max(64, 65536 * 16 * 64 // (c["B"] * H * max(D, 32) * (1 if c["L"] <= 4 and dtype != "f32" else 4)))
        c["M"] = _log(rng, 8, min(room, 40000))
        c["valid"] = c["M"] if rng.random() < 0.6 else rng.randint(0, c["M"])
        c["C"] = rng.choice([200, 1000, 1000, c["M"] + c["L"]])
    else:
        c["L"] = _log(rng, 17, 400)
        c["M"] = _log(rng, 16, 1500)
        c["B"] = _log(rng, 1, max(1, min(8, 2500000000 // (H * c["L"] * (c["M"] + c["L"]) * D))))
        c["valid"] = c["M"] if rng.random() < 0.6 else rng.randint(0, c["M"])
        c["C"] = rng.choice([200, 1000, c["M"] + c["L"]])
        if dtype == "f32":
            c["L"], c["B"] = min(c["L"], 128), min(c["B"], 2)
    c["wp"] = rng.randint(0, c["M"] - 1)
    return c


def work(c):
    B, H, D, L, M = c["B"], c["H"], c["D"], c["L"], c["M"]
    e = 4 if c["dtype"] == "f32" else 2
    G = (D + GROUP - 1) // GROUP
    row = 2 * (G * GROUP * c["bits"] // 8 + 4 * G)          # codes and parameters of a position's K and V
    if c["op"] == "push":                                   # read k, v; write codes; write them read back
        return {"bytes": B * H * L * (2 * D * e + row + 2 * D * e), "flops": 8 * B * H * L * D}
    if c["op"] == "read":
        return {"bytes": B * H * L * (row + 2 * D * e), "flops": 4 * B * H * L * D}
    n_rows = min(M + L, c["C"] + 1)
    pairs = L * c["valid"] + L * (L + 1) // 2
    return {"bytes": B * H * c["valid"] * row + H * n_rows * D * e + 4 * B * H * L * D * e,
            "flops": 6 * B * H * pairs * D}


# ------------------------------------------------------------------------------------ inputs
def _dtype(c):
    return torch.float32 if c["dtype"] == "f32" else torch.bfloat16


def _tensor(c, gen, T):
    """[B, T, H, D] ~ N(0, 1) with heads `hs` elements apart."""
    store = torch.empty(c["B"], T, c["H"], c["hs"], dtype=_dtype(c), device="cuda")
    for b in range(c["B"]):
        store[b] = torch.randn(T, c["H"], c["hs"], generator=gen, device="cuda")
    return store[..., : c["D"]]


def _inputs(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, H, D, L, M = c["B"], c["H"], c["D"], c["L"], c["M"]
    x = {}
    if c["op"] != "push":
        # the positions the memory holds, oldest first; some channels larger than the others
        gain = 0.5 + torch.rand(H, D, generator=gen, device="cuda") * 1.5
        for n in ("k_hist", "v_hist"):
            x[n] = _tensor(c, gen, c["valid"])
            x[n].mul_(gain.to(x[n].dtype))
    if c["op"] != "read":
        x["k"], x["v"] = _tensor(c, gen, L), _tensor(c, gen, L)
    if c["op"] in ("decode", "segment"):
        x["q"] = _tensor(c, gen, L)
        x["u"] = 0.02 * torch.randn(H, D, generator=gen, device="cuda")
        x["vb"] = 0.02 * torch.randn(H, D, generator=gen, device="cuda")
        # r = R W_R for distances 0 .. n_rows-1, R the interleaved sinusoid
        n_rows, dm = min(M + L, c["C"] + 1), 128
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
    B, H, D, M = c["B"], c["H"], c["D"], c["M"]
    s = dict(c=c, x=x)
    if own:
        import transformer_xl_relative_gb300 as txl
        s["txl"] = txl
        mem = txl.QuantMemory.empty(B, M, H, D, bits=c["bits"])
        mem.restore((c["wp"] - c["valid"]) % M, 0)
        if c["op"] == "push":
            mem.restore(c["wp"], c["valid"])
        elif c["valid"]:
            txl.qmem_push(mem, x["k_hist"], x["v_hist"])
        s["mem"] = mem
        if c["op"] in ("push", "read"):
            s["out"] = torch.empty(2, B, c["L"], H, D, dtype=_dtype(c), device="cuda")
        else:
            s["out"] = torch.zeros(B, c["L"], H, c["hs"], dtype=_dtype(c), device="cuda")[..., :D]
            need = txl.rel_attn_qmem_workspace_size(x["q"], mem)
            s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    else:
        G = (D + GROUP - 1) // GROUP
        s["ring"] = {n: (torch.zeros(B, H, M, G * GROUP * c["bits"] // 8, dtype=torch.uint8, device="cuda"),
                         torch.zeros(B, H, M, G, 2, dtype=torch.bfloat16, device="cuda")) for n in "kv"}
        if c["op"] != "push":
            slots = _slots(c, M - c["valid"], c["valid"])
            for n in "kv":
                _store(s["ring"][n], slots, x[n + "_hist"], c["bits"])
    return s


# ------------------------------------------------------------------------------------ plain form
def _slots(c, j0, n, wp=None):
    """Slots of the logical positions j0 .. j0+n-1 of the ring."""
    return ((c["wp"] if wp is None else wp) + j0 + torch.arange(n, device="cuda")) % c["M"]


def _bf16_toward(x, up):
    """x (fp32) rounded to bf16 toward +inf (up) or -inf."""
    bits = x.view(torch.int32)
    cut = bits & -65536
    t = cut.view(torch.float32)
    away = (t < x) if up else (t > x)
    return torch.where(away, (cut + 65536).view(torch.float32), t).bfloat16()


def _quantise(x, bits):
    """[..., D] -> codes (uint8 [..., G*32], zeros past D) and (step, lo) bf16 [..., G, 2]."""
    n, D = 2 ** bits - 1, x.shape[-1]
    G = (D + GROUP - 1) // GROUP
    x = torch.nn.functional.pad(x.float(), (0, G * GROUP - D), value=math.nan).unflatten(-1, (G, GROUP))
    pad = torch.isnan(x)
    lo = _bf16_toward(torch.where(pad, math.inf, x).amin(-1), up=False)
    span = torch.where(pad, -math.inf, x).amax(-1).double() - lo.double()
    step = _bf16_toward((span / n).float(), up=True)
    # quotient and conversion were rounded: one bf16 up or down where that crossed the exact value
    bits_of = step.view(torch.int16)
    step = torch.where(step.double() * n < span, (bits_of + 1).view(torch.bfloat16), step)
    less = (step.view(torch.int16) - 1).clamp(min=0).view(torch.bfloat16)
    step = torch.where(less.double() * n >= span, less, step)
    d = x.double() - lo.double()[..., None]
    code = torch.round(d / step.double()[..., None])
    code = torch.where(pad | (step == 0)[..., None], 0.0, code).to(torch.uint8)
    return code.flatten(-2), torch.stack((step, lo), -1)


def _store(ring, slots, x, bits):
    """Quantise x [B, n, H, D] into the slots of a ring (packed codes, parameters)."""
    for b in range(x.shape[0]):
        code, par = _quantise(x[b].transpose(0, 1), bits)
        if bits == 4:
            code = code[..., 0::2] | (code[..., 1::2] << 4)
        ring[0][b, :, slots] = code
        ring[1][b, :, slots] = par


def _load(ring, slots, D, bits):
    """The values the slots stand for, fp32 [B, H, n, D]."""
    code, par = ring[0][:, :, slots], ring[1][:, :, slots].float()
    if bits == 4:
        code = torch.stack((code & 15, code >> 4), -1).flatten(-2)
    x = code.float().unflatten(-1, (-1, GROUP)) * par[..., 0:1] + par[..., 1:2]
    return x.flatten(-2)[..., :D]


def _attend_plain(c, q, k, v, u, vb, r):
    """Relative attention of q [B, L, H, D] over keys k, v fp32 [B, H, K, D] (the last L the
    segment's own), all visible but those after the query."""
    D, L, K = c["D"], c["L"], k.shape[2]
    q = q.float().transpose(1, 2)
    dist = (K - L) + torch.arange(L, device="cuda")[:, None] - torch.arange(K, device="cuda")
    row = dist.clamp(0, c["C"])
    bd = (q + vb[:, None]) @ r[..., :D].float().permute(1, 2, 0)
    s = (q + u[:, None]) @ k.transpose(-1, -2) + bd.gather(-1, row.expand(*bd.shape[:2], L, K))
    s = torch.where(dist < 0, -math.inf, s / math.sqrt(D))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    return ((p @ v) / p.sum(-1, keepdim=True)).transpose(1, 2).to(_dtype(c))


def run(state):
    c, x = state["c"], state["x"]
    return _run_own(state, c, x) if own else _run_plain(state, c, x)


def _run_plain(state, c, x):
    ring, D, bits = state["ring"], c["D"], c["bits"]
    if c["op"] == "push":
        slots = _slots(c, 0, c["L"])
        for n in "kv":
            _store(ring[n], slots, x[n], bits)
        return torch.stack([_load(ring[n], slots, D, bits).transpose(1, 2).to(_dtype(c)) for n in "kv"])
    if c["op"] == "read":
        slots = _slots(c, c["M"] - c["L"], c["L"])
        return torch.stack([_load(ring[n], slots, D, bits).transpose(1, 2).to(_dtype(c)) for n in "kv"])
    slots = _slots(c, c["M"] - c["valid"], c["valid"])
    k, v = (torch.cat((_load(ring[n], slots, D, bits), x[n].float().transpose(1, 2)), 2) for n in "kv")
    return _attend_plain(c, x["q"], k, v, x["u"], x["vb"], x["r"])


def _run_own(state, c, x):
    txl, mem, out = state["txl"], state["mem"], state["out"]
    if c["op"] == "push":
        mem.restore(c["wp"], c["valid"])                    # the same slots on every pass
        txl.qmem_push(mem, x["k"], x["v"])
        txl.qmem_read(mem, c["M"] - c["L"], c["L"], out[0], out[1])
        return out
    if c["op"] == "read":
        txl.qmem_read(mem, c["M"] - c["L"], c["L"], out[0], out[1])
        return out
    return txl.rel_attn_qmem(x["q"], mem, x["k"], x["v"], x["u"], x["vb"], x["r"], x["r"].shape[0], c["C"], out,
                             workspace=state["ws"])


# ------------------------------------------------------------------------------------ 64 bits
def _grid8(x, up):
    """x >= 0 to 8 significant bits, up or down (bf16's subnormals apart); fp64."""
    m, e = torch.frexp(x)
    unit = ((e.long() - 8 + 1023) << 52).view(torch.float64)      # 2^(e-8), exactly
    return (torch.ceil(m * 256.0) if up else torch.floor(m * 256.0)) * unit


def _held(x, bits):
    """What the memory holds for x [B, n, H, D]: every group of 32 channels on its grid, fp64."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    n = 2 ** bits - 1
    for d0 in range(0, x.shape[-1], GROUP):
        g = x[..., d0:d0 + GROUP].double()
        least, most = torch.aminmax(g, dim=-1, keepdim=True)
        lo = torch.where(least < 0, -_grid8(-least, up=True), _grid8(least, up=False))
        # (division by a tensor: by a number the device multiplies with its rounded reciprocal)
        step = _grid8((most - lo) / torch.full_like(lo, n), up=True)
        at = torch.where(step > 0, ((g - lo) / step).round(), 0.0)
        out[..., d0:d0 + GROUP] = lo + at * step
    return out


def exact(case, seed):
    c, x = case, _inputs(case, seed)
    if c["op"] == "push":
        return torch.stack([_held(x[n], c["bits"]) for n in "kv"])
    if c["op"] == "read":
        return torch.stack([_held(x[n][:, c["valid"] - c["L"]:], c["bits"]) for n in ("k_hist", "v_hist")])
    B, H, D, L, C = c["B"], c["H"], c["D"], c["L"], c["C"]
    K = c["valid"] + L
    out = torch.empty(B, L, H, D, dtype=torch.float64, device="cuda")
    i, j = torch.arange(L, device="cuda")[:, None], torch.arange(K, device="cuda")[None]
    delta = c["valid"] + i - j
    hidden = delta < 0
    delta = delta.clamp(0, C)
    for b in range(B):
        k = torch.cat((_held(x["k_hist"][b:b + 1], c["bits"])[0], x["k"][b].double()))
        v = torch.cat((_held(x["v_hist"][b:b + 1], c["bits"])[0], x["v"][b].double()))
        for h in range(H):
            q = x["q"][b, :, h].double()
            content = torch.einsum("id,jd->ij", q + x["u"][h].double(), k[:, h])
            position = torch.einsum("id,nd->in", q + x["vb"][h].double(), x["r"][:, h, :D].double())
            s = (content + torch.gather(position, 1, delta)) * D ** -0.5
            out[b, :, h] = torch.softmax(s.masked_fill(hidden, -math.inf), -1) @ v[:, h]
    return out
