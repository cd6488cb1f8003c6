"""The measured cases of the operators around the grouped (mixture-of-experts)
products: tokens sorted by expert and back with their gradients, the gated
activation with its 8-bit checkpoint, and the checkpoint by itself.

`run` computes a case in plain torch where `own` is false and through the
framework's binding where it is true; `exact` is the definition in 64 bits.

The kinds of case, one pass each:
  route        expert ids -> the sort's plan, and the tokens in expert order;
  combine      expert outputs back in token order, weighted (or a plain sum:
               the gradient of the dispatch);
  combine_bwd  gradients of the expert outputs and of the weights;
  ckpt         a tensor saved in 8 bits and restored;
  gated        silu(gate) * up forward, its inputs kept in 8 bits, and the
               backward pass from those.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
BLOCK = 32


def listed():
    return [
        # one token of a decoding step through the 64-expert layer: latency alone
        dict(name="route_token", kind="route", tokens=1, topk=6, experts=64, hidden=2048, x="bf16", ids="int64",
             dropped=0.0),
        # the training step of the 64-expert, top-6 layer
        dict(name="route_step", kind="route", tokens=16384, topk=6, experts=64, hidden=2048, x="bf16", ids="int64",
             dropped=0.0),
        # a long batch of wide tokens over the most experts, some of its tokens padding (no expert)
        dict(name="route_long", kind="route", tokens=65536, topk=2, experts=256, hidden=8192, x="bf16", ids="int32",
             dropped=0.04),
        # a small uneven batch, rows of odd length, bf16 expert outputs
        dict(name="combine_ragged", kind="combine", tokens=1021, topk=8, experts=64, hidden=1001, y="bf16",
             out="fp32", weighted=True, dropped=0.1),
        # the training step's way back: fp32 products of the grouped GEMM to the bf16 stream
        dict(name="combine_step", kind="combine", tokens=16384, topk=6, experts=64, hidden=2048, y="fp32", out="bf16",
             weighted=True, dropped=0.0),
        # the dispatch's gradient: the sum over a token's experts, without weights
        dict(name="dispatch_grad", kind="combine", tokens=8192, topk=4, experts=32, hidden=4096, y="fp32", out="fp32",
             weighted=False, dropped=0.02),
        # a short sequence's backward pass
        dict(name="combine_bwd_short", kind="combine_bwd", tokens=128, topk=6, experts=64, hidden=2048, y="fp32",
             dout="bf16", dy="bf16", dropped=0.0),
        # the training step's backward pass
        dict(name="combine_bwd_step", kind="combine_bwd", tokens=16384, topk=6, experts=64, hidden=2048, y="fp32",
             dout="bf16", dy="bf16", dropped=0.01),
        # a small activation, rows that end inside a block
        dict(name="ckpt_small", kind="ckpt", rows=256, cols=1000, x="fp32", fmt="e4m3"),
        # the widest activation of the dense configurations
        dict(name="ckpt_wide", kind="ckpt", rows=65536, cols=8192, x="bf16", fmt="int8"),
        # a few hundred routed tokens through narrow experts
        dict(name="gated_short", kind="gated", rows=493, cols=1408, x="bf16", h="bf16", dh="fp32", dx="fp32",
             fmt="e4m3"),
        # all routed tokens of the training step: fp32 products in, bf16 operands out
        dict(name="gated_step", kind="gated", rows=98304, cols=1408, x="fp32", h="bf16", dh="fp32", dx="bf16",
             fmt="int8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        t = lambda: rng.choice(["bf16", "fp32"])  # noqa: E731
        kind = rng.choice(["route", "combine", "combine_bwd", "ckpt", "gated"])
        if kind in ("ckpt", "gated"):
            c = dict(kind=kind, rows=_log(rng, 1, 131072), cols=_log(rng, 16, 8192), x=t(),
                     fmt=rng.choice(["int8", "e4m3"]))
            if kind == "gated":
                c.update(h=t(), dh=t(), dx=t())
        else:
            experts = _log(rng, 2, 256)
            c = dict(kind=kind, tokens=_log(rng, 1, 65536), topk=rng.randint(1, min(8, experts)), experts=experts,
                     hidden=_log(rng, 16, 8192), dropped=round(rng.choice([0.0, rng.uniform(0.0, 0.2)]), 3))
            if kind == "route":
                c.update(x=t(), ids=rng.choice(["int32", "int64"]))
            elif kind == "combine":
                c.update(y=t(), out=t(), weighted=rng.random() < 0.7)
            else:
                c.update(y=t(), dout=t(), dy=t())
        # most sizes are those of models (multiples of 16), some are not
        for n in ("hidden", "cols"):
            if n in c and rng.random() < 0.6:
                c[n] = (c[n] + 15) // 16 * 16
        if work(c)["bytes"] <= most:
            return c


def work(case):
    """Bytes of inputs read once and outputs written once (a checkpoint is
    written by the forward and read by the backward), and flops."""
    if case["kind"] in ("ckpt", "gated"):
        n = case["rows"] * case["cols"]
        kept = n + case["rows"] * -(-case["cols"] // BLOCK)
        s = SIZE[case["x"]]
        if case["kind"] == "ckpt":
            return {"bytes": 2 * n * s + 2 * kept, "flops": 4 * n}
        return {"bytes": n * (2 * s + SIZE[case["h"]] + SIZE[case["dh"]] + 2 * SIZE[case["dx"]]) + 4 * kept,
                "flops": 20 * n}
    t, h = case["tokens"], case["hidden"]
    n = t * case["topk"]
    if case["kind"] == "route":
        return {"bytes": n * (4 if case["ids"] == "int32" else 8) + (t + n) * h * SIZE[case["x"]] + 8 * n +
                16 * case["experts"], "flops": 0}
    if case["kind"] == "combine":
        return {"bytes": n * h * SIZE[case["y"]] + t * h * SIZE[case["out"]] + n * (8 if case["weighted"] else 4),
                "flops": 2 * n * h}
    return {"bytes": n * h * (SIZE[case["y"]] + SIZE[case["dy"]]) + t * h * SIZE[case["dout"]] + 12 * n,
            "flops": 3 * n * h}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _routing(case, g):
    """Each token's experts (distinct, of a skewed distribution) and weights;
    a `dropped` part of the tokens is padding and goes nowhere (id -1)."""
    t, k, e = case["tokens"], case["topk"], case["experts"]
    popular = torch.randn(e, generator=g, device="cuda")
    u = torch.rand(t, e, generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
    logits = popular - torch.log(-torch.log(u))
    top, ids = torch.topk(logits, k, dim=1)
    weights = torch.softmax(top, dim=1)
    if case["dropped"] > 0:
        ids = torch.where((torch.rand(t, generator=g, device="cuda") < case["dropped"])[:, None], -1, ids)
    return ids, weights


def _plan(ids, experts):
    """The stable counting sort of the slots by expert: place of each slot,
    slot of each place, counts and offsets (dropped slots last)."""
    n = ids.numel()
    e = ids.reshape(-1).to(torch.int64)
    e = torch.where((e < 0) | (e >= experts), experts, e)
    hit = e[None, :] == torch.arange(experts + 1, device=e.device)[:, None]
    counts = hit.sum(1)
    start = counts.cumsum(0) - counts
    before = hit.to(torch.int32).cumsum(1, dtype=torch.int32)
    slot = torch.arange(n, device=e.device)
    pos = start[e] + before[e, slot] - 1
    src = torch.empty(n, dtype=torch.int32, device=e.device)
    src[pos] = slot.to(torch.int32)
    offsets = torch.cat([start, start.new_tensor([n])])
    return {"pos": pos.to(torch.int32).view(ids.shape), "src": src, "counts": counts[:experts],
            "offsets": offsets[:experts + 1].contiguous()}


def prepare(case, seed):
    g, kind = _gen(seed), case["kind"]
    s = {"case": case}
    if kind in ("ckpt", "gated"):
        shape = (case["rows"], case["cols"])
        # rows of differing size and a few columns far above the others
        scale = torch.exp2(torch.randint(-3, 3, (case["rows"], 1), generator=g, device="cuda").float())
        heavy = torch.where(torch.rand(case["cols"], generator=g, device="cuda") < 0.002, 20.0, 1.0)
        make = lambda: _normal(g, shape, 1.0, torch.float32).mul_(scale).mul_(heavy).to(DTYPES[case["x"]])  # noqa: E731
        if kind == "ckpt":
            s["x"] = make()
        else:
            s["gate"], s["up"] = make(), make()
            s["dh"] = _normal(g, shape, 1e-3, DTYPES[case["dh"]])
        return s
    t, h = case["tokens"], case["hidden"]
    n = t * case["topk"]
    ids, weights = _routing(case, g)
    if kind == "route":
        s["ids"] = ids.to(torch.int32) if case["ids"] == "int32" else ids
        s["x"] = _normal(g, (t, h), 1.0, DTYPES[case["x"]])
        return s
    # what the sort of the forward pass left
    s["plan"] = _plan(ids, case["experts"])
    s["weights"] = weights
    s["y"] = _normal(g, (n, h), 1.0, DTYPES[case["y"]])
    if kind == "combine_bwd":
        s["dout"] = _normal(g, (t, h), 1e-3, DTYPES[case["dout"]])
    return s


# -------------------------------------------------------------- plain forms
def _cut(x, fmt):
    """x through 8 bits and back, fp32: one power-of-two scale per 32
    elements of a row."""
    rows, cols = x.shape
    pad = -cols % BLOCK
    v = torch.nn.functional.pad(x.float(), (0, pad)).view(rows, -1, BLOCK)
    bits = v.abs().amax(-1, keepdim=True).contiguous().view(torch.int32)
    b = (bits >> 23) - (6 if fmt == "int8" else 8)
    if fmt == "e4m3":
        b = b + ((bits & 0x7FFFFF) > 0x600000)
    b = b.clamp(0, 248 if fmt == "int8" else 246)            # restored values stay finite in fp32
    v = v * ((254 - b) << 23).view(torch.float32)            # 2^(127 - b)
    v = v.round().clamp(-127, 127) if fmt == "int8" else v.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    v = v * torch.where(b > 0, b << 23, 0x400000).view(torch.float32)
    return v.view(rows, -1)[:, :cols]


def _run_plain(s):
    case, kind = s["case"], s["case"]["kind"]
    if kind == "ckpt":
        return {"x": _cut(s["x"], case["fmt"]).to(s["x"].dtype)}
    if kind == "gated":
        gate, up = s["gate"].float(), s["up"].float()
        h = (gate / (1 + torch.exp(-gate)) * up).to(DTYPES[case["h"]])
        gate, up, dh = _cut(gate, case["fmt"]), _cut(up, case["fmt"]), s["dh"].float()
        sig = 1 / (1 + torch.exp(-gate))
        out = DTYPES[case["dx"]]
        return {"h": h, "dgate": (dh * up * sig * (1 + gate * (1 - sig))).to(out), "dup": (dh * gate * sig).to(out)}
    if kind == "route":
        p = _plan(s["ids"], case["experts"])
        routed = torch.arange(p["src"].numel(), device="cuda")[:, None] < p["offsets"][-1]
        p["xs"] = torch.where(routed, s["x"][(p["src"] // case["topk"]).long()], 0)
        return p
    p = s["plan"]
    pos = p["pos"].long()
    routed = pos < p["offsets"][-1]
    y = torch.where(routed[:, :, None], s["y"][pos].float(), 0.0)
    if kind == "combine":
        if case["weighted"]:
            y = y * s["weights"][:, :, None]
        return {"out": y.sum(1).to(DTYPES[case["out"]])}
    dout = s["dout"].float()[:, None, :]
    w = torch.where(routed, s["weights"], 0.0)
    dy = torch.empty(s["y"].shape, dtype=DTYPES[case["dy"]], device="cuda")
    dy[pos] = (w[:, :, None] * dout).to(dy.dtype)
    return {"dy": dy, "dw": (dout * y).sum(2)}


# --------------------------------------------------- the framework's kernels
def _run_own(s):
    from fp4_quantized_numerics_gb300 import ufp4 as U
    case, kind = s["case"], s["case"]["kind"]
    if kind in ("ckpt", "gated"):
        fmt = U.UFP4_CKPT_INT8 if case["fmt"] == "int8" else U.UFP4_CKPT_E4M3
        if kind == "ckpt":
            return {"x": U.ufp4_ckpt_load(U.ufp4_ckpt_save(s["x"], fmt), dtype=s["x"].dtype)}
        h, kept_gate, kept_up = U.ufp4_swiglu(s["gate"], s["up"], ckpt=fmt, dtype=DTYPES[case["h"]])
        dgate, dup = U.ufp4_swiglu_bwd(s["dh"], kept_gate, kept_up, dtype=DTYPES[case["dx"]])
        return {"h": h, "dgate": dgate, "dup": dup}
    if kind == "route":
        p = U.ufp4_moe_sort(s["ids"], case["experts"])
        return {"pos": p.pos, "src": p.src, "counts": p.counts, "offsets": p.offsets,
                "xs": U.ufp4_moe_dispatch(s["x"], p)}
    p = U.MoePlan(**s["plan"])
    if kind == "combine":
        w = s["weights"] if case["weighted"] else None
        return {"out": U.ufp4_moe_combine(s["y"], p, w, dtype=DTYPES[case["out"]])}
    dy, dw = U.ufp4_moe_combine_bwd(s["dout"], s["y"], p, s["weights"], dtype=DTYPES[case["dy"]])
    return {"dy": dy, "dw": dw}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------- in 64 bits
def _grid(x, fmt):
    """The 8-bit values nearest to x, block by block, in 64 bits: spacing of
    the grid at each element by its own and its block's binary exponent."""
    rows, cols = x.shape
    out = torch.empty(rows, cols, dtype=torch.float64, device=x.device)
    for c in range(0, cols, BLOCK):
        v = x[:, c:c + BLOCK].double()
        top = v.abs().amax(1, keepdim=True)
        m, e = torch.frexp(top)                              # top = m 2^e, m in [1/2, 1)
        e = e.double() - 1
        if fmt == "int8":
            step = torch.exp2(torch.clamp(e - 6, min=-127.0))
            q = torch.clamp(torch.round(v / step), -127, 127) * step
        else:
            unit = torch.exp2(torch.clamp(e - 8 + (2 * m > 1.75), min=-127.0, max=119.0))
            r = torch.clamp(v / unit, -448, 448)             # 3 bits behind the leading one, 2^-9 at least
            own_e = torch.clamp(torch.frexp(r)[1].double() - 1, min=-6.0)
            step = torch.exp2(own_e - 3)
            q = torch.round(r / step) * step * unit
        out[:, c:c + BLOCK] = torch.where(top > 0, q, 0.0)
    return out


def exact(case, seed):
    s, kind = prepare(case, seed), case["kind"]
    if kind == "ckpt":
        return {"x": _grid(s["x"], case["fmt"])}
    if kind == "gated":
        gate, up = s["gate"].double(), s["up"].double()
        h = gate * torch.sigmoid(gate) * up
        gate, up, dh = _grid(s["gate"], case["fmt"]), _grid(s["up"], case["fmt"]), s["dh"].double()
        sig = torch.sigmoid(gate)
        dup = gate.mul(sig).mul_(dh)
        dgate = (sig + gate * sig * torch.sigmoid(-gate)).mul_(up).mul_(dh)
        return {"h": h, "dgate": dgate, "dup": dup}
    k, e = case["topk"], case["experts"]
    if kind == "route":
        ids = s["ids"].cpu().numpy().reshape(-1).astype(np.int64)
        ids = np.where((ids < 0) | (ids >= e), e, ids)
        src = np.argsort(ids, kind="stable")
        pos = np.empty_like(src)
        pos[src] = np.arange(src.size)
        ends = np.cumsum(np.bincount(ids, minlength=e + 1)[:e])
        xs = s["x"][torch.from_numpy(src // k).cuda()].double()
        xs[int(ends[-1]):] = 0
        return {"pos": pos.reshape(s["ids"].shape), "src": src, "counts": np.diff(ends, prepend=0),
                "offsets": np.concatenate([[0], ends]), "xs": xs}
    # over the sorted rows, not over the tokens
    p = s["plan"]
    routed = int(p["offsets"][-1])
    src = p["src"].long()[:routed]
    token = src // k
    if kind == "combine":
        y = s["y"][:routed].double()
        if case["weighted"]:
            y = y.mul_(s["weights"].reshape(-1)[src].double()[:, None])
        out = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device="cuda")
        return {"out": out.index_add_(0, token, y)}
    dout, w = s["dout"].double(), s["weights"].reshape(-1).double()
    dy = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros_like(w)
    for a in range(0, routed, 1 << 15):
        at = slice(a, min(routed, a + (1 << 15)))
        d = dout[token[at]]
        dy[at] = w[src[at]][:, None] * d
        dw[src[at]] = torch.einsum("ph,ph->p", d, s["y"][at].double())
    return {"dy": dy, "dw": dw.view(s["weights"].shape)}
