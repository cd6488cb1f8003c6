"""The measured cases of the operators that answer with a model held in 4 bits:
products of a few tokens with quantised weights (dense, and by expert), a cache
of keys and values quantised as it is written, and the attention of new tokens
(one, a run or a tree of drafted ones a sequence) over it.

`run` computes a case in plain torch where `own` is false and through the
framework's binding where it is true; `exact` is the definition in 64 bits.

The kinds of case, one pass each:
  gemv     tokens times a quantised matrix;
  experts  routed tokens times their experts' quantised matrices, with the plan
           of the sort at hand;
  cache    keys and values of new tokens written to the cache, and read back;
  attn     the attention of the new tokens over the cache.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
QMAX = {"e2m1": 6.0, "e1m2": 3.5}
GRID = {"e2m1": 0, "e1m2": 1}
VALUES = {"e2m1": [0, 0.5, 1, 1.5, 2, 3, 4, 6], "e1m2": [0, 0.5, 1, 1.5, 2, 2.5, 3, 3.5]}
SEED = 2                                 # of the rotation's signs


def listed():
    return [
        # one token through a square projection: latency alone
        dict(name="gemv_token", kind="gemv", tokens=1, rows=2048, k=2048, grid="e1m2", rht=True, x="bf16", out="bf16"),
        # a few sequences through the dense layer's first product, all in fp32
        dict(name="gemv_few", kind="gemv", tokens=4, rows=5632, k=2048, grid="e2m1", rht=True, x="fp32", out="fp32"),
        # sizes that fill no tile, inner dimension off the 64 of the packed layout
        dict(name="gemv_odd", kind="gemv", tokens=13, rows=1001, k=1040, grid="e1m2", rht=False, x="bf16", out="fp32"),
        # the largest matrix of a model, a vocabulary's, for one token
        dict(name="gemv_vocabulary", kind="gemv", tokens=1, rows=131072, k=8192, grid="e2m1", rht=False, x="bf16",
             out="fp32"),
        # one token through its 6 of 64 experts, read where it lies (not sorted)
        dict(name="experts_token", kind="experts", tokens=1, topk=6, experts=64, rows=2816, k=2048, grid="e1m2",
             rht=True, x="bf16", out="bf16", gather=True, dropped=0.0),
        # a batch of sequences: the second product, from sorted rows, some of them padding
        dict(name="experts_batch", kind="experts", tokens=64, topk=6, experts=64, rows=2048, k=1408, grid="e1m2",
             rht=True, x="bf16", out="fp32", gather=False, dropped=0.05),
        # a step of 64 sequences written and read
        dict(name="cache_step", kind="cache", tokens=64, heads=8, dim=128, page=64, grid="e1m2", rht=True, x="bf16",
             out="bf16", skipped=0.0),
        # long prompts written and read, in the other grid
        dict(name="cache_prompt", kind="cache", tokens=32768, heads=8, dim=128, page=64, grid="e2m1", rht=False,
             x="fp32", out="fp32", skipped=0.02),
        # one short sequence: latency alone
        dict(name="attn_token", kind="attn", batch=1, m=1, tree=False, heads=32, kv=8, dim=128, page=64, ctx=1000,
             idle=0, grid="e1m2", rht=True, x="bf16", out="bf16"),
        # a batch of sequences of differing length, a token each
        dict(name="attn_batch", kind="attn", batch=32, m=1, tree=False, heads=64, kv=8, dim=128, page=64, ctx=8192,
             idle=1, grid="e1m2", rht=True, x="bf16", out="bf16"),
        # one very long sequence, one token
        dict(name="attn_long", kind="attn", batch=1, m=1, tree=False, heads=32, kv=4, dim=128, page=64, ctx=262111,
             idle=0, grid="e2m1", rht=False, x="fp32", out="fp32"),
        # trees of 32 drafted tokens
        dict(name="attn_tree", kind="attn", batch=8, m=32, tree=True, heads=32, kv=8, dim=128, page=64, ctx=16384,
             idle=0, grid="e1m2", rht=True, x="bf16", out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    every = [work(c) for c in listed()]
    most = {n: max(w[n] for w in every) for n in ("bytes", "flops")}
    while True:
        t = lambda: rng.choice(["bf16", "fp32"])  # noqa: E731
        kind = rng.choice(["gemv", "experts", "cache", "attn"])
        c = dict(kind=kind, grid=rng.choice(["e2m1", "e1m2"]), rht=rng.random() < 0.6, x=t(), out=t())
        if kind in ("gemv", "experts"):
            c["k"] = 16 * _log(rng, 4, 1024)
            if kind == "gemv":
                c.update(tokens=_log(rng, 1, 64), rows=_log(rng, 16, 65536))
            else:
                experts = _log(rng, 2, 128)
                c.update(experts=experts, topk=rng.randint(1, min(8, experts)), tokens=_log(rng, 1, 128),
                         rows=_log(rng, 64, 4096), gather=rng.random() < 0.5,
                         dropped=round(rng.choice([0.0, rng.uniform(0.0, 0.2)]), 3))
            # most sizes are those of models, some are not
            if rng.random() < 0.6:
                c["rows"], c["k"] = (c["rows"] + 127) // 128 * 128, (c["k"] + 63) // 64 * 64
        else:
            c.update(dim=rng.choice([64, 80, 128, 128, 256]), page=rng.choice([16, 32, 64, 128]))
            if kind == "cache":
                c.update(tokens=_log(rng, 1, 65536), heads=rng.randint(1, 16),
                         skipped=round(rng.choice([0.0, rng.uniform(0.0, 0.1)]), 3))
            else:
                kv, batch = rng.randint(1, 16), _log(rng, 1, 64)
                c.update(kv=kv, heads=kv * rng.randint(1, 8), batch=batch, m=rng.choice([1, 1, _log(rng, 2, 64)]),
                         tree=rng.random() < 0.5, ctx=_log(rng, 64, 131072),
                         idle=0 if batch == 1 else rng.randint(0, batch // 4))
        w = work(c)
        if c.get("experts", 0) * c.get("rows", 0) * c["k" if "k" in c else "dim"] > 1 << 29:
            continue
        if all(w[n] <= most[n] for n in most):
            return c


def _lens(case):
    """Lengths of the sequences, the new tokens included (in no order)."""
    live = case["batch"] - case["idle"]
    n = case["ctx"] - (np.arange(live) * (case["ctx"] // 2)) // live
    return np.concatenate([np.maximum(n, case["m"]), np.zeros(case["idle"], dtype=np.int64)])


def _row_bytes(dim):
    """A row of the cache: codes, block scales, its own scale."""
    return dim / 2 + dim / 16 + 4


def work(case):
    """Bytes of inputs read once and outputs written once, and flops."""
    if case["kind"] == "gemv":
        t, n, k = case["tokens"], case["rows"], case["k"]
        return {"bytes": n * k * 0.5625 + t * k * SIZE[case["x"]] + t * n * SIZE[case["out"]], "flops": 2 * t * n * k}
    if case["kind"] == "experts":
        slots = case["tokens"] * case["topk"]
        # experts that some token goes to, were they all as likely
        used = case["experts"] * (1 - (1 - case["topk"] / case["experts"]) ** case["tokens"])
        read = (case["tokens"] if case["gather"] else slots) * case["k"] * SIZE[case["x"]]
        return {"bytes": used * case["rows"] * case["k"] * 0.5625 + read + slots * case["rows"] * SIZE[case["out"]],
                "flops": 2 * slots * case["rows"] * case["k"]}
    if case["kind"] == "cache":
        rows = 2 * case["tokens"] * case["heads"]
        return {"bytes": rows * (case["dim"] * (SIZE[case["x"]] + SIZE[case["out"]]) + 2 * _row_bytes(case["dim"])) +
                16 * case["tokens"], "flops": 8 * rows * case["dim"]}
    seen = int(_lens(case).sum())
    io = case["batch"] * case["m"] * case["heads"] * (case["dim"] * (SIZE[case["x"]] + SIZE[case["out"]]) + 4)
    return {"bytes": 2 * seen * case["kv"] * _row_bytes(case["dim"]) + io,
            "flops": 4 * seen * case["m"] * case["heads"] * case["dim"]}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _signs(seed):
    """The rotation's 16 signs: low bits of the first word of Philox4x32-10
    with this key, counter 0."""
    c, key, low = [0, 0, 0, 0], [seed & 0xFFFFFFFF, seed >> 32], 0xFFFFFFFF
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ key[0], b & low, (a >> 32) ^ c[3] ^ key[1], a & low]
        key = [(key[0] + 0x9E3779B9) & low, (key[1] + 0xBB67AE85) & low]
    return torch.tensor([-1.0 if c[0] >> j & 1 else 1.0 for j in range(16)], device="cuda")


def _stage(x, s):
    """One stage of the Walsh-Hadamard butterflies over the last 16."""
    v = x.reshape(*x.shape[:-1], 8 // s, 2, s)
    a, b = v[..., 0, :], v[..., 1, :]
    return torch.stack([a + b, a - b], dim=-2).reshape(x.shape)


def _hadamard(x):
    return _stage(_stage(_stage(_stage(x, 1), 2), 4), 8) * 0.25


def _rotate(x, signs):
    v = x.reshape(*x.shape[:-1], -1, 16)
    return _hadamard(v * signs).reshape(x.shape)


def _rotate_back(x, signs):
    v = x.reshape(*x.shape[:-1], -1, 16)
    return (_hadamard(v) * signs).reshape(x.shape)


def _nearest(a, grid):
    """Index of the grid value nearest to the magnitude a, ties to the even index."""
    if grid == "e1m2":
        return torch.round(a * 2).clamp(max=7).to(torch.uint8)
    m = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    return m.to(torch.uint8)


def _quantize(y, amax, grid):
    """y [..., k] fp32 with the largest magnitude amax [..., 1] of what shares a
    scale: packed codes [..., kpad / 2], block scales (E4M3 bytes) [..., kpad / 16]
    and that scale [..., 1]."""
    # (tensors: a division by a number is made a product with its reciprocal)
    qmax, top = (torch.full((), t * QMAX[grid], device=y.device) for t in (1, 448))
    y = torch.nn.functional.pad(y, (0, -y.shape[-1] % 64))
    enc = torch.where(amax > 0, (top / amax).clamp(max=torch.finfo(torch.float32).max), 1.0)
    dec = torch.where(amax > 0, amax / top, 1.0)
    v = y.reshape(*y.shape[:-1], -1, 16)
    e = (v.abs().amax(-1) / qmax * enc).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = e.float().unsqueeze(-1)
    q = v * torch.where(f > 0, enc.unsqueeze(-1) / f, 0.0)
    code = _nearest(q.abs(), grid) | (torch.signbit(q).to(torch.uint8) << 3)
    code = torch.where(f > 0, code, 0).reshape(y.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), e.view(torch.uint8), dec


def _to_atoms(scales):
    """Block scales [rows, blocks] as the tensor cores' atoms of 128 rows x 4 blocks."""
    rows, blocks = scales.shape
    s = torch.nn.functional.pad(scales, (0, 0, 0, -rows % 128))
    return s.view(-1, 4, 32, blocks // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _weights(g, case, segments, rows):
    """Quantised weights of `segments` matrices, each rows x k with its own
    scale, each from a row that is a multiple of 128."""
    k = case["k"]
    padded = (rows + 127) // 128 * 128 if segments > 1 else rows
    w = _normal(g, (segments, rows, k), k ** -0.5)
    # rows of differing size, some input channels far above the others
    w *= torch.exp2(torch.randint(-2, 3, (segments, rows, 1), generator=g, device="cuda").float())
    w *= torch.where(torch.rand(k, generator=g, device="cuda") < 0.004, 12.0, 1.0)
    w = w.to(torch.bfloat16).float()
    if case["rht"]:
        w = _rotate(w, _signs(SEED))
    codes, e, dec = _quantize(w, w.abs().amax((1, 2), keepdim=True), case["grid"])
    if padded > rows:
        codes = torch.nn.functional.pad(codes, (0, 0, 0, padded - rows))
        e = torch.nn.functional.pad(e, (0, 0, 0, padded - rows))
    return {"codes": codes.reshape(-1), "scales": _to_atoms(e.reshape(segments * padded, -1)),
            "tensor_scale": dec.reshape(-1).contiguous(), "rows": segments * padded, "k": k, "segment": padded}


def _routing(case, g):
    """Each token's experts (distinct, of a skewed distribution); a `dropped`
    part of the tokens is padding and goes nowhere (id -1)."""
    t, k, e = case["tokens"], case["topk"], case["experts"]
    popular = torch.randn(e, generator=g, device="cuda")
    u = torch.rand(t, e, generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
    ids = torch.topk(popular - torch.log(-torch.log(u)), k, dim=1).indices
    if case["dropped"] > 0:
        ids = torch.where((torch.rand(t, generator=g, device="cuda") < case["dropped"])[:, None], -1, ids)
    return ids


def _plan(ids, experts):
    """The stable sort of the slots by expert (dropped slots last)."""
    n = ids.numel()
    e = torch.where((ids < 0) | (ids >= experts), experts, ids).reshape(-1)
    src = torch.argsort(e, stable=True)
    pos = torch.empty_like(src)
    pos[src] = torch.arange(n, device=e.device)
    counts = (e[None, :] == torch.arange(experts, device=e.device)[:, None]).sum(1)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return {"pos": pos.to(torch.int32).view(ids.shape), "src": src.to(torch.int32), "counts": counts,
            "offsets": offsets}


def _keys(g, shape, dtype):
    """Keys or values of [.., heads, dim]: tokens of differing size, a few
    channels of each head far above the others."""
    x = _normal(g, shape, 1.0)
    x *= torch.exp2(torch.randint(-1, 2, shape[:-2] + (1, 1), generator=g, device="cuda").float())
    x *= torch.where(torch.rand(shape[-2:], generator=g, device="cuda") < 0.02, 6.0, 1.0)
    return x.to(dtype)


def _cache(case, heads, pages):
    """An empty cache: for keys and values, packed codes, block scales and each row's scale."""
    pad = (case["dim"] + 63) // 64 * 64
    new = lambda *tail, dtype=torch.uint8: torch.zeros((pages, heads, case["page"]) + tail, dtype=dtype,  # noqa: E731
                                                       device="cuda")
    return {n: {"codes": new(pad // 2), "scales": new(pad // 16), "row_scale": new(dtype=torch.float32)} for n in "kv"}


def _write(half, x, slots, case, signs):
    """Rows x [tokens, heads, dim] quantised to the places `slots` of one half of the cache."""
    y = x.float()
    if case["rht"]:
        y = _rotate(y, signs)
    codes, e, dec = _quantize(y, y.abs().amax(-1, keepdim=True), case["grid"])
    at = (slots // case["page"], slice(None), slots % case["page"])
    half["codes"][at], half["scales"][at], half["row_scale"][at] = codes, e, dec.squeeze(-1)


def prepare(case, seed):
    g, kind = _gen(seed), case["kind"]
    s = {"case": case, "signs": _signs(SEED)}
    if kind == "gemv":
        s["x"] = _normal(g, (case["tokens"], case["k"]), 1.0, DTYPES[case["x"]])
        s["w"] = _weights(g, case, 1, case["rows"])
        return s
    if kind == "experts":
        s["plan"] = _plan(_routing(case, g), case["experts"])
        n = case["tokens"] * (1 if case["gather"] else case["topk"])
        s["x"] = _normal(g, (n, case["k"]), 1.0, DTYPES[case["x"]])
        s["w"] = _weights(g, case, case["experts"], case["rows"])
        return s
    dim, page = case["dim"], case["page"]
    if kind == "cache":
        pages = -(-case["tokens"] // page) * 5 // 4 + 2
        s["cache"] = _cache(case, case["heads"], pages)
        # places in no order, the last page left free
        slots = torch.randperm((pages - 1) * page, generator=g, device="cuda")[:case["tokens"]]
        skip = torch.rand(case["tokens"], generator=g, device="cuda") < case["skipped"]
        s["slots"] = torch.where(skip, -1, slots)
        s["k"], s["v"] = (_keys(g, (case["tokens"], case["heads"], dim), DTYPES[case["x"]]) for _ in range(2))
        return s
    batch, m = case["batch"], case["m"]
    rng = np.random.RandomState(int(seed) % (1 << 31))
    lens = rng.permutation(_lens(case))
    width = max(-(-int(lens.max()) // page), 1)
    s["lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    pages = batch * width
    s["table"] = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(batch, width)
    s["cache"] = _cache(case, case["kv"], pages)
    every = torch.arange(pages * page, device="cuda")
    for part in torch.split(every, 1 << 16):
        for n in "kv":
            _write(s["cache"][n], _keys(g, (part.numel(), case["kv"], dim), torch.bfloat16), part, case, s["signs"])
    s["q"] = _keys(g, (batch * m, case["heads"], dim), DTYPES[case["x"]])
    s["mask"] = None
    if case["tree"]:
        # every drafted token follows an earlier one, or the sequence itself
        mask = np.zeros((batch, m), dtype=np.uint64)
        for i in range(m):
            before = rng.randint(-1, i, size=batch) if i else np.full(batch, -1)
            mask[:, i] = np.where(before >= 0, mask[np.arange(batch), before], 0) | np.uint64(1 << i)
        s["mask"] = torch.from_numpy(mask.view(np.int64)).cuda()
    return s


# -------------------------------------------------------------- plain forms
def _decode(codes, scales, scale, grid):
    """Packed codes [..., kpad / 2] and block scales [..., kpad / 16] as the values that they stand for."""
    m = torch.stack([codes & 15, codes >> 4], dim=-1)
    table = torch.tensor(VALUES[grid] + [-v for v in VALUES[grid]], device=codes.device)
    v = table[m.reshape(*codes.shape[:-1], -1, 16).int()]
    v = v * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)
    return (v * scale.unsqueeze(-1)).flatten(-2)


def _plain_weights(w, grid):
    """The weights [segments, rows of a segment, k] in fp32."""
    pad = (w["k"] + 63) // 64 * 64
    n = w["tensor_scale"].numel()
    s = w["scales"].view(-1, pad // 64, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, pad // 16)[:w["rows"]]
    codes = w["codes"].view(n, w["segment"], pad // 2)
    v = _decode(codes, s.reshape(n, w["segment"], pad // 16), w["tensor_scale"][:, None, None], grid)
    return v[..., :w["k"]]


def _read(half, at, case, signs):
    """Rows of one half of the cache, in fp32: [..., heads, dim]."""
    v = _decode(half["codes"][at], half["scales"][at], half["row_scale"][at].unsqueeze(-1), case["grid"])
    v = v[..., :case["dim"]]
    return _rotate_back(v, signs) if case["rht"] else v


def _run_plain(s):
    case, kind = s["case"], s["case"]["kind"]
    out = DTYPES[case["out"]]
    if kind in ("gemv", "experts"):
        x = s["x"].float()
        if case["rht"]:
            x = _rotate(x, s["signs"])
        w = _plain_weights(s["w"], case["grid"])
        if kind == "gemv":
            return {"y": (x @ w[0].T).to(out)}
        # each expert's rows behind one another, as many places as there are tokens
        p, t = s["plan"], case["tokens"]
        place = torch.arange(t * case["topk"], device="cuda")
        expert = torch.searchsorted(p["offsets"][1:], place, right=True)
        dropped = place >= p["offsets"][-1]
        expert = torch.where(dropped, 0, expert)
        at = torch.where(dropped, t, place - p["offsets"][expert])      # (behind the places)
        rows = x[(p["src"] // case["topk"]).long()] if case["gather"] else x
        xs = torch.zeros(case["experts"], t + 1, case["k"], device="cuda")
        xs[expert, at] = rows
        y = torch.bmm(xs, w[:, :case["rows"]].transpose(1, 2))[expert, at]
        return {"y": torch.where(dropped[:, None], 0.0, y).to(out)}
    page = case["page"]
    if kind == "cache":
        live = s["slots"] >= 0
        free = s["cache"]["k"]["codes"].shape[0] * page - 1              # a place that nobody has
        slots = torch.where(live, s["slots"], free)
        r = {}
        for n in "kv":
            half = s["cache"][n]
            _write(half, s[n], slots, case, s["signs"])
            v = _read(half, (slots // page, slice(None), slots % page), case, s["signs"])
            r[n] = torch.where(live[:, None, None], v, 0.0).to(out)
        return r
    b, m, kv, dim = case["batch"], case["m"], case["kv"], case["dim"]
    table, lens = s["table"].long(), s["lens"].long()
    place = torch.arange(table.shape[1] * page, device="cuda")
    at = (table[:, place // page], slice(None), (place % page).expand(b, -1))
    k, v = (_read(s["cache"][n], at, case, s["signs"]).transpose(1, 2) for n in "kv")      # [b, kv, L, dim]
    q = s["q"].float().view(b, m, kv, -1, dim).permute(0, 2, 3, 1, 4)                     # [b, kv, group, m, dim]
    x = torch.matmul(q.reshape(b, kv, -1, dim), k.transpose(2, 3)).view(b, kv, -1, m, place.numel()) * dim ** -0.5
    tail = place[None, :] - (lens[:, None] - m)                          # place among the new tokens
    tail_at = tail.clamp(0, m - 1)
    node = torch.arange(m, device="cuda")
    if s["mask"] is None:
        sees = tail_at[:, None, :] <= node[:, None]
    else:
        sees = (s["mask"][:, :, None] >> tail_at[:, None, :]) & 1 == 1
    sees = torch.where((tail < 0)[:, None, :], True, sees) & (place[None, :] < lens[:, None])[:, None, :]
    x = torch.where(sees[:, None, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, kv, -1, place.numel()), v).view(b, kv, -1, m, dim)
    o = torch.where(z > 0, o / z, 0.0)
    lse = (torch.log(z) + top).squeeze(-1)
    return {"out": o.permute(0, 3, 1, 2, 4).reshape(b * m, case["heads"], dim).to(out),
            "lse": lse.permute(0, 3, 1, 2).reshape(b * m, case["heads"])}


# --------------------------------------------------- the framework's kernels
def _run_own(s):
    from fp4_quantized_numerics_gb300 import ufp4 as U
    case, kind = s["case"], s["case"]["kind"]
    out, grid = DTYPES[case["out"]], GRID[case["grid"]]
    rotation = dict(rht=case["rht"], rht_seed=SEED)
    if kind in ("gemv", "experts"):
        w = s["w"]
        q = U.QTensor(w["codes"], w["scales"], w["tensor_scale"], w["rows"], w["k"], grid)
        if kind == "gemv":
            return {"y": U.ufp4_gemv(s["x"], q, dtype=out, **rotation)}
        plan = U.MoePlan(**s["plan"])
        return {"y": U.ufp4_gemv_grouped(s["x"], q, plan, case["rows"], gather=case["gather"], dtype=out, **rotation)}
    k, v = s["cache"]["k"], s["cache"]["v"]
    cache = U.Cache(k["codes"], k["scales"], k["row_scale"], v["codes"], v["scales"], v["row_scale"], case["dim"], grid,
                    **rotation)
    if kind == "cache":
        U.ufp4_cache_append(s["k"], s["v"], s["slots"], cache)
        k, v = U.ufp4_cache_load(cache, s["slots"], dtype=out)
        return {"k": k, "v": v}
    o, lse = U.ufp4_cache_attn(s["q"], cache, s["table"], s["lens"], mask=s["mask"], dtype=out, lse=True)
    return {"out": o, "lse": lse}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------- in 64 bits
def _e4m3(byte):
    """The value of an E4M3 byte (none here is negative or NaN)."""
    e, f = (byte >> 3).double(), (byte & 7).double()
    return torch.where(e > 0, torch.exp2(e - 7) * (1 + f / 8), torch.exp2(torch.full_like(f, -6.0)) * f / 8)


def _values(codes, scales, grid):
    """Codes and block scales (int) as values without the outermost scale."""
    n = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.uint8, device=codes.device)
    n[..., 0::2], n[..., 1::2] = codes % 16, codes // 16
    m = (n % 8).double()
    v = m / 2 if grid == "e1m2" else torch.where(m < 4, m / 2, torch.where(m < 7, m - 2, 6.0))
    v = torch.where(n >= 8, -v, v)
    return v * _e4m3(scales).repeat_interleave(16, dim=-1)


def _matrix(signs):
    """The rotation as a matrix: y = R x."""
    i = np.arange(16)
    h = np.array([[(-1.0) ** bin(a & b).count("1") for b in i] for a in i]) / 4
    return torch.from_numpy(h).cuda() * signs.double()[None, :]


def _turn(x, r):
    return (x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16) @ r.T).reshape(x.shape)


def _expert_rows(s, e, case):
    """Rows of the result that expert e (or matrix 0) has, and their inputs."""
    if case["kind"] == "gemv":
        return slice(None), s["x"].double()
    a, b = (int(v) for v in s["plan"]["offsets"][e:e + 2])
    rows = s["plan"]["src"][a:b].long() // case["topk"] if case["gather"] else torch.arange(a, b, device="cuda")
    return slice(a, b), s["x"][rows].double()


def _half(half, pages, case, r):
    """Rows of some pages of the cache, [heads, rows, dim]."""
    v = _values(half["codes"][pages], half["scales"][pages], case["grid"])[..., :case["dim"]]
    v = v * half["row_scale"][pages].double().unsqueeze(-1)
    v = _turn(v, r.T) if case["rht"] else v
    return v.permute(1, 0, 2, 3).reshape(v.shape[1], -1, case["dim"])


def _steps(y, case):
    """The values nearest to the rows y in 64 bits (what the format's
    definition rounds to fp32 on the way, rounded there)."""
    f32 = lambda t: t.float().double()  # noqa: E731
    qmax = QMAX[case["grid"]]
    amax = y.abs().amax(-1, keepdim=True)
    enc = torch.where(amax > 0, f32(448 * qmax / amax), 1.0).unsqueeze(-1)
    dec = torch.where(amax > 0, f32(amax / (448 * qmax)), 1.0).unsqueeze(-1)
    v = y.reshape(*y.shape[:-1], -1, 16)
    top = f32(f32(v.abs().amax(-1, keepdim=True) / qmax) * enc).clamp(max=448)
    unit = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -6))) - 3)
    e = torch.round(top / unit) * unit
    q = torch.where(e > 0, f32(v * f32(enc / e)), 0.0)
    a = q.abs().clamp(max=qmax)
    step = 0.5 if case["grid"] == "e1m2" else torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    g = torch.round(a / step) * step
    return (torch.where(q < 0, -g, g) * e * dec).reshape(y.shape)


def exact(case, seed):
    s, kind = prepare(case, seed), case["kind"]
    r = _matrix(s["signs"])
    if kind in ("gemv", "experts"):
        w, rows, pad = s["w"], case["rows"], (case["k"] + 63) // 64 * 64
        n = case["tokens"] * case.get("topk", 1)
        y = torch.zeros(n, rows, dtype=torch.float64, device="cuda")
        at = torch.arange(pad // 16, device="cuda")
        for e in range(w["tensor_scale"].numel()):
            to, x = _expert_rows(s, e, case)
            x = _turn(x, r) if case["rht"] else x
            for a in range(0, rows if x.shape[0] else 0, 1 << 13):
                local = torch.arange(a, min(rows, a + (1 << 13)), device="cuda")
                row = (local + e * w["segment"])[:, None]
                # a scale's byte by the layout's formula
                byte = (row // 128 * (pad // 64) + at // 4) * 512 + row % 32 * 16 + row % 128 // 32 * 4 + at % 4
                v = _values(w["codes"].view(-1, pad // 2)[row[:, 0]], w["scales"][byte], case["grid"])[:, :case["k"]]
                y[to, a:a + local.numel()] = x @ v.T * float(w["tensor_scale"][e])
        return {"y": y}
    if kind == "cache":
        if case["rht"] and case["out"] == "fp32":
            return None           # a rotated value next to a border may fall on either side of it
        live = (s["slots"] >= 0)[:, None, None]
        got = {}
        for n in "kv":
            y = s[n].double()
            got[n] = _turn(_steps(_turn(y, r), case), r.T) if case["rht"] else _steps(y, case)
        return {n: torch.where(live, t, 0.0) for n, t in got.items()}
    b, m, kv, dim, page = case["batch"], case["m"], case["kv"], case["dim"], case["page"]
    group = case["heads"] // kv
    out = torch.zeros(b * m, case["heads"], dim, dtype=torch.float64, device="cuda")
    lse = torch.full((b * m, case["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        pages = s["table"][i, :-(-n // page)].long()
        k, v = (_half(s["cache"][h], pages, case, r)[:, :n] for h in "kv")
        bits = np.arange(m)
        if s["mask"] is None:
            sees = bits[None, :] <= bits[:, None]
        else:
            sees = s["mask"][i].cpu().numpy().view(np.uint64)[:, None] >> bits.astype(np.uint64)[None, :] & np.uint64(1)
        hidden = torch.zeros(m, n, dtype=torch.bool, device="cuda")
        hidden[:, n - m:] = torch.from_numpy(np.asarray(sees) == 0).cuda()
        for h in range(kv):
            q = s["q"][i * m:(i + 1) * m, h * group:(h + 1) * group].double().transpose(0, 1)
            x = (q @ k[h].T / math.sqrt(dim)).masked_fill(hidden, -math.inf)
            out[i * m:(i + 1) * m, h * group:(h + 1) * group] = (torch.softmax(x, -1) @ v[h]).transpose(0, 1)
            lse[i * m:(i + 1) * m, h * group:(h + 1) * group] = torch.logsumexp(x, -1).T
    return {"out": out, "lse": lse}
