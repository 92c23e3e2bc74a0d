"""Cases, inputs and plain forms of the window-side operators: the append of exact rows,
the append of indexer keys, and attention of new tokens over a sliding window of exact
rows with a few first tokens that stay visible.

``run`` computes a case in elementary torch operations, or with the library's calls
where ``own`` is true.
"""
from __future__ import annotations

import math

import torch

own = False

LATENT, ROPE, DQK, PAGE = 512, 64, 576, 64
EPS = 1e-6
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the newest token of every sequence of a serving batch
        dict(name="rows decode", op="rows", n=64, rows=64 * 128, norm=True, half=False, scaling="none", top=262144),
        # a ragged prompt, some rows of it padding
        dict(name="rows ragged", op="rows", n=5003, rows=6016, norm=False, half=True, scaling="parts", top=1 << 20),
        # a prompt slab
        dict(name="rows slab", op="rows", n=131072, rows=131072, norm=True, half=False, scaling="linear", top=131072),
        # the newest indexer key of every sequence
        dict(name="keys decode e4m3", op="keys", kind="e4m3", n=64, rows=64 * 64, dim=128, offset=0, rot=64, half=True,
             norm="layer", scaling="none", top=262144),
        # indexer keys of a ragged prompt in FP4
        dict(name="keys ragged fp4", op="keys", kind="fp4", n=5003, rows=6016, dim=128, offset=64, rot=64, half=False,
             norm="rms", scaling="parts", top=1 << 20),
        # indexer keys of a million positions
        dict(name="keys million e4m3", op="keys", kind="e4m3", n=1 << 20, rows=1 << 20, dim=128, offset=0, rot=64,
             half=True, norm="layer", scaling="parts", top=1 << 20),
        # one token, few heads
        dict(name="attend one token", op="attend", heads=16, batch=1, q_lo=1, q_hi=1, c_lo=200, c_hi=200, window=128,
             sinks=0, join=False, paged=True),
        # a serving batch's newest tokens, joined with the rest of the layer
        dict(name="attend decode batch", op="attend", heads=64, batch=64, q_lo=1, q_hi=1, c_lo=8192, c_hi=262144,
             window=128, sinks=0, join=True, paged=True),
        # the window of a whole model's layers, one token a sequence: few rows, a long axis
        dict(name="attend decode long", op="attend", heads=64, batch=8, q_lo=1, q_hi=1, c_lo=131072, c_hi=131072,
             window=2048, sinks=4, join=False, paged=True),
        # draft tokens of a ragged batch, first tokens kept
        dict(name="attend drafts", op="attend", heads=64, batch=16, q_lo=1, q_hi=5, c_lo=30, c_hi=16384, window=128,
             sinks=4, join=True, paged=True),
        # ragged whole prompts
        dict(name="attend prompts", op="attend", heads=64, batch=4, q_lo=1001, q_hi=3000, c_lo=0, c_hi=0, window=128,
             sinks=0, join=False, paged=True),
        # a prompt's chunk late in a context, long window
        dict(name="attend chunk long", op="attend", heads=64, batch=1, q_lo=2048, q_hi=2048, c_lo=30720, c_hi=30720,
             window=2048, sinks=4, join=False, paged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rows", "keys", "attend", "attend"])
    scaling, top, half = rng.choice(["none", "linear", "parts"]), rng.choice([4096, 131072, 1 << 20]), rng.random() < 0.5
    if op == "rows":
        n = _log(rng, 1, 131072)
        return dict(op="rows", n=n, rows=-(-(n + rng.randint(0, 500)) // 64) * 64, norm=rng.random() < 0.7, half=half,
                    scaling=scaling, top=top)
    if op == "keys":
        n, kind = _log(rng, 1, 1 << 20), rng.choice(["e4m3", "e4m3", "fp4", "fp32"])
        dim = 64 if kind == "fp32" else 128
        offset, rot = rng.choice([(0, 64), (0, 32), (dim - 32, 32), (0, dim), (6, 20)])
        return dict(op="keys", kind=kind, n=n, rows=-(-(n + rng.randint(0, 500)) // 64) * 64, dim=dim, offset=offset,
                    rot=rot, half=half, norm=rng.choice(["none", "rms", "layer"]), scaling=scaling, top=top)
    heads = rng.choice([7, 16, 24, 64, 64])
    form = rng.choice(["decode", "drafts", "chunk", "prompt"])
    window, sinks = _log(rng, 16, 2048), rng.choice([0, 0, 1, 4, 64])
    batch = _log(rng, 1, 128) if form in ("decode", "drafts") else rng.randint(1, 4)
    q = {"decode": 1, "drafts": rng.randint(2, 9)}.get(form) or _log(rng, 10, 2048)
    q = max(1, min(q, 2048 * 2052 // (batch * (window + sinks))))
    c = 0 if form == "prompt" else _log(rng, 64, 262144)
    return dict(op="attend", heads=heads, batch=batch, q_lo=max(1, q // 3), q_hi=q, c_lo=c // 3, c_hi=c, window=window,
                sinks=sinks, join=rng.random() < 0.5, paged=c > 20000 or rng.random() < 0.7)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _frequencies(rot, scaling):
    """Angle per position of each pair, in 64 bits (theta 10000)."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / 8.0
    if scaling == "parts":                    # factor 16 from 65536 positions, ramp from 1 to 32 turns
        turns = 65536.0 * f / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0, 1)
        f = f * keep + f / 16.0 * (1 - keep)
    return f


def _mscale(scaling):
    return 1.25 if scaling == "parts" else 1.0


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _lengths(case):
    """New tokens and contexts (with them) of the case's sequences, spread over its bounds."""
    g = torch.Generator()
    g.manual_seed(1000003 * case["batch"] + 1009 * case["q_hi"] + case["c_hi"])
    q = torch.randint(case["q_lo"], case["q_hi"] + 1, (case["batch"],), generator=g)
    c = torch.randint(case["c_lo"], case["c_hi"] + 1, (case["batch"],), generator=g)
    return q.tolist(), (c + q).tolist()


def _places(case, s, g):
    """The rows' positions and places: whole pages in any order, padding without a place."""
    n = case["n"]
    s["pos"] = torch.randint(0, case["top"], (n,), generator=g, device="cuda", dtype=torch.int32)
    pages = torch.randperm(case["rows"] // PAGE, generator=g, device="cuda")
    dst = (pages[:, None] * PAGE + torch.arange(PAGE, device="cuda")).reshape(-1)[:n]
    if n % 2:
        dst[torch.randperm(n, generator=g, device="cuda")[:n // 50]] = -1
    s["dst"] = dst.contiguous()


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "rows":
        s["x"] = (_normal(g, case["n"], DQK) * torch.exp(0.5 * _normal(g, DQK))).to(torch.bfloat16)
        s["w"] = (1 + 0.1 * _normal(g, LATENT)).to(torch.bfloat16) if case["norm"] else None
        _places(case, s, g)
        s["kv"] = torch.zeros(case["rows"], DQK, dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "keys":
        n, rows, dim = case["n"], case["rows"], case["dim"]
        dt = torch.float32 if case["kind"] == "fp32" else torch.bfloat16
        s["x"] = (_normal(g, n, dim) * torch.exp(0.5 * _normal(g, dim)) + 0.3 * _normal(g, dim)).to(dt)
        s["w"] = (1 + 0.1 * _normal(g, dim)).to(dt) if case["norm"] != "none" else None
        s["b"] = (0.1 * _normal(g, dim)).to(dt) if case["norm"] == "layer" else None
        _places(case, s, g)
        if case["kind"] == "fp32":
            s["keys"] = torch.zeros(rows, dim, device="cuda")
        elif case["kind"] == "e4m3":
            s["keys"] = torch.zeros(rows, dim, dtype=torch.uint8, device="cuda")
        else:                                 # codes [rows][64], scales [rows][8]
            s["keys"] = torch.zeros(rows * 72, dtype=torch.uint8, device="cuda")
            s["values"] = torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda")
    else:
        ql, cl = _lengths(case)
        heads, window, sinks = case["heads"], case["window"], case["sinks"]
        starts = [0]
        for v in ql:
            starts.append(starts[-1] + v)
        total, width = starts[-1], -(-max(cl) // PAGE)
        if case["paged"]:
            # pages that no new token sees any more have gone back to the pool
            keep = torch.zeros(len(cl), width, dtype=torch.bool)
            for b, (q, c) in enumerate(zip(ql, cl)):
                keep[b, max(0, c - q - window + 1) // PAGE:(c - 1) // PAGE + 1] = True
                keep[b, :-(-min(sinks, c) // PAGE)] = True
            pages = int(keep.sum()) + 3
            table = torch.full((len(cl), width), -1, dtype=torch.int32)
            g2 = torch.Generator()
            g2.manual_seed(seed)
            table[keep] = torch.randperm(pages, generator=g2)[:pages - 3].to(torch.int32)
            s["table"], s["pages"] = table.cuda(), pages
            rows = pages * PAGE
        else:
            s["table"], s["pages"], rows = None, 0, len(cl) * width * PAGE
        s["width"], s["total"] = width, total
        s["kv"] = (_normal(g, rows, DQK) * torch.exp(0.5 * _normal(g, DQK))).to(torch.bfloat16)
        s["q"] = _normal(g, total, heads, DQK).to(torch.bfloat16)
        s["ctx"] = torch.tensor(cl, dtype=torch.int32, device="cuda")
        s["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        s["scale"] = 1.0 / math.sqrt(DQK)
        s["prev"], s["prev_lse"] = None, None
        if case["join"]:                      # what attention over the layer's other rows gave
            s["prev"] = (0.3 * _normal(g, total, heads, LATENT)).to(torch.bfloat16)
            s["prev_lse"] = 5.5 + _normal(g, total, heads)
        s["out"] = torch.empty(total, heads, LATENT, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(total, heads, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _plan(s):
    """What a user's program sets up once: the rotary configuration, or the dimensions and the workspace."""
    from compressed_sparse_attention_fp4_gb300 import csa2
    if "plan" not in s:
        if s["op"] == "attend":
            dims = csa2.Dims(heads=s["heads"], max_pages=s["width"] if s["pages"] else 0, num_pages=s["pages"],
                             max_ctx=s["width"] * PAGE)
            s["plan"] = dims, csa2.alloc_window_attn_workspace(dims, s["batch"], s["total"])
        else:
            kind = {"none": csa2.ROPE_PLAIN, "linear": csa2.ROPE_LINEAR, "parts": csa2.ROPE_PARTS}[s["scaling"]]
            s["plan"] = csa2.Rope(rot=s.get("rot", ROPE), theta=10000.0, scaling=kind,
                                  layout=csa2.ROPE_HALF if s["half"] else csa2.ROPE_INTERLEAVED,
                                  factor={"none": 1.0, "linear": 8.0, "parts": 16.0}[s["scaling"]], orig_ctx=65536.0,
                                  turns_lo=1.0, turns_hi=32.0, mscale=_mscale(s["scaling"]))
    return csa2, s["plan"]


def run(s):
    return {"rows": _run_rows, "keys": _run_keys, "attend": _run_attend}[s["op"]](s)


def _rotate(x, pos, case, rot):
    """x [n, rot] by the angles of pos."""
    a = (pos.double()[:, None] * _frequencies(rot, case["scaling"]).to(x.device)) % (2 * math.pi)
    m = _mscale(case["scaling"])
    cos, sin = (torch.cos(a) * m).to(x.dtype), (torch.sin(a) * m).to(x.dtype)
    if case["half"]:
        u, v = x[..., :rot // 2], x[..., rot // 2:]
        return torch.cat([u * cos - v * sin, u * sin + v * cos], dim=-1)
    u, v = x[..., 0::2], x[..., 1::2]
    return torch.stack([u * cos - v * sin, u * sin + v * cos], dim=-1).flatten(-2)


def _run_rows(s):
    if own:
        csa2, cfg = _plan(s)
        csa2.csa2_window_append(cfg, s["x"], s["pos"], s["dst"], s["kv"], norm_w=s["w"], eps=EPS)
        return s["kv"]
    x = s["x"][:, :LATENT].float()
    if s["w"] is not None:
        x = x * s["w"].float() / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    row = torch.cat([x, _rotate(s["x"][:, LATENT:].float(), s["pos"], s, ROPE)], dim=-1).to(torch.bfloat16)
    keep = s["dst"] >= 0
    s["kv"][s["dst"][keep]] = row[keep]
    return s["kv"]


def _power(e):
    """2^e in 64 bits, exactly (an integer's bits in place of a power function)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(v):
    """Non-negative 64-bit values rounded to E4M3, saturating at 448."""
    _, e = torch.frexp(v)
    step = _power(e.clamp(min=-5) - 4)
    return (torch.round(v / step) * step).clamp(max=448.0)


def _fp4(row):
    """bf16-valued 64-bit rows as the values that FP4 with a scale per 16 channels holds."""
    x = row.view(row.shape[0], -1, 16)
    sc = _e4m3(x.abs().amax(-1, keepdim=True) / 6.0)
    r = torch.where(sc > 0, x.abs() / torch.where(sc > 0, sc, torch.ones_like(sc)), torch.zeros_like(x)).clamp(max=6.0)
    step = torch.where(r < 2, 0.5, torch.where(r < 4, 1.0, 2.0))
    return (torch.round(r / step) * step * sc * torch.sign(x)).view(row.shape)


def _run_keys(s):
    if own:
        csa2, cfg = _plan(s)
        kind = {"e4m3": csa2.IDXK_E4M3, "fp4": csa2.IDXK_FP4, "fp32": csa2.IDXK_F32}[s["kind"]]
        norm = {"none": csa2.IDX_NORM_NONE, "rms": csa2.IDX_NORM_RMS, "layer": csa2.IDX_NORM_LAYER}[s["norm"]]
        csa2.csa2_idx_k_append(cfg, kind, s["x"], s["pos"], s["dst"], s["keys"], s["rows"], offset=s["offset"], norm=norm,
                               norm_w=s["w"], norm_b=s["b"], eps=EPS)
        if s["kind"] == "fp4":
            codes, scales = csa2.fp4_idx_k_planes(s["keys"], s["rows"])
            return csa2.fp4_kv_dequantize(codes.view(-1, 256), scales.view(-1, 32), s["values"].view(-1, LATENT)).view(-1, s["dim"])
        return s["keys"].view(torch.float8_e4m3fn) if s["kind"] == "e4m3" else s["keys"]
    # in 64 bits for FP4: values next to a border of its grid, whose steps are wide
    x = s["x"].double() if s["kind"] == "fp4" else s["x"].float()
    wide = x.dtype
    if s["norm"] == "layer":
        x = x - x.mean(-1, keepdim=True)
    if s["norm"] != "none":
        x = x * s["w"].to(wide) / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    if s["norm"] == "layer":
        x = x + s["b"].to(wide)
    a, b = s["offset"], s["offset"] + s["rot"]
    x = torch.cat([x[:, :a], _rotate(x[:, a:b], s["pos"], s, s["rot"]), x[:, b:]], dim=-1)
    keep = s["dst"] >= 0
    if s["kind"] == "fp4":
        s["values"][s["dst"][keep]] = _fp4(x.to(torch.bfloat16).double())[keep].to(torch.bfloat16)
        return s["values"]
    if s["kind"] == "e4m3":
        key = x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        s["keys"][s["dst"][keep]] = key.view(torch.uint8)[keep]
        return s["keys"].view(torch.float8_e4m3fn)
    s["keys"][s["dst"][keep]] = x[keep]
    return s["keys"]


def _run_attend(s):
    W, S = s["window"], s["sinks"]
    if own:
        csa2, (dims, ws) = _plan(s)
        csa2.csa2_window_attn_chunk(dims, s["batch"], s["q"], s["q_start"], s["kv"], s["table"], s["ctx"], s["scale"], W,
                                    s["out"], s["lse"], ws, sinks=S, prev_out=s["prev"], prev_lse=s["prev_lse"])
        return s["out"], s["lse"]
    dev = s["q"].device
    # every token's sequence and position, and the positions that it may see: the first S, then its last W
    t = torch.arange(s["total"], device=dev)
    b = torch.searchsorted(s["q_start"][1:].long(), t, right=True)
    pos = (s["ctx"].long()[b] - s["q_start"].long()[b + 1] + t)[:, None]
    sink, last = torch.arange(S, device=dev).expand(s["total"], S), pos - W + 1 + torch.arange(W, device=dev)
    at = torch.cat([sink, last.clamp(min=0)], dim=1)
    see = torch.cat([sink <= pos, last >= S], dim=1)
    if s["table"] is None:
        rows = b[:, None] * (s["width"] * PAGE) + at
    else:
        rows = s["table"].long()[b[:, None], at // PAGE].clamp(min=0) * PAGE + at % PAGE
    key = s["kv"][rows].float()                                                  # [total, S + W, 576]
    logit = torch.bmm(s["q"].float(), key.transpose(1, 2)) * s["scale"]
    logit.masked_fill_(~see[:, None], -math.inf)
    top = logit.amax(-1, keepdim=True)
    p = torch.exp(logit - top)
    del logit
    out = torch.bmm(p, key[..., :LATENT])
    total = p.sum(-1)
    out, lse = out / total[..., None], top[..., 0] + torch.log(total)
    if s["prev"] is not None:
        most = torch.maximum(lse, s["prev_lse"])
        u, v = torch.exp(lse - most), torch.exp(s["prev_lse"] - most)
        out = (out * u[..., None] + s["prev"].float() * v[..., None]) / (u + v)[..., None]
        lse = most + torch.log(u + v)
    s["out"].copy_(out.to(torch.bfloat16))
    s["lse"].copy_(lse)
    return s["out"], s["lse"]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "rows":
        return {"bytes": case["n"] * (4 * DQK + 12), "flops": case["n"] * 5 * DQK}
    if case["op"] == "keys":
        n, dim, kind = case["n"], case["dim"], case["kind"]
        size = {"e4m3": 3 * dim, "fp4": 2 * dim + 72, "fp32": 8 * dim}[kind] + 12
        back = case["rows"] * (72 + 2 * dim) if kind == "fp4" else 0              # read back as values
        return {"bytes": n * size + back, "flops": n * 10 * dim}
    W, S, H = case["window"], case["sinks"], case["heads"]
    read = seen = rows = 0
    for q, c in zip(*_lengths(case)):
        rows += q
        first = max(0, c - q - W + 1)
        read += c - first + min(S, first)
        for p in range(c - q, c):
            low = max(0, p - W + 1)
            seen += p - low + 1 + min(S, low)
    per = 2 * DQK + 2 * LATENT + 4 + (2 * LATENT + 4 if case["join"] else 0)
    return {"bytes": read * 2 * DQK + rows * H * per, "flops": H * seen * 2 * (DQK + LATENT)}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _turn64(x, pos, case, rot):
    """Pairs as complex numbers times m e^(i angle)."""
    n = rot // 2
    z = torch.complex(x[:, :n], x[:, n:]) if case["half"] else torch.view_as_complex(x.unflatten(-1, (n, 2)).contiguous())
    a = torch.outer(pos.double(), _frequencies(rot, case["scaling"]).to(x.device))
    z = z * torch.polar(torch.full_like(a, _mscale(case["scaling"])), a)
    return torch.cat([z.real, z.imag], -1) if case["half"] else torch.view_as_real(z).flatten(-2)


def _nearest(v, grid):
    """Non-negative values on an ascending grid, ties to the even place."""
    mid = (grid[1:] + grid[:-1]) / 2
    k = torch.bucketize(v, mid)               # a tie stays with the lower place ...
    tie = (k < len(mid)) & (v == mid[k.clamp(max=len(mid) - 1)]) & (k % 2 == 1)
    return grid[k + tie.long()]               # ... unless that is odd


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rows":
        x = s["x"].double()
        lat = x[:, :LATENT]
        if s["w"] is not None:
            lat = lat * torch.rsqrt((lat * lat).sum(1, keepdim=True) / LATENT + EPS) * s["w"].double()
        row = torch.cat([lat, _turn64(x[:, LATENT:].contiguous(), s["pos"], case, ROPE)], 1)
        kv = torch.zeros(case["rows"], DQK, dtype=torch.float64, device="cuda")
        ok = (s["dst"] >= 0).nonzero()[:, 0]
        kv[s["dst"][ok]] = row[ok]
        return kv
    if case["op"] == "keys":
        keys = torch.zeros(case["rows"], case["dim"], dtype=torch.float64, device="cuda")
        grid8 = torch.arange(127, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn).double()
        for i in range(0, case["n"], 1 << 17):
            x, dst, pos = s["x"][i:i + (1 << 17)].double(), s["dst"][i:i + (1 << 17)], s["pos"][i:i + (1 << 17)]
            if case["norm"] == "layer":
                var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
                x = (x - mean) * torch.rsqrt(var + EPS) * s["w"].double() + s["b"].double()
            elif case["norm"] == "rms":
                x = x * torch.rsqrt((x * x).sum(1, keepdim=True) / case["dim"] + EPS) * s["w"].double()
            a, b = case["offset"], case["offset"] + case["rot"]
            y = x.clone()
            y[:, a:b] = _turn64(x[:, a:b].contiguous(), pos, case, case["rot"])
            if case["kind"] == "e4m3":
                y = _nearest(y.abs(), grid8) * torch.sign(y)
            elif case["kind"] == "fp4":
                # 8 significant bits, as bf16 has, by adding and taking away 3/2 2^(e + 44) (made from its bits)
                big = ((torch.frexp(y)[1].long() + 44 + 1023 << 52) + (1 << 51)).view(torch.float64)
                y = ((y + big) - big).view(len(y), -1, 16)
                sc = _nearest(y.abs().amax(2) / 6, grid8)[..., None]
                grid4 = torch.tensor(LEVELS, device="cuda", dtype=torch.float64)
                y = (_nearest(y.abs() / sc.clamp(min=1e-300), grid4) * sc * torch.sign(y)).view(len(y), -1)
            ok = (dst >= 0).nonzero()[:, 0]
            keys[dst[ok]] = y[ok]
        return keys
    # attention, one sequence and a few tokens at a time
    if work(case)["flops"] > 1.2e13:
        return None
    W, S = case["window"], case["sinks"]
    out = torch.empty(s["total"], s["heads"], LATENT, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["total"], s["heads"], dtype=torch.float64, device="cuda")
    starts = s["q_start"].tolist()
    for b, n in enumerate(s["ctx"].tolist()):
        t0, t1 = starts[b], starts[b + 1]
        first = max(0, n - (t1 - t0) - W + 1)
        at = torch.cat([torch.arange(min(S, first), device="cuda"), torch.arange(first, n, device="cuda")])
        if s["table"] is None:
            k = s["kv"][b * s["width"] * PAGE + at].double()
        else:
            k = s["kv"].view(-1, PAGE, DQK)[s["table"][b].long()[at // PAGE], at % PAGE].double()
        few = max(1, (1 << 28) // (len(at) * s["heads"]))
        for t in range(t0, t1, few):
            e = min(t + few, t1)
            p = torch.arange(t, e, device="cuda")[:, None] - t1 + n
            seen = (at <= p) & ((at > p - W) | (at < S))
            x = torch.einsum("thd,nd->thn", s["q"][t:e].double(), k) * s["scale"]
            x = torch.where(seen[:, None], x, -math.inf)
            lse[t:e] = torch.logsumexp(x, 2)
            out[t:e] = torch.einsum("thn,nd->thd", torch.softmax(x, 2), k[:, :LATENT])
    if case["join"]:
        both = torch.logaddexp(lse, s["prev_lse"].double())
        out = out * torch.exp(lse - both)[..., None] + s["prev"].double() * torch.exp(s["prev_lse"].double() - both)[..., None]
        lse = both
    return out, lse
