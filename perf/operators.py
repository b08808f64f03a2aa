"""Workloads of the routing and block-scaled 8-bit expert operators.

Each case is one call of one operator (``op``):

* ``route``: scores (softmax or sigmoid) plus a balance bias, expert groups,
  top-k, renormalised weights, and the per-expert token lists;
* ``quantize``: e4m3 values with a power-of-two scale per block of 128
  columns of one row (activations) or of 128 rows (weights);
* ``gemm``: the block-scaled product of list entries with their experts'
  weights;
* ``ffn``: the SwiGLU expert FFN on block-scaled e4m3 weights.

``run`` computes the plain form with elementary torch operations, or, where
``own`` is true, calls the library.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# Expert layers (hidden size, experts, experts per token, intermediate size)
# as in moe_synth.SHAPES.
SHAPES = {"e64": (2048, 64, 8, 1024), "q30b": (2048, 128, 8, 768), "q235b": (4096, 128, 8, 1536)}


# ---------------------------------------------------------------- cases --
def _route(name, T, E, k, score, groups=1, top_groups=1, best=1, bias=True, masked=0.0, scale=1.0, renorm=True):
    c = {"op": "route", "T": T, "E": E, "k": k, "score": score, "groups": groups, "top_groups": top_groups,
         "best": best, "bias": bias, "masked": masked, "scale": scale, "renorm": renorm}
    return dict(c, name=name) if name else c


def _quantize(name, batch, rows, cols, block_rows, src):
    c = {"op": "quantize", "batch": batch, "rows": rows, "cols": cols, "block_rows": block_rows, "src": src}
    return dict(c, name=name) if name else c


def _gemm(name, T, d, E, k, N, out="bf16"):
    c = {"op": "gemm", "T": T, "d": d, "E": E, "k": k, "F": N, "padded": 0.0, "out": out}
    return dict(c, name=name) if name else c


def _ffn(name, T, d, E, k, F, padded=0.0, src="bf16"):
    c = {"op": "ffn", "T": T, "d": d, "E": E, "k": k, "F": F, "padded": padded, "src": src}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of a decode step: latency only
        _route("route_1_sigmoid_grouped", 1, 256, 8, "sigmoid", 8, 4, 2, scale=2.5),
        # a decode batch of odd size; some experts are not resident
        _route("route_77_softmax_masked", 77, 128, 8, "softmax", bias=False, masked=0.1),
        # a prefill chunk's tokens
        _route("route_8192_sigmoid_grouped", 8192, 256, 8, "sigmoid", 8, 4, 2, scale=2.5),
        # a prefill chunk's activations before a product
        _quantize("quantize_rows_4096", 1, 4096, 2048, 1, "bf16"),
        # a layer's expert matrices when the weights are loaded
        _quantize("quantize_weights_128", 128, 768, 2048, 128, "bf16"),
        # one projection of an expert layer for a ragged decode batch
        _gemm("gemm_33_tokens", 33, 2048, 64, 8, 1024, "f32"),
        # a dense layer (one expert that every token takes) in prefill
        _gemm("gemm_2000_dense", 2000, 4096, 1, 1, 4096),
        # decode of one request
        _ffn("ffn_1_q30b", 1, *SHAPES["q30b"]),
        # a decode batch
        _ffn("ffn_16_q30b", 16, *SHAPES["q30b"]),
        # a small decode batch on the largest layer
        _ffn("ffn_8_q235b", 8, *SHAPES["q235b"]),
        # a mixed batch of odd size with padded tokens, fp32 activations
        _ffn("ffn_333_e64_padded", 333, *SHAPES["e64"], padded=0.1, src="f32"),
        # a prefill chunk
        _ffn("ffn_4096_q30b", 4096, *SHAPES["q30b"]),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "quantize", "gemm", "ffn", "ffn"])
    if op == "route":
        E = rng.choice([16, 48, 64, 128, 160, 256])
        k = rng.randint(1, 8)
        groups, top, best = 1, 1, 1
        if rng.random() < 0.5:
            groups = rng.choice([g for g in (2, 4, 8) if E % g == 0])
            best = rng.choice([1, 2])
            top = rng.randint(max(1, -(-k * groups // E)), groups)
        return _route(None, _log(rng, 1, 8192), E, k, rng.choice(["softmax", "sigmoid"]), groups, top, best,
                      rng.random() < 0.7, rng.choice([0.0, 0.0, 0.1, 0.5]), rng.choice([1.0, 2.5]),
                      rng.random() < 0.8)
    if op == "quantize":
        src = rng.choice(["bf16", "f32"])
        if rng.random() < 0.6:
            return _quantize(None, 1, _log(rng, 1, 8192), 16 * _log(rng, 4, 256), 1, src)
        return _quantize(None, _log(rng, 1, 32), 16 * _log(rng, 4, 64), 16 * _log(rng, 4, 128), 128, src)
    E = rng.choice([8, 16, 60, 64, 128])
    if op == "gemm":
        if rng.random() < 0.3:
            return _gemm(None, _log(rng, 1, 2000), 16 * _log(rng, 8, 256), 1, 1, 16 * _log(rng, 8, 256),
                         rng.choice(["bf16", "f32"]))
        return _gemm(None, _log(rng, 1, 1000), 16 * _log(rng, 8, 128), E, rng.randint(1, 8), 16 * _log(rng, 8, 64),
                     rng.choice(["bf16", "f32"]))
    return _ffn(None, _log(rng, 1, 3000), 16 * _log(rng, 16, 128), E, rng.randint(1, 8), 16 * _log(rng, 8, 64),
                rng.choice([0.0, 0.0, 0.2]), rng.choice(["bf16", "f32"]))


# --------------------------------------------------------------- inputs --
def _choice(T, E, k, padded, seed):
    """Experts [T][k] and weights [T][k] of a skewed softmax router, on the
    CPU; padded tokens hold no expert."""
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g) + 0.5 * torch.randn(E, generator=g)
    w, e = torch.softmax(logits, 1).topk(k, 1)
    w = w / w.sum(1, keepdim=True)
    n_pad = int(padded * T)
    if n_pad:
        at = torch.randperm(T, generator=g)[:n_pad]
        e[at], w[at] = -1, 0.0
    return e.to(torch.int32), w


def _make_lists(e, w, E):
    """Per-expert token lists of a choice, as the library's re-selection and
    routing write them."""
    T, k = e.shape
    flat = e.reshape(-1).long()
    flat = torch.where(flat < 0, torch.full_like(flat, E), flat)
    order = torch.argsort(flat, stable=True)
    count = torch.zeros(E + 1, dtype=torch.long, device=e.device).scatter_add_(0, flat, torch.ones_like(flat))[:E]
    ids = torch.argsort((count == 0).to(torch.int32), stable=True)
    n_active = (count > 0).sum().reshape(1)
    slot = torch.arange(E, device=e.device)
    active = torch.where(slot < n_active, ids, torch.full_like(ids, -1))
    ends = torch.cumsum(torch.where(slot < n_active, count[ids], torch.zeros_like(count)), 0)
    offsets = torch.cat([torch.zeros(1, dtype=torch.long, device=e.device), ends])
    real = torch.arange(T * k, device=e.device) < ends[-1]
    tok = torch.where(real, order // k, torch.full_like(order, -1))
    lw = torch.where(real, w.reshape(-1)[order], torch.zeros_like(w.reshape(-1)))
    i32 = torch.int32
    return {"n_active": n_active.to(i32), "active": active.to(i32), "offsets": offsets.to(i32), "tok": tok.to(i32),
            "w": lw}


def _weights(gen, E, rows, cols):
    """e4m3 expert matrices [E][rows][cols] with one fp32 scale (largest
    magnitude / 448) per block of 128 x 128, as checkpoints hold them."""
    q = torch.empty(E, rows, cols, dtype=F8, device="cuda")
    rb, cb = -(-rows // BLOCK), -(-cols // BLOCK)
    scale = torch.empty(E, rb, cb, device="cuda")
    for e in range(E):
        w = torch.zeros(rb * BLOCK, cb * BLOCK, device="cuda")
        w[:rows, :cols] = torch.randn(rows, cols, device="cuda", generator=gen) * 0.02
        blocks = w.view(rb, BLOCK, cb, BLOCK)
        s = blocks.abs().amax((1, 3)) / E4M3_MAX
        scale[e] = s
        q[e] = (blocks / s[:, None, :, None]).view(rb * BLOCK, cb * BLOCK)[:rows, :cols].to(F8)
    return q, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "route":
        T, E = case["T"], case["E"]
        logits = torch.randn(T, E, device="cuda", generator=gen) * 1.5
        if case["masked"]:
            off = torch.rand(E, device="cuda", generator=gen) < case["masked"]
            pad = torch.rand(T, 1, device="cuda", generator=gen) < case["masked"] / 2  # tokens that are padding
            logits = torch.where(off | pad, torch.full_like(logits, -math.inf), logits)
        bias = torch.randn(E, device="cuda", generator=gen) * 0.05 if case["bias"] else None
        return {"case": case, "logits": logits, "bias": bias}
    if op == "quantize":
        shape = (case["batch"], case["rows"], case["cols"])
        x = torch.empty(shape, dtype=TYPES[case["src"]], device="cuda")
        for b in range(case["batch"]):  # columns of different size, as activations have them
            x[b] = torch.randn(shape[1:], device="cuda", generator=gen) * torch.exp(
                torch.randn(shape[2], device="cuda", generator=gen))
        return {"case": case, "x": x}
    T, d, E, k, F = (case[n] for n in ("T", "d", "E", "k", "F"))
    e, w = _choice(T, E, k, case["padded"], seed)
    most = int(torch.bincount(e[e >= 0].reshape(-1).long(), minlength=E).max()) if bool((e >= 0).any()) else 1
    state = {"case": case, "most": most, "lists": _make_lists(e.cuda(), w.cuda(), E)}
    x = torch.randn(T, d, device="cuda", generator=gen) * torch.exp(0.5 * torch.randn(d, device="cuda", generator=gen))
    if op == "gemm":
        state["q"], state["scale"] = _quantize_plain(x.view(1, T, d), 1)
        state["q"], state["scale"] = state["q"][0].contiguous(), state["scale"][0].contiguous()
        state["W"] = _weights(gen, E, F, d)
        return state
    state["x"] = x.to(TYPES[case["src"]])
    state["W"] = (*_weights(gen, E, F, d), *_weights(gen, E, F, d), *_weights(gen, E, d, F))
    return state


# ----------------------------------------------------------- plain forms --
def _padded_blocks(x, block_rows):
    """x [batch][rows][cols] as [batch][row blocks][block_rows][column
    blocks][128], zeros past the ends."""
    b, r, c = x.shape
    rb, cb = -(-r // block_rows), -(-c // BLOCK)
    if (rb * block_rows, cb * BLOCK) != (r, c):
        x = torch.nn.functional.pad(x, (0, cb * BLOCK - c, 0, rb * block_rows - r))
    return x.view(b, rb, block_rows, cb, BLOCK)


def _quantize_plain(x, block_rows):
    b, r, c = x.shape
    blocks = _padded_blocks(x.float(), block_rows)
    top = blocks.abs().amax((2, 4))
    # the exponent of top / 448 rounded up: 448 = 1.75 * 2^8
    m, ex = torch.frexp(top)
    ex = ex - 9 + (m > 0.875).to(torch.int32)
    scale = torch.where(top > 0, torch.ldexp(torch.ones_like(top), ex), torch.ones_like(top))
    q = (blocks / scale[:, :, None, :, None]).reshape(b, blocks.shape[1] * block_rows, -1)[:, :r, :c]
    return q.to(F8), scale


def _dequantized(q, scale):
    """fp32 values of e4m3 matrices [n][rows][cols] with a scale per 128 x
    128 block."""
    n, r, c = q.shape
    s = scale.repeat_interleave(BLOCK, 1)[:, :r].repeat_interleave(BLOCK, 2)[:, :, :c]
    return q.float().mul_(s)


def _route_plain(state):
    c = state["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    l = state["logits"].double()
    open_ = l > -math.inf
    if c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        top = l.amax(1, keepdim=True)
        p = torch.where(open_, torch.exp(l - torch.where(top > -math.inf, top, torch.zeros_like(top))),
                        torch.zeros_like(l))
        s = p / p.sum(1, keepdim=True).clamp_min(1e-300)
    rank = s if state["bias"] is None else s + state["bias"].double()
    rank = torch.where(open_, rank, torch.full_like(rank, -math.inf))
    if G > 1:
        best = rank.view(T, G, E // G).sort(dim=2, descending=True)[0][:, :, :c["best"]]
        some = best[:, :, :1] > -math.inf
        gscore = torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(2, keepdim=True)
        gscore = torch.where(some, gscore, torch.full_like(gscore, -math.inf))[:, :, 0]
        gsel = gscore.sort(dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, gsel, True)
        rank = torch.where(keep.repeat_interleave(E // G, 1), rank, torch.full_like(rank, -math.inf))
    val, idx = rank.sort(dim=1, descending=True, stable=True)
    val, idx = val[:, :k], idx[:, :k]
    held = val > -math.inf
    w = torch.where(held, s.gather(1, idx), torch.zeros_like(val))
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    w = (w * c["scale"]).float()
    sel = torch.where(held, idx, torch.full_like(idx, -1)).to(torch.int32)
    return {"sel": sel, "w": w, "lists": _make_lists(sel, w, E)}


def _slots(state):
    """Expert slots of a call (padded to the most a batch can activate),
    their experts, and the rank of each list entry within its expert."""
    c, l = state["case"], state["lists"]
    slots = min(c["E"], c["T"] * c["k"])
    active = l["active"][:slots].long().clamp_min(0)
    ends = l["offsets"][1:slots + 1].long()
    at = torch.arange(c["T"] * c["k"], device="cuda")
    slot = torch.searchsorted(ends, at, right=True).clamp_max(slots - 1)
    rank = (at - l["offsets"].long()[slot]).clamp(0, state["most"] - 1)
    return slots, active, slot, rank, l["tok"] >= 0


def _by_expert(x, state):
    """Rows of x dispatched as [slot][rank][columns], and the place of each
    list entry in it."""
    slots, active, slot, rank, real = _slots(state)
    out = torch.zeros(slots, state["most"], x.shape[1], device="cuda")
    tok = state["lists"]["tok"].long().clamp_min(0)
    rows = torch.where(real[:, None], x[tok], torch.zeros((), device="cuda"))
    out.index_put_((slot, rank), rows, accumulate=True)
    return out, active, slot, rank, real


def _gemm_plain(state):
    x = _dequantized_rows(state["q"], state["scale"])
    xe, active, slot, rank, real = _by_expert(x, state)
    q, scale = state["W"]
    y = torch.bmm(xe, _dequantized(q[active], scale[active]).transpose(1, 2))[slot, rank]
    return torch.where(real[:, None], y, torch.zeros((), device="cuda")).to(TYPES[state["case"]["out"]])


def _dequantized_rows(q, scale):
    return q.float() * scale.repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _rounded_rows(x):
    """x [..][cols] after rounding to block-scaled e4m3."""
    flat = x.reshape(1, -1, x.shape[-1])
    q, scale = _quantize_plain(flat, 1)
    return _dequantized_rows(q[0], scale[0]).view(x.shape)


def _ffn_plain(state):
    Wg, Sg, Wu, Su, Wd, Sd = state["W"]
    xe, active, slot, rank, real = _by_expert(_rounded_rows(state["x"].float()), state)
    g = torch.bmm(xe, _dequantized(Wg[active], Sg[active]).transpose(1, 2))
    u = torch.bmm(xe, _dequantized(Wu[active], Su[active]).transpose(1, 2))
    h = _rounded_rows(g / (1.0 + torch.exp(-g)) * u)
    y = torch.bmm(h, _dequantized(Wd[active], Sd[active]).transpose(1, 2))[slot, rank]
    y = torch.where(real[:, None], y, torch.zeros((), device="cuda")) * state["lists"]["w"][:, None]
    out = torch.zeros(state["x"].shape, device="cuda")
    return out.index_add_(0, state["lists"]["tok"].long().clamp_min(0), y).to(torch.bfloat16)


# ------------------------------------------------------------------ runs --
def _run_own(state):
    import aware_expert_routing_moe_b200 as moe
    c = state["case"]
    if c["op"] == "route":
        if "ws" not in state:  # kept from call to call, as a serving loop does
            T, E, k = c["T"], c["E"], c["k"]
            state["ws"] = moe.new_route_workspace(T, E, k)
            state["lists"] = moe.alloc_lists(T, E, k)
            state["out"] = (torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda"))
        sel, w, lists = moe.moe_route_scored(
            state["logits"], c["k"], moe.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else moe.MOE_SCORE_SOFTMAX,
            bias=state["bias"], groups=c["groups"], top_groups=c["top_groups"], group_best=c["best"],
            renorm=c["renorm"], scale=c["scale"], out=state["out"], lists=state["lists"], ws=state["ws"])
        return {"sel": sel, "w": w, "lists": dict(lists, n_active=lists["n_active"][:1])}
    if c["op"] == "quantize":
        q, scale = moe.moe_quantize_blocks(state["x"], c["block_rows"])
        return {"q": q, "scale": scale}
    if "ws" not in state:
        state["ws"] = (moe.new_gemm_workspace() if c["op"] == "gemm"
                       else moe.new_blocks_workspace(c["T"], c["d"], c["E"], c["k"], c["F"]))
    if c["op"] == "gemm":
        if "y" not in state:  # rows past the last list entry stay as they are
            state["y"] = torch.zeros(c["T"] * c["k"], c["F"], dtype=TYPES[c["out"]], device="cuda")
        return {"y": moe.moe_expert_gemm_blocks(state["q"], state["scale"], *state["W"], state["lists"], c["k"],
                                                ws=state["ws"], y=state["y"])}
    return {"y": moe.moe_expert_ffn_blocks(state["x"], *state["W"], state["lists"], c["k"], ws=state["ws"],
                                           y_dtype=torch.bfloat16)}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "route":
        return _route_plain(state)
    if op == "quantize":
        q, scale = _quantize_plain(state["x"], state["case"]["block_rows"])
        return {"q": q.contiguous(), "scale": scale}
    return {"y": _gemm_plain(state) if op == "gemm" else _ffn_plain(state)}


# ----------------------------------------------------------------- work --
def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * 4 + (E * 4 if case["bias"] else 0) + T * k * 16 + E * 8, "flops": 20 * T * E}
    if op == "quantize":
        n = case["batch"] * case["rows"] * case["cols"]
        size = 2 if case["src"] == "bf16" else 4
        blocks = case["batch"] * -(-case["rows"] // case["block_rows"]) * -(-case["cols"] // BLOCK)
        return {"bytes": n * (size + 1) + blocks * 4, "flops": 3 * n}
    T, d, E, k, F = (case[n] for n in ("T", "d", "E", "k", "F"))
    e, _ = _choice(T, E, k, case["padded"], 0)
    pairs = int((e >= 0).sum())
    n_active = int(torch.unique(e[e >= 0]).numel())
    scales = -(-d // BLOCK) * -(-F // BLOCK) * 4
    if op == "gemm":
        return {"bytes": n_active * (d * F + scales) + T * (d + 4 * -(-d // BLOCK)) + pairs * F * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * pairs * d * F}
    return {"bytes": n_active * 3 * (d * F + scales) + T * d * ((2 if case["src"] == "bf16" else 4) + 2) + pairs * 8,
            "flops": 6 * pairs * d * F}


# ---------------------------------------------------------------- exact --
def _e4m3_nearest(v):
    """Nearest e4m3 value (ties to even) of each 64-bit value, |v| <= 448."""
    ex = torch.frexp(v)[1].double() - 1.0
    step = torch.exp2(torch.clamp_min(ex, -6.0) - 3.0)
    return torch.round(v / step) * step


def _rounded64(x, block_rows=1):
    """(values on the e4m3 grid, scales) of x [rows][cols] in 64 bits."""
    r, c = x.shape
    v, rows = torch.zeros_like(x), []
    for i in range(0, r, block_rows):
        cols = []
        for j in range(0, c, BLOCK):
            b = x[i:i + block_rows, j:j + BLOCK] if block_rows > 1 else x[:, j:j + BLOCK]
            top = b.abs().amax(None if block_rows > 1 else 1, keepdim=True).reshape(-1, 1)
            s = torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX)))
            # a border case of log2 is put right by comparison
            s = torch.where(s * E4M3_MAX < top, s * 2, torch.where(s / 2 * E4M3_MAX >= top, s / 2, s))
            s = torch.where(top > 0, s, torch.ones_like(s))
            (v[i:i + block_rows, j:j + BLOCK] if block_rows > 1 else v[:, j:j + BLOCK]).copy_(_e4m3_nearest(b / s))
            cols.append(s)
        rows.append(torch.cat(cols, 1))
        if block_rows == 1:
            break
    return v, torch.cat(rows, 0)


def _matrix64(q, scale, e):
    m = q[e].double()
    for i in range(scale.shape[1]):
        for j in range(scale.shape[2]):
            m[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] *= scale[e, i, j].double()
    return m


def _rows64(v, s):
    out = v.clone()
    for j in range(s.shape[1]):
        out[:, j * BLOCK:(j + 1) * BLOCK] *= s[:, j:j + 1]
    return out


def _exact_weights(state):
    """The weights of the routing cases, token by token: by slot [T][k] and
    in list order [T * k]."""
    c = state["case"]
    l = state["logits"].double().cpu()
    bias = torch.zeros(c["E"], dtype=torch.double) if state["bias"] is None else state["bias"].double().cpu()
    w = torch.zeros(c["T"], c["k"], dtype=torch.double)
    entries = []
    per = c["E"] // c["groups"]
    score = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)
    for t in range(c["T"]):
        pool = [e for e in range(c["E"]) if l[t, e] > -math.inf]
        r, s = (score[t] + bias).tolist(), score[t].tolist()
        if c["groups"] > 1:
            members = {}
            for e in pool:
                members.setdefault(e // per, []).append(r[e])
            order = sorted(members, key=lambda g: (-math.fsum(sorted(members[g])[-c["best"]:]), g))
            kept = set(order[:c["top_groups"]])
            pool = [e for e in pool if e // per in kept]
        pool = sorted(pool, key=lambda e: (-r[e], e))[:c["k"]]
        total = math.fsum(s[e] for e in pool) if c["renorm"] else 1.0
        for i, e in enumerate(pool):
            w[t, i] = s[e] / total * c["scale"]
            entries.append((e, t, float(w[t, i])))
    in_lists = torch.zeros(c["T"] * c["k"], dtype=torch.double)
    in_lists[:len(entries)] = torch.tensor([v for _, _, v in sorted(entries)], dtype=torch.double)
    return w, in_lists


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "route":
        w, in_lists = _exact_weights(state)
        return {"sel": None, "w": w, "lists": {"w": in_lists}}
    if op == "quantize":
        b, r, c = state["x"].shape
        if b * r * c > 1 << 25 and case["block_rows"] > 1:
            return None
        got = [_rounded64(x.double(), case["block_rows"]) for x in state["x"]]
        return {"q": torch.stack([v for v, _ in got]), "scale": torch.stack([s for _, s in got])}
    lists = {n: v.cpu().tolist() for n, v in state["lists"].items()}
    T, d, k, F = (case[n] for n in ("T", "d", "k", "F"))
    if op == "gemm":
        x = _rows64(state["q"].double(), state["scale"].double())
        y = torch.zeros(T * k, F, dtype=torch.double, device="cuda")
    else:
        x = _rows64(*_rounded64(state["x"].double()))
        y = torch.zeros(T, d, dtype=torch.double, device="cuda")
    W = state["W"]
    for i in range(lists["n_active"][0]):
        e, lo, hi = lists["active"][i], lists["offsets"][i], lists["offsets"][i + 1]
        tok = torch.tensor(lists["tok"][lo:hi], device="cuda")
        if op == "gemm":
            y[lo:hi] = x[tok] @ _matrix64(W[0], W[1], e).T
            continue
        g, u = x[tok] @ _matrix64(W[0], W[1], e).T, x[tok] @ _matrix64(W[2], W[3], e).T
        h = _rows64(*_rounded64(g * torch.sigmoid(g) * u))
        y[tok] += state["lists"]["w"][lo:hi].double()[:, None] * (h @ _matrix64(W[4], W[5], e).T)
    return {"y": y}
