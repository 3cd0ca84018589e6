"""Cases of the operators in front of and beside the budgeted KV cache.

A layer's step begins with the projection's rows: the query and key heads are
normed and rotated and laid out per unit (``norm``).  A prompt, or a layer that
keeps all of its tokens, lives in a cache of pages: rows are quantised as they
are written (``write``), one new token is appended and attends over the pages
(``attend``), and the rows that a selection keeps are read back for the budgeted
cache (``read``).  ``run`` makes one of these calls, in elementary torch
operations or, where ``own`` is set, through the library's entry points.

A unit is one (sequence, layer, KV head); its G query heads share the KV head.
Pages belong to a sequence and hold ``heads`` units each; with ``heads`` = 1
every unit has a table and a length of its own.
"""
import math

import torch

own = False

D = 128                      # head dimension
SCALE = 1.0 / math.sqrt(D)
INF = float("inf")
E4M3_MAX = 448.0
TINY = 2.0 ** -126           # least scale of a row


# ---------------------------------------------------------------------- cases

def _norm(name, seqs, T, heads, G, rot=D, interleaved=False, norm=True, base=1e6, far=40960):
    return dict(name=name, op="norm", seqs=seqs, T=T, heads=heads, G=G, rot=rot,
                interleaved=interleaved, norm=norm, base=base, far=far)


def _write(name, seqs, heads, T, n, page, e4m3, ragged=0.0):
    return dict(name=name, op="write", seqs=seqs, heads=heads, T=T, n=n, page=page, e4m3=e4m3,
                ragged=ragged)


def _read(name, seqs, heads, m, n, page, e4m3, ragged=0.0):
    return dict(name=name, op="read", seqs=seqs, heads=heads, m=m, n=n, page=page, e4m3=e4m3,
                ragged=ragged)


def _attend(name, seqs, heads, G, n, page, e4m3, ragged=0.0, append=True):
    return dict(name=name, op="attend", seqs=seqs, heads=heads, G=G, n=n, page=page, e4m3=e4m3,
                ragged=ragged, append=append)


def listed():
    return [
        # one token of one sequence, 32 query heads over 8 KV heads: the latency of a call
        _norm("norm-token", 1, 1, 8, 4),
        # drafted trees of a batch of 16 sequences, 24 tokens each and fewer in some
        _norm("norm-tree", 16, 24, 8, 4),
        # a whole prompt
        _norm("norm-prompt", 1, 32768, 8, 4),
        # accepted drafted tokens of a batch behind prompts of different lengths
        _write("write-accepted", 16, 8, 6, 3277, 16, True, ragged=0.4),
        # a whole prompt, quantised as it is written
        _write("write-prompt", 1, 8, 32768, 0, 64, True),
        # a 10 % selection out of the prompts of 4 sequences, a list per unit
        _read("read-kept", 4, 8, 3277, 32768, 16, True, ragged=0.4),
        # the whole of a long prompt, as the prefill scorer takes it
        _read("read-prompt", 1, 8, 131071, 131071, 64, True),
        # one sequence, one layer, a short prompt: the latency of a call
        _attend("attend-token", 1, 8, 4, 64, 16, False),
        # one layer of a batch of 16 sequences that keep their whole prompts
        _attend("attend-batch", 16, 8, 4, 32768, 64, True, ragged=0.4),
        # every layer of 4 sequences in one call, a budget and a table per unit
        _attend("attend-units", 1024, 1, 4, 1024, 16, True, ragged=0.5),
        # one layer of a batch at a 10 % budget, 64 query heads
        _attend("attend-group", 16, 8, 8, 3277, 32, False, ragged=0.4),
        # one layer of one sequence over its long prompt
        _attend("attend-long", 1, 8, 4, 131071, 128, False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["norm", "write", "read", "attend", "attend"])
    heads = rng.choice([1, 2, 4, 8, 8])
    G, page = rng.choice([1, 2, 4, 8]), rng.choice([16, 32, 64, 128])
    e4m3, ragged = rng.random() < 0.6, rng.choice([0.0, 0.4, 1.0])
    if op == "norm":
        tokens = _log(rng, 1, 32768 * 48 // (heads * (G + 2)))
        seqs = min(tokens, _log(rng, 1, 64))
        case = _norm("", seqs, max(1, tokens // seqs), heads, G, rng.choice([32, 64, 96, 128, 128]),
                     rng.random() < 0.4, rng.random() < 0.7, rng.choice([1e4, 5e5, 1e6]),
                     rng.choice([4096, 40960, 131072, 1 << 20]))
    else:
        seqs = _log(rng, 1, 1024 // heads)
        n = min(_log(rng, 1, 131071), (1 << (22 if e4m3 else 21)) // (seqs * heads))
        if op == "write":
            T = min(_log(rng, 1, 32768), max(1, (1 << 18) // (seqs * heads)))
            case = _write("", seqs, heads, T, n, page, e4m3, ragged)
        elif op == "read":
            n = min(n, max(1, (1 << 20) // (seqs * heads)))
            m = n if rng.random() < 0.3 else _log(rng, 1, n)
            case = _read("", seqs, heads, m, n, page, e4m3, ragged)
        else:
            case = _attend("", seqs, heads, G, n, page, e4m3, ragged, rng.random() < 0.8)
    del case["name"]
    return case


# --------------------------------------------------------------------- inputs

def _spread(n, count, ragged, least):
    """`count` whole numbers over [(1 - ragged) n, n], `least` and above."""
    return [max(least, n - int(ragged * n * ((i * 0.6180339887) % 1.0))) for i in range(count)]


def _lengths(case):
    """Slots in use per sequence, before what the call adds."""
    least = 0 if case["op"] == "write" or case.get("append") else 1
    return _spread(case["n"], case["seqs"], case["ragged"], least)


def _counts(case):
    """Rows per sequence (written), per unit (read), live tokens per sequence (normed)."""
    if case["op"] == "norm":
        return _spread(case["T"], case["seqs"], 0.25, 1)
    if case["op"] == "write":
        return _spread(case["T"], case["seqs"], case["ragged"], 1)
    lens = _lengths(case)
    counts = _spread(case["m"], case["seqs"] * case["heads"], case["ragged"], 1)
    return [min(c, lens[u // case["heads"]]) for u, c in enumerate(counts)]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _quantise(x):
    """Rows of x as e4m3 values and a scale each: the largest magnitude becomes 448."""
    x = x.float()
    # by a tensor: torch multiplies by the reciprocal of a number, which is off by an ulp in some rows
    scale = (x.abs().amax(-1) / torch.full((), E4M3_MAX, device=x.device)).clamp_min(TINY)
    y = (x * (1.0 / scale).unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX)
    return y.to(torch.float8_e4m3fn), scale


def _rows(g, n, bias):
    """Rows that share a direction, as a head's keys and values do."""
    x = torch.randn(n, bias.numel(), generator=g, device="cuda")
    return (x + bias).to(torch.bfloat16)


def _fill(s, g, n_pages, heads, page, e4m3):
    """The pool of pages, every row of it an older token's."""
    shape = (n_pages, heads, page, D)
    for name in ("K", "V"):
        bias = torch.randn(D, generator=g, device="cuda") * (1.0 if name == "K" else 0.5)
        pool = torch.empty(shape, dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16, device="cuda")
        scale = torch.empty(shape[:3], device="cuda") if e4m3 else None
        flat, rows = pool.view(-1, D), n_pages * heads * page
        for at in range(0, rows, 1 << 20):
            m = min(1 << 20, rows - at)
            x = _rows(g, m, bias)
            if e4m3:
                flat[at:at + m], scale.view(-1)[at:at + m] = _quantise(x)
            else:
                flat[at:at + m] = x
        s[name], s[name + "_scale"], s[name + "_bias"] = pool, scale, bias


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] == "norm":
        _prepare_norm(s, g)
    else:
        _prepare_pages(s, g)
    return s


def _prepare_norm(s, g):
    case = s["case"]
    B, T, H, G, rot = case["seqs"], case["T"], case["heads"], case["G"], case["rot"]
    dev, bf = "cuda", torch.bfloat16
    width = H * (G + 2) * D
    s["qkv"] = torch.empty(B, T, width, dtype=bf, device=dev)
    flat = s["qkv"].view(B * T, width)
    for at in range(0, B * T, 4096):
        m = min(4096, B * T - at)
        flat[at:at + m] = (2.0 * torch.randn(m, width, generator=g, device=dev)).to(bf)
    live = _counts(case)
    s["n"] = _i32(live)
    first = torch.randint(0, max(1, case["far"] - T), (B, 1), generator=g, device=dev)
    s["pos"] = (first + torch.arange(T, device=dev)).to(torch.int32).contiguous()
    weight = lambda: (1.0 + 0.3 * torch.randn(D, generator=g, device=dev)).to(bf)
    s["q_weight"], s["k_weight"] = (weight(), weight()) if case["norm"] else (None, None)
    i = torch.arange(rot // 2, dtype=torch.float64, device=dev)
    s["inv_freq"] = case["base"] ** (-2.0 * i / rot)
    s["q"] = torch.zeros(B * H, T, G, D, dtype=bf, device=dev)
    s["k"] = torch.zeros(B * H, T, D, dtype=bf, device=dev)
    s["v"] = torch.zeros(B * H, T, D, dtype=bf, device=dev)
    if own:
        from kv_cache_eviction_kvc_gb300 import kvc
        s["rope"] = kvc.make_rope(H * G, H, s["inv_freq"], s["q_weight"], s["k_weight"], eps=1e-6,
                                  interleaved=case["interleaved"])


def _prepare_pages(s, g):
    case = s["case"]
    B, H, page, e4m3 = case["seqs"], case["heads"], case["page"], case["e4m3"]
    U, dev, bf = B * H, "cuda", torch.bfloat16
    lens, counts = _lengths(case), None
    added = [0] * B
    if case["op"] == "write":
        counts = added = _counts(case)
    elif case["op"] == "attend":
        added = [int(case["append"])] * B
    elif case["op"] == "read":
        counts = _counts(case)
    need = [-(-(n + a) // page) for n, a in zip(lens, added)]
    n_pages, stride = sum(need) + 3, max(need) + 1
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table, at = torch.full((B, stride), -1, dtype=torch.int32), 0
    order = order.cpu()
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    s["table"], s["len"] = table.to(dev), _i32(lens)
    _fill(s, g, n_pages, H, page, e4m3)
    if case["op"] == "write":
        T = case["T"]
        s["first"], s["count"] = _i32(lens), _i32(counts)
        s["k"] = _rows(g, U * T, s["K_bias"]).view(U, T, D)
        s["v"] = _rows(g, U * T, s["V_bias"]).view(U, T, D)
    elif case["op"] == "read":
        m = case["m"]
        s["slots"] = None
        if m < case["n"]:
            # a list per unit, ascending, spread over the sequence
            n = s["len"].repeat_interleave(H).unsqueeze(-1)
            gap = torch.rand(U, m + 1, generator=g, device=dev, dtype=torch.float64) + 0.01
            c = _i32(counts).unsqueeze(-1)
            gap = torch.where(torch.arange(m + 1, device=dev) <= c, gap, 0.0)
            at = gap.cumsum(1)
            at = at[:, :m] / at[:, -1:] * (n - c).double()
            s["slots"] = (at.long() + torch.arange(m, device=dev)).clamp_max(n.long() - 1)
            s["slots"] = s["slots"].to(torch.int32).contiguous()
        s["count"] = _i32(counts)
        s["k_out"] = torch.zeros(U, m, D, dtype=bf, device=dev)
        s["v_out"] = torch.zeros(U, m, D, dtype=bf, device=dev)
    else:
        G = case["G"]
        s["q"] = (1.5 * torch.randn(U, G, D, generator=g, device=dev)).to(bf)
        s["k"] = s["v"] = None
        if case["append"]:
            s["k"], s["v"] = _rows(g, U, s["K_bias"]), _rows(g, U, s["V_bias"])
        s["o"] = torch.zeros(U, G, D, dtype=bf, device=dev)
        s["lse"] = torch.zeros(U, G, device=dev)
    if own:
        # what a serving program keeps beside its cache: the descriptor and a workspace
        from kv_cache_eviction_kvc_gb300 import kvc
        s["pages"] = kvc.make_pages(s["K"], s["V"], s["K_scale"], s["V_scale"], s["table"], s["len"])
        s["ws"] = torch.zeros(kvc.kvc_page_workspace_size(s["pages"], case.get("G", 1)),
                              dtype=torch.uint8, device=dev)


# ---------------------------------------------------------------- plain forms

def _rotate(x, cos, sin, rot, interleaved):
    """The first `rot` dimensions of the last axis, in pairs (i, i + rot/2) or (2i, 2i + 1)."""
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    c, d = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([c, d], -1).flatten(-2) if interleaved else torch.cat([c, d], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _norm_plain(s):
    case = s["case"]
    B, T, H, G, rot = case["seqs"], case["T"], case["heads"], case["G"], case["rot"]
    x = s["qkv"].view(B, T, H * (G + 2), D)
    angle = s["pos"].double().unsqueeze(-1) * s["inv_freq"]
    cos, sin = angle.cos().float().unsqueeze(2), angle.sin().float().unsqueeze(2)
    live = (torch.arange(T, device="cuda") < s["n"].unsqueeze(-1)).view(B, 1, T, 1)

    def heads(at, count, weight, rotated):
        y = x[:, :, at:at + count].float()
        if rotated:
            if weight is not None:
                y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * weight.float()
            y = _rotate(y, cos, sin, rot, case["interleaved"])
        return y.to(torch.bfloat16)

    q = heads(0, H * G, s["q_weight"], True).view(B, T, H, G * D).transpose(1, 2)
    k = heads(H * G, H, s["k_weight"], True).transpose(1, 2)
    v = heads(H * (G + 1), H, None, False).transpose(1, 2)
    for name, y in (("q", q), ("k", k), ("v", v)):
        out = s[name].view(B, H, T, -1)
        out.copy_(torch.where(live, y, out))
    return {"q": s["q"], "k": s["k"], "v": s["v"]}


def _where(s, slots):
    """Row index in the pool, by unit, of slots [U][m] (clamped into the table)."""
    case = s["case"]
    H, page = case["heads"], case["page"]
    U = case["seqs"] * H
    u = torch.arange(U, device="cuda")
    slots = slots.long().clamp(0, s["table"].shape[1] * page - 1)
    block = torch.gather(s["table"].long().repeat_interleave(H, 0), 1, slots // page).clamp_min(0)
    return (block * H + (u % H).unsqueeze(-1)) * page + slots % page


def _store(s, at, keep, k, v):
    """Rows k, v [U][m][d] into pool rows at [U][m] where `keep` holds."""
    at = at[keep]
    for name, x in (("K", k), ("V", v)):
        x = x[keep]
        if s["case"]["e4m3"]:
            y, scale = _quantise(x)
            s[name].view(torch.uint8).view(-1, D)[at] = y.view(torch.uint8)
            s[name + "_scale"].view(-1)[at] = scale
        else:
            s[name].view(-1, D)[at] = x


def _load(s, name, at):
    """Pool rows at [U][m] in fp32."""
    if s["case"]["e4m3"]:
        rows = s[name].view(torch.uint8).view(-1, D)[at].view(torch.float8_e4m3fn).float()
        return rows * s[name + "_scale"].view(-1)[at].unsqueeze(-1)
    return s[name].view(-1, D)[at].float()


def _pool(s):
    out = {"K": s["K"], "V": s["V"]}
    if s["case"]["e4m3"]:
        out |= {"K_scale": s["K_scale"], "V_scale": s["V_scale"]}
    return out


def _write_plain(s):
    H, T = s["case"]["heads"], s["case"]["T"]
    i = torch.arange(T, device="cuda")
    slots = s["first"].repeat_interleave(H).unsqueeze(-1) + i
    keep = i < s["count"].repeat_interleave(H).unsqueeze(-1)
    _store(s, _where(s, slots), keep, s["k"], s["v"])
    return _pool(s)


def _read_plain(s):
    i = torch.arange(s["case"]["m"], device="cuda")
    slots = s["slots"] if s["slots"] is not None else i.expand(s["k_out"].shape[0], -1)
    keep = (i < s["count"].unsqueeze(-1)).unsqueeze(-1)
    at = _where(s, slots)
    for name, out in (("K", s["k_out"]), ("V", s["v_out"])):
        out.copy_(torch.where(keep, _load(s, name, at).to(torch.bfloat16), out))
    return {"k": s["k_out"], "v": s["v_out"]}


def _attend_plain(s):
    case = s["case"]
    H, U = case["heads"], case["seqs"] * case["heads"]
    n = s["len"].long().repeat_interleave(H).unsqueeze(-1)
    if s["k"] is not None:
        always = torch.ones(U, 1, dtype=torch.bool, device="cuda")
        _store(s, _where(s, n), always, s["k"].unsqueeze(1), s["v"].unsqueeze(1))
        n = n + 1
    i = torch.arange(case["n"] + int(case["append"]), device="cuda")
    at = _where(s, i.expand(U, -1))
    x = torch.matmul(s["q"].float(), _load(s, "K", at).transpose(1, 2)) * SCALE
    x = x.masked_fill((i >= n).unsqueeze(1), -INF)
    top = x.amax(-1, keepdim=True)
    x = (x - top).exp_()
    z = x.sum(-1, keepdim=True)
    # rows behind a sequence are another's: their weight is zero
    f = torch.matmul(x, _load(s, "V", at)) / z
    s["o"].copy_(f)
    s["lse"].copy_((z.log() + top).squeeze(-1))
    return {"o": s["o"], "lse": s["lse"]} | _pool(s)


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from kv_cache_eviction_kvc_gb300 import kvc
        case = s["case"]
        if op == "norm":
            kvc.kvc_qk_norm_rope(s["rope"], s["qkv"], s["pos"], s["n"], s["q"], s["k"], s["v"])
            return {"q": s["q"], "k": s["k"], "v": s["v"]}
        if op == "write":
            kvc.kvc_page_write(s["pages"], s["first"], s["count"], s["k"], s["v"], s["ws"])
            return _pool(s)
        if op == "read":
            kvc.kvc_page_read(s["pages"], s["slots"], s["count"], s["k_out"], s["v_out"], s["ws"])
            return {"k": s["k_out"], "v": s["v_out"]}
        kvc.kvc_page_attend(s["pages"], case["n"] + int(case["append"]), s["q"], s["k"], s["v"],
                            s["o"], s["lse"], s["ws"])
        return {"o": s["o"], "lse": s["lse"]} | _pool(s)
    return {"norm": _norm_plain, "write": _write_plain, "read": _read_plain,
            "attend": _attend_plain}[op](s)


# ----------------------------------------------------------------------- work

def work(case):
    H = case["heads"]
    if case["op"] == "norm":
        tokens = sum(_counts(case))
        rows = tokens * H * (case["G"] + 2)
        return {"bytes": rows * 4 * D + tokens * 4 + case["rot"] * 4,
                "flops": tokens * H * (case["G"] + 1) * (7 * D if case["norm"] else 3 * case["rot"])}
    row = 2 * D + 8 if case["e4m3"] else 4 * D           # a slot's key and value in the pool
    if case["op"] == "write":
        rows = sum(_counts(case)) * H
        return {"bytes": rows * (4 * D + row), "flops": rows * 4 * D}
    if case["op"] == "read":
        rows = sum(_counts(case))
        listed_ = 4 * rows if case["m"] < case["n"] else 0
        return {"bytes": rows * (4 * D + row) + listed_, "flops": rows * 2 * D}
    slots, U, G = sum(_lengths(case)) * H, case["seqs"] * H, case["G"]
    new = U * int(case["append"])
    return {"bytes": slots * row + new * (4 * D + row) + U * G * (4 * D + 4),
            "flops": (slots + new) * G * 4 * D}


# ---------------------------------------------------------------------- exact

def exact(case, seed):
    """The definitions in 64 bits."""
    s = prepare(case, seed)
    return {"norm": _exact_norm, "write": _exact_write, "read": _exact_read,
            "attend": _exact_attend}[case["op"]](s)


def _exact_norm(s):
    case = s["case"]
    H, G, rot = case["heads"], case["G"], case["rot"]
    q, k, v = (s[name].double() for name in ("q", "k", "v"))
    for b, n in enumerate(s["n"].tolist()):
        step = 4096
        for t in range(0, n, step):
            m = min(step, n - t)
            x = s["qkv"][b, t:t + m].double().view(m, -1, D)
            turn = torch.exp(1j * (s["pos"][b, t:t + m].double()[:, None] * s["inv_freq"]))[:, None]
            for h in range(H * (G + 1)):
                y = x[:, h:h + 1]
                w = s["q_weight"] if h < H * G else s["k_weight"]
                if w is not None:
                    y = w.double() * y / torch.sqrt(y.square().sum(-1, keepdim=True) / D + 1e-6)
                y = y.clone()
                pair = ((slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else
                        (slice(0, rot // 2), slice(rot // 2, rot)))
                z = torch.complex(y[..., pair[0]], y[..., pair[1]]) * turn
                y[..., pair[0]], y[..., pair[1]] = z.real, z.imag
                if h < H * G:
                    q[b * H + h // G, t:t + m, h % G] = y[:, 0]
                else:
                    k[b * H + h - H * G, t:t + m] = y[:, 0]
            for h in range(H):
                v[b * H + h, t:t + m] = x[:, H * (G + 1) + h]
    return {"q": q, "k": k, "v": v}


def _exact_scale(x):
    """A row's scale is held in fp32; what it stands for is the row over the scale."""
    scale = (x.abs().amax(-1) / E4M3_MAX).float().clamp_min(TINY)
    return scale, x / scale.double().unsqueeze(-1)


def _exact_put(s, out, b, slots, k, v):
    """Rows k, v [heads][m][d] of sequence b behind one another at slots [m]."""
    page = s["case"]["page"]
    blocks, rows = s["table"][b].long()[slots // page], slots % page
    for name, x in (("K", k), ("V", v)):
        x = x.double().transpose(0, 1)
        if s["case"]["e4m3"]:
            out[name + "_scale"][blocks, :, rows], x = _exact_scale(x)
        out[name][blocks, :, rows] = x


def _exact_write(s):
    H = s["case"]["heads"]
    out = {name: x.double() for name, x in _pool(s).items()}
    for name in ("K_scale", "V_scale"):
        if name in out:
            out[name] = out[name].float()
    for b, (first, n) in enumerate(zip(s["first"].tolist(), s["count"].tolist())):
        slots = torch.arange(first, first + n, device="cuda")
        _exact_put(s, out, b, slots, s["k"][b * H:(b + 1) * H, :n], s["v"][b * H:(b + 1) * H, :n])
    return {name: x.double() for name, x in out.items()}


def _exact_rows(s, name, b, slots):
    """[heads][m][d] of sequence b in 64 bits."""
    page = s["case"]["page"]
    blocks, rows = s["table"][b].long()[slots // page], slots % page
    pool = s[name].view(torch.uint8) if s["case"]["e4m3"] else s[name]
    x = pool[blocks, :, rows].transpose(0, 1)
    if s["case"]["e4m3"]:
        scale = s[name + "_scale"][blocks, :, rows].transpose(0, 1)
        return x.contiguous().view(torch.float8_e4m3fn).double() * scale.double().unsqueeze(-1)
    return x.double()


def _exact_read(s):
    H, m = s["case"]["heads"], s["case"]["m"]
    out = {"k": s["k_out"].double(), "v": s["v_out"].double()}
    for u, n in enumerate(s["count"].tolist()):
        slots = torch.arange(m, device="cuda") if s["slots"] is None else s["slots"][u].long()
        for name, x in (("K", out["k"]), ("V", out["v"])):
            for at in range(0, n, 1 << 16):
                part = slots[at:min(n, at + (1 << 16))]
                x[u, at:at + len(part)] = _exact_rows(s, name, u // H, part)[u % H]
    return out


def _exact_attend(s):
    case = s["case"]
    H, U = case["heads"], case["seqs"] * case["heads"]
    o, lse = s["o"].double(), s["lse"].double()
    out = {name: x.double() for name, x in _pool(s).items()}
    for name in ("K_scale", "V_scale"):
        if name in out:
            out[name] = out[name].float()
    for b, n in enumerate(s["len"].tolist()):
        slots = torch.arange(n, device="cuda")
        k, v = _exact_rows(s, "K", b, slots), _exact_rows(s, "V", b, slots)
        us = slice(b * H, (b + 1) * H)
        if s["k"] is not None:
            new = [x[us].double().unsqueeze(1) for x in (s["k"], s["v"])]
            _exact_put(s, out, b, torch.tensor([n], device="cuda"), *new)
            if case["e4m3"]:
                # the token attends its own row as it is stored
                for i, x in enumerate(new):
                    scale, _ = _exact_scale(x)
                    y = x.float() * (1.0 / scale).unsqueeze(-1)
                    y = y.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
                    new[i] = y.double() * scale.double().unsqueeze(-1)
            k, v = torch.cat([k, new[0]], 1), torch.cat([v, new[1]], 1)
        x = s["q"][us].double() @ k.transpose(1, 2) / math.sqrt(D)
        lse[us] = torch.logsumexp(x, -1)
        o[us] = torch.softmax(x, -1) @ v
    return {"o": o, "lse": lse} | {name: x.double() for name, x in out.items()}
