"""What the sequence-state operators are measured on: the short causal convolution, the selective state
space scan (prompts, single tokens, training) and the page operations of a cache of recurrent states.

`run` computes each case in plain torch operations, or, where `own` is true, through the framework's
entry points.  `exact` computes the same from the definition in float64, token by token.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a training step of the convolution in front of a layer of width 2048, the batch of the 1B layer
        {"name": "conv_train_1b", "op": "conv_train", "dtype": "bf16", "B": 8, "L": 2048, "D": 2048, "W": 4},
        # the same on a small odd model in float32, kernel width 3
        {"name": "conv_train_f32_odd", "op": "conv_train", "dtype": "f32", "B": 3, "L": 515, "D": 1000, "W": 3},
        # a serving batch of ragged prompts of the 125M layer's width, states in pages of a pool
        {"name": "prompt_packed_125m", "op": "prompt", "dtype": "bf16", "lens": "1 700 17 2048 333 0 1901",
         "D": 768, "N": 16, "G": 1, "W": 4, "P": 24},
        # a larger batch of ragged prompts of width 2048
        {"name": "prompt_packed_1b", "op": "prompt", "dtype": "bf16",
         "lens": "512 37 1024 5 2000 815 64 1 1333 256 777 1200", "D": 2048, "N": 16, "G": 1, "W": 4, "P": 40},
        # the prefill of a batch: 8 prompts of 2048 tokens
        {"name": "scan_batch_1b", "op": "scan", "dtype": "bf16", "B": 8, "L": 2048, "D": 2048, "N": 16, "G": 1, "z": True},
        # one long document, the only sequence on the GPU
        {"name": "scan_long_one", "op": "scan", "dtype": "bf16", "B": 1, "L": 8200, "D": 2048, "N": 16, "G": 1, "z": True},
        # a training step through the scan (forward and all gradients), the 1B layer's width
        {"name": "scan_train_1b", "op": "scan_train", "dtype": "bf16", "B": 8, "L": 2048, "D": 2048, "N": 16, "G": 1, "z": True},
        # a small float32 training step: two groups of B and C, 8 states, odd length, no gate
        {"name": "scan_train_f32_groups", "op": "scan_train", "dtype": "f32", "B": 2, "L": 333, "D": 772, "N": 8, "G": 2, "z": False},
        # one decode step (convolution and scan) of 128 sequences, the decode workload's batch, states in pages
        {"name": "step_128", "op": "step", "dtype": "bf16", "B": 128, "D": 4096, "N": 16, "G": 1, "W": 4, "P": 160},
        # one decode step of 3 sequences: latency
        {"name": "step_3", "op": "step", "dtype": "bf16", "B": 3, "D": 768, "N": 16, "G": 1, "W": 4, "P": 8},
        # beam search forks 48 sequences of the 1B layer's TTT cache (32 heads, dense format)
        {"name": "cache_fork_48", "op": "fork", "H": 32, "P": 128, "live": 64, "n": 48},
        # a third of 96 sequences of the 125M layer's cache end; the rest move to the front for the decode step
        {"name": "cache_compact_96", "op": "compact", "H": 12, "P": 128, "live": 96, "n": 32},
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv_train", "prompt", "scan", "scan_train", "step", "fork", "compact"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    if op in ("fork", "compact"):
        H = rng.choice([1, 3, 12, 16, 32])
        P = _logint(rng, 8, 160)
        live = rng.randint(2, P - 2)
        n = rng.randint(1, min(live, P - live) if op == "fork" else live)
        return {"op": op, "H": H, "P": P, "live": live, "n": n}
    D = _logint(rng, 64, 4096)
    if rng.random() < 0.5:
        D = -(-D // 8) * 8
    N = rng.choice([3, 4, 8, 16, 16, 16, 24, 32, 64])
    G = rng.choice([1, 1, 1, 2, 4])
    D = -(-D // G) * G
    W = rng.choice([2, 3, 4, 4])
    if op == "step":
        B = _logint(rng, 1, 256)
        B = max(1, min(B, (128 * 4096 * 16) // (D * N)))
        return {"op": op, "dtype": dt, "B": B, "D": D, "N": N, "G": G, "W": W, "P": B + rng.randint(0, 40)}
    if op == "conv_train":
        B = rng.randint(1, 16)
        L = max(1, min(_logint(rng, 1, 8200), (8 * 2048 * 2048) // (B * D)))
        return {"op": op, "dtype": dt, "B": B, "L": L, "D": D, "W": W}
    most = (8 * 2048 * 2048 * 16) // (D * N * (1 if op != "scan_train" else 2))
    if op == "prompt":
        n = rng.randint(1, 16)
        lens, left = [], min(most, 8200)
        for _ in range(n):
            k = min(left, _logint(rng, 1, 2500) - rng.choice([0, 0, 1]))
            lens.append(k)
            left -= k
        if sum(lens) == 0:
            lens[0] = 1
        return {"op": op, "dtype": dt, "lens": " ".join(map(str, lens)), "D": D, "N": N, "G": G, "W": W, "P": n + rng.randint(0, 20)}
    B = rng.randint(1, 8)
    L = max(1, min(_logint(rng, 1, 8200), most // B))
    return {"op": op, "dtype": dt, "B": B, "L": L, "D": D, "N": N, "G": G, "z": rng.random() < 0.6}


def _lens(c):
    return [int(k) for k in c["lens"].split()]


def _scan_inputs(g, shape, c, dt):
    """Inputs of the scan as a layer makes them: delta before its softplus around log(1e-3 .. 1e-1), A = -(1 .. N)."""
    dev = "cuda"
    rn = lambda *s: torch.randn(*s, device=dev, generator=g)
    D, N, G = c["D"], c["N"], c["G"]
    step = torch.exp(torch.rand(D, device=dev, generator=g) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
    s = {"u": rn(*shape, D).to(dt), "delta": (rn(*shape, D) * 0.5).to(dt),
         "B": rn(*shape, G, N).to(dt), "C": rn(*shape, G, N).to(dt),
         "A": -(torch.arange(1, N + 1, device=dev).float().repeat(D, 1) * (1 + 0.1 * torch.rand(D, N, device=dev, generator=g))),
         "Dskip": 1 + 0.1 * rn(D), "bias": torch.log(torch.expm1(step))}
    s["z"] = rn(*shape, D).to(dt) if c.get("z", True) else None
    return s


def _conv_inputs(g, shape, c, dt):
    rn = lambda *s: torch.randn(*s, device="cuda", generator=g)
    return {"x": rn(*shape, c["D"]).to(dt), "w": rn(c["D"], c["W"]) / math.sqrt(c["W"]), "cb": 0.1 * rn(c["D"])}


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = c["op"]
    s = {"c": c}
    rn = lambda *sh: torch.randn(*sh, device="cuda", generator=g)
    if op in ("fork", "compact"):
        P, H, live, n = c["P"], c["H"], c["live"], c["n"]
        s["pool"] = [rn(P, H, 64, 64), rn(P, H, 64), rn(P, H, 64, 64), rn(P, H, 64)]
        rows = torch.randperm(P, device="cuda", generator=g)
        pages = torch.randperm(P, device="cuda", generator=g)
        table = torch.full((P,), -1, device="cuda", dtype=torch.int32)
        owner = torch.full((P,), -1, device="cuda", dtype=torch.int32)
        table[rows[:live]] = pages[:live].int()
        owner[pages[:live]] = rows[:live].int()
        s["table0"], s["owner0"] = table, owner
        s["table"], s["owner"] = table.clone(), owner.clone()
        if op == "fork":
            s["parents"] = rows[torch.randint(0, live, (n,), device="cuda", generator=g)].int()
            s["children"] = rows[live:live + n].int().contiguous()
        else:
            s["rows"] = rows[:n].int().contiguous()
        return s
    dt = DTYPES[c["dtype"]]
    if op == "step":
        s |= _scan_inputs(g, (c["B"],), c, dt) | _conv_inputs(g, (c["B"],), c, dt)
        s["conv_state"] = rn(c["P"], c["W"] - 1, c["D"]).to(dt)
        s["state"] = rn(c["P"], c["D"], c["N"]) * 0.3
        s["pages"] = torch.randperm(c["P"], device="cuda", generator=g)[:c["B"]].int()
    elif op == "prompt":
        lens = _lens(c)
        T = sum(lens)
        s |= _scan_inputs(g, (T,), c, dt) | _conv_inputs(g, (T,), c, dt)
        s["conv_state"] = rn(c["P"], c["W"] - 1, c["D"]).to(dt)
        s["state"] = rn(c["P"], c["D"], c["N"]) * 0.3
        s["conv_out"], s["state_out"] = torch.zeros_like(s["conv_state"]), torch.zeros_like(s["state"])
        s["pages"] = torch.randperm(c["P"], device="cuda", generator=g)[:len(lens)].int()
        s["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
        s["max_len"] = max(lens)
    else:
        shape = (c["B"], c["L"])
        if op == "conv_train":
            s |= _conv_inputs(g, shape, c, dt)
        else:
            s |= _scan_inputs(g, shape, c, dt)
        s["dout"] = rn(*shape, c["D"]).to(dt)
    return s


# ---- the plain form ---------------------------------------------------------------------------

def _recur(a, b):
    """h with h[:, t] = a[:, t] h[:, t-1] + b[:, t] and h before the start zero, by doubling; a and b are used up."""
    k = 1
    while k < b.shape[1]:
        b[:, k:] += a[:, k:] * b[:, :-k]
        a[:, k:] = a[:, k:] * a[:, :-k]
        k *= 2
    return b


def _silu_grad(x):
    g = torch.sigmoid(x)
    return g * (1 + x * (1 - g))


def _plain_scan(s, first=None, h0=None):
    """The scan over [B, L, ...]; rows of `first` start a sequence from h0's rows.  Returns what the gradients need too."""
    u, delta = s["u"].float(), s["delta"].float() + s["bias"]
    r = u.shape[-1] // s["B"].shape[-2]
    Bm, Cm = (s[k].float().repeat_interleave(r, -2) for k in ("B", "C"))
    dt = torch.nn.functional.softplus(delta, threshold=60.0)
    a = torch.exp(dt.unsqueeze(-1) * s["A"])
    b = (dt * u).unsqueeze(-1) * Bm
    if first is not None:
        b[:, first] += a[:, first] * h0
        a[:, first] = 0
    h = _recur(a.clone(), b)
    y = (h * Cm).sum(-1) + s["Dskip"] * u
    z = None if s["z"] is None else s["z"].float()
    out = (y if z is None else y * z * torch.sigmoid(z)).to(s["u"].dtype)
    return out, dict(u=u, delta=delta, dt=dt, a=a, h=h, Bm=Bm, Cm=Cm, y=y, z=z, r=r)


def _plain_scan_grads(s, v):
    u, dt, a, h, dtype = v["u"], v["dt"], v["a"], v["h"], s["u"].dtype
    dout = s["dout"].float()
    g = {}
    dy = dout
    if v["z"] is not None:
        g["dz"] = (dout * v["y"] * _silu_grad(v["z"])).to(dtype)
        dy = dout * v["z"] * torch.sigmoid(v["z"])
    group = lambda t: t.unflatten(-2, (-1, v["r"])).sum(-2).to(dtype)
    g["dC"] = group(dy.unsqueeze(-1) * h)
    after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1).flip(1)
    dh = _recur(after, (dy.unsqueeze(-1) * v["Cm"]).flip(1)).flip(1)
    g["dB"] = group(dh * (dt * u).unsqueeze(-1))
    along = (dh * v["Bm"]).sum(-1)
    back = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1).mul_(a).mul_(dh)
    g["dA"] = (back * dt.unsqueeze(-1)).sum((0, 1))
    ddt = (back * s["A"]).sum(-1) + along * u
    ddelta = ddt * torch.sigmoid(v["delta"])
    g["ddelta"], g["ddelta_bias"] = ddelta.to(dtype), ddelta.sum((0, 1))
    g["du"] = (dy * s["Dskip"] + dt * along).to(dtype)
    g["dD"] = (dy * u).sum((0, 1))
    return g


def _plain_conv(x, w, cb):
    """The convolution of rows x [..., L + W - 1, D], the first W - 1 of them what came before."""
    return (x.float().unfold(-2, w.shape[1], 1) * w).sum(-1) + cb


def _plain_conv_train(s):
    x, w, W = s["x"], s["w"], s["w"].shape[1]
    wide = torch.nn.functional.pad(x.float(), (0, 0, W - 1, 0))
    pre = _plain_conv(wide, w, s["cb"])
    dpre = s["dout"].float() * _silu_grad(pre)
    ahead = torch.nn.functional.pad(dpre, (0, 0, 0, W - 1))
    dx = (ahead.unfold(-2, W, 1) * w.flip(1)).sum(-1)
    dw = (wide.unfold(-2, W, 1) * dpre.unsqueeze(-1)).double().sum((0, 1)).float()
    return {"out": (pre * torch.sigmoid(pre)).to(x.dtype), "dx": dx.to(x.dtype), "dweight": dw,
            "dbias": dpre.double().sum((0, 1)).float()}


def _plain_prompt(s):
    cu, pages, W = s["cu"].long(), s["pages"].long(), s["w"].shape[1]
    x, T = s["x"], s["x"].shape[0]
    lens = cu[1:] - cu[:-1]
    t = torch.arange(T, device=x.device)
    seq = torch.searchsorted(cu[1:], t, right=True)
    back = torch.arange(1 - W, 1, device=x.device)
    at = (t - cu[seq]).unsqueeze(1) + back                          # position in its sequence of each tap
    before = s["conv_state"][pages]                                 # [n, W-1, D]
    take = lambda n, pos: torch.where((pos < 0).unsqueeze(-1), before[n, (pos + W - 1).clamp(0, W - 2)],
                                      x[(cu[n] + pos).clamp(0, T - 1)])
    pre = (take(seq.unsqueeze(1).expand_as(at), at).float() * s["w"].t()).sum(1) + s["cb"]
    n = torch.arange(len(lens), device=x.device).unsqueeze(1)
    s["conv_out"][pages] = take(n.expand(-1, W - 1), lens.unsqueeze(1) + back[:-1])
    alive = (lens > 0).nonzero().squeeze(1)
    packed = {k: (v.unsqueeze(0) if k in ("u", "delta", "B", "C", "z") else v) for k, v in s.items()}
    out, v = _plain_scan(packed, cu[:-1][alive], s["state"][pages[alive]])
    s["state_out"][pages] = s["state"][pages]
    s["state_out"][pages[alive]] = v["h"][0, cu[1:][alive] - 1]
    return [(pre * torch.sigmoid(pre)).to(x.dtype), s["conv_out"], out[0], s["state_out"]]


def _plain_step(s):
    pages = s["pages"].long()
    wide = torch.cat([s["conv_state"][pages], s["x"].unsqueeze(1)], 1)
    pre = _plain_conv(wide, s["w"], s["cb"]).squeeze(1)
    s["conv_state"][pages] = wide[:, 1:]
    one = {k: (v.unsqueeze(1) if k in ("u", "delta", "B", "C", "z") else v) for k, v in s.items()}
    first = torch.zeros(1, dtype=torch.long, device=pages.device)
    out, v = _plain_scan(one, first, s["state"][pages].unsqueeze(1))
    s["state"][pages] = v["h"][:, 0]
    return [(pre * torch.sigmoid(pre)).to(s["x"].dtype), s["conv_state"], out[:, 0], s["state"]]


def _copy_pages(pool, src, dst):
    pool[0][dst], pool[1][dst], pool[2][dst], pool[3][dst] = pool[0][src], pool[1][src], pool[2][src], pool[3][src]


def _plain_fork(s):
    table, owner, parents, children = s["table"], s["owner"], s["parents"].long(), s["children"].long()
    src = table[parents].long()
    free = torch.sort((owner >= 0).to(torch.int8), stable=True).indices   # the free pages, lowest first
    dst = free[:len(children)]
    table[children] = dst.int()
    owner[dst] = s["children"]
    _copy_pages(s["pool"], src, dst)
    return [dst.int(), table, owner, *s["pool"]]


def _plain_compact(s):
    table, owner, rows = s["table"], s["owner"], s["rows"].long()
    owner[table[rows].long()] = -1
    table[rows] = -1
    held = owner >= 0
    count = held.sum()
    low = torch.arange(len(owner), device=owner.device) < count
    src, dst = (held & ~low).nonzero().squeeze(1), (~held & low).nonzero().squeeze(1)
    _copy_pages(s["pool"], src, dst)
    owner[dst] = owner[src]
    owner[src] = -1
    table[owner[dst].long()] = dst.int()
    return [count.int(), table, owner, *s["pool"]]


def _plain(s):
    op = s["c"]["op"]
    if op == "conv_train":
        return _plain_conv_train(s)
    if op == "prompt":
        return _plain_prompt(s)
    if op == "scan":
        return [_plain_scan(s)[0]]
    if op == "scan_train":
        out, v = _plain_scan(s)
        return {"out": out, **_plain_scan_grads(s, v)}
    if op == "step":
        return _plain_step(s)
    return _plain_fork(s) if op == "fork" else _plain_compact(s)


# ---- through the framework --------------------------------------------------------------------

def _own(s):
    import test_rnn_layers_b200 as ttt
    c = s["c"]
    op = c["op"]
    if op == "conv_train":
        out = ttt.ttt_causal_conv_forward(s["x"], s["w"], s["cb"])
        return {"out": out, **ttt.ttt_causal_conv_backward(s["x"], s["w"], s["dout"], s["cb"])}
    if op in ("scan", "scan_train"):
        args = (s["u"], s["delta"], s["A"], s["B"], s["C"])
        more = dict(D=s["Dskip"], z=s["z"], delta_bias=s["bias"])
        if op == "scan":
            return [ttt.ttt_selective_scan_forward(*args, **more)]
        n = ttt.ttt_selective_scan_ckpt_bytes(c["B"], c["L"], c["D"], c["N"])
        ckpt = torch.empty(n // 4, device="cuda")
        out = ttt.ttt_selective_scan_forward(*args, **more, ckpt=ckpt)
        return {"out": out, **ttt.ttt_selective_scan_backward(*args, s["dout"], ckpt, **more)}
    if op == "prompt":
        y = ttt.ttt_causal_conv_forward(s["x"], s["w"], s["cb"], state_in=s["conv_state"], state_out=s["conv_out"],
                                        pages=s["pages"], cu_seqlens=s["cu"])
        out = ttt.ttt_selective_scan_forward(s["u"], s["delta"], s["A"], s["B"], s["C"], D=s["Dskip"], z=s["z"],
                                             delta_bias=s["bias"], state_in=s["state"], state_out=s["state_out"],
                                             pages=s["pages"], cu_seqlens=s["cu"], max_seqlen=s["max_len"])
        return [y, s["conv_out"], out, s["state_out"]]
    if op == "step":
        y = ttt.ttt_causal_conv_step(s["x"], s["conv_state"], s["w"], s["cb"], pages=s["pages"])
        out = ttt.ttt_selective_scan_step(s["u"], s["delta"], s["A"], s["B"], s["C"], s["state"], D=s["Dskip"],
                                          z=s["z"], delta_bias=s["bias"], pages=s["pages"])
        return [y, s["conv_state"], out, s["state"]]
    if op == "fork":
        pages = ttt.ttt_cache_fork(s["pool"], s["table"], s["owner"], s["parents"], s["children"])
        return [pages, s["table"], s["owner"], *s["pool"]]
    ttt.ttt_cache_free(s["table"], s["owner"], s["rows"])
    count, _ = ttt.ttt_cache_compact(s["pool"], s["table"], s["owner"])
    return [count, s["table"], s["owner"], *s["pool"]]


def run(state):
    if state["c"]["op"] in ("fork", "compact"):  # each pass starts from the same bookkeeping
        state["table"].copy_(state["table0"])
        state["owner"].copy_(state["owner0"])
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without --------------------------------------------------------------

def work(case):
    c = case
    op = c["op"]
    if op in ("fork", "compact"):
        page = c["H"] * (2 * 64 * 64 + 2 * 64) * 4
        if op == "fork":
            moved = c["n"]
        else:  # live pages that lie past the new end: they are drawn at random, so their expected number
            left = c["live"] - c["n"]
            moved = left * (c["P"] - left) / c["P"]
        return {"bytes": 2 * moved * page + 16 * c["P"], "flops": 0}
    e = 2 if c["dtype"] == "bf16" else 4
    D, W = c["D"], c.get("W", 0)
    if op == "conv_train":
        td = c["B"] * c["L"] * D
        return {"bytes": 4 * td * e + 8 * D * (W + 1), "flops": td * (6 * W + 12)}
    N, G = c["N"], c["G"]
    if op == "step":
        td = c["B"] * D
        return {"bytes": td * (6 * e + 2 * (W - 1) * e + 8 * N) + 2 * c["B"] * G * N * e + 4 * D * (N + W + 3),
                "flops": td * (7 * N + 2 * W + 12)}
    T = sum(_lens(c)) if op == "prompt" else c["B"] * c["L"]
    td = T * D
    gate = 1 if c.get("z", True) else 0
    params = 4 * D * (N + 2)
    if op == "scan_train":
        return {"bytes": td * e * (6 + 2 * gate) + 4 * T * G * N * e + 2 * params, "flops": td * (26 * N + 40)}
    b = td * e * (3 + gate) + 2 * T * G * N * e + params
    f = td * (7 * N + 8)
    if op == "prompt":
        n = len(_lens(c))
        b += td * e * 2 + 4 * D * (W + 1) + n * D * (2 * (W - 1) * e + 8 * N)
        f += td * (2 * W + 4)
    return {"bytes": b, "flops": f}


# ---- the definition in 64 bits, token by token ------------------------------------------------------

def _exact_scan(s, starts, h0):
    """Over [T, B, D]-ordered rows: (out, h of every token) with the state reset to h0[i] at token starts[i]."""
    u, delta, Bm, Cm = (s[k].double() for k in ("u", "delta", "B", "C"))
    r = u.shape[-1] // Bm.shape[-2]
    pre = delta + s["bias"].double()
    dt = torch.clamp(pre, min=0) + torch.log1p(torch.exp(-pre.abs()))
    A = s["A"].double()
    hs, ys = [], []
    h = torch.zeros(*u.shape[1:], A.shape[1], dtype=torch.float64, device=u.device)
    for t in range(u.shape[0]):
        if t in starts:
            h = h0[starts[t]]
        bt, ct = Bm[t].repeat_interleave(r, -2), Cm[t].repeat_interleave(r, -2)
        h = torch.exp(dt[t].unsqueeze(-1) * A) * h + (dt[t] * u[t]).unsqueeze(-1) * bt
        ys.append((h * ct).sum(-1))
        hs.append(h if s.get("keep", True) else None)
    y = torch.stack(ys) + s["Dskip"].double() * u
    z = None if s["z"] is None else s["z"].double()
    return (y if z is None else y * z / (1 + torch.exp(-z))), hs, y, dt, pre, h


def _exact_grads(s, hs, y, dt, pre):
    u, Bm, Cm, dout, A = (s[k].double() for k in ("u", "B", "C", "dout", "A"))
    T, r = u.shape[0], u.shape[-1] // Bm.shape[-2]
    g = {}
    dy = dout
    if s["z"] is not None:
        z = s["z"].double()
        sg = 1 / (1 + torch.exp(-z))
        g["dz"] = dout * y * (sg + z * sg * (1 - sg))
        dy = dout * z * sg
    du, ddt, dB, dC = torch.empty_like(u), torch.empty_like(u), torch.empty_like(Bm), torch.empty_like(Cm)
    dA = torch.zeros_like(A)
    carry = torch.zeros_like(hs[0])
    for t in range(T - 1, -1, -1):
        bt, ct = Bm[t].repeat_interleave(r, -2), Cm[t].repeat_interleave(r, -2)
        dh = carry + dy[t].unsqueeze(-1) * ct
        dC[t] = (dy[t].unsqueeze(-1) * hs[t]).unflatten(-2, (-1, r)).sum(-2)
        dB[t] = (dh * (dt[t] * u[t]).unsqueeze(-1)).unflatten(-2, (-1, r)).sum(-2)
        carry = dh * torch.exp(dt[t].unsqueeze(-1) * A)
        q = (dh * bt).sum(-1)
        du[t] = dy[t] * s["Dskip"].double() + dt[t] * q
        ddt[t] = u[t] * q
        if t:
            p = carry * hs[t - 1]
            ddt[t] += (p * A).sum(-1)
            dA += (p * dt[t].unsqueeze(-1)).sum(0)
    ddelta = ddt / (1 + torch.exp(-pre))
    return {**g, "dC": dC, "dB": dB, "dA": dA, "ddelta": ddelta, "ddelta_bias": ddelta.sum((0, 1)), "du": du,
            "dD": (dy * u).sum((0, 1))}


def _exact_conv(rows, w, cb):
    """Outputs before the activation for rows [..., L + W - 1, D]."""
    W = w.shape[1]
    L = rows.shape[-2] - W + 1
    return sum(rows[..., k:k + L, :] * w[:, k].double() for k in range(W)) + cb.double()


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    op = c["op"]
    if op in ("fork", "compact"):
        return None
    acts = ("u", "delta", "B", "C", "z", "dout")
    if op == "conv_train":
        w, W = s["w"].double(), c["W"]
        rows = torch.cat([torch.zeros(c["B"], W - 1, c["D"], dtype=torch.float64, device="cuda"), s["x"].double()], 1)
        pre = _exact_conv(rows, s["w"], s["cb"])
        sg = 1 / (1 + torch.exp(-pre))
        dpre = s["dout"].double() * (sg + pre * sg * (1 - sg))
        drows = torch.zeros_like(rows)
        for k in range(W):
            drows[:, k:k + c["L"]] += dpre * w[:, k]
        dw = torch.stack([(dpre * rows[:, k:k + c["L"]]).sum((0, 1)) for k in range(W)], 1)
        return {"out": pre * sg, "dx": drows[:, W - 1:], "dweight": dw, "dbias": dpre.sum((0, 1))}
    if op in ("scan", "scan_train"):
        t = {k: (v.transpose(0, 1) if k in acts and v is not None else v) for k, v in s.items()}
        t["keep"] = op == "scan_train"
        out, hs, y, dt, pre, _ = _exact_scan(t, {}, None)
        if op == "scan":
            return [out.transpose(0, 1)]
        g = _exact_grads(t, hs, y, dt, pre)
        rows = ("dz", "dC", "dB", "ddelta", "du")
        g = {k: (v.transpose(0, 1) if k in rows else v) for k, v in g.items()}
        return {"out": out.transpose(0, 1), **g}
    pages = s["pages"].long()
    if op == "step":
        rows = torch.cat([s["conv_state"][pages], s["x"].unsqueeze(1)], 1).double()
        pre = _exact_conv(rows, s["w"], s["cb"])[:, 0]
        s["conv_state"][pages] = rows[:, 1:].to(s["conv_state"].dtype)
        t = {k: (v.unsqueeze(0) if k in acts and v is not None else v) for k, v in s.items()}
        state = s["state"].double()
        out, _, _, _, _, h = _exact_scan(t, {0: 0}, [state[pages]])
        state[pages] = h
        return [pre / (1 + torch.exp(-pre)), s["conv_state"].double(), out[0], state]
    cu, W, lens = s["cu"].tolist(), c["W"], _lens(c)
    y = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
    for i, n in enumerate(lens):
        rows = torch.cat([s["conv_state"][pages[i]], s["x"][cu[i]:cu[i + 1]]]).double()
        if n:
            pre = _exact_conv(rows, s["w"], s["cb"])
            y[cu[i]:cu[i + 1]] = pre / (1 + torch.exp(-pre))
        s["conv_out"][pages[i]] = rows[n:].to(s["conv_out"].dtype)
    alive = [i for i, n in enumerate(lens) if n]
    h0 = [s["state"][pages[i]].double() for i in range(len(lens))]
    out, hs, _, _, _, _ = _exact_scan(s, {cu[i]: i for i in alive}, h0)
    state = s["state_out"].double()
    for i in range(len(lens)):
        state[pages[i]] = hs[cu[i + 1] - 1] if i in alive else h0[i]
    return [y, s["conv_out"].double(), out, state]
