"""Plain float64 forms of the causal convolution, the selective scan, their gradients and the cache's
page operations, token by token and request by request, on the CPU.

`scan` and `scan_grads` also run on magnitudes: with every operand replaced by its absolute value (and
the decay factors as they are) they give, entry by entry, the sum M of the absolute values of all
terms of a result.  A result whose terms each pass through at most c roundings of float32 is off by at
most c 2^-24 M, whatever the order of its sums, and then by half a step of the type it is stored in.
"""
import math

import torch

F32 = 2.0 ** -24  # half a step of float32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def sequences(n_seq, L, cu):
    """(first row, length) pairs into rows flattened over the batch."""
    if cu is None:
        return [(b * L, L) for b in range(n_seq)]
    return [(cu[b], cu[b + 1] - cu[b]) for b in range(n_seq)]


def conv(x, w, bias, state, silu=True):
    """One sequence: x [len, D], w [D, W], state [W-1, D] -> (out, state after, pre, M of pre)."""
    W = w.shape[1]
    rows = torch.cat([state, x])
    taps = [rows[k:k + len(x)] * w[:, k] for k in range(W)]
    pre = sum(taps) + bias
    mag = sum(t.abs() for t in taps) + bias.abs()
    out = pre * torch.sigmoid(pre) if silu else pre
    return out, rows[len(x):], pre, mag


def step_sizes(delta, bias, softplus):
    x = delta + bias
    return (torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs())), torch.sigmoid(x)) if softplus else (x, torch.ones_like(x))


def scan(u, dt, a, B, C, D, gate, h0):
    """One sequence: u, dt, gate [len, D], a [len, D, N], B, C [len, D, N] (per channel), h0 [D, N] ->
    (out, y, states [len + 1, D, N])."""
    hs, ys = [h0], []
    for t in range(len(u)):
        h = a[t] * hs[-1] + (dt[t] * u[t])[:, None] * B[t]
        hs.append(h)
        ys.append((C[t] * h).sum(-1) + D * u[t])
    y = torch.stack(ys) if ys else torch.zeros_like(u)
    return y * gate, y, torch.stack(hs)


def scan_grads(u, dt, a, A, B, C, D, dy, hs, dh_last):
    """Gradients of one sequence: dict of dB, dC (per channel), du, ddt, dA, dD, dstate_in."""
    n = len(u)
    g = {k: torch.zeros_like(B) for k in ("dB", "dC")} | {k: torch.zeros_like(u) for k in ("du", "ddt")}
    dA, carry = torch.zeros_like(A), dh_last.clone()
    for t in range(n - 1, -1, -1):
        dh = carry + dy[t][:, None] * C[t]
        g["dC"][t] = dy[t][:, None] * hs[t + 1]
        g["dB"][t] = dh * (dt[t] * u[t])[:, None]
        through = (dh * B[t]).sum(-1)
        carry = dh * a[t]
        back = carry * hs[t]
        g["du"][t] = D * dy[t] + dt[t] * through
        g["ddt"][t] = (back * A).sum(-1) + u[t] * through
        dA += back * dt[t][:, None]
    return g | {"dA": dA, "dD": (dy * u).sum(0), "dstate_in": carry}


class Scan:
    """Inputs of a scan (dense or packed rows, float64 copies of what the kernel sees), its results and
    their magnitudes; gradients on demand."""

    def __init__(self, u, delta, A, B, C, D, z, bias, softplus, h0, n_seq, L, cu):
        d = lambda t: None if t is None else t.detach().double().cpu()
        flat = lambda t, k: None if t is None else d(t).reshape(-1, *t.shape[t.dim() - k:])
        self.u, self.delta, self.z = flat(u, 1), flat(delta, 1), flat(z, 1)
        r = u.shape[-1] // B.shape[-2]
        self.B, self.C = (flat(t, 2).repeat_interleave(r, 1) for t in (B, C))
        self.A, self.r, self.seqs = d(A), r, sequences(n_seq, L, cu)
        zero = torch.zeros(u.shape[-1], dtype=torch.float64)
        self.D, self.bias = (zero if t is None else d(t) for t in (D, bias))
        self.dt, self.slope = step_sizes(self.delta, self.bias, softplus)
        self.a = torch.exp(self.dt[..., None] * self.A)
        s = torch.ones_like(self.u) if z is None else self.z * torch.sigmoid(self.z)
        self.gate = s
        self.h0 = torch.zeros(n_seq, *self.A.shape, dtype=torch.float64) if h0 is None else d(h0)
        self.out, self.y, self.out_mag = torch.zeros_like(self.u), torch.zeros_like(self.u), torch.zeros_like(self.u)
        self.hs, self.hs_mag, self.last, self.last_mag = [], [], [], []
        for b, (t0, n) in enumerate(self.seqs):
            k = slice(t0, t0 + n)
            self.out[k], self.y[k], hs = scan(self.u[k], self.dt[k], self.a[k], self.B[k], self.C[k], self.D, s[k], self.h0[b])
            om, _, hm = scan(self.u[k].abs(), self.dt[k].abs(), self.a[k], self.B[k].abs(), self.C[k].abs(), self.D.abs(),
                             s[k].abs(), self.h0[b].abs())
            self.out_mag[k] = om
            self.hs.append(hs), self.hs_mag.append(hm), self.last.append(hs[-1]), self.last_mag.append(hm[-1])
        longest = max([n for _, n in self.seqs] + [0])
        # roundings that a term of a state or of its gradient passes through: a token's decay factor is
        # within 2^-22 of exp(dt A) for the dt A it is given, which is off by 8 roundings (dt: softplus
        # within 6, the two products), and is multiplied and added (2); 64 for what is done once (the
        # products, the gate's sigmoid, sums over up to 64 states, the sums over lanes and blocks)
        m = float((self.dt[..., None] * self.A).abs().max()) if self.dt.numel() else 0.0
        self.c = 64 + longest * (4 + 8 * m + 2)

    def grads(self, dout, dlast):
        """(gradients, magnitudes) for the gradients of out and of the states after the sequences."""
        dout = dout.detach().double().cpu().reshape(self.u.shape)
        dlast = [torch.zeros_like(self.A)] * len(self.seqs) if dlast is None else dlast.detach().double().cpu()
        shapes = {"du": self.u, "ddelta": self.u, "dz": self.u, "dB": self.B, "dC": self.B}
        both = []
        for mag in (False, True):
            f = (lambda t: t.abs()) if mag else (lambda t: t)
            g = {k: torch.zeros_like(v) for k, v in shapes.items()}
            g |= {"dA": torch.zeros_like(self.A), "dD": torch.zeros_like(self.D), "dstate_in": torch.zeros_like(self.h0)}
            dy = f(dout * self.gate)
            for b, (t0, n) in enumerate(self.seqs):
                k = slice(t0, t0 + n)
                hs = (self.hs_mag if mag else self.hs)[b]
                r = scan_grads(f(self.u[k]), f(self.dt[k]), self.a[k], f(self.A), f(self.B[k]), f(self.C[k]), f(self.D),
                               dy[k], hs, f(dlast[b]))
                for n_ in ("du", "dB", "dC"):
                    g[n_][k] = r[n_]
                g["ddelta"][k] = r["ddt"] * self.slope[k]
                g["dA"] += r["dA"]
                g["dD"] += r["dD"]
                g["dstate_in"][b] = r["dstate_in"]
            if self.z is not None:
                sg = torch.sigmoid(self.z)
                slope = sg * (1 + self.z * (1 - sg))
                y = self.y
                if mag:  # y without its gate
                    y = torch.zeros_like(self.u)
                    for b, (t0, n) in enumerate(self.seqs):
                        k = slice(t0, t0 + n)
                        y[k] = (self.hs_mag[b][1:] * self.C[k].abs()).sum(-1) + (self.D * self.u[k]).abs()
                # 1 + z (1 - sigmoid): both terms, where they cancel
                g["dz"] = f(dout) * y * (sg * (1 + self.z.abs() * (1 - sg)) if mag else slope)
            else:
                g.pop("dz")
            g["ddelta_bias"] = g["ddelta"].sum(0)
            for n_ in ("dB", "dC"):
                g[n_] = g[n_].unflatten(1, (-1, self.r)).sum(2)
            both.append(g)
        return both


def check(name, got, want, mag, c, dtype):
    """got within c roundings of float32 of each term, and half a step of its own type."""
    got = got.detach().double().cpu().reshape(want.shape)
    assert torch.isfinite(got).all(), name
    tol = c * F32 * mag + (half_step(dtype) * want.abs() if dtype != torch.float32 else 0) + 1e-30
    if dtype != torch.float32:  # what is rounded is the kernel's value, itself off by the first term
        tol = tol * (1 + half_step(dtype))
    off = ((got - want).abs() / tol).max().item() if got.numel() else 0.0
    assert off <= 1.0, f"{name}: {off:.3g} times the bound"


def fork(table, owner, parents, children, n_pages):
    """Books of ttt_cache_fork on lists, in place: (pages, [(source or -1, page)])."""
    before, pages, moves, claimed = list(table), [], [], set()
    for p, c in zip(parents, children):
        ok = 0 <= c < len(table) and before[c] < 0 and c not in claimed and (p == -1 or (0 <= p < len(table) and before[p] >= 0))
        page = -1
        if ok:
            claimed.add(c)
            free = [k for k in range(n_pages) if owner[k] < 0]
            if free:
                page = free[0]
                owner[page], table[c] = c, page
                moves.append((before[p] if p >= 0 else -1, page))
        pages.append(page)
    return pages, moves


def compact(table, owner):
    """Books of ttt_cache_compact on lists, in place: (live, new_page, [(source, destination)])."""
    live = sum(o >= 0 for o in owner)
    holes = [k for k in range(live) if owner[k] < 0]
    late = [k for k in range(live, len(owner)) if owner[k] >= 0]
    new = [k if o >= 0 else -1 for k, o in enumerate(owner)]
    for src, dst in zip(late, holes):
        owner[dst], owner[src] = owner[src], -1
        table[owner[dst]] = dst
        new[src] = dst
    return live, new, list(zip(late, holes))
