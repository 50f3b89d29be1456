"""The selective scan (prompts, single tokens, gradients) against its float64 form; the tolerances
count roundings (seq_ref.Scan.c, seq_ref.check)."""
import math

import pytest
import torch

import seq_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def inputs(lead, D, N, G, dt, seed, z=True, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)
    step = torch.exp(torch.rand(D, generator=g) * math.log(100.0) + math.log(1e-3))
    s = dict(u=rn(*lead, D).to(dt), delta=(scale * rn(*lead, D)).to(dt), A=-(1 + rn(D, N).abs() * 4),
             B=rn(*lead, G, N).to(dt), C=rn(*lead, G, N).to(dt), D=rn(D), z=rn(*lead, D).to(dt) if z else None,
             delta_bias=torch.log(torch.expm1(step)))
    return {k: v if v is None else v.cuda() for k, v in s.items()}


def positional(s):
    return [s[k] for k in ("u", "delta", "A", "B", "C")], dict(D=s["D"], z=s["z"], delta_bias=s["delta_bias"])


CASES = [  # n_seq, L, D, N, G, dtype, z
    (1, 1, 1, 1, 1, "f32", False), (2, 7, 5, 3, 1, "f32", True), (1, 16, 64, 16, 1, "bf16", True),
    (2, 17, 72, 16, 2, "bf16", True), (3, 40, 10, 4, 1, "f32", False), (2, 33, 12, 8, 4, "bf16", True),
    (1, 65, 130, 16, 1, "f32", True), (2, 24, 70, 24, 2, "bf16", False), (1, 50, 9, 32, 3, "f32", True),
    (2, 31, 6, 64, 1, "bf16", True), (1, 23, 33, 33, 1, "f32", True), (1, 100, 300, 2, 1, "f32", True),
]


def want_of(s, n_seq, L, cu=None, h0=None, softplus=True):
    return ref.Scan(s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"], s["delta_bias"], softplus, h0, n_seq, L, cu)


@pytest.mark.parametrize("n_seq,L,D,N,G,dt,z", CASES)
@pytest.mark.parametrize("softplus", [True, False])
def test_forward_and_state(libttt, n_seq, L, D, N, G, dt, z, softplus):
    s = inputs((n_seq, L), D, N, G, DT[dt], 3, z)
    if not softplus:
        s["delta"], s["delta_bias"] = s["delta"].abs() * 0.1, None
    pool = torch.randn(n_seq + 2, D, N, generator=torch.Generator().manual_seed(9)).cuda()
    pages = torch.randperm(n_seq + 2, generator=torch.Generator().manual_seed(3))[:n_seq]
    want = want_of(s, n_seq, L, h0=pool[pages.cuda()], softplus=softplus)
    a, k = positional(s)
    after = pool.clone()
    out = libttt.ttt_selective_scan_forward(*a, **k, softplus=softplus, state_in=after, state_out=after, pages=pages.int().cuda())
    ref.check("out", out, want.out, want.out_mag, want.c, DT[dt])
    ref.check("state", after[pages.cuda()], torch.stack(want.last), torch.stack(want.last_mag), want.c, torch.float32)
    rest = [p for p in range(n_seq + 2) if p not in pages.tolist()]
    assert torch.equal(after[rest], pool[rest])
    plain = want_of(s, n_seq, L, softplus=softplus)
    out = libttt.ttt_selective_scan_forward(*a, **k, softplus=softplus)
    ref.check("out without a state", out, plain.out, plain.out_mag, plain.c, DT[dt])


@pytest.mark.parametrize("L", [255, 256, 400, 1000])
@pytest.mark.parametrize("N,G,D,n_seq", [(16, 1, 40, 2), (5, 2, 6, 1), (64, 1, 8, 1)])
def test_long_sequences_in_spans(libttt, L, N, G, D, n_seq):
    """Lengths where the work is cut into spans of tokens, in place on the state pages."""
    if L >= 400:
        assert libttt.ttt_selective_scan_workspace_bytes(n_seq, L, D, N, G) > 0
    s = inputs((n_seq, L), D, N, G, torch.float32, 4)
    pool = torch.randn(n_seq, D, N, generator=torch.Generator().manual_seed(9)).cuda()
    want = want_of(s, n_seq, L, h0=pool)
    a, k = positional(s)
    n = libttt.ttt_selective_scan_ckpt_bytes(n_seq, L, D, N)
    ckpt = torch.empty(n // 4, device="cuda")
    out = libttt.ttt_selective_scan_forward(*a, **k, state_in=pool, state_out=pool, ckpt=ckpt)
    ref.check("out", out, want.out, want.out_mag, want.c, torch.float32)
    ref.check("state", pool, torch.stack(want.last), torch.stack(want.last_mag), want.c, torch.float32)
    kept = torch.stack([h[:L:8] for h in want.hs])
    ref.check("ckpt", ckpt.view(kept.shape), kept, torch.stack([h[:L:8] for h in want.hs_mag]), want.c, torch.float32)


@pytest.mark.parametrize("lens", [[9], [0, 1, 70, 0, 3, 16, 64, 2], [17, 0], [1] * 7, [700, 5, 300]])
@pytest.mark.parametrize("dt,D,N,G", [("bf16", 40, 16, 1), ("f32", 9, 6, 3)])
@pytest.mark.parametrize("known", [True, False])
def test_packed(libttt, lens, dt, D, N, G, known):
    n, T = len(lens), sum(lens) + 3
    s = inputs((T,), D, N, G, DT[dt], 6)
    cu = [0]
    for m in lens:
        cu.append(cu[-1] + m)
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    pool = torch.randn(n, D, N, generator=torch.Generator().manual_seed(9)).cuda()
    pages = torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda")
    want = want_of(s, n, T, cu, h0=pool.flip(0))
    a, k = positional(s)
    out = torch.full_like(s["u"], 9.0)
    libttt.ttt_selective_scan_forward(*a, **k, state_in=pool, state_out=pool, pages=pages, cu_seqlens=cut, out=out,
                                      max_seqlen=max(lens) if known else 0)
    assert (out[cu[-1]:] == 9.0).all()
    ref.check("out", out[:cu[-1]], want.out[:cu[-1]], want.out_mag[:cu[-1]], want.c, DT[dt])
    ref.check("state", pool.flip(0), torch.stack(want.last), torch.stack(want.last_mag), want.c, torch.float32)


def check_grads(lib, s, n_seq, L, dt, cu=None, cut=None, h0=None, dlast=None, seed=8):
    a, k = positional(s)
    lead = s["u"].shape[:-1]
    D, N = s["A"].shape
    packed = cu is not None
    ckpt = torch.empty(lib.ttt_selective_scan_ckpt_bytes(n_seq, L, D, N, packed) // 4, device="cuda")
    more = {} if h0 is None else dict(state_in=h0)
    lib.ttt_selective_scan_forward(*a, **k, **more, ckpt=ckpt, cu_seqlens=cut)
    dout = torch.randn(*lead, D, generator=torch.Generator().manual_seed(seed)).to(dt).cuda()
    g = lib.ttt_selective_scan_backward(*a, dout, ckpt, **k, d_state_out=dlast, state_in_grad=True, cu_seqlens=cut)
    want, mag = want_of(s, n_seq, L, cu, h0).grads(dout, dlast)
    w = want_of(s, n_seq, L, cu, h0)
    rows = cu[-1] if packed else n_seq * L
    # a gradient's terms are the product of a state's and of an adjoint's roundings (2 c), and the
    # sums over rows, channels and sequences add one a term
    c = 2 * w.c + rows + D
    for name in want:
        t = torch.float32 if name in ("dA", "dD", "ddelta_bias", "dstate_in") else dt
        got = g[name]
        if got is None:
            assert s["z"] is None and name == "dz"
            continue
        x, m = want[name], mag[name]
        if name in ("du", "ddelta", "dz", "dB", "dC"):
            got = got.reshape(-1, *got.shape[got.dim() - (x.dim() - 1):])[:rows]
            x, m = x[:rows], m[:rows]
        ref.check(name, got, x, m, c, t)
    return g, dout


@pytest.mark.parametrize("n_seq,L,D,N,G,dt,z", CASES)
def test_backward(libttt, n_seq, L, D, N, G, dt, z):
    s = inputs((n_seq, L), D, N, G, DT[dt], 12, z)
    gen = torch.Generator().manual_seed(2)
    h0, dlast = torch.randn(n_seq, D, N, generator=gen).cuda(), torch.randn(n_seq, D, N, generator=gen).cuda()
    check_grads(libttt, s, n_seq, L, DT[dt], h0=h0, dlast=dlast)
    check_grads(libttt, s, n_seq, L, DT[dt])


@pytest.mark.parametrize("lens", [[9], [0, 1, 70, 0, 3, 16, 64, 2], [17, 0]])
@pytest.mark.parametrize("dt,D,N,G", [("bf16", 40, 16, 1), ("f32", 9, 6, 3)])
def test_backward_packed(libttt, lens, dt, D, N, G):
    n, T = len(lens), sum(lens) + 3
    s = inputs((T,), D, N, G, DT[dt], 13)
    cu = [0]
    for m in lens:
        cu.append(cu[-1] + m)
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    gen = torch.Generator().manual_seed(2)
    h0, dlast = torch.randn(n, D, N, generator=gen).cuda(), torch.randn(n, D, N, generator=gen).cuda()
    g, _ = check_grads(libttt, s, n, T, DT[dt], cu, cut, h0, dlast)
    for name in ("du", "ddelta", "dz", "dB", "dC"):
        assert (g[name][cu[-1]:] == 0).all(), name


def test_gradient_against_differences(libttt):
    """d <out, R> + <state, S> along random directions: central differences of the float32 kernel.  With a
    step of 1e-2 and loss terms of order 1, the difference is off by about 1e-4 (third derivatives) and
    L D 2^-24 / 1e-2 ~ 5e-4 (rounding of the loss); 5e-3 of the sum of magnitudes covers both."""
    n_seq, L, D, N, G = 2, 19, 12, 8, 2
    s = inputs((n_seq, L), D, N, G, torch.float32, 21)
    a, k = positional(s)
    ckpt = torch.empty(libttt.ttt_selective_scan_ckpt_bytes(n_seq, L, D, N) // 4, device="cuda")
    gen = torch.Generator().manual_seed(5)
    rn = lambda t: torch.randn(t.shape, generator=gen).cuda()
    h0, R = rn(torch.empty(n_seq, D, N)), rn(s["u"])
    S = rn(h0)
    libttt.ttt_selective_scan_forward(*a, **k, state_in=h0, ckpt=ckpt)
    g = libttt.ttt_selective_scan_backward(*a, R, ckpt, **k, d_state_out=S, state_in_grad=True)

    def loss(s, h):
        a, k = positional(s)
        end = torch.empty_like(h)
        out = libttt.ttt_selective_scan_forward(*a, **k, state_in=h, state_out=end)
        return (out.double() * R.double()).sum() + (end.double() * S.double()).sum()

    for name in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias", "state_in"):
        x = h0 if name == "state_in" else s[name]
        v = rn(x) * (0.1 if name == "A" else 1.0)
        eps = 1e-2
        lo, hi = ((({**s}, h0 + e * v) if name == "state_in" else ({**s, name: x + e * v}, h0)) for e in (-eps, eps))
        num = (loss(*hi) - loss(*lo)) / (2 * eps)
        got = (g["d" + name].double() * v.double())
        assert abs(got.sum() - num) <= 5e-3 * got.abs().sum(), name


@pytest.mark.parametrize("D,N,G,dt", [(1, 1, 1, "f32"), (37, 16, 1, "bf16"), (64, 8, 2, "f32"), (12, 64, 3, "bf16"), (10, 20, 1, "f32")])
def test_steps_continue_a_prompt(libttt, D, N, G, dt):
    n_seq, L, split = 4, 21, 9
    s = inputs((n_seq, L), D, N, G, DT[dt], 15)
    pool = torch.randn(7, D, N, generator=torch.Generator().manual_seed(9)).cuda()
    pages = torch.tensor([5, 0, 6, 2], dtype=torch.int32, device="cuda")
    want = want_of(s, n_seq, L, h0=pool[pages.long()])
    cut = lambda f: {k: (f(v) if k in ("u", "delta", "B", "C", "z") else v) for k, v in s.items()}
    a, k = positional(cut(lambda v: v[:, :split]))
    out = [libttt.ttt_selective_scan_forward(*a, **k, state_in=pool, state_out=pool, pages=pages)]
    for t in range(split, L):
        a, k = positional(cut(lambda v: v[:, t]))
        out.append(libttt.ttt_selective_scan_step(*a, pool, **k, pages=pages).unsqueeze(1))
    ref.check("out", torch.cat(out, 1), want.out, want.out_mag, want.c, DT[dt])
    ref.check("state", pool[pages.long()], torch.stack(want.last), torch.stack(want.last_mag), want.c, torch.float32)


def test_step_without_a_page_gives_zeros(libttt):
    s = inputs((3,), 16, 16, 1, torch.bfloat16, 37)
    a, k = positional(s)
    pool = torch.randn(4, 16, 16, device="cuda")
    out, before = torch.full((3, 16), 5.0, device="cuda").bfloat16(), pool.clone()
    libttt.ttt_selective_scan_step(*a, pool, **k, pages=torch.tensor([1, -1, 99], dtype=torch.int32, device="cuda"), out=out)
    assert (out[1:] == 0).all() and (out[0] != 5).any()
    assert torch.equal(pool[[0, 2, 3]], before[[0, 2, 3]]) and not torch.equal(pool[1], before[1])


def test_views_and_broadcast_rows(libttt):
    """u and z as halves of one projection, B and C as slices at an odd offset, one gate row for all."""
    n_seq, L, D, N = 2, 37, 24, 16
    s = inputs((n_seq, L), D, N, 1, torch.bfloat16, 41)
    wide = torch.cat([s["u"], s["delta"]], -1)
    tail = torch.cat([torch.zeros(n_seq, L, 5, device="cuda").bfloat16(), s["B"].flatten(2), s["C"].flatten(2)], -1)
    v = {**s, "u": wide[..., :D], "delta": wide[..., D:], "B": tail[..., 5:5 + N].unflatten(-1, (1, N)),
         "C": tail[..., 5 + N:].unflatten(-1, (1, N)), "z": s["z"][:1, :1].expand(n_seq, L, D)}
    c = {**s, "z": v["z"].contiguous()}
    outs = []
    for q in (v, c):
        a, k = positional(q)
        ckpt = torch.empty(libttt.ttt_selective_scan_ckpt_bytes(n_seq, L, D, N) // 4, device="cuda")
        out = libttt.ttt_selective_scan_forward(*a, **k, ckpt=ckpt)
        outs.append([out, *libttt.ttt_selective_scan_backward(*a, s["u"], ckpt, **k).values()])
    for x, y in zip(*outs):
        assert (x is None and y is None) or torch.equal(x, y)
    a, k = positional(s)
    into = torch.zeros(L, n_seq, 2 * D, device="cuda").bfloat16()  # token-outer output rows with gaps
    libttt.ttt_selective_scan_forward(*a, **k, out=into.transpose(0, 1)[..., :D])
    assert torch.equal(into.transpose(0, 1)[..., :D], libttt.ttt_selective_scan_forward(*a, **k))
    assert (into[..., D:] == 0).all()


def test_extreme_steps(libttt):
    """Steps so long that a state is forgotten at once, so short that nothing changes, and an infinite
    step: exp(-inf) is 0 and the state holds what the last token put there."""
    s = inputs((1, 20), 8, 16, 1, torch.float32, 51, z=False)
    s["delta_bias"] = None
    s["delta"][:, :, 0], s["delta"][:, :, 1], s["delta"][:, :, 2] = 300.0, -300.0, 60.0
    want = want_of(s, 1, 20)
    a, k = positional(s)
    out = libttt.ttt_selective_scan_forward(*a, **k)
    ref.check("out", out, want.out, want.out_mag, want.c, torch.float32)
    s["delta"][0, 5, 3] = float("inf")
    out = libttt.ttt_selective_scan_forward(*a, **k)
    assert torch.isfinite(out[0, :5]).all() and not torch.isfinite(out[0, 5, 3]) and torch.isfinite(out[0, :, 4:]).all()
    s["delta"][0, 5, 3], s["u"][0, 7, 4] = 0.0, float("nan")
    out = libttt.ttt_selective_scan_forward(*a, **k)
    assert torch.isnan(out[0, 7:, 4]).all() and torch.isfinite(out[0, :7]).all() and torch.isfinite(out[0, :, 5:]).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("mask", ["lowest", "-inf"])
def test_masked_steps(libttt, dt, mask):
    """Tokens switched off by their delta, the type's lowest value or -inf: softplus of it is 0, so the state
    passes through them unchanged and their delta has no gradient."""
    n_seq, L, D, N = 2, 37, 12, 16
    s = inputs((n_seq, L), D, N, 1, DT[dt], 71)
    off = torch.tensor([0, 5, 6, 16, 31, 32, 36], device="cuda")
    s["delta"][:, off] = torch.finfo(DT[dt]).min if mask == "lowest" else -math.inf
    s["delta"][1] = s["delta"][0, 0, 0]  # a sequence with nothing left
    h0 = torch.randn(n_seq, D, N, generator=torch.Generator().manual_seed(5)).cuda()
    want = want_of(s, n_seq, L, h0=h0)
    a, k = positional(s)
    end = h0.clone()
    out = libttt.ttt_selective_scan_forward(*a, **k, state_in=end, state_out=end)
    ref.check("out", out, want.out, want.out_mag, want.c, DT[dt])
    ref.check("state", end, torch.stack(want.last), torch.stack(want.last_mag), want.c, torch.float32)
    assert torch.equal(end[1], h0[1])
    g, _ = check_grads(libttt, s, n_seq, L, DT[dt], h0=h0, dlast=h0.flip(0).contiguous())
    assert (g["ddelta"][:, off] == 0).all() and (g["ddelta"][1] == 0).all()
    pool, t = h0.clone(), {n_: v[:, 5] if n_ in ("u", "delta", "B", "C", "z") else v for n_, v in s.items()}
    a, k = positional(t)
    y = libttt.ttt_selective_scan_step(*a, pool, **k)
    assert torch.equal(pool, h0) and torch.isfinite(y).all()


def test_empty_sequences(libttt):
    s = inputs((2, 0), 8, 16, 1, torch.bfloat16, 51)
    a, k = positional(s)
    pool, end = torch.randn(2, 8, 16, device="cuda"), torch.empty(2, 8, 16, device="cuda")
    out = libttt.ttt_selective_scan_forward(*a, **k, state_in=pool, state_out=end)
    assert out.shape == (2, 0, 8) and torch.equal(end, pool)
    ckpt = torch.empty(1 << 12, device="cuda")
    g = libttt.ttt_selective_scan_backward(*a, out, ckpt, **k, d_state_out=pool, state_in_grad=True)
    assert torch.equal(g["dstate_in"], pool) and (g["dA"] == 0).all() and (g["dD"] == 0).all()
