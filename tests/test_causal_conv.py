"""The causal convolution (prompts, single tokens, gradients) against its float64 form.

Tolerances: `pre` is a sum of W + 1 terms, each rounded at most W + 2 times; silu and its derivative
take 8 more roundings relative to values no larger than those of the terms (their slopes are at most
1.1), 64 covers both; sums over rows add one rounding a row of the block and one a block.
"""
import pytest
import torch

import seq_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def inputs(n_seq, L, D, W, dt, seed, packed_rows=None, view=False):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)
    lead = (n_seq, L) if packed_rows is None else (packed_rows,)
    x = rn(*lead, 2 * D + 3).to(dt).cuda()[..., 1:1 + D] if view else rn(*lead, D).to(dt).cuda()
    return x, (rn(D, W) / W).cuda(), (0.3 * rn(D)).cuda(), rn(n_seq + 3, W - 1, D).to(dt).cuda(), rn(*lead, D).to(dt).cuda()


CASES = [  # n_seq, L, D, W, dtype, silu, view
    (1, 1, 1, 2, "f32", True, False), (2, 2, 7, 4, "bf16", True, False), (3, 33, 64, 3, "bf16", False, False),
    (2, 31, 256, 4, "f32", True, False), (1, 129, 1032, 4, "bf16", True, False), (2, 40, 24, 4, "bf16", True, True),
    (5, 3, 130, 4, "bf16", True, False), (2, 65, 20, 2, "f32", False, True), (1, 3000, 8, 4, "bf16", True, False),
]


@pytest.mark.parametrize("n_seq,L,D,W,dt,silu,view", CASES)
@pytest.mark.parametrize("state", ["none", "apart", "in place"])
def test_forward(libttt, n_seq, L, D, W, dt, silu, view, state):
    x, w, b, pool, _ = inputs(n_seq, L, D, W, DT[dt], 11, view=view)
    pages = torch.tensor([(2 * k + 1) % (n_seq + 3) for k in range(n_seq)][:n_seq], dtype=torch.int32)
    pages = torch.randperm(n_seq + 3, generator=torch.Generator().manual_seed(3))[:n_seq].int()
    before = pool.clone()
    after = None if state == "none" else pool if state == "in place" else torch.full_like(pool, 7.0)
    out = libttt.ttt_causal_conv_forward(x, w, b, silu=silu, state_in=None if state == "none" else pool, state_out=after,
                                         pages=pages.cuda())
    for k in range(n_seq):
        s = torch.zeros(W - 1, D).double() if state == "none" else before[pages[k]].double().cpu()
        want, last, _, mag = ref.conv(x[k].double().cpu(), w.double().cpu(), b.double().cpu(), s, silu)
        ref.check("out", out[k], want, mag, 64, DT[dt])
        if state != "none":
            assert torch.equal(after[pages[k]].double().cpu(), last)
    if after is not None:  # the other pages are as they were
        rest = [p for p in range(n_seq + 3) if p not in pages.tolist()]
        assert torch.equal(after[rest], before[rest] if state == "in place" else torch.full_like(before[rest], 7.0))


@pytest.mark.parametrize("lens", [[5], [0, 1, 70, 0, 3, 32, 64, 2], [33, 0], [1] * 9])
@pytest.mark.parametrize("dt,D,W", [("bf16", 40, 4), ("f32", 9, 3)])
def test_packed_and_backward(libttt, lens, dt, D, W):
    n, T = len(lens), sum(lens) + 4  # 4 rows past the last sequence
    x, w, b, pool, dout = inputs(n, 0, D, W, DT[dt], 5, packed_rows=T)
    cu = [0]
    for k in lens:
        cu.append(cu[-1] + k)
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    pages = torch.arange(n, dtype=torch.int32)
    pages[n // 2] = -1  # one sequence without a page
    out = torch.full_like(x, 9.0)
    before = pool.clone()
    libttt.ttt_causal_conv_forward(x, w, b, state_in=pool, state_out=pool, pages=pages.cuda(), cu_seqlens=cut, out=out)
    assert (out[cu[-1]:] == 9.0).all()
    for k, (t0, m) in enumerate(ref.sequences(n, 0, cu)):
        s = before[k].double().cpu() if pages[k] >= 0 else torch.zeros(W - 1, D).double()
        want, last, _, mag = ref.conv(x[t0:t0 + m].double().cpu(), w.double().cpu(), b.double().cpu(), s)
        ref.check("out", out[t0:t0 + m], want, mag, 64, DT[dt])
        assert torch.equal(pool[k], before[k]) if pages[k] < 0 else torch.equal(pool[k].double().cpu(), last)
    backward(libttt, x, w, b, before[:n].contiguous(), dout, torch.flip(before[:n], (0,)).contiguous(), cut, ref.sequences(n, 0, cu), DT[dt], True)


def backward(lib, x, w, b, state, dout, dlast, cut, seqs, dt, silu):
    g = lib.ttt_causal_conv_backward(x, w, dout, b, silu=silu, state_in=state, d_state_out=dlast, cu_seqlens=cut)
    D, W = w.shape
    xf, df = x.double().cpu().reshape(-1, D), dout.double().cpu().reshape(-1, D)
    total = {"dx": torch.zeros_like(xf), "dw": torch.zeros(D, W).double(), "db": torch.zeros(D).double()}
    mags = {k: v.clone() for k, v in total.items()}
    for i, (t0, m) in enumerate(seqs):
        leaves = [t.double().cpu().requires_grad_() for t in (xf[t0:t0 + m], w, b, state[i])]
        out, last, pre, pmag = ref.conv(*leaves, silu)
        loss = (out * df[t0:t0 + m]).sum() + (last * dlast[i].double().cpu()).sum()
        gx, gw, gb, gs = torch.autograd.grad(loss, leaves, allow_unused=True)
        gx = torch.zeros_like(leaves[0]) if gx is None else gx
        # magnitudes: |dpre| <= |d_out| 1.1 (1 + what an error of pre does to silu', slope at most 0.5)
        with torch.no_grad():
            sens = df[t0:t0 + m].abs() * (1.1 + (0.5 * pmag if silu else 0))
            rows = torch.cat([state[i].double().cpu(), xf[t0:t0 + m]]).abs()
            mrows = torch.zeros_like(rows)
            for k in range(W):
                mrows[k:k + m] += sens * w[:, k].abs().double().cpu()
                mags["dw"][:, k] += (sens * rows[k:k + m]).sum(0)
            mrows[m:] += dlast[i].double().cpu().abs()
            mags["dx"][t0:t0 + m] = mrows[W - 1:]
            mags["db"] += sens.sum(0)
        total["dx"][t0:t0 + m] = gx
        total["dw"] += 0 if gw is None else gw
        total["db"] += 0 if gb is None else gb
        ref.check("dstate_in", g["dstate_in"][i], gs, mrows[:W - 1], 64, dt)
    ref.check("dx", g["dx"], total["dx"], mags["dx"], 64, dt)
    blocks = sum(m // 8 + 1 for _, m in seqs)
    ref.check("dweight", g["dweight"], total["dw"], mags["dw"], 64 + 64 + blocks, torch.float32)
    ref.check("dbias", g["dbias"], total["db"], mags["db"], 64 + 64 + blocks, torch.float32)


@pytest.mark.parametrize("n_seq,L,D,W,dt,silu,view", CASES)
def test_backward(libttt, n_seq, L, D, W, dt, silu, view):
    x, w, b, pool, dout = inputs(n_seq, L, D, W, DT[dt], 17, view=view)
    backward(libttt, x, w, b, pool[:n_seq].contiguous(), dout, torch.flip(pool[:n_seq], (0,)).contiguous(), None,
             ref.sequences(n_seq, L, None), DT[dt], silu)


def test_backward_repeats_bit_for_bit_and_broadcast_gradient(libttt):
    x, w, b, _, _ = inputs(3, 200, 96, 4, torch.bfloat16, 23)
    dout = torch.randn(96, device="cuda").bfloat16().expand(3, 200, 96)  # strides 0
    one = libttt.ttt_causal_conv_backward(x, w, dout, b)
    two = libttt.ttt_causal_conv_backward(x, w, dout.contiguous(), b)
    assert all(torch.equal(one[k], two[k]) for k in ("dx", "dweight", "dbias"))
    assert one["dstate_in"] is None


@pytest.mark.parametrize("D,W,dt", [(1, 4, "f32"), (37, 3, "bf16"), (256, 4, "bf16"), (2048, 2, "f32")])
def test_steps_continue_a_prompt(libttt, D, W, dt):
    """A prompt in one piece, and the same as a prompt, then single tokens: the same bits."""
    x, w, b, pool, _ = inputs(4, 9, D, W, DT[dt], 31)
    pages = torch.tensor([5, 0, 6, 2], dtype=torch.int32, device="cuda")
    whole, end = libttt.ttt_causal_conv_forward(x, w, b, state_in=pool, state_out=(end := pool.clone()), pages=pages), end
    part = pool.clone()
    out = [libttt.ttt_causal_conv_forward(x[:, :4], w, b, state_in=part, state_out=part, pages=pages)]
    for t in range(4, 9):
        out.append(libttt.ttt_causal_conv_step(x[:, t], part, w, b, pages=pages).unsqueeze(1))
    assert torch.equal(torch.cat(out, 1), whole) and torch.equal(part, end)


def test_step_without_a_page_gives_zeros(libttt):
    x, w, b, pool, _ = inputs(3, 1, 16, 4, torch.bfloat16, 37)
    out, before = torch.full((3, 16), 5.0, device="cuda").bfloat16(), pool.clone()
    libttt.ttt_causal_conv_step(x[:, 0], pool, w, b, pages=torch.tensor([1, -1, 99], dtype=torch.int32, device="cuda"), out=out)
    assert (out[1:] == 0).all() and (out[0] != 5).any()
    keep = [0, 2, 3, 4, 5]
    assert torch.equal(pool[keep], before[keep]) and not torch.equal(pool[1], before[1])
