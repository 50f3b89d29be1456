"""The convolution, the scan and the cache's pages together, as a program that serves or trains uses
them: prompts into pages, steps, forks, ends, compaction, the TTT decode step on the dense pages, graphs,
two streams, autograd."""
import pytest
import torch

import seq_ref as ref

pytestmark = pytest.mark.gpu

DIM, N, W = 48, 16, 4


class Layer:
    """A convolution and a scan whose delta, B and C come from the convolution's output by fixed maps."""

    def __init__(self, seed=3):
        g = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g).cuda()
        self.w, self.cb = rn(DIM, W) / W, 0.1 * rn(DIM)
        self.A, self.D, self.bias = -(1 + rn(DIM, N).abs() * 3), rn(DIM), rn(DIM) - 3
        self.proj = (rn(DIM, DIM + 2 * N) / DIM ** 0.5)

    def split(self, v):
        o = v @ self.proj
        return o[..., :DIM], o[..., DIM:DIM + N].unflatten(-1, (1, N)), o[..., DIM + N:].unflatten(-1, (1, N))

    def prompt(self, lib, x, cu, conv, state, pages, longest):
        v = lib.ttt_causal_conv_forward(x, self.w, self.cb, state_in=conv, state_out=conv, pages=pages, cu_seqlens=cu)
        d, B, C = self.split(v)
        return lib.ttt_selective_scan_forward(v, d, self.A, B, C, D=self.D, delta_bias=self.bias, state_in=state,
                                              state_out=state, pages=pages, cu_seqlens=cu, max_seqlen=longest)

    def step(self, lib, x, conv, state, pages):
        v = lib.ttt_causal_conv_step(x, conv, self.w, self.cb, pages=pages)
        d, B, C = self.split(v)
        return lib.ttt_selective_scan_step(v, d, self.A, B, C, state, D=self.D, delta_bias=self.bias, pages=pages)

    def whole(self, x):
        """The float64 outputs of one whole sequence x [L, DIM]."""
        dd = lambda t: t.double().cpu()
        v, _, _, _ = ref.conv(dd(x), dd(self.w), dd(self.cb), torch.zeros(W - 1, DIM).double())
        o = v @ dd(self.proj)
        d, B, C = o[:, :DIM], o[:, DIM:DIM + N], o[:, DIM + N:]
        wide = lambda t: t[:, None, :].expand(-1, DIM, -1)
        dt, _ = ref.step_sizes(d, dd(self.bias), True)
        a = torch.exp(dt[..., None] * dd(self.A))
        return ref.scan(v, dt, a, wide(B), wide(C), dd(self.D), torch.ones_like(v), torch.zeros(DIM, N).double())[0]


def close(got, want):
    # float32 throughout and sequences of under 100 tokens; the maps from v to delta, B, C are matrix
    # products of 48 terms, each rounded (48 + 100 * (4 + 8 * 5)) 2^-24 ~ 3e-4 of the values' scale, at most
    if want.numel() == 0:
        return
    scale = want.abs().max()
    assert (got.double().cpu() - want).abs().max() <= 3e-4 * scale + 1e-6


def test_serving_run(libttt):
    """Three prompts, steps, a fork, an end, compaction, more steps: every output is that of its own whole
    token sequence."""
    torch.backends.cuda.matmul.allow_tf32 = False
    layer, g = Layer(), torch.Generator().manual_seed(5)
    n_pages, n_rows = 7, 6
    conv, state = torch.full((n_pages, W - 1, DIM), 9.0, device="cuda"), torch.full((n_pages, DIM, N), 9.0, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table, owner = i32([-1] * n_rows), i32([-1] * n_pages)
    said = {}          # row -> list of its tokens
    fresh = lambda n: torch.randn(n, DIM, generator=g).cuda()

    def pages(rows):   # as a program would: a lookup on the device
        return table[torch.tensor(rows, device="cuda")]

    def step(rows):
        x = fresh(len(rows))
        out = layer.step(libttt, x, conv, state, pages(rows))
        for i, r in enumerate(rows):
            said[r] = torch.cat([said[r], x[i:i + 1]])
            close(out[i], layer.whole(said[r])[-1])

    got = libttt.ttt_cache_fork([conv, state], table, owner, i32([-1, -1, -1]), i32([4, 0, 2]))
    assert got.tolist() == [0, 1, 2]
    lens, rows = [13, 1, 70], [4, 0, 2]
    x = fresh(sum(lens))
    cu = i32([0, 13, 14, 84])
    out = layer.prompt(libttt, x, cu, conv, state, pages(rows), max(lens))
    for r, part, o in zip(rows, x.split(lens), out.split(lens)):
        said[r] = part
        close(o, layer.whole(part))
    for _ in range(3):
        step(rows)
    got = libttt.ttt_cache_fork([conv, state], table, owner, i32([2, 2, 0]), i32([1, 3, 5]))
    assert got.tolist() == [3, 4, 5]
    said[1], said[3], said[5] = said[2], said[2], said[0]
    for _ in range(2):
        step([4, 0, 2, 1, 3, 5])
    assert int(libttt.ttt_cache_free(table, owner, i32([4, 0]))) == 2
    live, new = libttt.ttt_cache_compact([conv, state], table, owner)
    assert int(live) == 4 and new.tolist() == [-1, -1, 2, 3, 0, 1, -1]
    order = owner[:4].tolist()
    assert order == [3, 5, 2, 1] and table.tolist() == [-1, 3, 2, 0, -1, 1]
    step(order)
    # the first pages are a dense batch now: the same step without page indexes
    x = fresh(4)
    out = layer.step(libttt, x, conv, state, None)
    for i, r in enumerate(order):
        said[r] = torch.cat([said[r], x[i:i + 1]])
        close(out[i], layer.whole(said[r])[-1])
    # a second part of a prompt, from the pages
    more = [5, 0, 33, 2]
    x = fresh(sum(more))
    out = layer.prompt(libttt, x, i32([0, 5, 5, 38, 40]), conv, state, pages(order), 33)
    for r, part, o in zip(order, x.split(more), out.split(more)):
        said[r] = torch.cat([said[r], part])
        close(o, layer.whole(said[r])[len(said[r]) - len(part):])


@pytest.mark.parametrize("hist", [False, True])
def test_ttt_decode_on_compacted_pages(libttt, hist):
    """The TTT decode step on a cache whose sequences were forked, freed and compacted gives the bits of
    the sequences on their own."""
    H, K, g = 2, 16, torch.Generator().manual_seed(9)
    rn = lambda *s: torch.randn(*s, generator=g).cuda()
    make = lambda n: [rn(n, H, 64, 64) * 0.02, rn(n, H, 64) * 0.1, torch.zeros(n, H, K, 2, 64, device="cuda") if hist else torch.zeros(n, H, 64, 64, device="cuda"),
                      torch.zeros(n, H, 64, device="cuda")]
    lnw, lnb = 1 + 0.1 * rn(H, 64), 0.1 * rn(H, 64)
    fn = libttt.ttt_linear_decode_step_hist if hist else libttt.ttt_linear_decode_step
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    pool = make(6)
    alone = {r: [t[r:r + 1].clone() for t in pool] for r in range(4)}  # rows 0 .. 3 start in pages 0 .. 3
    table, owner = i32([0, 1, 2, 3, -1, -1]), i32([0, 1, 2, 3, -1, -1])
    off = {r: 0 for r in range(4)}

    def step(order):
        n = len(order)
        q, k, v = ((rn(n, H, 64) / 8).bfloat16() for _ in range(3))
        lr = torch.rand(n, H, generator=g).cuda() / 64
        out = fn(q, k, v, lr, lnw, lnb, *[t[:n] for t in pool], off[order[0]])
        for i, r in enumerate(order):
            own = fn(q[i:i + 1], k[i:i + 1], v[i:i + 1], lr[i:i + 1], lnw, lnb, *alone[r], off[r])
            assert torch.equal(own[0], out[i])
            off[r] += 1

    for _ in range(5):
        step([0, 1, 2, 3])
    assert libttt.ttt_cache_fork(pool, table, owner, i32([2]), i32([5])).tolist() == [4]
    alone[5], off[5] = [t.clone() for t in alone[2]], off[2]
    libttt.ttt_cache_free(table, owner, i32([1, 0]))
    live, _ = libttt.ttt_cache_compact(pool, table, owner)
    order = owner[:int(live)].tolist()
    assert order == [3, 5, 2]
    for _ in range(13):  # past a commit
        step(order)
    for i, r in enumerate(order):
        for t, a in zip(pool, alone[r]):
            assert torch.equal(t[i], a[0])


def test_step_and_prompt_in_a_graph(libttt):
    """A captured step and a captured (cut up) prompt with its gradient, replayed on other values."""
    layer = Layer()
    conv, state = torch.zeros(4, W - 1, DIM, device="cuda"), torch.zeros(4, DIM, N, device="cuda")
    x, pages = torch.randn(3, DIM, device="cuda"), torch.tensor([2, 0, 3], dtype=torch.int32, device="cuda")
    L = 600
    assert libttt.ttt_selective_scan_workspace_bytes(1, L, DIM, N) > 0
    u, d = torch.randn(1, L, DIM, device="cuda"), torch.randn(1, L, DIM, device="cuda")
    B, C = torch.randn(1, L, 1, N, device="cuda"), torch.randn(1, L, 1, N, device="cuda")
    ckpt = torch.empty(libttt.ttt_selective_scan_ckpt_bytes(1, L, DIM, N) // 4, device="cuda")

    def work():
        out = layer.step(libttt, x, conv, state, pages)
        y = libttt.ttt_selective_scan_forward(u, d, layer.A, B, C, D=layer.D, delta_bias=layer.bias, ckpt=ckpt)
        g = libttt.ttt_selective_scan_backward(u, d, layer.A, B, C, y, ckpt, D=layer.D, delta_bias=layer.bias)
        c = libttt.ttt_causal_conv_backward(u, layer.w, y, layer.cb)
        return [out, y, *g.values(), *c.values()]

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        held = work()
    for seed in (1, 2):
        torch.manual_seed(seed)
        for t in (x, u, d, B, C):
            t.copy_(torch.randn_like(t))
        conv.zero_(), state.zero_(), pages.copy_(torch.randperm(4)[:3].int())
        graph.replay()
        got = [None if t is None else t.clone() for t in held] + [conv.clone(), state.clone()]
        conv.zero_(), state.zero_()
        want = work() + [conv, state]
        assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(got, want))


def test_two_streams_at_once(libttt):
    """The same calls on two streams with their own inputs: nothing is shared between them."""
    L, streams, ins, outs = 700, [torch.cuda.Stream(), torch.cuda.Stream()], [], [[], []]
    layer = Layer()
    for k in range(2):
        torch.manual_seed(k)
        ins.append([torch.randn(1, L, DIM, device="cuda"), torch.randn(1, L, DIM, device="cuda"),
                    torch.randn(1, L, 1, N, device="cuda"), torch.randn(1, L, 1, N, device="cuda")])

    def run(k, stream):
        u, d, B, C = ins[k]
        v = libttt.ttt_causal_conv_forward(u, layer.w, layer.cb, stream=stream)
        y = libttt.ttt_selective_scan_forward(v, d, layer.A, B, C, D=layer.D, delta_bias=layer.bias, stream=stream)
        g = libttt.ttt_causal_conv_backward(u, layer.w, y, layer.cb, stream=stream)
        return [v, y, g["dx"], g["dweight"], g["dbias"]]

    want = [run(k, None) for k in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for k in range(2):
            outs[k].append(run(k, streams[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for o in outs[k]:
            assert all(torch.equal(a, b) for a, b in zip(o, want[k]))


def test_bad_cu_seqlens_stay_in_bounds(libttt):
    """An array that decreases or points outside the rows: no row outside the buffers is touched (guard
    rows around them keep their values), and a correct call afterwards is correct."""
    L, n = 40, 3
    layer = Layer()
    big = torch.full((3 * L, DIM), 7.0, device="cuda")
    x = torch.randn(L, DIM, device="cuda")
    u, d = torch.randn(L, DIM, device="cuda"), torch.randn(L, DIM, device="cuda")
    B, C = torch.randn(L, 1, N, device="cuda"), torch.randn(L, 1, N, device="cuda")
    ckpt = torch.empty(libttt.ttt_selective_scan_ckpt_bytes(n, L, DIM, N, True) // 4 + 1024, device="cuda")
    ckpt[-1024:] = 5.0
    for cu in ([0, 30, 20, 40], [-5, 10, 90, 1 << 30], [40, 0, 40, 0], [50, 50, 50, 50]):
        cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
        libttt.ttt_causal_conv_forward(x, layer.w, layer.cb, cu_seqlens=cut, out=big[L:2 * L])
        libttt.ttt_selective_scan_forward(u, d, layer.A, B, C, cu_seqlens=cut, out=big[L:2 * L], ckpt=ckpt)
        libttt.ttt_selective_scan_backward(u, d, layer.A, B, C, u, ckpt, cu_seqlens=cut)
        libttt.ttt_causal_conv_backward(x, layer.w, u, layer.cb, cu_seqlens=cut)
        assert (big[:L] == 7).all() and (big[2 * L:] == 7).all() and (ckpt[-1024:] == 5).all()
    cut = torch.tensor([0, 7, 7, 40], dtype=torch.int32, device="cuda")
    out = libttt.ttt_causal_conv_forward(x, layer.w, layer.cb, cu_seqlens=cut)
    for t0, m in ref.sequences(n, 0, [0, 7, 7, 40]):
        want, _, _, mag = ref.conv(x[t0:t0 + m].double().cpu(), layer.w.double().cpu(), layer.cb.double().cpu(), torch.zeros(W - 1, DIM).double())
        ref.check("out", out[t0:t0 + m], want, mag, 64, torch.float32)


def test_autograd_through_the_layer(libttt):
    """torch.autograd through convolution and scan (with states carried from one part to the next) gives the
    gradients of the float64 form."""
    from test_rnn_layers_b200.autograd import causal_conv, selective_scan
    torch.backends.cuda.matmul.allow_tf32 = False
    layer, L = Layer(), 30
    x = torch.randn(2, L, DIM, device="cuda")
    names = ("w", "cb", "A", "D", "bias", "proj")

    def run(p, x, conv, scan):
        v = conv(x, p["w"], p["cb"])
        o = v @ p["proj"]
        d, B, C = o[..., :DIM], o[..., DIM:DIM + N].unflatten(-1, (1, N)), o[..., DIM + N:].unflatten(-1, (1, N))
        return scan(v, d, p["A"], B, C, p["D"], torch.tanh(v), p["bias"])

    def scan32(v, d, A, B, C, D, z, bias):
        k = 13
        y1, s = selective_scan(v[:, :k], d[:, :k], A, B[:, :k], C[:, :k], D, z[:, :k], bias, return_state=True)
        y2, s = selective_scan(v[:, k:], d[:, k:], A, B[:, k:], C[:, k:], D, z[:, k:], bias, state_in=s, return_state=True)
        return torch.cat([y1, y2], 1), s

    def conv64(x, w, b):
        return torch.stack([ref.conv(t, w, b, torch.zeros(W - 1, DIM).double())[0] for t in x])

    def scan64(v, d, A, B, C, D, z, bias):
        outs, last = [], []
        for i in range(2):
            dt, _ = ref.step_sizes(d[i], bias, True)
            out, _, hs = ref.scan(v[i], dt, torch.exp(dt[..., None] * A), B[i].expand(-1, DIM, -1), C[i].expand(-1, DIM, -1), D,
                                  z[i] * torch.sigmoid(z[i]), torch.zeros(DIM, N).double())
            outs.append(out), last.append(hs[-1])
        return torch.stack(outs), torch.stack(last)

    grads = []
    R, S = torch.randn(2, L, DIM, device="cuda"), torch.randn(2, DIM, N, device="cuda")
    for f64 in (False, True):
        cast = (lambda t: t.detach().double().cpu().requires_grad_()) if f64 else (lambda t: t.detach().clone().requires_grad_())
        p = {n: cast(getattr(layer, n)) for n in names}
        xi = cast(x)
        out, s = run(p, xi, conv64 if f64 else causal_conv, scan64 if f64 else scan32)
        ((out * R.to(out)).sum() + (s * S.to(s)).sum()).backward()
        grads.append([xi.grad, *[p[n].grad for n in names]])
    for a, b in zip(*grads):
        close(a, b)
    # an upstream gradient whose rows and channels are one repeated number
    p = layer.w.detach().clone().requires_grad_()
    causal_conv(x, p, layer.cb).sum().backward()
    want = layer.w.detach().double().cpu().requires_grad_()
    conv64(x.double().cpu(), want, layer.cb.double().cpu()).sum().backward()
    close(p.grad, want.grad)


def test_autograd_in_a_graph(libttt):
    """Forward and gradients captured together (by torch.autograd.grad), replayed on other values, while
    an eager pass over the same leaves has its own graph."""
    from test_rnn_layers_b200.autograd import causal_conv
    x = torch.randn(2, 50, DIM, device="cuda", requires_grad=True)
    w = (torch.randn(DIM, W, device="cuda") / W).requires_grad_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            torch.autograd.grad(causal_conv(x, w).square().sum(), (x, w))
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        held = torch.autograd.grad(causal_conv(x, w).square().sum(), (x, w))
    with torch.no_grad():
        x.copy_(torch.randn_like(x))
    graph.replay()
    want = torch.autograd.grad(causal_conv(x, w).square().sum(), (x, w))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_a_cache_of_many_tensors(libttt):
    """All layers' states in one call: 24 layers of 4 tensors, one of them with pages of odd sizes."""
    g = torch.Generator(device="cuda").manual_seed(2)
    pool = [torch.randn(9, 3 + k % 7 * 40, device="cuda", generator=g) for k in range(96)]
    pool[50] = torch.randint(0, 255, (9, 333), device="cuda", generator=g, dtype=torch.uint8)
    before = [t.clone() for t in pool]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table, owner = i32([8, 2, -1, -1, -1]), i32([-1, -1, 1, -1, -1, -1, -1, -1, 0])
    assert libttt.ttt_cache_fork(pool, table, owner, i32([0, -1]), i32([3, 4])).tolist() == [0, 1]
    live, new = libttt.ttt_cache_compact(pool, table, owner)
    assert int(live) == 4 and new.tolist() == [0, 1, 2, -1, -1, -1, -1, -1, 3] and owner.tolist() == [3, 4, 1, 0] + [-1] * 5
    for t, b in zip(pool, before):
        assert torch.equal(t[0], b[8]) and (t[1] == 0).all() and torch.equal(t[2], b[2]) and torch.equal(t[3], b[8])
    with pytest.raises(libttt.TTTError):
        libttt.ttt_cache_fork(pool * 6, table, owner, i32([0]), i32([2]))


def test_binding_refuses(libttt):
    x, w = torch.randn(2, 8, 12, device="cuda"), torch.randn(12, 4, device="cuda")
    assert torch.equal(libttt.ttt_causal_conv_forward(x=x, weight=w), libttt.ttt_causal_conv_forward(x, w))  # by name, too
    for bad in (dict(x=x.half()), dict(x=x[0]), dict(x=x.transpose(1, 2)), dict(weight=w.bfloat16()), dict(weight=w[:5]), dict(weight=w.cpu()),
                dict(x=x.cpu()), dict(bias=w[0]), dict(out=x[:1]), dict(state_in=x), dict(pages=torch.zeros(2, dtype=torch.int64, device="cuda"))):
        with pytest.raises((TypeError, ValueError)):
            libttt.ttt_causal_conv_forward(**(dict(x=x, weight=w) | bad))
    u, A = x, -torch.rand(12, 16, device="cuda")
    B = torch.randn(2, 8, 1, 16, device="cuda")
    assert libttt.ttt_selective_scan_forward(u=u, delta=u, A=A, B=B, C=B).shape == u.shape
    for bad in (dict(delta=x[:, :4]), dict(A=A[:5]), dict(B=B[:, :, 0]), dict(C=B.bfloat16()), dict(D=w), dict(z=x.bfloat16()),
                dict(state_in=A), dict(ckpt=torch.empty(8, device="cuda")), dict(C=None), dict(delta=None)):
        with pytest.raises((TypeError, ValueError)):
            libttt.ttt_selective_scan_forward(**(dict(u=u, delta=u, A=A, B=B, C=B) | bad))
    with pytest.raises((TypeError, ValueError, libttt.TTTError)):
        libttt.ttt_selective_scan_forward(u, u, A, B, B, workspace=torch.empty(4, device="cuda"))
    t = torch.zeros(4, 3, device="cuda")
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in ((t, i.long(), i), ([t], i.long(), i), ([t], i, i.cpu()), ([t.t()], i, i), ([], i, i)):
        with pytest.raises((TypeError, ValueError)):
            libttt.ttt_cache_copy(*bad)
