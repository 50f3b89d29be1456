"""The entry points of the causal convolution, the selective scan and the cache's pages on the host: bad
arguments give the documented codes before any CUDA call (fake pointers are never dereferenced)."""
import ctypes

import pytest

A = 1 << 24  # fake device addresses, far enough apart for the sizes below


def strides(*v):
    return None if not v else (ctypes.c_longlong * len(v))(*v)


def conv(lib, **k):
    a = dict(x=A, w=2 * A, b=3 * A, s=None, cu=None, si=4 * A, so=5 * A, pages=6 * A, np=8, n=3, L=40, D=64, W=4, dt=1, f=16, out=7 * A)
    a.update(k)
    return lib.ttt_causal_conv_forward(a["x"], a["w"], a["b"], a["s"], a["cu"], a["si"], a["so"], a["pages"], a["np"], a["n"],
                                       a["L"], a["D"], a["W"], a["dt"], a["f"], a["out"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), -1), (dict(L=-1), -1), (dict(L=1 << 30), -1), (dict(D=0), -1), (dict(W=0), -1), (dict(W=1), -6), (dict(W=5), -6),
    (dict(dt=2), -1), (dict(f=1), -1), (dict(f=8), -1), (dict(x=None), -1), (dict(w=None), -1), (dict(out=None), -1),
    (dict(x=A + 1), -2), (dict(w=2 * A + 2), -2), (dict(cu=9 * A + 2), -2), (dict(pages=6 * A + 1), -2), (dict(so=5 * A + 1), -2),
    (dict(np=0), -1), (dict(pages=None, np=2), -1), (dict(out=A), -3), (dict(so=4 * A + 64), -3), (dict(so=A), -3), (dict(out=4 * A), -3),
    (dict(s=strides(2560, -64, 2560, 64)), -1), (dict(s=strides(2560, 64, 2560, 32)), -1), (dict(s=strides(2560, 64, 64, 64)), -1),
    (dict(s=strides(0, 0, 0, 64)), -1), (dict(n=1 << 25), -1), (dict(D=(1 << 24) + 1), -1),
])
def test_conv_forward_rejects(libttt, kw, code):
    lib = libttt.lib()
    assert conv(lib, **kw) == code
    assert lib.ttt_last_error_message()


def conv_step(lib, **k):
    a = dict(x=A, w=2 * A, b=None, s=None, st=4 * A, pages=6 * A, np=8, n=3, D=64, W=4, dt=0, f=0, out=7 * A)
    a.update(k)
    return lib.ttt_causal_conv_step(a["x"], a["w"], a["b"], a["s"], a["st"], a["pages"], a["np"], a["n"], a["D"], a["W"], a["dt"],
                                    a["f"], a["out"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(st=None), -1), (dict(out=None), -1), (dict(n=0), -1), (dict(W=6), -6), (dict(np=0), -1),
    (dict(pages=None, np=2), -1), (dict(st=4 * A + 2), -2), (dict(out=4 * A), -3), (dict(out=A), -3), (dict(s=strides(64, 32)), -1),
    (dict(f=2), -1),
])
def test_conv_step_rejects(libttt, kw, code):
    assert conv_step(libttt.lib(), **kw) == code


def conv_bwd(lib, **k):
    a = dict(x=A, w=2 * A, b=3 * A, s=None, cu=None, si=None, n=3, L=40, D=64, W=4, dt=1, f=16, do=4 * A, dso=None, dx=5 * A, dw=6 * A,
             db=7 * A, dsi=None, ws=8 * A, wb=1 << 22)
    a.update(k)
    return lib.ttt_causal_conv_backward(a["x"], a["w"], a["b"], a["s"], a["cu"], a["si"], a["n"], a["L"], a["D"], a["W"], a["dt"], a["f"],
                                        a["do"], a["dso"], a["dx"], a["dw"], a["db"], a["dsi"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(do=None), -1), (dict(dx=None), -1), (dict(dw=None), -1), (dict(ws=None), -1), (dict(wb=16), -1), (dict(ws=8 * A + 16), -2),
    (dict(dx=A), -3), (dict(dx=4 * A), -3), (dict(dw=2 * A), -3), (dict(db=6 * A), -3), (dict(ws=5 * A), -3), (dict(L=-2), -1),
    (dict(W=8), -6), (dict(f=64), -1),
])
def test_conv_backward_rejects(libttt, kw, code):
    assert conv_bwd(libttt.lib(), **kw) == code


def scan(lib, **k):
    a = dict(u=A, d=2 * A, A=3 * A, B=4 * A, C=5 * A, D=6 * A, z=7 * A, bias=8 * A, s=None, cu=None, ml=0, si=9 * A, so=10 * A, pages=11 * A,
             np=8, n=3, L=40, dim=64, G=2, N=16, dt=1, f=8, out=12 * A, ck=13 * A, ws=14 * A, wb=1 << 22)
    a.update(k)
    return lib.ttt_selective_scan_forward(a["u"], a["d"], a["A"], a["B"], a["C"], a["D"], a["z"], a["bias"], a["s"], a["cu"], a["ml"],
                                          a["si"], a["so"], a["pages"], a["np"], a["n"], a["L"], a["dim"], a["G"], a["N"], a["dt"],
                                          a["f"], a["out"], a["ck"], a["ws"], a["wb"], None)


OK = (2560, 64) * 2 + (1280, 32) * 2


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(L=-1), -1), (dict(dim=0), -1), (dict(G=0), -1), (dict(G=3), -1), (dict(N=0), -1), (dict(N=65), -6),
    (dict(dt=9), -1), (dict(f=1), -1), (dict(f=16), -1), (dict(u=None), -1), (dict(d=None), -1), (dict(A=None), -1), (dict(B=None), -1),
    (dict(C=None), -1), (dict(out=None), -1), (dict(A=3 * A + 4), -2), (dict(si=9 * A + 8), -2), (dict(ck=13 * A + 8), -2),
    (dict(u=A + 1), -2), (dict(z=7 * A + 1), -2), (dict(np=0), -1), (dict(pages=None, np=2), -1), (dict(ml=-1), -1),
    (dict(out=A), -3), (dict(out=7 * A), -3), (dict(so=9 * A + 16), -3), (dict(ck=4 * A), -3), (dict(so=12 * A), -3),
    (dict(s=strides(*OK, 2560, 64, 2560, 63)), -1), (dict(s=strides(*OK, 2560, -1, 2560, 64)), -1), (dict(s=strides(*OK, 2560, 64, 0, 64)), -1),
    (dict(n=1, L=9000, wb=16), -1), (dict(n=1, L=9000, ws=None), -1), (dict(n=1, L=9000, ws=14 * A + 128, wb=1 << 30, np=1), -2),
])
def test_scan_forward_rejects(libttt, kw, code):
    lib = libttt.lib()
    if kw.get("L") == 9000:  # long enough to be cut into spans, so a workspace is needed
        assert lib.ttt_selective_scan_workspace_bytes(1, 9000, 0, 0, 64, 2, 16) > 0
        kw = dict(kw, u=A, d=A << 4, A=A << 5, B=A << 6, C=A << 7, z=A << 8, out=A << 9, ck=None)
    assert scan(lib, **kw) == code
    assert lib.ttt_last_error_message()


def scan_step(lib, **k):
    a = dict(u=A, d=2 * A, A=3 * A, B=4 * A, C=5 * A, D=None, z=None, bias=None, s=None, st=9 * A, pages=11 * A, np=8, n=3, dim=64, G=2,
             N=16, dt=1, f=8, out=12 * A)
    a.update(k)
    return lib.ttt_selective_scan_step(a["u"], a["d"], a["A"], a["B"], a["C"], a["D"], a["z"], a["bias"], a["s"], a["st"], a["pages"],
                                       a["np"], a["n"], a["dim"], a["G"], a["N"], a["dt"], a["f"], a["out"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(u=None), -1), (dict(st=None), -1), (dict(B=None), -1), (dict(N=65), -6), (dict(G=5), -1), (dict(st=9 * A + 4), -2),
    (dict(out=9 * A), -3), (dict(out=2 * A), -3), (dict(np=0), -1), (dict(s=strides(64, 64, 32, 32, 64, 8)), -1), (dict(f=4), -1),
])
def test_scan_step_rejects(libttt, kw, code):
    assert scan_step(libttt.lib(), **kw) == code


def scan_bwd(lib, **k):
    a = dict(u=A, d=2 * A, A=3 * A, B=4 * A, C=5 * A, D=6 * A, z=7 * A, bias=8 * A, s=None, cu=None, ck=9 * A, n=3, L=40, dim=64, G=2, N=16,
             dt=1, f=8, do=10 * A, dso=None, du=11 * A, dd=12 * A, dA=13 * A, dB=14 * A, dC=15 * A, dD=16 * A, dz=17 * A, db=18 * A, dsi=None,
             ws=19 * A, wb=1 << 23)
    a.update(k)
    return lib.ttt_selective_scan_backward(a["u"], a["d"], a["A"], a["B"], a["C"], a["D"], a["z"], a["bias"], a["s"], a["cu"], a["ck"],
                                           a["n"], a["L"], a["dim"], a["G"], a["N"], a["dt"], a["f"], a["do"], a["dso"], a["du"],
                                           a["dd"], a["dA"], a["dB"], a["dC"], a["dD"], a["dz"], a["db"], a["dsi"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(ck=None), -1), (dict(do=None), -1), (dict(du=None), -1), (dict(dA=None), -1), (dict(dz=None), -1), (dict(z=None), -1),
    (dict(ws=None), -1), (dict(wb=64), -1), (dict(ws=19 * A + 64), -2), (dict(ck=9 * A + 4), -2), (dict(dso=20 * A + 4), -2),
    (dict(du=A), -3), (dict(dB=14 * A, dC=14 * A), -3), (dict(ws=9 * A), -3), (dict(dA=3 * A), -3), (dict(N=70), -6), (dict(G=7), -1),
])
def test_scan_backward_rejects(libttt, kw, code):
    assert scan_bwd(libttt.lib(), **kw) == code


def cache(lib, what, tensors=((A, 256), (2 * A, 64)), n_pages=10, n_rows=6, n=4, **k):
    ptrs = (ctypes.c_void_p * max(1, len(tensors)))(*[t[0] for t in tensors])
    sizes = (ctypes.c_longlong * max(1, len(tensors)))(*[t[1] for t in tensors])
    a = dict(table=3 * A, owner=4 * A, a=5 * A, b=6 * A, out=7 * A, live=8 * A, ws=9 * A)
    a.update(k)
    if what == "copy":
        return lib.ttt_cache_copy(ptrs, sizes, len(tensors), n_pages, a["a"], a["b"], n, a["out"], a["ws"], None)
    if what == "fork":
        return lib.ttt_cache_fork(ptrs, sizes, len(tensors), n_pages, a["table"], n_rows, a["owner"], a["a"], a["b"], n, a["out"], a["ws"], None)
    if what == "free":
        return lib.ttt_cache_free(a["table"], n_rows, a["owner"], n_pages, a["a"], n, a["out"], None)
    return lib.ttt_cache_compact(ptrs, sizes, len(tensors), n_pages, a["table"], n_rows, a["owner"], a["live"], a["out"], a["ws"], None)


@pytest.mark.parametrize("what,kw,code", [
    ("copy", dict(n_pages=0), -1), ("copy", dict(n=11), -1), ("copy", dict(n=-1), -1), ("copy", dict(a=None), -1), ("copy", dict(out=None), -1),
    ("copy", dict(tensors=((A, 0),)), -1), ("copy", dict(tensors=((None, 4),)), -1), ("copy", dict(tensors=((A, 4),) * 513), -6),
    ("copy", dict(tensors=((A, 64), (A + 64, 64))), -3), ("copy", dict(out=5 * A), -3), ("copy", dict(ws=A), -3), ("copy", dict(ws=9 * A + 2), -2),
    ("fork", dict(table=None), -1), ("fork", dict(owner=None), -1), ("fork", dict(n_rows=0), -1), ("fork", dict(n=-1), -1), ("fork", dict(b=None), -1),
    ("fork", dict(b=6 * A + 1), -2), ("fork", dict(table=4 * A), -3), ("fork", dict(out=6 * A), -3), ("fork", dict(a=2 * A), -3),
    ("free", dict(n_pages=0), -1), ("free", dict(table=None), -1), ("free", dict(a=None), -1), ("free", dict(out=None), -1), ("free", dict(out=5 * A), -3),
    ("compact", dict(live=None), -1), ("compact", dict(ws=None), -1), ("compact", dict(out=None), -1), ("compact", dict(table=4 * A), -3),
    ("compact", dict(live=9 * A), -3), ("compact", dict(n_pages=-2), -1), ("compact", dict(owner=4 * A + 1), -2),
])
def test_cache_rejects(libttt, what, kw, code):
    assert cache(libttt.lib(), what, **kw) == code


@pytest.mark.parametrize("kw", [
    dict(D=(1 << 22) + 1, s=strides(0, 1 << 23, 1 << 40, 1 << 23)),  # more channels than a grid's second axis takes
    dict(n=1 << 20, s=strides(1 << 44, 64, 2560, 64)),                # sizes that pass 64 bits on the host: the aliasing
    dict(s=strides(0, 1 << 48, 2560, 64)),                            # check would be made on their remainders
])
def test_conv_refuses_sizes_past_its_arithmetic(libttt, kw):
    assert conv(libttt.lib(), si=None, so=None, pages=None, **kw) == -1


def test_scan_and_step_refuse_sizes_past_their_arithmetic(libttt):
    wide = strides(*([0, 1 << 48] + [2560, 64] * 5))
    assert scan(libttt.lib(), s=wide) == -1
    assert conv_step(libttt.lib(), n=1 << 20, np=1 << 20, s=strides(1 << 44, 64)) == -1


def test_cache_refuses_sizes_past_its_arithmetic(libttt):
    lib = libttt.lib()
    assert cache(lib, "copy", tensors=((A, 1 << 40),), n_pages=1 << 30) == -1
    assert cache(lib, "compact", tensors=((A, 1 << 40),), n_pages=1 << 24) == -1
    # every copy by index is compared with all others of its call
    assert cache(lib, "copy", tensors=((1 << 40, 4),), n_pages=1 << 20, n=(1 << 14) + 1) == -6


def test_nothing_to_do_is_fine(libttt):
    lib = libttt.lib()
    assert cache(lib, "copy", n=0, a=None, b=None) == 0
    assert cache(lib, "fork", n=0, a=None, b=None) == 0
    assert conv(lib, L=0, x=None, out=None, so=None) == 0
    assert scan(lib, L=0, u=None, d=None, B=None, C=None, z=None, out=None, so=None) == 0


def test_byte_counts(libttt):
    # the state before every 8th token; packed sequences: a slot for each started chunk, whatever the lengths
    assert libttt.ttt_selective_scan_ckpt_bytes(2, 17, 5, 3) == 2 * 3 * 5 * 3 * 4
    assert libttt.ttt_selective_scan_ckpt_bytes(2, 17, 5, 3, packed=True) == (17 // 8 + 2) * 5 * 3 * 4
    assert libttt.ttt_selective_scan_workspace_bytes(8, 2048, 2048, 16) == 0  # fills the GPU: no spans
    assert libttt.ttt_selective_scan_workspace_bytes(1, 8200, 2048, 16) > 0
    assert libttt.ttt_causal_conv_backward_workspace_bytes(1, 0, 8, 4) > 0
    for bad in (dict(d_state=0), dict(d_state=65), dict(dim=0), dict(L=-1)):
        with pytest.raises(libttt.TTTError):
            libttt.ttt_selective_scan_backward_workspace_bytes(**(dict(n_seq=1, L=8, dim=8, d_state=8) | bad))


def test_slots_of_packed_sequences_never_collide():
    """The numbering that the kernels use for pieces of packed sequences (slot_base): every piece of every
    sequence has a slot of its own below T // span + n, found again by the search, for random lengths."""
    import random
    rng = random.Random(7)
    for _ in range(300):
        span, n = rng.choice([8, 16, 32, 64, 464]), rng.randint(1, 20)
        lens = [rng.choice([0, 1, rng.randint(0, 9), rng.randint(0, 1500)]) for _ in range(n)]
        cu = [0]
        for k in lens:
            cu.append(cu[-1] + k)
        T = cu[-1] + rng.choice([0, 5])
        base = [cu[b] // span + b for b in range(n)]
        seen = {}
        for b in range(n):
            for tile in range(max(1, -(-lens[b] // span))):
                slot = base[b] + tile
                assert slot not in seen and slot < T // span + n
                seen[slot] = (b, tile)
        for slot in range(T // span + n):
            lo, hi = 0, n - 1
            while lo < hi:
                mid = (lo + hi + 1) >> 1
                lo, hi = (mid, hi) if base[mid] <= slot else (lo, mid - 1)
            tile = slot - base[lo]
            found = tile == 0 or (tile > 0 and tile * span < lens[lo])
            assert (seen.get(slot) == (lo, tile)) == found
