"""Acceptance of a verified path: moved blocks and new lengths against plain
indexing, refusals on the CPU."""
import ctypes as C

import numpy as np
import pytest

A, A2, MIS = 0x10000, 0x20000, 0x10004


@pytest.fixture(scope="module")
def T():
    import long_context_attention_tbq4_b200 as pkg
    return pkg


def _call(paged=False, **kw):
    from long_context_attention_tbq4_b200._lib import lib as L
    a = dict(k=[A], v=[A2], n=None, ctx=A, path=A, acc=A, max_path=4, B=2, Hkv=2, cap=64, table=A,
             max_pages=2, page=32, n_pages=8, new=A2)
    a.update(kw)

    def ptrs(v):
        return None if v is None else (C.c_void_p * max(len(v), 1))(*v)
    n = len(a["k"] or [0]) if a["n"] is None else a["n"]
    p = [C.c_void_p(a[x]) if a[x] is not None else None for x in ("ctx", "path", "acc", "new", "table")]
    if paged:
        return L.tbq4_tree_accept_paged(ptrs(a["k"]), ptrs(a["v"]), n, p[4], a["max_pages"], a["page"],
                                        a["n_pages"], p[0], p[1], p[2], a["max_path"], a["B"], a["Hkv"], p[3], None)
    return L.tbq4_tree_accept(ptrs(a["k"]), ptrs(a["v"]), n, p[0], p[1], p[2], a["max_path"], a["B"], a["Hkv"],
                              a["cap"], p[3], None)


@pytest.mark.parametrize("paged", [False, True])
def test_refusals(paged):
    def r(**kw):
        return _call(paged, **kw)
    assert r(k=None) == 1
    assert r(k=[None]) == 1
    assert r(ctx=None) == 1
    assert r(path=None) == 1
    assert r(acc=None) == 1
    assert r(k=[MIS]) == 2
    assert r(path=0x10002) == 2
    assert r(n=0) == 3
    assert r(max_path=0) == 3
    assert r(max_path=65) == 3
    assert r(B=0) == 3
    assert r(new=A) == 3                              # the new lengths over the old ones
    assert r(acc=0x18000, new=0x18004) == 3           # over the counts
    assert r(path=0x18000, new=0x1801c) == 3          # over the path
    assert r(v=[A]) == 3                              # a cache given twice
    assert r(k=[A, 0x30000], v=[A2, A]) == 3
    if paged:
        assert r(table=None) == 1
        assert r(page=40) == 3
        assert r(max_pages=1 << 27) == 4               # more slots than 32 bits number
    else:
        assert r(cap=60) == 4
        assert r(cap=1 << 31) == 4


@pytest.mark.gpu
@pytest.mark.parametrize("layers,B,Hkv,cap,page,T_,max_path", [
    (1, 1, 1, 8, 0, 1, 1), (2, 3, 4, 64, 0, 20, 7), (5, 6, 2, 96, 32, 40, 12), (65, 2, 1, 128, 64, 64, 64),
    (1, 40, 8, 256, 0, 64, 33), (3, 2, 3, 128, 128, 64, 64)])
def test_moves(T, layers, B, Hkv, cap, page, T_, max_path):
    import torch
    rng = np.random.default_rng(layers * 100 + B)
    if page:
        mp = cap // page
        table = rng.permutation(B * mp + 1)[: B * mp].reshape(B, mp)
        shape = (B * mp + 1, Hkv, page, 66)
    else:
        shape = (B, Hkv, cap, 66)
    caches = [rng.integers(0, 256, shape).astype(np.uint8) for _ in range(2 * layers)]
    ctx = rng.integers(0, cap - T_ + 1, B).astype(np.int32)
    for kind in ("path", "any"):
        acc = rng.integers(0, max_path + 1, B).astype(np.int32)
        acc[0] = max_path
        if kind == "path":
            path = np.stack([np.sort(rng.permutation(T_)[:max_path]) for _ in range(B)]).astype(np.int32)
        else:                                           # any order, repeats
            path = rng.integers(0, T_, (B, max_path)).astype(np.int32)
        dev = [torch.from_numpy(c).cuda() for c in caches]
        t = {n: torch.from_numpy(x).cuda() for n, x in dict(ctx=ctx, path=path, acc=acc).items()}
        if page:
            tb = torch.from_numpy(table.astype(np.int32)).cuda()
            new = T.tbq4_tree_accept_paged(dev[::2], dev[1::2], tb, t["ctx"], t["path"], t["acc"])
        else:
            new = T.tbq4_tree_accept(dev[::2], dev[1::2], t["ctx"], t["path"], t["acc"])
        assert T.tbq4_get_device_status() == 0
        np.testing.assert_array_equal(new.cpu().numpy(), ctx + acc)
        for c, d in zip(caches, dev):
            want = c.copy()
            for b in range(B):
                to, src = ctx[b] + np.arange(acc[b]), ctx[b] + path[b, : acc[b]]
                if page:
                    want[table[b, to // page], :, to % page] = c[table[b, src // page], :, src % page]
                else:
                    want[b, :, to] = c[b, :, src]
            np.testing.assert_array_equal(d.cpu().numpy(), want)


@pytest.mark.gpu
def test_bad_counts_and_nodes(T):
    import torch
    dev = "cuda"
    base = torch.randint(0, 256, (3, 2, 16, 66), device=dev).to(torch.uint8)

    def run(ctx, path, acc):
        k, v = base.clone(), base.clone()
        t = [torch.tensor(x, dtype=torch.int32, device=dev) for x in (ctx, path, acc)]
        new = T.tbq4_tree_accept([k], [v], *t)
        return k, new.tolist(), T.tbq4_get_device_status()
    # a count above max_path, one below 0, one without room: nothing moves there
    k, new, status = run([4, 4, 15], [[1, 2]] * 3, [3, -1, 2])
    assert status == 4 and new == [4, 4, 15] and torch.equal(k, base)
    # a node outside the cache is skipped, the others move
    k, new, status = run([4, 4, 4], [[1, 2], [1, 50], [-7, 3]], [2, 2, 2])
    assert status == 4 and new == [6, 6, 6]
    assert torch.equal(k[1, :, 4], base[1, :, 5]) and torch.equal(k[1, :, 5], base[1, :, 5])
    assert torch.equal(k[2, :, 4], base[2, :, 4]) and torch.equal(k[2, :, 5], base[2, :, 7])


@pytest.mark.parametrize("paged", [False, True])
def test_refuses_caches_that_overlap(paged):
    # one cache's blocks would move while another's are read
    size = (8 * 32 if paged else 2 * 64) * 2 * 66
    assert _call(paged, k=[A], v=[A + size - 16]) == 3
    assert _call(paged, k=[A, 0x80000], v=[A2, 0x80000 + size - 16]) == 3
    assert _call(paged, k=[A + 4 * size], v=[A + 3 * size + 16]) == 3
    assert _call(paged, new=A2 + 64) == 3                # the new lengths in a cache
    if paged:
        assert _call(True, new=A + 8) == 3               # or in the block table
