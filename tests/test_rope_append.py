"""Rotary embedding fused with quantise-append: cache bytes bit for bit against
the oracle's encoder on rows rotated in 64 bits, rotated queries against the
64-bit values within half a step of their type, refusals on the CPU."""
import ctypes as C

import numpy as np
import pytest

from tree_helpers import encoded, rope

SEED = 11
A, A2, MIS = C.c_void_p(0x10000), C.c_void_p(0x20000), C.c_void_p(0x10004)


@pytest.fixture(scope="module")
def T():
    import long_context_attention_tbq4_b200 as pkg
    return pkg


def _call(paged=False, **kw):
    from long_context_attention_tbq4_b200._lib import lib as L
    a = dict(q=A, qs=(256, 128), k=A, ks=(256, 128), v=A, vs=(256, 128), dtype=2, n=4, B=2, Hq=4,
             Hkv=2, ids=A, slots=A, pos=A, freq=A, rot=128, inter=0, cap=64, table=A, max_pages=4,
             page=32, n_pages=8, seed=0, kc=A, vc=A2, qo=A, stream=None)
    a.update(kw)
    head = (a["q"], *a["qs"], a["k"], *a["ks"], a["v"], *a["vs"], a["dtype"], a["n"], a["B"], a["Hq"],
            a["Hkv"], a["ids"], a["slots"], a["pos"], a["freq"], a["rot"], a["inter"])
    tail = (a["seed"], a["kc"], a["vc"], a["qo"], a["stream"])
    if paged:
        return L.tbq4_rope_append_paged(*head, a["table"], a["max_pages"], a["page"], a["n_pages"], *tail)
    return L.tbq4_rope_append(*head, a["cap"], *tail)


@pytest.mark.parametrize("paged", [False, True])
def test_refusals(paged):
    def r(**kw):
        return _call(paged, **kw)
    for name in ("q", "k", "v", "slots", "kc", "vc", "qo", "freq"):
        assert r(**{name: None}) == 1, name
    for name in ("q", "k", "v", "kc", "vc", "qo", "freq"):
        assert r(**{name: MIS}) == 2, name
    assert r(ks=(252, 128)) == 2                       # rows off a 16-byte boundary
    assert r(vs=(256, 68)) == 2
    assert r(qs=(-256, 128)) == 2
    assert r(dtype=3) == 3
    assert r(B=0) == 3
    assert r(Hkv=0) == 3
    assert r(n=-1) == 3
    assert r(rot=12) == 3                              # not a multiple of 8
    assert r(rot=136) == 3
    assert r(vc=A) == 3                                # K and V in one cache
    assert r(ids=None, n=5) == 3                       # 5 tokens over 2 sequences
    assert r(n=0) == 0                                 # nothing to do, nothing launched
    if paged:
        assert r(table=None) == 1
        assert r(page=48) == 3
        assert r(n_pages=0) == 3
    else:
        assert r(cap=60) == 4


def test_refuses_queries_written_over_rows_that_are_read():
    far = dict(k=C.c_void_p(0x100000), v=C.c_void_p(0x200000))
    at = 4 * 4 * 128 * 2                               # bytes of q_out
    assert _call(q=C.c_void_p(0x300000), k=C.c_void_p(0x10000 + at - 16), v=far["v"]) == 3
    assert _call(q=C.c_void_p(0x300000), k=far["k"], v=C.c_void_p(0x10000 - 3 * 512 - 512 + 16)) == 3
    assert _call(q=A, qs=(512, 256), **far) == 3       # q itself, but its rows lie elsewhere
    assert _call(q=A, qs=(1024, 128), **far) == 3
    assert _call(q=C.c_void_p(0x10000 + 256), qs=(512, 128), **far) == 3


def test_binding_refuses_cpu_tensors(T):
    import torch
    kc = torch.zeros((1, 2, 8, 66), dtype=torch.uint8)
    x = torch.zeros((1, 2, 128))
    with pytest.raises(TypeError):
        T.tbq4_rope_append(x, x, torch.zeros(1, dtype=torch.int32), None, kc, kc.clone())


def _frequencies(rot, base=1e4):
    return base ** (-np.arange(0, rot, 2) / max(rot, 1))


def _run(T, n, B, Hq, Hkv, dtype, rot, interleaved, paged, far=0, fused=True, seed=0, pad=0,
         order="ids", positions=True):
    """One call on random rows; checks caches (written and untouched bytes) and q."""
    import torch
    rng = np.random.default_rng(1000 + seed)
    x = rng.standard_normal((n, Hq + 2 * Hkv, 128)).astype(np.float32)
    x[:, Hq: Hq + Hkv, 5] *= 12.0
    x = torch.from_numpy(x).to(dtype).cuda()
    if fused:
        q, k, v = x[:, :Hq], x[:, Hq: Hq + Hkv], x[:, Hq + Hkv:]
    else:                                               # head-major storage, tokens inside
        q, k, v = (t.transpose(0, 1).contiguous().transpose(0, 1)
                   for t in (x[:, :Hq], x[:, Hq: Hq + Hkv], x[:, Hq + Hkv:]))
    per = -(-n // B)
    ids = np.arange(n) // per if order == "ids" else rng.integers(0, B, n)
    slots = np.zeros(n, np.int64)
    for b in range(B):                                  # distinct slots, not in order
        at = np.flatnonzero(ids == b)
        slots[at] = rng.permutation(len(at) + 3)[: len(at)] + 2
    pos = (far + rng.integers(0, 5000, n)).astype(np.int64)
    ids[n - pad:] = -1
    cap = int(slots.max() + 8) // 8 * 8 + 8
    freq = _frequencies(rot)

    def dev(a, t=torch.int32):
        return torch.from_numpy(np.ascontiguousarray(a)).to(t).cuda()
    fill = 0xA5
    args = dict(q=q if Hq else None, positions=dev(pos) if positions else None, seq_ids=dev(ids),
                interleaved=interleaved, sign_seed=SEED)
    inv = dev(freq, torch.float64) if rot else None
    if Hq:
        args["q_out"] = torch.full((n, Hq, 128), 7.0, dtype=dtype, device="cuda")
    if paged:
        size = paged
        mp = -(-cap // size)
        table = rng.permutation(B * mp + 2)[: B * mp].reshape(B, mp)
        kc, vc = (torch.full((B * mp + 2, Hkv, size, 66), fill, dtype=torch.uint8, device="cuda") for _ in "kv")
        got_q = T.tbq4_rope_append_paged(k, v, dev(slots), inv, dev(table), kc, vc, **args)
    else:
        kc, vc = (torch.full((B, Hkv, cap, 66), fill, dtype=torch.uint8, device="cuda") for _ in "kv")
        got_q = T.tbq4_rope_append(k, v, dev(slots), inv, kc, vc, **args)
    assert T.tbq4_get_device_status() == 0
    real = ids >= 0
    p = pos if positions else slots
    for rows, cache in ((rope(k.float().cpu().numpy(), p, freq[: rot // 2], interleaved), kc),
                        (v.float().cpu().numpy(), vc)):
        want = np.full(tuple(cache.shape), fill, np.uint8)
        enc = encoded(rows, SEED)
        for t in np.flatnonzero(real):
            if paged:
                want[table[ids[t], slots[t] // size], :, slots[t] % size] = enc[t]
            else:
                want[ids[t], :, slots[t]] = enc[t]
        np.testing.assert_array_equal(cache.cpu().numpy(), want)
    if Hq:
        # 64-bit rotation; the kernel's angle is exact to binary32 and its three
        # operations round once each: 2 (|x1| + |x2|) 2^-24 and some, then half
        # a step of the type
        theta = p.astype(np.float64)[:, None] * freq
        xq = q.double().cpu().numpy()
        want = xq.copy()
        h = rot // 2
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, h), slice(h, rot))
        c, s = np.cos(theta)[:, None], np.sin(theta)[:, None]
        want[..., a] = xq[..., a] * c - xq[..., b] * s
        want[..., b] = xq[..., b] * c + xq[..., a] * s
        size_ = np.zeros_like(want)
        size_[..., a] = size_[..., b] = np.abs(xq[..., a]) + np.abs(xq[..., b])
        half = torch.finfo(dtype).eps / 2
        tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
        bound = 4 * 2.0 ** -24 * size_ + half * (np.abs(want) + 4 * 2.0 ** -24 * size_) + tiny
        got = got_q.double().cpu().numpy()
        assert (np.abs(got - want)[real] <= bound[real]).all()
        assert (got[~real] == 7.0).all()                # padding is left as it was


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 8, 64, 96, 128])
def test_types_and_pairs(T, dtype, interleaved, rot):
    import torch
    _run(T, 13, 2, 6, 2, getattr(torch, dtype), rot, interleaved, 0, seed=rot)
    _run(T, 13, 2, 6, 2, getattr(torch, dtype), rot, interleaved, 32, seed=rot + 1, fused=False)


@pytest.mark.gpu
@pytest.mark.parametrize("n,B,Hq,Hkv", [(1, 1, 4, 1), (1, 1, 24, 4), (2, 2, 1, 1), (7, 3, 8, 8), (64, 1, 24, 4),
                                        (130, 5, 40, 5), (1000, 16, 12, 2), (2050, 1, 24, 4), (33, 1, 0, 3)])
def test_sizes(T, n, B, Hq, Hkv):
    import torch
    _run(T, n, B, Hq, Hkv, torch.bfloat16, 128, False, 64 if n % 2 else 0, seed=n, pad=min(3, n - 1))


@pytest.mark.gpu
def test_scattered_sequences_and_default_positions(T):
    import torch
    _run(T, 200, 7, 8, 2, torch.float16, 128, False, 96, order="random", seed=5, pad=9)
    _run(T, 200, 7, 8, 2, torch.float32, 64, True, 0, order="random", seed=6, positions=False)


@pytest.mark.gpu
@pytest.mark.parametrize("far", [262144, 1 << 24, (1 << 31) - 6000])
def test_far_positions(T, far):
    # angles of up to 2^31 radians: an angle kept in 32 bits would be off by 100
    import torch
    _run(T, 65, 1, 4, 2, torch.float32, 128, False, 0, far=far, seed=far % 97)


@pytest.mark.gpu
@pytest.mark.parametrize("rot,interleaved,dtype", [(128, False, "bfloat16"), (128, True, "float32"), (96, False, "float16")])
def test_every_bit_of_many_rows(T, rot, interleaved, dtype):
    # 24,000 rows a case: a product and a sum rounded once instead of twice
    # changes an index in a million, and a binary32 query in ten
    import torch
    n, Hq, Hkv = 3000, 2, 4
    gen = torch.Generator("cuda").manual_seed(rot + interleaved)
    x = torch.randn((n, Hq + 2 * Hkv, 128), generator=gen, device="cuda").to(getattr(torch, dtype))
    pos = torch.arange(n, dtype=torch.int32, device="cuda") * 37 % 200003
    freq = _frequencies(rot, 1e6)
    kc, vc = (torch.zeros((1, Hkv, n, 66), dtype=torch.uint8, device="cuda") for _ in "kv")
    q = T.tbq4_rope_append(x[:, Hq: Hq + Hkv], x[:, Hq + Hkv:], torch.arange(n, dtype=torch.int32, device="cuda"),
                           torch.from_numpy(freq).cuda(), kc, vc, q=x[:, :Hq], positions=pos,
                           interleaved=interleaved, sign_seed=SEED)
    rows = x.float().cpu().numpy()
    want_q = torch.from_numpy(rope(rows[:, :Hq], pos.cpu().numpy(), freq, interleaved)).to(x.dtype)
    assert torch.equal(q.cpu(), want_q)
    for got, r in ((kc, rope(rows[:, Hq: Hq + Hkv], pos.cpu().numpy(), freq, interleaved)), (vc, rows[:, Hq + Hkv:])):
        np.testing.assert_array_equal(got[0].cpu().numpy().transpose(1, 0, 2), encoded(r, SEED))


@pytest.mark.gpu
def test_no_tokens(T):
    import torch
    x = torch.zeros((0, 2, 128), device="cuda", dtype=torch.bfloat16)
    kc, vc = (torch.full((2, 2, 8, 66), 9, dtype=torch.uint8, device="cuda") for _ in "kv")
    q = T.tbq4_rope_append(x, x, torch.zeros(0, dtype=torch.int32, device="cuda"), None, kc, vc,
                           q=torch.zeros((0, 4, 128), device="cuda", dtype=torch.bfloat16))
    assert q.shape == (0, 4, 128)
    assert bool((kc == 9).all()) and bool((vc == 9).all())


@pytest.mark.gpu
def test_in_place_queries_and_implied_sequences(T):
    import torch
    g = torch.Generator("cuda").manual_seed(3)
    q = torch.randn((6, 4, 128), generator=g, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.randn((6, 2, 128), generator=g, device="cuda", dtype=torch.bfloat16) for _ in "kv")
    slots = torch.tensor([4, 5, 0, 1, 9, 8], dtype=torch.int32, device="cuda")
    inv = torch.from_numpy(_frequencies(128)).cuda()
    kc, vc, kc2, vc2 = (torch.zeros((3, 2, 16, 66), dtype=torch.uint8, device="cuda") for _ in range(4))
    ids = torch.tensor([0, 0, 1, 1, 2, 2], dtype=torch.int32, device="cuda")
    want = T.tbq4_rope_append(k, v, slots, inv, kc, vc, q=q, seq_ids=ids)
    got = T.tbq4_rope_append(k, v, slots, inv, kc2, vc2, q=q, q_out=q)
    assert got.data_ptr() == q.data_ptr()
    assert torch.equal(got, want) and torch.equal(kc, kc2) and torch.equal(vc, vc2)


@pytest.mark.gpu
def test_bad_slots_ids_and_pages_are_skipped_and_flagged(T):
    import torch
    dev = "cuda"
    x = torch.randn((4, 2, 128), device=dev)
    for slots, ids in (([3, 16, 1, 0], [0, 0, 0, 0]), ([3, -1, 1, 0], [0, 0, 0, 0]), ([3, 2, 1, 0], [0, 1, 0, 0])):
        kc, vc = (torch.zeros((1, 2, 16, 66), dtype=torch.uint8, device=dev) for _ in "kv")
        T.tbq4_rope_append(x, x, torch.tensor(slots, dtype=torch.int32, device=dev), None, kc, vc,
                           seq_ids=torch.tensor(ids, dtype=torch.int32, device=dev))
        assert T.tbq4_get_device_status() == 4
        written = kc[0, 0].any(-1).cpu().numpy()
        assert written[[3, 1, 0]].all() and written.sum() == 3
    table = torch.tensor([[1, 7]], dtype=torch.int32, device=dev)      # page 7 of 3: none
    kc, vc = (torch.zeros((3, 2, 32, 66), dtype=torch.uint8, device=dev) for _ in "kv")
    T.tbq4_rope_append_paged(x, x, torch.tensor([0, 31, 32, 40], dtype=torch.int32, device=dev), None, table, kc, vc)
    assert T.tbq4_get_device_status() == 4
    assert kc[1, 0].any(-1).sum() == 2 and not kc[0].any() and not kc[2].any()


@pytest.mark.gpu
def test_equals_separate_quantize_append(T):
    # without a rotation the fused call writes what two quantise-appends write
    import torch
    k, v = (torch.randn((40, 4, 128), device="cuda") for _ in "kv")
    a = [torch.zeros((1, 4, 64, 66), dtype=torch.uint8, device="cuda") for _ in range(4)]
    T.tbq4_rope_append(k, v, torch.arange(5, 45, dtype=torch.int32, device="cuda"), None, a[0], a[1], sign_seed=9)
    start = torch.tensor([5], dtype=torch.int32, device="cuda")
    T.tbq4_quantize_append(k[None], start, a[2], 9)
    T.tbq4_quantize_append(v[None], start, a[3], 9)
    assert torch.equal(a[0], a[2]) and torch.equal(a[1], a[3])


@pytest.mark.gpu
@pytest.mark.parametrize("rot,interleaved", [(0, False), (128, False), (64, True), (96, False)])
def test_every_scale_of_rows(T, rot, interleaved):
    # rows of zeros, of scales that round to 0 or are subnormal in fp16, that
    # saturate at 65504 or fall just short of it: the encoder's rare branch
    import torch
    n, Hkv = 240, 3
    gen = torch.Generator("cuda").manual_seed(rot + interleaved)
    x = torch.randn((n, 2 * Hkv, 128), generator=gen, device="cuda")
    size = torch.tensor([0.0, 1e-9, 2e-8, 3e-8, 1e-7, 1e-6, 2e-5, 1.0, 2e4, 3e4, 1e6, 1e30], device="cuda")
    x *= size[torch.arange(n, device="cuda") % 12][:, None, None]
    x[5, 0] = 0.0
    x[5, 0, 7] = 65504.0                                # spread evenly: 65504 / sqrt(128) everywhere
    pos = np.arange(n) * 11
    freq = _frequencies(rot, 1e5)
    kc, vc = (torch.full((1, Hkv, n, 66), 0xA5, dtype=torch.uint8, device="cuda") for _ in "kv")
    T.tbq4_rope_append(x[:, :Hkv], x[:, Hkv:], torch.arange(n, dtype=torch.int32, device="cuda"),
                       torch.from_numpy(freq).cuda() if rot else None, kc, vc,
                       positions=torch.from_numpy(pos).to(torch.int32).cuda(), interleaved=interleaved, sign_seed=SEED)
    assert T.tbq4_get_device_status() == 0
    rows = x.cpu().numpy()
    for got, r in ((kc, rope(rows[:, :Hkv], pos, freq[: rot // 2], interleaved)), (vc, rows[:, Hkv:])):
        got = got[0].cpu().numpy().transpose(1, 0, 2)
        scales = got[..., :2].copy().view(np.uint16)
        assert (scales == 0).any() and ((scales > 0) & (scales < 0x400)).any() and (scales == 0x7BFF).any()
        np.testing.assert_array_equal(got, encoded(r, SEED))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq", [1, 4, 7])
@pytest.mark.parametrize("rot,interleaved", [(128, False), (128, True), (64, False), (64, True), (96, False), (0, False)])
@pytest.mark.parametrize("n", [1, 9, 6000])
def test_in_place_queries(T, n, rot, interleaved, Hq):
    # a pair's halves are read again from the row that is written over: with one
    # row to a half-warp, an odd count, and as many warps to a token as it has
    # pairs of rows, or one
    import torch
    g = torch.Generator("cuda").manual_seed(n + rot + Hq)
    for dtype in (torch.float32, torch.bfloat16):
        q = torch.randn((n, Hq, 128), generator=g, device="cuda").to(dtype)
        k, v = (torch.randn((n, 1, 128), generator=g, device="cuda").to(dtype) for _ in "kv")
        slots = torch.arange(n, dtype=torch.int32, device="cuda")
        inv = torch.from_numpy(_frequencies(rot)).cuda() if rot else None
        caches = [torch.zeros((1, 1, (n + 7) // 8 * 8, 66), dtype=torch.uint8, device="cuda") for _ in range(4)]
        want = T.tbq4_rope_append(k, v, slots, inv, *caches[:2], q=q, interleaved=interleaved)
        got = T.tbq4_rope_append(k, v, slots, inv, *caches[2:], q=q, q_out=q, interleaved=interleaved)
        assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)
        assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


@pytest.mark.parametrize("paged", [False, True])
def test_refuses_caches_that_overlap(paged):
    far = dict(q=C.c_void_p(0x300000), k=C.c_void_p(0x400000), v=C.c_void_p(0x500000), qo=C.c_void_p(0x600000))
    size = (8 * 32 if paged else 2 * 64) * 2 * 66
    assert _call(paged, **{**far, "vc": C.c_void_p(0x10000 + size - 16)}) == 3
    assert _call(paged, **{**far, "vc": C.c_void_p(0x10000 - size + 16)}) == 3
    # rotated queries over a cache
    assert _call(paged, **{**far, "qo": C.c_void_p(0x10000 + size - 16)}) == 3
    assert _call(paged, **{**far, "qo": C.c_void_p(0x20000 - 16)}) == 3
