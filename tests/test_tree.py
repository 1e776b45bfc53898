"""Tree attention over TBQ4 caches against its definition in 64 bits, and a
speculative step as it is used: rope-append, tree attention, acceptance and
the next step."""
import ctypes as C

import numpy as np
import pytest

from tree_helpers import check_tree, dequantised, random_tree, rope, rotation, tree_attention

SEED = 5
SCALE = 128 ** -0.5
A, A2, MIS = C.c_void_p(0x10000), C.c_void_p(0x20000), C.c_void_p(0x10004)


@pytest.fixture(scope="module")
def T():
    import long_context_attention_tbq4_b200 as pkg
    return pkg


# ---- host checks ------------------------------------------------------------

def _call(paged=False, **kw):
    from long_context_attention_tbq4_b200._lib import lib as L
    a = dict(q=A, qt=2, k=A, v=A, table=A, max_pages=4, page=32, n_pages=8, ctx=A, nn=A, mask=A, ms=4, B=2, T=4,
             Hq=8, Hkv=2, cap=64, scale=0.1, seed=0, ws=A2, wb=1 << 30, out=A, ot=2, stream=None)
    a.update(kw)
    mid = (a["ctx"], a["nn"], a["mask"], a["ms"], a["B"], a["T"], a["Hq"], a["Hkv"])
    tail = (a["scale"], a["seed"], a["ws"], a["wb"], a["out"], a["ot"], a["stream"])
    if paged:
        return L.tbq4_attn_tree_paged(a["q"], a["qt"], a["k"], a["v"], a["table"], a["max_pages"], a["page"],
                                      a["n_pages"], *mid, *tail)
    return L.tbq4_attn_tree(a["q"], a["qt"], a["k"], a["v"], *mid, a["cap"], *tail)


@pytest.mark.parametrize("paged", [False, True])
def test_refusals(paged):
    def r(**kw):
        return _call(paged, **kw)
    for name in ("q", "k", "v", "ctx", "mask", "ws", "out"):
        assert r(**{name: None}) == 1, name
    for name in ("q", "k", "v", "mask", "ws", "out"):
        assert r(**{name: MIS}) == 2, name
    assert r(qt=3) == 3
    assert r(ot=0) == 3                                # no fp32 output
    assert r(B=0) == 3
    assert r(B=1025) == 3
    assert r(T=0) == 3
    assert r(T=65, ms=65) == 3
    assert r(Hq=7) == 3
    assert r(Hq=18) == 3
    assert r(ms=3) == 3                                # masks that overlap
    assert r(scale=float("nan")) == 3
    assert r(wb=16) == 5
    assert r(qt=0) == 3                                # out over wider queries
    assert r(out=C.c_void_p(0x10000 + 256)) == 3       # out over q, but not in its place
    if paged:
        assert r(table=None) == 1
        assert r(page=48) == 3
        assert r(max_pages=1 << 26) == 4               # more tokens than 32 bits number
    else:
        assert r(cap=60) == 4
        assert r(cap=1 << 31) == 4
        assert r(cap=(1 << 31) - 512, B=1024, Hkv=64, Hq=64) == 3    # more tiles than 32 bits number


def test_workspace_query(T):
    assert T.tbq4_tree_workspace_bytes(1, 4, 24, 4) > 0
    for bad in ((0, 4, 24, 4), (1, 0, 24, 4), (1, 65, 24, 4), (1, 4, 23, 4), (1, 4, 36, 4), (1025, 4, 24, 4)):
        assert T.tbq4_tree_workspace_bytes(*bad) == 0


def test_tree_mask(T):
    import torch
    assert T.tree_mask([-1, 0, 0, 1]).tolist() == [1, 3, 5, 11]
    assert T.tree_mask(torch.tensor([[-1, -1], [-1, 0], [1, -1]])).tolist() == [[1, 2], [1, 3], [3, 2]]
    chain = T.tree_mask(torch.arange(64) - 1)
    assert chain[63].item() == -1 and chain[62].item() == 2 ** 63 - 1
    for bad in ([0], [1, 0], [-2], [1], [-1] * 65):
        with pytest.raises(ValueError):
            T.tree_mask(bad)


# ---- the operator -----------------------------------------------------------

def make(T, seed, B, nodes, Hkv, G, ctx, counts=None, page=0, dtype="bfloat16", out="bfloat16", kind="random",
         gain=1.0, shared=False, outliers=False):
    """Caches (by quantise-append of random rows), queries and masks."""
    import torch
    rng = np.random.default_rng(seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    cap = (max(ctx) + nodes + 7) // 8 * 8
    rows = {}
    for n in "kv":
        x = torch.randn((B, cap, Hkv, 128), generator=gen, device="cuda")
        if outliers and n == "k":
            x[..., [3, 77]] *= 10.0
        if outliers and n == "v":
            x *= torch.exp(2.0 * torch.randn((B, cap, Hkv, 1), generator=gen, device="cuda"))
        rows[n] = x
    start = torch.zeros(B, dtype=torch.int32, device="cuda")
    if page:
        mp = -(-cap // page)
        table = torch.from_numpy(rng.permutation(B * mp + 2)[: B * mp].reshape(B, mp).astype(np.int32)).cuda()
        kc, vc = (torch.full((B * mp + 2, Hkv, page, 66), 0xFF, dtype=torch.uint8, device="cuda") for _ in "kv")
        T.tbq4_quantize_append_paged(rows["k"], start, table, kc, SEED)
        T.tbq4_quantize_append_paged(rows["v"], start, table, vc, SEED)
    else:
        table = None
        kc, vc = (torch.full((B, Hkv, cap, 66), 0xFF, dtype=torch.uint8, device="cuda") for _ in "kv")
        T.tbq4_quantize_append(rows["k"], start, kc, SEED)
        T.tbq4_quantize_append(rows["v"], start, vc, SEED)
    q = (torch.randn((B, nodes, Hkv * G, 128), generator=gen, device="cuda") * gain).to(getattr(torch, dtype))
    trees = np.stack([random_tree(rng, nodes, kind) for _ in range(1 if shared else B)])
    mask = T.tree_mask(torch.from_numpy(trees[0] if shared else trees)).cuda()
    counts = [nodes] * B if counts is None else counts
    return dict(q=q, kc=kc, vc=vc, table=table, ctx=torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                n=torch.tensor(counts, dtype=torch.int32, device="cuda"), mask=mask, out=getattr(torch, out))


def call(T, s, fill=None, **kw):
    import torch
    out = None if fill is None else torch.full(s["q"].shape, fill, dtype=s["out"], device="cuda")
    args = dict(sign_seed=SEED, n_nodes=s["n"], out=out, out_dtype=s["out"])
    args.update(kw)
    if s["table"] is None:
        return T.tbq4_attn_tree(s["q"], s["kc"], s["vc"], s["ctx"], s["mask"], SCALE, **args)
    return T.tbq4_attn_tree_paged(s["q"], s["kc"], s["vc"], s["table"], s["ctx"], s["mask"], SCALE, **args)


def check(T, s):
    """One call against 64 bits; rows of absent nodes stay as they were."""
    import torch
    got = call(T, s, fill=3.5)
    assert T.tbq4_get_device_status() == 0
    want, eps, amp = tree_attention(s["q"], s["kc"], s["vc"], s["ctx"], s["n"], s["mask"], SCALE, SEED, s["table"])
    real = torch.arange(s["q"].shape[1], device="cuda") < s["n"][:, None]
    assert bool((got[~real] == 3.5).all())
    check_tree(got[real], want[real], eps[real], amp[real])
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("nodes,G", [(1, 1), (1, 8), (2, 3), (5, 6), (16, 6), (21, 8), (33, 2), (64, 1), (64, 8), (43, 6)])
def test_rows(T, nodes, G):
    # query rows from 1 to 512: one partial block to several
    check(T, make(T, nodes * 10 + G, 1, nodes, 2, G, [1000]))
    check(T, make(T, nodes * 10 + G + 1, 1, nodes, 1, G, [300], out="float16", dtype="float32"))


@pytest.mark.gpu
@pytest.mark.parametrize("ctx", [0, 1, 2, 31, 32, 120, 127, 128, 129, 255, 256, 2047, 20001])
def test_lengths(T, ctx):
    # the tree inside a tile, across a tile's border, alone without a context
    check(T, make(T, ctx, 1, 9, 2, 4, [ctx]))
    check(T, make(T, ctx + 1, 1, 1, 1, 6, [ctx], out="float16"))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("out", ["float16", "bfloat16"])
def test_types(T, dtype, out):
    s = make(T, 77, 2, 12, 2, 6, [700, 130], dtype=dtype, out=out, page=32)
    assert check(T, s).dtype == s["out"]


@pytest.mark.gpu
@pytest.mark.parametrize("page", [0, 32, 96, 128, 4096])
@pytest.mark.parametrize("out", ["float16", "bfloat16"])
def test_ragged_batch(T, page, out):
    ctx = [0, 5000, 1, 127, 640, 3000, 64]
    counts = [20, 7, 20, 1, 0, 13, 20]                 # one sequence without a tree
    check(T, make(T, 9 + page, 7, 20, 2, 6, ctx, counts, page=page, out=out))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["chain", "star"])
@pytest.mark.parametrize("shared", [False, True])
def test_masks(T, kind, shared):
    check(T, make(T, 21, 3, 30, 2, 4, [200, 31, 77], kind=kind, shared=shared))


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["float16", "bfloat16"])
def test_peaked_and_wide_scales(T, out):
    # logits of tens; K with outlier channels, V scales over several decades
    check(T, make(T, 31, 1, 6, 2, 6, [4000], gain=8.0, out=out))
    check(T, make(T, 32, 2, 10, 1, 6, [4000, 900], gain=3.0, outliers=True, out=out))


@pytest.mark.gpu
@pytest.mark.parametrize("rows", ["tiny", "huge"])
def test_scales_of_queries(T, rows):
    # one query row far larger or smaller than its neighbours in the block
    s = make(T, 33, 1, 4, 1, 4, [500], dtype="float32", out="float16")
    s["q"][0, 1, 2] *= 1e-4 if rows == "tiny" else 50.0
    check(T, s)


@pytest.mark.gpu
def test_large_v_scales_late(T):
    # V scales that grow by 2^20 along the context, and blocks of zeros
    import torch
    s = make(T, 34, 1, 5, 1, 6, [3000], out="float16")
    sc = torch.exp2(torch.linspace(-10, 10, s["vc"].shape[2], device="cuda")).half()
    s["vc"][..., :2] = sc.view(torch.uint8).view(-1, 2)
    check(T, s)
    s["vc"][..., :2] = 0
    assert not call(T, s, fill=1.0).any()
    s["kc"][..., :2] = 0                               # every logit 0: the plain mean
    s["vc"][..., :2] = sc.view(torch.uint8).view(-1, 2)
    check(T, s)


@pytest.mark.gpu
def test_rows_that_see_nothing(T):
    # a mask of 0 sees the context alone; without a context, nothing: zero rows
    import torch
    s = make(T, 41, 2, 8, 2, 3, [0, 200])
    s["mask"][:, 3] = 0
    s["mask"][:, 5] = 1 << 6                           # not itself
    got = check(T, s)
    assert not got[0, 3].any() and got[1, 3].any()
    s["mask"][:] = 0
    got = check(T, s)
    assert not got[0].any()
    # bits of nodes that are not there count for nothing
    s["n"][:] = 4
    s["mask"][:] = -1
    check(T, s)


@pytest.mark.gpu
@pytest.mark.parametrize("poison", [0x7E00, 0x7C00, 0xFC00])
@pytest.mark.parametrize("out", ["float16", "bfloat16"])
def test_poison_behind_masks_and_ends(T, poison, out):
    # NaN and infinite scales in a node that only node 6 sees, and in every slot
    # behind the nodes: no other row may change
    import torch
    s = make(T, 51, 1, 10, 2, 6, [250], counts=[9], out=out)
    s["mask"][0] &= ~(1 << 4)
    clean = call(T, s, fill=0.0)
    bits = torch.tensor([poison & 0xFF, poison >> 8], dtype=torch.uint8, device="cuda")
    for c in (s["kc"], s["vc"]):
        c[:, :, 250 + 4, :2] = bits
        c[:, :, 259:, :2] = bits
        c[:, :, 259:, 2:] = 0x5A
    s["mask"][0, 6] |= 1 << 4
    got = call(T, s, fill=0.0)
    rows = [i for i in range(9) if i != 6]
    assert torch.equal(got[0, rows], clean[0, rows])
    assert not bool(torch.isfinite(got[0, 6]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_queries_stay_in_their_rows(T, bad):
    import torch
    s = make(T, 52, 1, 6, 2, 4, [300])
    clean = call(T, s)
    s["q"][0, 2, 1, 17] = bad
    got = call(T, s)
    ok = torch.ones((6, 8), dtype=torch.bool, device="cuda")
    ok[2, 1] = False
    assert torch.equal(got[0][ok], clean[0][ok])


@pytest.mark.gpu
def test_clamped_lengths_are_flagged(T):
    import torch
    s = make(T, 61, 2, 4, 1, 2, [60, 60])
    for ctx, n in (([60, 1000], [4, 4]), ([-3, 60], [4, 4]), ([60, 60], [4, 5]), ([60, 60], [4, -1])):
        s["ctx"].copy_(torch.tensor(ctx))
        s["n"].copy_(torch.tensor(n))
        call(T, s)
        assert T.tbq4_get_device_status() == 4
    assert T.tbq4_get_device_status() == 0


@pytest.mark.gpu
def test_bad_page_reads_page_zero_and_is_flagged(T):
    s = make(T, 62, 1, 4, 1, 2, [100], page=32)
    s["table"][0, 1] = 99
    call(T, s)
    assert T.tbq4_get_device_status() == 4


@pytest.mark.gpu
def test_offsets_past_32_bits(T):
    # the last KV heads of a cache of 5.5 GB, and the last pages of such a pool
    import torch
    cap = 5_200_000
    s = make(T, 63, 1, 5, 16, 2, [400])
    for n in ("kc", "vc"):
        big = torch.empty((1, 16, cap, 66), dtype=torch.uint8, device="cuda")
        big[:, :, :408] = s[n]
        s[n] = big
    check(T, s)
    s = make(T, 64, 1, 5, 2, 2, [400], page=64)
    pages = 660_000
    for n in ("kc", "vc"):
        big = torch.empty((pages, 2, 64, 66), dtype=torch.uint8, device="cuda")
        big[-s[n].shape[0]:] = s[n]
        s[n] = big
    s["table"] += pages - 9
    assert s["table"].max() < pages
    check(T, s)


@pytest.mark.gpu
def test_long_context(T):
    check(T, make(T, 65, 1, 16, 4, 6, [131000]))
    check(T, make(T, 66, 1, 3, 4, 6, [131000], out="float16"))


@pytest.mark.gpu
def test_many_short_sequences(T):
    rng = np.random.default_rng(4)
    B = 300
    check(T, make(T, 67, B, 5, 1, 2, rng.integers(0, 400, B).tolist(), rng.integers(0, 6, B).tolist(), page=32))


@pytest.mark.gpu
def test_same_bits_on_every_call_and_stream(T):
    import torch
    s = make(T, 71, 3, 17, 2, 6, [3000, 10, 777])
    ref = call(T, s)
    sides = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(6):                                  # two streams at once, a workspace each
        with torch.cuda.stream(sides[i % 2]):
            got.append(call(T, s))
    torch.cuda.synchronize()
    assert all(torch.equal(ref, g) for g in got)


@pytest.mark.gpu
def test_memory_of_a_call_on_another_stream(T):
    # what a call on another stream allocates must not be memory that pending
    # work of the current stream still uses
    import torch
    s = make(T, 73, 1, 16, 2, 6, [9000])
    ref = call(T, s)
    size = T.tbq4_tree_workspace_bytes(1, 16, 12, 2)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = torch.full((size,), 7, dtype=torch.uint8, device="cuda")
    held_out = torch.full(s["q"].shape, 7, dtype=s["out"], device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                       # some 10 ms
    seen, seen_out = held.clone(), held_out.clone()
    del held, held_out
    got = call(T, s, stream=other)
    torch.cuda.synchronize()
    assert torch.equal(got, ref)
    assert bool((seen == 7).all()) and bool((seen_out == 7).all())


@pytest.mark.gpu
def test_out_in_place_of_queries(T):
    import torch
    for ctx in ([2000, 3], [200000, 1]):                # whole works, and joined ones
        s = make(T, 74, 2, 9, 2, 6, ctx)
        want = call(T, s)
        got = call(T, s, out=s["q"])
        assert got.data_ptr() == s["q"].data_ptr() and torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["float16", "bfloat16"])
def test_a_single_visible_token_of_any_logit(T, out):
    # softmax over one token is 1 whatever the logit: rows that see themselves only
    import torch
    s = make(T, 75, 1, 16, 2, 3, [0], out=out, dtype="float32")
    s["mask"] = torch.ones(16, dtype=torch.int64, device="cuda") << torch.arange(16, device="cuda")
    s["q"] *= torch.logspace(-30, 33, 16, device="cuda")[None, :, None, None]
    got = call(T, s)
    v = dequantised(s["vc"][0, :, :16]) @ rotation(SEED, "cuda")       # [Hkv][16][128]
    want = v.repeat_interleave(3, 0).transpose(0, 1)[None]
    amp = dequantised(s["vc"][0, :, :16]).abs().sum(-1).repeat_interleave(3, 0).T[None, ..., None] / 128 ** 0.5
    check_tree(got, want, torch.zeros_like(amp[..., 0]), amp)


@pytest.mark.gpu
def test_first_call_inside_a_capture():
    # in a process of its own: nothing of the library has run before the capture
    import subprocess
    import sys
    code = """
import torch, long_context_attention_tbq4_b200 as T
B, n, Hq, Hkv, cap = 1, 8, 12, 2, 512
dev = dict(device="cuda")
x = torch.randn((n, Hq + 2 * Hkv, 128), dtype=torch.bfloat16, **dev)
ctx = torch.full((B,), 300, dtype=torch.int32, **dev)
slots = torch.arange(300, 308, dtype=torch.int32, **dev)
inv = 1e4 ** (-torch.arange(64, dtype=torch.float64, **dev) / 64)
mask = torch.full((n,), 255, dtype=torch.int64, **dev)
path = torch.tensor([[0, 3, 5]], dtype=torch.int32, **dev)
acc = torch.tensor([3], dtype=torch.int32, **dev)

def step(kc, vc):
    q = T.tbq4_rope_append(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], slots, inv, kc, vc, q=x[:, :Hq])
    o = T.tbq4_attn_tree(q.view(B, n, Hq, 128), kc, vc, ctx, mask, 0.09)
    return o, T.tbq4_tree_accept([kc], [vc], ctx, path, acc)

caches = [torch.zeros((B, Hkv, cap, 66), dtype=torch.uint8, **dev) for _ in range(4)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    o, new = step(caches[0], caches[1])
g.replay()
o2, new2 = step(caches[2], caches[3])
torch.cuda.synchronize()
assert torch.equal(o, o2) and torch.equal(new, new2) and int(new) == 303
assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)


@pytest.mark.gpu
def test_one_capture_serves_any_lengths(T):
    import torch
    s = make(T, 72, 2, 12, 2, 6, [2000, 2000])
    ws = torch.empty(T.tbq4_tree_workspace_bytes(2, 12, 12, 2), dtype=torch.uint8, device="cuda")
    out = torch.zeros(s["q"].shape, dtype=s["out"], device="cuda")
    call(T, s, out=out, workspace=ws)                   # first call outside a capture
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call(T, s, out=out, workspace=ws)
    for ctx, n in (([2000, 2000], [12, 12]), ([0, 1], [1, 12]), ([1999, 130], [0, 7]), ([77, 1500], [12, 3])):
        s["ctx"].copy_(torch.tensor(ctx))
        s["n"].copy_(torch.tensor(n))
        out.fill_(2.0)
        graph.replay()
        assert torch.equal(out, call(T, s, fill=2.0))


@pytest.mark.gpu
def test_chain_agrees_with_multi_query_decode(T):
    # drafts in a row are the multi-query decode's case
    import torch
    s = make(T, 73, 2, 4, 2, 6, [1500, 40], kind="chain", dtype="float32", out="float16")
    got = check(T, s)
    lens = s["ctx"] + 4
    ref = T.tbq4_attn_decode_mq(s["q"], s["kc"], s["vc"], lens, int(lens.max()), SCALE, SEED)
    # both are rounded to fp16 from values within 2^-12 of each other's
    assert (got.double() - ref.double()).norm() <= 2.0 ** -10 * ref.double().norm()


# ---- a run of the three -----------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("page", [0, 64])
def test_speculative_steps(T, page):
    """Three steps of two sequences: prompt, draft trees, acceptance.  A shadow
    of every accepted row is kept in fp32 and, at the end, the caches' accepted
    tokens must be the bytes of a plain append of the rotated rows, and the
    attention of the last step the 64-bit one over them."""
    import torch
    rng = np.random.default_rng(8)
    B, N, Hkv, G, cap, layers = 2, 9, 2, 3, 512, 2
    freq = 1e4 ** (-np.arange(0, 128, 2) / 128)
    inv = torch.from_numpy(freq).cuda()
    if page:
        mp = cap // page
        table = torch.from_numpy(rng.permutation(B * mp).reshape(B, mp).astype(np.int32)).cuda()
        caches = [torch.zeros((B * mp, Hkv, page, 66), dtype=torch.uint8, device="cuda") for _ in range(2 * layers)]
    else:
        table = None
        caches = [torch.zeros((B, Hkv, cap, 66), dtype=torch.uint8, device="cuda") for _ in range(2 * layers)]
    shadow = [[[] for _ in range(B)] for _ in range(2 * layers)]
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")

    def append(layer, qkv, slots, positions, ids):
        q, k, v = qkv.split([Hkv * G, Hkv, Hkv], 1)
        args = dict(q=q, positions=positions, seq_ids=ids, sign_seed=SEED)
        kc, vc = caches[2 * layer: 2 * layer + 2]
        if page:
            return T.tbq4_rope_append_paged(k, v, slots, inv, table, kc, vc, **args)
        return T.tbq4_rope_append(k, v, slots, inv, kc, vc, **args)

    def rows(n):
        return torch.from_numpy(rng.standard_normal((n, Hkv * (G + 2), 128)).astype(np.float32)).to(torch.bfloat16).cuda()

    def dev(x):
        return torch.from_numpy(np.ascontiguousarray(x)).to(torch.int32).cuda()

    def note(layer, qkv, positions, ids, order):
        _, k, v = qkv.float().cpu().split([Hkv * G, Hkv, Hkv], 1)
        k = rope(k.numpy(), positions, freq, False)
        for t in order:
            shadow[2 * layer][ids[t]].append(k[t])
            shadow[2 * layer + 1][ids[t]].append(v.numpy()[t])

    # prompts of 150 and 70 tokens in one call
    ids = np.repeat([0, 1], [150, 70])
    pos = np.concatenate([np.arange(150), np.arange(70)])
    for layer in range(layers):
        x = rows(220)
        append(layer, x, dev(pos), dev(pos), dev(ids))
        note(layer, x, pos, ids, range(220))
    lens.copy_(torch.tensor([150, 70]))
    for step in range(3):
        ctx = lens.cpu().numpy()
        trees = np.stack([random_tree(rng, N) for _ in range(B)])
        depth = np.zeros((B, N), np.int64)
        for b in range(B):
            for i in range(N):
                depth[b, i] = 0 if trees[b, i] < 0 else depth[b, trees[b, i]] + 1
        ids = np.repeat(np.arange(B), N)
        slots = (ctx[:, None] + np.arange(N)).ravel()
        pos = (ctx[:, None] + depth).ravel()
        mask = T.tree_mask(torch.from_numpy(trees)).cuda()
        paths, acc = np.zeros((B, N), np.int32), np.zeros(B, np.int32)
        for b in range(B):
            i, path = int(rng.integers(0, N)), []
            while i >= 0:
                path.append(i)
                i = int(trees[b, i])
            paths[b, : len(path)], acc[b] = path[::-1], len(path)
        for layer in range(layers):
            x = rows(B * N)
            q = append(layer, x, dev(slots), dev(pos), dev(ids)).view(B, N, Hkv * G, 128)
            s = dict(q=q, kc=caches[2 * layer], vc=caches[2 * layer + 1], table=table, ctx=lens, mask=mask,
                     n=torch.full((B,), N, dtype=torch.int32, device="cuda"), out=torch.bfloat16)
            check(T, s)
            note(layer, x, pos, ids, [b * N + j for b in range(B) for j in paths[b, : acc[b]]])
        accept = T.tbq4_tree_accept_paged if page else T.tbq4_tree_accept
        args = (caches[::2], caches[1::2], *((table,) if page else ()), lens, dev(paths), dev(acc))
        lens = accept(*args)
        np.testing.assert_array_equal(lens.cpu().numpy(), ctx + acc)
    assert T.tbq4_get_device_status() == 0
    from tree_helpers import encoded, tokens_of
    for c, sh in zip(caches, shadow):
        for b in range(B):
            want = encoded(np.stack(sh[b]), SEED)
            n = int(lens[b])
            assert n == len(want)
            got = np.stack([tokens_of(c.cpu(), b, g, n, None if table is None else table.cpu()).numpy()
                            for g in range(Hkv)], 1)
            np.testing.assert_array_equal(got, want)
