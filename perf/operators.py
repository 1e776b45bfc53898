"""Speculative decoding with drafted token trees over TBQ4 caches: the operators and what is measured of them.

Three operators, in the order in which a decoding step calls them:

  rope_append   rotate the new tokens' queries and keys by their positions, quantise keys and values, and write them into
                the (contiguous or paged) caches: `tbq4_rope_append`, `tbq4_rope_append_paged`
  attn_tree     attention of a tree of drafted tokens over the cached context and over its own visible nodes:
                `tbq4_attn_tree`, `tbq4_attn_tree_paged`
  tree_accept   keep the accepted path: move its blocks to the front of the drafted region in every layer's caches and
                count the new lengths: `tbq4_tree_accept`, `tbq4_tree_accept_paged`

`run` computes them in plain torch operations, or, with `own` set, by the package's entry points.  A block of a cache is
returned as its scale (fp16 values) and its packed 4-bit indices (whole numbers), both views of the caches themselves.
"""
import math

import torch

own = False

D = 128
BLOCK = 66
SEED = 0                       # seed of the rotation's signs
DTYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}


# --------------------------------------------------------------------------------------------------------------- cases

def listed():
    rope = dict(op="rope_append", pages=64, rot=128, pairs="halves", pad=0)
    tree = dict(op="attn_tree", pages=0, ragged=False)
    accept = dict(op="tree_accept", pages=64)
    return [
        # one new token of one sequence in a decoding step: nothing but latency
        dict(rope, name="rope 1 token", B=1, n=1, q_heads=24, kv_heads=4, dtype="bfloat16", base=1e7, far=200000),
        # a draft tree of 25 nodes for each of 8 ragged sequences, with rows of padding behind the last
        dict(rope, name="rope 8 trees", B=8, n=200, q_heads=24, kv_heads=4, dtype="float16", base=1e6, far=98304, pad=7),
        # an odd prompt in fp32, interleaved pairs, half of each head rotated, contiguous caches
        dict(rope, name="rope 1999 fp32", B=1, n=1999, q_heads=8, kv_heads=8, dtype="float32", base=1e4, far=0, pages=0,
             rot=64, pairs="neighbours"),
        # prompt chunks of 16 sequences at once, behind long contexts
        dict(rope, name="rope 16 x 1024", B=16, n=16384, q_heads=24, kv_heads=4, dtype="bfloat16", base=1e7, far=261000),
        # the smallest tree: two layers of drafts behind a short context
        dict(tree, name="tree 7 at 1K", B=1, nodes=7, q_heads=4, kv_heads=1, ctx=1000, dtype="float32", out="float16"),
        # single-token serving through the tree's entry point
        dict(tree, name="tree 1 at 32K", B=1, nodes=1, q_heads=24, kv_heads=4, ctx=32767, dtype="bfloat16", out="bfloat16"),
        # a ragged batch over pages
        dict(tree, name="tree 8 x 25 paged", B=8, nodes=25, q_heads=24, kv_heads=4, ctx=98304, dtype="bfloat16", out="bfloat16",
             pages=64, ragged=True),
        # a small tree behind the longest context, fp16 out
        dict(tree, name="tree 5 at 262K fp16", B=1, nodes=5, q_heads=24, kv_heads=4, ctx=262000, dtype="float16", out="float16"),
        # an ordinary and the largest tree behind the longest context
        dict(tree, name="tree 16 at 262K", B=1, nodes=16, q_heads=24, kv_heads=4, ctx=262000, dtype="bfloat16", out="bfloat16"),
        dict(tree, name="tree 64 at 262K", B=1, nodes=64, q_heads=24, kv_heads=4, ctx=262080, dtype="bfloat16", out="bfloat16"),
        # one sequence, the four layers of a small model, contiguous caches
        dict(accept, name="accept 1 x 4 layers", layers=4, B=1, kv_heads=4, nodes=8, path=4, cap=1024, pages=0),
        # a serving batch through all layers
        dict(accept, name="accept 64 x 28 layers", layers=28, B=64, kv_heads=4, nodes=25, path=9, cap=256),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, evenly spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["rope_append", "attn_tree", "attn_tree", "tree_accept"])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 6, 8])
    pages = rng.choice([0, 32, 64, 96, 256])
    dtype = rng.choice(list(DTYPES))
    if op == "rope_append":
        n = _spread(rng, 1, 4096 * 4 * 8 // (kv * (group + 2)))
        return dict(op=op, B=rng.randint(1, min(n, 16)), n=n, q_heads=kv * group, kv_heads=kv, dtype=dtype, pages=pages,
                    rot=rng.choice([32, 64, 96, 128]), pairs=rng.choice(["halves", "neighbours"]), pad=rng.randint(0, min(n - 1, 9)),
                    base=rng.choice([1e4, 5e5, 1e7]), far=_spread(rng, 1, 1000000))
    if op == "attn_tree":
        B, nodes = _spread(rng, 1, 24), _spread(rng, 1, 64)
        most = min(262080, (1 << 20) // (B * kv), 384 * (1 << 20) // (B * kv * nodes * group))
        return dict(op=op, B=B, nodes=nodes, q_heads=kv * group, kv_heads=kv, ctx=_spread(rng, 1, most), dtype=dtype,
                    out=rng.choice(["bfloat16", "bfloat16", "float16"]), pages=pages, ragged=rng.choice([True, False]))
    nodes = _spread(rng, 1, 64)
    return dict(op=op, layers=rng.randint(1, 28), B=_spread(rng, 1, 64), kv_heads=min(kv, 4), nodes=nodes,
                path=rng.randint(1, min(nodes, 10)), cap=rng.choice([128, 192, 256]), pages=rng.choice([0, 32, 64]))


# -------------------------------------------------------------------------------------------------------------- inputs

def _lengths(B, most, ragged):
    """Context lengths: all alike, or evenly spread from a sixth of the longest up to it."""
    return [most if not ragged or B == 1 else max(1, most - b * (5 * most) // (6 * (B - 1))) for b in range(B)]


def _counts(case):
    """Drafted nodes of each sequence: all of them, or every other sequence somewhat fewer."""
    return [case["nodes"] - (case["nodes"] // 3 if case["ragged"] and b % 2 else 0) for b in range(case["B"])]


def _generator(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _table(gen, B, per_seq, spare=3):
    """A block table [B][per_seq] whose pages lie scattered over a pool, and the pool's pages."""
    n = B * per_seq + spare
    order = torch.randperm(n, generator=gen, device="cuda")
    return order[: B * per_seq].reshape(B, per_seq).to(torch.int32).contiguous(), n


def _blocks(gen, shape, outliers=False):
    """Random cache blocks as the encoder leaves them: gaussian rows in the rotated domain, scaled and indexed."""
    out = torch.empty((*shape, BLOCK), dtype=torch.uint8, device="cuda")
    flat = out.view(-1, BLOCK)
    for at in range(0, flat.shape[0], 1 << 20):
        part = flat[at: at + (1 << 20)]
        x = torch.randn((part.shape[0], D), generator=gen, device="cuda")
        if outliers:                     # a few rows are much larger than the others
            x *= torch.exp(0.3 * torch.randn((part.shape[0], 1), generator=gen, device="cuda"))
        s = x.abs().amax(-1, keepdim=True).half()
        i = torch.round(x / s.float() * 7.5 + 7.5).clamp(0, 15).to(torch.uint8)
        part[:, :2] = s.view(torch.uint8)
        part[:, 2:] = i[:, 0::2] | (i[:, 1::2] << 4)
    return out


def _parents(gen, nodes):
    """Random trees: node i hangs below one of the nodes just before it, node 0 is the root."""
    i = torch.arange(nodes, device="cuda")
    back = torch.randint(1, 5, (nodes,), generator=gen, device="cuda")
    return torch.where(i > 0, (i - back).clamp(min=0), -1)


def prepare(case, seed):
    gen = _generator(seed)
    st = {"case": case}
    if case["op"] == "rope_append":
        B, n, H, K = case["B"], case["n"], case["q_heads"], case["kv_heads"]
        per = -(-n // B)
        i = torch.arange(n, device="cuda")
        ids = i // per
        offset = torch.randint(0, 40, (B,), generator=gen, device="cuda")
        st["slots"] = (offset[ids] + i % per).to(torch.int32)
        # drafted siblings share a position: every fifth token sits beside the one before it
        st["positions"] = (case["far"] + 3 * ids + i % per - (i % 5 == 4).long()).to(torch.int32)
        st["seq_ids"] = torch.where(i < n - case["pad"], ids, -1).to(torch.int32)
        qkv = torch.randn((n, (H + 2 * K), D), generator=gen, device="cuda")
        qkv[:, H: H + K, :4] *= 10.0                                    # keys with outlier channels
        qkv = qkv.to(DTYPES[case["dtype"]])
        st["q"], st["k"], st["v"] = qkv[:, :H], qkv[:, H: H + K], qkv[:, H + K:]     # slices of one projection
        st["q_out"] = torch.zeros((n, H, D), dtype=qkv.dtype, device="cuda")
        half = torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64)
        st["inv_freq"] = case["base"] ** (-half / case["rot"])
        need = per + 40
        if case["pages"]:
            st["table"], pages = _table(gen, B, -(-need // case["pages"]))
            shape = (pages, K, case["pages"], BLOCK)
        else:
            st["table"], shape = None, (B, K, (need + 7) // 8 * 8, BLOCK)
        st["kc"], st["vc"] = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2))
        return st
    if case["op"] == "attn_tree":
        B, T, H, K = case["B"], case["nodes"], case["q_heads"], case["kv_heads"]
        lens = _lengths(B, case["ctx"], case["ragged"])
        if case["pages"]:
            st["table"], pages = _table(gen, B, -(-(case["ctx"] + T) // case["pages"]))
            shape = (pages, K, case["pages"])
        else:
            st["table"], shape = None, (B, K, (case["ctx"] + T + 7) // 8 * 8)
        st["kc"], st["vc"] = _blocks(gen, shape), _blocks(gen, shape, True)
        st["ctx"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["n_nodes"] = torch.tensor(_counts(case), dtype=torch.int32, device="cuda")
        parents = _parents(gen, T)
        sees = torch.eye(T, dtype=torch.bool, device="cuda")
        at = parents
        for _ in range(T):                                              # ancestors, one generation at a time
            sees |= (at[:, None] == torch.arange(T, device="cuda")) & (at[:, None] >= 0)
            at = torch.where(at >= 0, parents[at.clamp(min=0)], -1)
        bits = torch.where(sees, torch.ones((), dtype=torch.int64, device="cuda") << torch.arange(T, device="cuda"), 0)
        st["mask"] = bits.sum(-1).expand(B, T).contiguous()
        # heads differ in how sharply they attend
        gain = 0.5 + 2.5 * torch.rand((H, 1), generator=gen, device="cuda")
        st["q"] = (torch.randn((B, T, H, D), generator=gen, device="cuda") * gain).to(DTYPES[case["dtype"]])
        st["out"] = torch.zeros((B, T, H, D), dtype=DTYPES[case["out"]], device="cuda")
        st["scale"] = D ** -0.5
        return st
    B, K, L = case["B"], case["kv_heads"], case["layers"]
    room = case["cap"] - case["nodes"]
    st["ctx"] = torch.randint(0, room + 1, (B,), generator=gen, device="cuda").to(torch.int32)
    if case["pages"]:
        st["table"], pages = _table(gen, B, -(-case["cap"] // case["pages"]))
        shape = (pages, K, case["pages"], BLOCK)
    else:
        st["table"], shape = None, (B, K, case["cap"], BLOCK)
    # finite scales, any indices
    st["caches"] = [torch.randint(0, 120, shape, generator=gen, device="cuda").to(torch.uint8) for _ in range(2 * L)]
    order = torch.rand((B, case["nodes"]), generator=gen, device="cuda").argsort(-1)[:, : case["path"]]
    st["path"] = order.sort(-1).values.to(torch.int32).contiguous()
    st["n_accept"] = torch.randint(1, case["path"] + 1, (B,), generator=gen, device="cuda").to(torch.int32)
    st["new_lens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    return st


# --------------------------------------------------------------------------------------------------------- plain forms

_signs = {}


def _sign_row(device):
    """The +-1 diagonal of the rotation: bits of the SplitMix64 stream of SEED, set means -1."""
    if device not in _signs:
        state, words = SEED, []
        for _ in range(2):
            state = (state + 0x9E3779B97F4A7C15) % 2 ** 64
            z = state
            z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9 % 2 ** 64
            z = (z ^ (z >> 27)) * 0x94D049BB133111EB % 2 ** 64
            words.append(z ^ (z >> 31))
        _signs[device] = torch.tensor([1.0 - 2.0 * (words[i // 64] >> (i % 64) & 1) for i in range(D)], device=device)
    return _signs[device]


def _rotate(x):
    """The Hadamard rotation in fp32: signs, butterflies of stride 1 .. 64, each rounded by itself, and one product."""
    x = x * _sign_row(x.device)
    for stride in (1, 2, 4, 8, 16, 32, 64):
        x = x.view(*x.shape[:-1], -1, 2, stride) if x.shape[-1] == D else x
        a, b = x[..., 0, :], x[..., 1, :]
        x = torch.stack((a + b, a - b), -2).flatten(-3)
    return x * torch.tensor(0x3DB504F3, dtype=torch.int32, device=x.device).view(torch.float32)


def _rope(x, cos, sin, rot, pairs):
    a, b = (x[..., : rot // 2], x[..., rot // 2: rot]) if pairs == "halves" else (x[..., 0:rot:2], x[..., 1:rot:2])
    y = (a * cos - b * sin, b * cos + a * sin)
    y = torch.cat(y, -1) if pairs == "halves" else torch.stack(y, -1).flatten(-2)
    return torch.cat((y, x[..., rot:]), -1)


def _rows_of(st, ids, slots):
    """The (page, row) or (sequence, row) of each slot of each sequence."""
    if st["table"] is None:
        return ids, slots
    size = st["case"]["pages"]
    return st["table"].long()[ids, slots // size], slots % size


def _encode(x):
    x = _rotate(x)
    s = x.abs().amax(-1, keepdim=True).clamp(max=65504.0).half()
    f = s.float()
    i = torch.round(x / f * 7.5 + 7.5).clamp(0, 15)
    i = torch.where(f == 0, torch.full_like(i, 8.0), i).to(torch.uint8)
    return torch.cat((s.view(torch.uint8), i[..., 0::2] | (i[..., 1::2] << 4)), -1)


def _plain_rope_append(st):
    case = st["case"]
    angle = st["positions"].double()[:, None] * st["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    real = st["seq_ids"] >= 0
    q = _rope(st["q"].float(), cos, sin, case["rot"], case["pairs"]).to(st["q"].dtype)
    st["q_out"].copy_(torch.where(real[:, None, None], q, st["q_out"]))
    at = _rows_of(st, st["seq_ids"].long()[real], st["slots"].long()[real])
    k = _rope(st["k"].float(), cos, sin, case["rot"], case["pairs"])
    st["kc"][at[0], :, at[1]] = _encode(k[real])
    st["vc"][at[0], :, at[1]] = _encode(st["v"].float()[real])


def _levels(blocks):
    s = blocks[..., :2].contiguous().view(torch.float16).float()
    i = torch.stack((blocks[..., 2:] & 15, blocks[..., 2:] >> 4), -1).flatten(-2)
    return s * (2.0 * i.float() - 15.0) / 15.0


def _gathered(st, cache, longest):
    """Blocks of the tokens 0 .. longest of every sequence: [B][Hkv][longest][66]."""
    if st["table"] is None:
        return cache[:, :, :longest]
    pages = cache[st["table"].long()]                       # [B][pages][Hkv][size][66]
    return pages.transpose(1, 2).flatten(2, 3)[:, :, :longest]


def _plain_attn_tree(st):
    case, ctx, count = st["case"], st["ctx"].long(), st["n_nodes"].long()
    B, T, H, K = case["B"], case["nodes"], case["q_heads"], case["kv_heads"]
    n = case["ctx"] + T
    q = _rotate(st["q"].float()).view(B, T, K, H // K, D).permute(0, 2, 1, 3, 4).flatten(2, 3)       # [B][K][T G][128]
    k = _levels(_gathered(st, st["kc"], n))
    s = (q @ k.transpose(-1, -2) * st["scale"]).view(B, K, T, H // K, -1)
    del k
    t = torch.arange(s.shape[-1], device=q.device)
    j = t - ctx[:, None]                                                                              # node at each token
    bit = (st["mask"][:, :, None] >> j.clamp(0, 63)[:, None]) & 1
    seen = (j < 0)[:, None] | ((bit == 1) & ((j >= 0) & (j < count[:, None]))[:, None])               # [B][T][n]
    s.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top.isinf(), 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    v = _levels(_gathered(st, st["vc"], n))
    o = (p.flatten(2, 3) @ v).view(B, K, T, H // K, D) / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 2, 1, 3, 4).flatten(2, 3)
    # back from the rotated domain: the rotation is symmetric up to its signs
    signs = _sign_row(o.device)
    o = _rotate(o * signs) * signs
    real = torch.arange(T, device=o.device) < count[:, None]
    st["out"].copy_(torch.where(real[:, :, None, None], o.to(st["out"].dtype), st["out"]))


def _plain_tree_accept(st):
    take = torch.arange(st["path"].shape[1], device="cuda") < st["n_accept"][:, None]
    ids = torch.arange(st["path"].shape[0], device="cuda")[:, None].expand_as(take)[take]
    base = st["ctx"].long()[:, None]
    to = (base + torch.arange(st["path"].shape[1], device="cuda")).expand_as(take)[take]
    to, src = _rows_of(st, ids, to), _rows_of(st, ids, (base + st["path"].long())[take])
    for c in st["caches"]:
        c[to[0], :, to[1]] = c[src[0], :, src[1]]
    st["new_lens"].copy_(st["ctx"] + st["n_accept"])


# ----------------------------------------------------------------------------------------------------------------- run

def _own_rope_append(st):
    import long_context_attention_tbq4_b200 as tbq4
    args = dict(q=st["q"], positions=st["positions"], seq_ids=st["seq_ids"], interleaved=st["case"]["pairs"] == "neighbours",
                sign_seed=SEED, q_out=st["q_out"])
    if st["table"] is None:
        tbq4.tbq4_rope_append(st["k"], st["v"], st["slots"], st["inv_freq"], st["kc"], st["vc"], **args)
    else:
        tbq4.tbq4_rope_append_paged(st["k"], st["v"], st["slots"], st["inv_freq"], st["table"], st["kc"], st["vc"], **args)


def _own_attn_tree(st):
    import long_context_attention_tbq4_b200 as tbq4
    args = dict(sign_seed=SEED, n_nodes=st["n_nodes"], out=st["out"])
    if st["table"] is None:
        tbq4.tbq4_attn_tree(st["q"], st["kc"], st["vc"], st["ctx"], st["mask"], st["scale"], **args)
    else:
        tbq4.tbq4_attn_tree_paged(st["q"], st["kc"], st["vc"], st["table"], st["ctx"], st["mask"], st["scale"], **args)


def _own_tree_accept(st):
    import long_context_attention_tbq4_b200 as tbq4
    k, v = st["caches"][0::2], st["caches"][1::2]
    if st["table"] is None:
        tbq4.tbq4_tree_accept(k, v, st["ctx"], st["path"], st["n_accept"], new_lens=st["new_lens"])
    else:
        tbq4.tbq4_tree_accept_paged(k, v, st["table"], st["ctx"], st["path"], st["n_accept"], new_lens=st["new_lens"])


def run(state):
    op = state["case"]["op"]
    if op == "rope_append":
        (_own_rope_append if own else _plain_rope_append)(state)
        return {"q": state["q_out"], "k_scale": state["kc"].view(torch.float16)[..., 0], "k_index": state["kc"][..., 2:],
                "v_scale": state["vc"].view(torch.float16)[..., 0], "v_index": state["vc"][..., 2:]}
    if op == "attn_tree":
        (_own_attn_tree if own else _plain_attn_tree)(state)
        return {"out": state["out"]}
    (_own_tree_accept if own else _plain_tree_accept)(state)
    return {"lens": state["new_lens"], "caches": state["caches"]}


def work(case):
    if case["op"] == "rope_append":
        n, size = case["n"] - case["pad"], DTYPES[case["dtype"]].itemsize
        row = case["q_heads"] * 2 * D * size + 2 * case["kv_heads"] * (D * size + BLOCK)
        # rotation by position, 7 butterfly stages, scale and index of each key and value
        return {"bytes": n * (row + 12) + case["rot"] * 4, "flops": n * D * (case["q_heads"] * 3 + case["kv_heads"] * (3 + 2 * 12))}
    if case["op"] == "attn_tree":
        lens, counts, K, G = _lengths(case["B"], case["ctx"], case["ragged"]), _counts(case), case["kv_heads"], case["q_heads"] // case["kv_heads"]
        tokens = sum(a + b for a, b in zip(lens, counts))
        rows = sum(counts) * case["q_heads"]
        pairs = sum((a + (b + 1) / 2) * b for a, b in zip(lens, counts)) * case["q_heads"]
        io = DTYPES[case["dtype"]].itemsize + DTYPES[case["out"]].itemsize
        return {"bytes": tokens * K * 2 * BLOCK + rows * D * io + sum(counts) * 8 + 8 * case["B"], "flops": pairs * 4 * D}
    moved = case["B"] * (1 + case["path"]) / 2 * case["kv_heads"] * 2 * case["layers"]
    return {"bytes": moved * 2 * BLOCK + case["B"] * (4 * case["path"] + 12), "flops": 0}


# --------------------------------------------------------------------------------------------------------------- exact

def _matrix():
    """The rotation H diag(s) / sqrt(128) in 64 bits, entry by entry: (-1)^popcount(i & j)."""
    i = torch.arange(D, device="cuda")
    both, ones = i[:, None] & i[None], torch.zeros((D, D), dtype=torch.int64, device="cuda")
    for b in range(7):
        ones += (both >> b) & 1
    return (1.0 - 2.0 * (ones % 2).double()) * _sign_row(i.device).double() / math.sqrt(D)


def _turn(x, angle, rot, pairs):
    """Rotates pairs of x's first `rot` channels by `angle`, as products of complex numbers."""
    x = x.double().clone()
    first = torch.arange(rot // 2, device="cuda") * (1 if pairs == "halves" else 2)
    second = first + (rot // 2 if pairs == "halves" else 1)
    z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(angle), angle)[:, None]
    x[..., first], x[..., second] = z.real, z.imag
    return x


def exact(case, seed):
    if case["op"] == "tree_accept":
        return None                                  # nothing is computed: blocks are moved
    st, R = prepare(case, seed), _matrix()
    if case["op"] == "rope_append":
        angle = st["positions"].double()[:, None] * st["inv_freq"]
        ids = st["seq_ids"].tolist()
        real = [i for i, b in enumerate(ids) if b >= 0]
        q = torch.zeros(st["q_out"].shape, dtype=torch.float64, device="cuda")
        q[real] = _turn(st["q"], angle, case["rot"], case["pairs"])[real]
        found = {"q": q, "k_index": None, "v_index": None}
        slots = st["slots"].long()[real]
        seq = torch.tensor([ids[i] for i in real], device="cuda")
        where = (seq, slots) if not case["pages"] else (st["table"].long()[seq, slots // case["pages"]], slots % case["pages"])
        for name, rows in (("k", _turn(st["k"], angle, case["rot"], case["pairs"])), ("v", st["v"].double())):
            scale = torch.zeros(st[name + "c"].shape[:-1], dtype=torch.float64, device="cuda")
            scale[where[0], :, where[1]] = (rows[real] @ R.T).abs().amax(-1)
            found[name + "_scale"] = scale
        return found
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    H, K = case["q_heads"], case["kv_heads"]
    level = (2.0 * torch.arange(16, device="cuda", dtype=torch.float64) - 15.0) / 15.0
    for b in range(case["B"]):
        c, n = int(st["ctx"][b]), int(st["n_nodes"][b])
        sees = (st["mask"][b, :n, None] >> torch.arange(n, device="cuda")) & 1 == 1
        for g in range(K):
            kv = []
            for cache in (st["kc"], st["vc"]):
                if case["pages"]:
                    rows = cache[st["table"][b].long(), g].reshape(-1, BLOCK)[: c + n]
                else:
                    rows = cache[b, g, : c + n]
                scale = (rows[:, 0].int() + 256 * rows[:, 1].int()).to(torch.int16).view(torch.float16).double()
                values = torch.empty((c + n, D), dtype=torch.float64, device="cuda")
                values[:, 0::2], values[:, 1::2] = level[(rows[:, 2:] % 16).long()], level[(rows[:, 2:] // 16).long()]
                kv.append(values * scale[:, None])
            for h in range(g * (H // K), (g + 1) * (H // K)):
                s = (st["q"][b, :n, h].double() @ R.T) @ kv[0].T * st["scale"]
                s[:, c:][~sees] = -math.inf
                out[b, :n, h] = torch.softmax(s, -1) @ kv[1] @ R
    return {"out": out}

