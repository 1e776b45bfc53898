"""Tree attention where bits could run out: hidden and unweighted tokens of
large V scales."""
import pytest

from test_tree import T, call, check, make  # noqa: F401  (T is a fixture)


def _bits(value):
    import torch
    return torch.tensor([value & 0xFF, value >> 8], dtype=torch.uint8, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["float16", "bfloat16"])
@pytest.mark.parametrize("scale", [0.02, 0.1, 2.5])
def test_a_hidden_node_of_the_largest_scale_changes_no_other_row(T, out, scale):  # noqa: F811
    # 65504 is what the encoder saturates at: a draft that overflowed.  Rows that
    # do not see it take it with weight 0, so nothing of theirs may change
    import torch
    s = make(T, 81, 1, 10, 2, 6, [250], out=out)
    mean = s["vc"][..., :2].contiguous().view(torch.float16).float().mean()
    sv = s["vc"][..., :2].contiguous().view(torch.float16).float() * (scale / mean)
    s["vc"][..., :2] = sv.half().view(torch.uint8)
    s["mask"][0] &= ~(1 << 4)
    clean = check(T, s)
    for c in (s["kc"], s["vc"]):
        c[:, :, 250 + 4, :2] = _bits(0x7BFF)
    assert torch.equal(call(T, s, fill=3.5), clean)
    s["kc"][:, :, 250 + 4, :2] = _bits(0x3C00)
    s["mask"][0, 6] |= 1 << 4                           # one row sees it, at an ordinary logit
    got = check(T, s)
    rows = [i for i in range(10) if i != 6]
    assert torch.equal(got[0, rows], clean[0, rows])


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["float16", "bfloat16"])
def test_a_token_of_the_largest_scale_and_no_weight(T, out):  # noqa: F811
    # token 3 has V scale 65504 and a logit of about -60: e^-60 of the others'
    # weight, so the row is the others' mean to 2^-70
    import torch
    s = make(T, 82, 1, 1, 2, 1, [700], out=out, dtype="float32")
    k = -60.0 * 128 ** 0.5 * s["q"][0, 0] / (s["q"][0, 0] ** 2).sum(-1, keepdim=True)
    T.tbq4_rope_append(k[None], k[None], torch.tensor([3], dtype=torch.int32, device="cuda"), None,
                       s["kc"], torch.empty_like(s["vc"]), sign_seed=5)
    sv = s["vc"][..., :2].contiguous().view(torch.float16).float() * 0.01
    s["vc"][..., :2] = sv.half().view(torch.uint8)
    s["vc"][:, :, 3, :2] = _bits(0x7BFF)
    check(T, s)


@pytest.mark.gpu
def test_many_small_weights_beside_a_large_one(T):  # noqa: F811
    # 32,767 tokens 20 below a token whose V is nearly 0: each weight is 2^-29
    # of the row's largest, and they make the row.  160 sequences share the
    # pages, so that CTAs hold whole sequences (a share of the tokens without
    # the large one would be easy)
    import torch
    from tree_helpers import check_tree, tree_attention
    n, B = 32767, 160
    gen = torch.Generator("cuda").manual_seed(83)
    q = torch.randn((1, 1, 1, 128), generator=gen, device="cuda")
    k = torch.randn((1, n + 1, 1, 128), generator=gen, device="cuda")
    k[0, 0, 0] = 20.0 * 128 ** 0.5 * q[0, 0, 0] / (q ** 2).sum()
    v = 100.0 + torch.randn((1, n + 1, 1, 128), generator=gen, device="cuda")
    v[0, 0] = 1e-6
    table = torch.arange(128, dtype=torch.int32, device="cuda")[None]
    s = dict(kc=torch.empty((128, 1, 256, 66), dtype=torch.uint8, device="cuda"), table=table.expand(B, 128).contiguous(),
             q=q.expand(B, 1, 1, 128).contiguous(), out=torch.float16,
             ctx=torch.full((B,), n, dtype=torch.int32, device="cuda"),
             n=torch.ones(B, dtype=torch.int32, device="cuda"),
             mask=torch.ones(1, dtype=torch.int64, device="cuda"))
    s["vc"] = torch.empty_like(s["kc"])
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    T.tbq4_quantize_append_paged(k, start, table, s["kc"], 5)
    T.tbq4_quantize_append_paged(v, start, table, s["vc"], 5)
    got = call(T, s)
    want, eps, amp = tree_attention(q, s["kc"], s["vc"], s["ctx"], s["n"], s["mask"], 128 ** -0.5, 5, table)
    assert T.tbq4_get_device_status() == 0
    check_tree(got, want.expand(B, 1, 1, 128), eps.expand(B, 1, 1), amp.expand(B, 1, 1, 1))


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["float16", "bfloat16"])
@pytest.mark.parametrize("size", [1e6, 1e12, 1e30])
def test_a_huge_query_changes_no_other_row(T, out, size):  # noqa: F811
    # finite, as memory that nobody wrote may hold in the rows of a padded tree;
    # the row itself is beyond what logits resolve, and its neighbours are not
    import torch
    from tree_helpers import check_tree, tree_attention
    for dtype in ("float32", "bfloat16"):
        s = make(T, 84, 1, 12, 2, 4, [300], dtype=dtype, out=out)
        want = tree_attention(s["q"], s["kc"], s["vc"], s["ctx"], s["n"], s["mask"], 128 ** -0.5, 5)
        s["q"][0, 2, 1] *= size
        s["q"][0, 5, 6] *= 1e-30                        # and a tiny one: the plain mean of what it sees
        tiny = s["q"].clone()
        tiny[0, 2, 1] = 0
        small = tree_attention(tiny, s["kc"], s["vc"], s["ctx"], s["n"], s["mask"], 128 ** -0.5, 5)
        got = call(T, s)
        ok = torch.ones(s["q"].shape[:3], dtype=torch.bool, device="cuda")
        ok[0, 2, 1] = ok[0, 5, 6] = False
        check_tree(got[ok], *(x[ok] for x in want))
        check_tree(got[0, 5, 6][None], *(x[0, 5, 6][None] for x in small))
        assert T.tbq4_get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "float16"])
@pytest.mark.parametrize("page", [0, 64])
def test_sharp_queries_of_more_than_bf16_bits(T, dtype, page):  # noqa: F811
    """Logits of some +-100 over 20,000 tokens, bf16 output.  Queries that carry
    more bits than bf16 go in as pairs: a logit is off by 2^-22 of the sum of
    |q_d k_d| (eps is 2^-11 of it), a weight by 2^-22 and by what that does to
    it, sums and exponentials by 2^-18; and the output is rounded once, by at
    most 2^-8 relative, uniformly, so that the 2-norm is within 2^-8 / sqrt(3)
    but for chance (9,216 elements: a few percent)."""
    import torch
    from tree_helpers import tree_attention
    s = make(T, 85, 1, 12, 2, 3, [20000], dtype=dtype, out="bfloat16", gain=30.0, page=page)
    got = call(T, s, fill=3.5).double()
    assert T.tbq4_get_device_status() == 0
    want, eps, amp = tree_attention(s["q"], s["kc"], s["vc"], s["ctx"], s["n"], s["mask"], 128 ** -0.5, 5, s["table"])
    x = torch.expm1(eps * 2.0 ** -11)[..., None] * (1 + 2.0 ** -22) + 2.0 ** -22 + 2.0 ** -18
    err = (got - want).abs()
    assert bool((err <= 2 * x * amp + 2.0 ** -8 * (want.abs() + 2 * x * amp)).all())
    rest = float((2 * x * amp).expand_as(want).norm() / want.norm())
    assert float(err.norm() / want.norm()) <= 1.05 * 2.0 ** -8 / 3 ** 0.5 + rest, (float(err.norm() / want.norm()), rest)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,out", [("bfloat16", "bfloat16"), ("float32", "bfloat16"), ("float16", "float16")])
@pytest.mark.parametrize("gain", [1.0, 6.0])
def test_error_of_ordinary_calls(T, dtype, out, gain):  # noqa: F811
    """The 2-norm of the error, from independent roundings.  A rounding by at most
    h is uniform, so its rms is h / sqrt(3).  The output's h is 2^-8 (bf16) or
    2^-11 relative; a query channel's and a weight's h 2^-11 relative for one
    term, 2^-22 for pairs, and 2^-18 for sums and exponentials.  A channel's
    moves logit t by scale q_d k_td of it; a weight off by x_t moves the row by
    p_t x_t (v_t - o).  Those add up in squares, with 10 % left for chance."""
    import torch
    from tree_helpers import dequantised, rotation, tree_attention
    s = make(T, 86, 1, 12, 2, 3, [3000], dtype=dtype, out=out, gain=gain)
    got = call(T, s, fill=3.5).double()
    want, _, _ = tree_attention(s["q"], s["kc"], s["vc"], s["ctx"], s["n"], s["mask"], 128 ** -0.5, 5)
    h = 2.0 ** -11 if dtype == out == "bfloat16" else 2.0 ** -22
    R, total = rotation(5, "cuda"), (torch.finfo(s["out"]).eps / 2) ** 2 / 3 * float(want.norm()) ** 2
    sees = torch.ones((12, 3012), dtype=torch.bool, device="cuda")
    sees[:, 3000:] = (s["mask"][0][:, None] >> torch.arange(12, device="cuda")) & 1 == 1
    for head in range(6):
        k, v = (dequantised(s[c][0, head // 3, :3012]) for c in ("kc", "vc"))
        q = s["q"][0, :, head].double() @ R.T
        p = ((q @ k.T) / 128 ** 0.5).masked_fill(~sees, float("-inf")).softmax(-1)
        x2 = (q ** 2) @ (k ** 2).T / 128 * h ** 2 / 3 + h ** 2 / 3 + 2.0 ** -36
        o = p @ v
        dist = (v ** 2).sum(-1)[None] - 2 * o @ v.T + (o ** 2).sum(-1, keepdim=True)
        total += float((p ** 2 * x2 * dist).sum())
    err = float((got - want).norm())
    print(f"error {err / float(want.norm()):.3e}, expected at most {(total ** 0.5) / float(want.norm()):.3e}")
    assert err <= 1.1 * total ** 0.5
