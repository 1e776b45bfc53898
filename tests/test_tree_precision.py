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
