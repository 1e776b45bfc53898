"""What the draft-tree calls of the binding refuse before the library sees it."""
import pytest


@pytest.fixture(scope="module")
def T():
    import long_context_attention_tbq4_b200 as pkg
    return pkg


def test_check_names_what_is_no_tensor(T):
    import torch
    for bad in (None, 3, [1, 2], "slots"):
        with pytest.raises(TypeError, match="slots"):
            T._check("slots", bad, torch.int32, 1, 0)
    with pytest.raises(TypeError, match="slots"):
        T._check("slots", torch.zeros(3, dtype=torch.int32), torch.int32, 1, 0)        # not on a GPU


@pytest.mark.gpu
def test_arguments_that_are_no_tensors(T):
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros((1, 2, 8, 66), dtype=torch.uint8, device="cuda") for _ in "kv")
    pool = [torch.zeros((2, 2, 32, 66), dtype=torch.uint8, device="cuda") for _ in "kv"]
    x, q = torch.zeros((1, 2, 128), device="cuda"), torch.zeros((1, 1, 4, 128), device="cuda")
    slots, ctx, mask = torch.zeros(1, **i32), torch.ones(1, **i32), torch.ones(1, dtype=torch.int64, device="cuda")
    path, table = torch.zeros((1, 1), **i32), torch.zeros((1, 1), **i32)
    for bad in (None, 5, [0]):
        if bad is not None:                             # None is a value of these
            for kw in (dict(positions=bad), dict(seq_ids=bad), dict(q=bad), dict(q=x, q_out=bad)):
                with pytest.raises(TypeError):
                    T.tbq4_rope_append(x, x, slots, None, kc, vc, **kw)
            with pytest.raises(TypeError):
                T.tbq4_rope_append(x, x, slots, bad, kc, vc)
            for kw in (dict(n_nodes=bad), dict(workspace=bad), dict(out=bad)):
                with pytest.raises(TypeError):
                    T.tbq4_attn_tree(q, kc, vc, ctx, mask, 0.1, **kw)
            with pytest.raises(TypeError):
                T.tbq4_tree_accept([kc], [vc], ctx, path, ctx, new_lens=bad)
        for at in (0, 1, 2, 4, 5):
            args = [x, x, slots, None, kc, vc]
            args[at] = bad
            with pytest.raises(TypeError):
                T.tbq4_rope_append(*args)
        for at in range(5):
            args = [q, kc, vc, ctx, mask]
            args[at] = bad
            with pytest.raises(TypeError):
                T.tbq4_attn_tree(*args, 0.1)
        with pytest.raises(TypeError):
            T.tbq4_attn_tree_paged(q, *pool, bad, ctx, mask, 0.1)
        with pytest.raises(TypeError):
            T.tbq4_rope_append_paged(x, x, slots, None, bad, *pool)
        with pytest.raises(TypeError):
            T.tbq4_tree_accept_paged(pool[:1], pool[1:], bad, ctx, path, ctx)
        for at in (2, 3, 4):
            args = [[kc], [vc], ctx, path, ctx]
            args[at] = bad
            with pytest.raises(TypeError):
                T.tbq4_tree_accept(*args)
        for ks, vs in (([bad], [vc]), ([kc], [bad])):
            with pytest.raises(TypeError):
                T.tbq4_tree_accept(ks, vs, ctx, path, ctx)
    assert T.tbq4_get_device_status() == 0
