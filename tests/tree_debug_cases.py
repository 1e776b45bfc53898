"""Runs the draft-tree entry points once on seeded inputs and saves the results
(cache bytes, outputs, the device status) to an .npz file; as a script:
``python tests/tree_debug_cases.py OUT.npz``, with TBQ4_DEBUG=1 on the debug
build.  ``test_tree_debug.py`` runs it both ways and compares."""
import os
import sys

import numpy as np


def run(path):
    import torch
    import long_context_attention_tbq4_b200 as T
    from long_context_attention_tbq4_b200 import _lib

    gen = torch.Generator("cuda").manual_seed(20261207)
    res = {"debug": np.array(int(_lib.DEBUG)), "lib": np.array(os.path.basename(_lib.LIB_PATH))}
    B, Hkv, Hq, N = 3, 4, 24, 20
    inv = 1e6 ** (-torch.arange(0, 128, 2, dtype=torch.float64, device="cuda") / 128)
    lens = torch.tensor([3000, 130, 700], dtype=torch.int32, device="cuda")
    order = torch.randperm(200, generator=gen, device="cuda")

    def rows(n, h, dtype):
        return torch.randn((n, h, 128), generator=gen, device="cuda").to(dtype)

    def bits(t):
        return t.cpu().contiguous().view(torch.int16).numpy()
    for name, page, dtype in (("flat", 0, torch.float32), ("paged", 64, torch.bfloat16)):
        if page:
            table = order[: B * 50].reshape(B, 50).to(torch.int32).contiguous()
            caches = [torch.zeros((200, Hkv, page, 66), dtype=torch.uint8, device="cuda") for _ in "kv"]
        else:
            caches = [torch.zeros((B, Hkv, 3200, 66), dtype=torch.uint8, device="cuda") for _ in "kv"]

        def append(n_of, start, freq, interleaved):
            ids = torch.repeat_interleave(torch.arange(B, device="cuda"), n_of).to(torch.int32)
            slots = torch.cat([s + torch.arange(int(n), device="cuda") for s, n in zip(start.tolist(), n_of.tolist())])
            n = int(n_of.sum())
            args = (rows(n, Hkv, dtype), rows(n, Hkv, dtype), slots.to(torch.int32), freq)
            kw = dict(q=rows(n, Hq, dtype), seq_ids=ids, interleaved=interleaved, sign_seed=3)
            if page:
                return T.tbq4_rope_append_paged(*args, table, *caches, **kw)
            return T.tbq4_rope_append(*args, *caches, **kw)
        append(lens.long(), torch.zeros(B, dtype=torch.int64), inv, False)          # the contexts
        q = append(torch.full((B,), N, device="cuda"), lens, inv[:40].contiguous(), bool(page))
        mask = T.tree_mask(torch.arange(N) // 2 - 1).cuda()
        nodes = torch.tensor([N, 7, N], dtype=torch.int32, device="cuda")
        q = q.view(B, N, Hq, 128)
        for out_dtype in (torch.float16, torch.bfloat16):
            out = torch.zeros(q.shape, dtype=out_dtype, device="cuda")
            kw = dict(sign_seed=3, n_nodes=nodes, out=out)
            if page:
                T.tbq4_attn_tree_paged(q, *caches, table, lens, mask, 0.088, **kw)
            else:
                T.tbq4_attn_tree(q, *caches, lens, mask, 0.088, **kw)
            res[f"{name}_{out_dtype}"] = bits(out)
        paths = torch.tensor([[0, 2, 6], [1, 3, 3], [0, 1, 2]], dtype=torch.int32, device="cuda")
        acc = torch.tensor([3, 2, 0], dtype=torch.int32, device="cuda")
        if page:
            new = T.tbq4_tree_accept_paged([caches[0]], [caches[1]], table, lens, paths, acc)
        else:
            new = T.tbq4_tree_accept([caches[0]], [caches[1]], lens, paths, acc)
        res[name + "_lens"] = new.cpu().numpy()
        res[name + "_k"], res[name + "_v"] = (c.cpu().numpy() for c in caches)
    torch.cuda.synchronize()
    res["status"] = np.array(T.tbq4_get_device_status())
    np.savez(path, **res)


if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    run(sys.argv[1])
