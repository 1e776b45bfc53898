"""Tree attention at the ends of its ranges: no nodes at all, the largest batch,
rows of every kind in one captured call."""
import numpy as np
import pytest

from test_tree import T, call, check, make  # noqa: F401  (T is a fixture)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 40])
@pytest.mark.parametrize("out", ["float16", "bfloat16"])
def test_no_nodes_at_all(T, B, out):  # noqa: F811
    s = make(T, 91, B, 5, 4, 2, [100] * B, counts=[0] * B, out=out)
    assert bool((call(T, s, fill=3.5) == 3.5).all())
    assert T.tbq4_get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_largest_batch(T, dtype):  # noqa: F811
    rng = np.random.default_rng(6)
    check(T, make(T, 92, 1024, 3, 1, 2, rng.integers(0, 300, 1024).tolist(), rng.integers(0, 4, 1024).tolist(),
                  page=32, dtype=dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("nodes,G,dtype", [(64, 8, "float16"), (64, 8, "bfloat16"), (11, 6, "float32"), (8, 8, "float32")])
def test_bf16_outputs_of_wider_queries(T, nodes, G, dtype):  # noqa: F811
    # two terms a weight: blocks of 64 rows, one full, one and two rows over
    check(T, make(T, 93, 2, nodes, 2, G, [700, 3], page=64, dtype=dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["float16", "bfloat16"])
def test_one_capture_serves_any_sizes_of_rows_and_scales(T, out):  # noqa: F811
    import torch
    s = make(T, 94, 2, 12, 2, 6, [2000, 300], out=out)
    ws = torch.empty(T.tbq4_tree_workspace_bytes(2, 12, 12, 2), dtype=torch.uint8, device="cuda")
    got = torch.zeros(s["q"].shape, dtype=s["out"], device="cuda")
    call(T, s, out=got, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call(T, s, out=got, workspace=ws)
    q, v = s["q"].clone(), s["vc"].clone()
    for kind in ("plain", "huge row", "zero rows", "nan row", "scales"):
        s["q"].copy_(q)
        s["vc"].copy_(v)
        if kind == "huge row":
            s["q"][1, 4, 3] = 1e30
        elif kind == "zero rows":
            s["q"][:, 2:5] = 0
        elif kind == "nan row":
            s["q"][0, 7, 1, 5] = float("nan")
            s["q"][0, 8, 1] *= 1e-9
        elif kind == "scales":
            sc = torch.exp2(torch.linspace(-24, 15, v.shape[2], device="cuda")).half()
            s["vc"][..., :2] = sc.view(torch.uint8).view(-1, 2)
        got.fill_(2.0)
        graph.replay()
        want = call(T, s, fill=2.0)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)), kind
        if kind in ("zero rows", "plain"):
            check(T, s)
        rest = torch.ones(s["q"].shape[:3], dtype=torch.bool, device="cuda")
        rest[1, 4, 3] = kind != "huge row"
        rest[0, 7, 1] = kind != "nan row"
        assert bool(torch.isfinite(got[rest]).all()) or kind == "scales", kind
    assert T.tbq4_get_device_status() == 0
