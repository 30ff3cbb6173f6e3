"""Layouts that the embedding and clipping calls take: ids that are slices or transposed, gradients that are dense but
not contiguous."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def bl():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import bit_linear_layers_b200 as m
    return m


@pytest.mark.parametrize("it", [torch.int32, torch.int64])
def test_ids_of_any_strides(bl, it):
    g = torch.Generator().manual_seed(1)
    ids = torch.randint(0, 50, (6, 9), generator=g).to(it).cuda()
    table = torch.randn(50, 24, generator=g).cuda()
    for view in (ids[:, :-1], ids[:, 1:], ids.t(), ids[::2], ids[:, 3], ids[:1].expand(4, 9), ids[2, 3], ids[:, 4:4]):
        want = table[view.long()]
        y = bl.embedding(view, table)
        assert y.shape == want.shape and y.is_contiguous() and torch.equal(y, want)
        dy = torch.randint(-4, 5, (*view.shape, 24), generator=g).float().cuda()
        got = bl.embedding_backward(view, dy, 50)
        assert torch.equal(got, torch.zeros(50, 24, device="cuda").index_add_(0, view.reshape(-1).long(), dy.reshape(-1, 24)))
    assert bl.device_error() == (0, 0)


def test_ids_of_any_strides_on_a_stream_and_in_a_graph(bl):
    g = torch.Generator().manual_seed(2)
    ids, table = torch.randint(0, 50, (64, 33), generator=g).cuda(), torch.randn(50, 24, generator=g).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [bl.embedding(ids[:, k:], table) for k in range(1, 8)]
    s.synchronize()
    assert all(torch.equal(y, table[ids[:, k:]]) for k, y in zip(range(1, 8), got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = bl.embedding(ids[:, :-1], table)
    for k in range(3):
        ids.copy_(torch.randint(0, 50, (64, 33), generator=g))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, table[ids[:, :-1]])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_dense_gradients_in_any_order(bl, dtype):
    g = torch.Generator().manual_seed(3)

    def make():
        g.manual_seed(3)
        return [torch.randn(40, 70, generator=g).to(dtype).cuda().t(), torch.randn(5, 6, 7, generator=g).to(dtype).cuda().permute(2, 0, 1),
                torch.randn(2, 3, 8, 8, generator=g).to(dtype).cuda().to(memory_format=torch.channels_last),
                torch.randn(100, generator=g).to(dtype).cuda(), torch.randn(1, 9, generator=g).to(dtype).cuda().t()]

    src = make()
    plain = [t.contiguous() for t in src]
    want = [torch.empty_like(t) for t in plain]
    n0, c0 = bl.grad_clip(plain, 1.0, out=want)
    for in_place in (False, True):
        ts = make()
        outs = ts if in_place else [torch.empty_like(t) for t in ts]
        n, c = bl.grad_clip(ts, 1.0, out=None if in_place else outs)
        # fp64 sums of fp32 squares in another order
        assert abs(float(n) / float(n0) - 1) < 1e-6 and abs(float(c) / float(c0) - 1) < 1e-6
        assert all(torch.allclose(o.float(), w.float(), rtol=2.0 ** -7 if dtype == BF16 else 1e-6, atol=0) for o, w in zip(outs, want))
        assert in_place or all(torch.equal(a, b) for a, b in zip(ts, src))


def test_layouts_refused(bl):
    t = torch.randn(8, 6, device="cuda")
    out = torch.zeros(6, 8, device="cuda")
    for call in (lambda: bl.grad_clip([t[:, :3]], 1.0), lambda: bl.grad_clip([t[::2]], 1.0),
                 lambda: bl.grad_clip([t[:1].expand(4, 6)], 1.0), lambda: bl.grad_clip([t.t()], 1.0, out=[out]),
                 lambda: bl.grad_clip([t], 1.0, out=[out.t()]), lambda: bl.grad_clip([t.to_sparse()], 1.0),
                 lambda: bl.embedding_backward(torch.zeros(8, dtype=torch.int64, device="cuda"), out.t(), 5)):
        with pytest.raises(ValueError):
            call()
    assert not bool(out.any())
