"""bl_embedding and bl_embedding_backward on the GPU: the lookup bit for bit
against its definition, the table's gradient against the fp64 statement of
tests/train_ref.py with the bound derived there. Token lists of every kind:
one token, all alike, all different, Zipf, padding, ids outside the table,
runs that end on, before and after every boundary of the 32-token chunks."""
import numpy as np
import pytest
import torch

import train_ref as R
from parity import guarded_empty, guards_intact

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
TYPES = [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)]


@pytest.fixture(scope="module")
def bl():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import bit_linear_layers_b200 as m
    return m


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _zipf(T, V, seed):
    rng = np.random.default_rng(seed)
    p = 1.0 / (np.arange(V) + 2.7)
    return torch.from_numpy(rng.permutation(V)[rng.choice(V, T, p=p / p.sum())])


def _plain(ids, table, scale, dtype):
    return (table[ids.long()].float() * scale).to(dtype)


@pytest.mark.parametrize("tt,yt", TYPES)
@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (1, 1000, 4096), (16, 300, 2048), (7, 50, 33), (300, 1000, 1000), (2000, 31, 8),
                                   (5, 9, 10000)])
def test_lookup(bl, T, V, D, tt, yt):
    table = torch.randn(V, D, generator=_gen(T + D)).to(tt).cuda()
    ids = _zipf(T, V, D).cuda()
    for it in (torch.int32, torch.int64):
        for scale in (1.0, 45.25483322143555, -0.3):
            out, buf, s = guarded_empty((T, D), yt, "cuda")
            y = bl.embedding(ids.to(it), table, scale=scale, out=out)
            assert torch.equal(y, _plain(ids, table, np.float32(scale).item(), yt))
            assert guards_intact(buf, T * D, sentinel=s)
    assert bl.device_error() == (0, 0)


def test_lookup_shapes_and_views(bl):
    table = torch.randn(40, 24, generator=_gen(1)).cuda()
    ids = torch.randint(0, 40, (3, 5), generator=_gen(2)).cuda()
    y = bl.embedding(ids, table, out_dtype=BF16)
    assert y.shape == (3, 5, 24) and y.dtype == BF16 and torch.equal(y, table[ids].to(BF16))
    # a table and an output that start between 16-byte boundaries
    flat = torch.randn(1 + 40 * 24, generator=_gen(3)).cuda()
    odd = flat[1:].view(40, 24)
    out = torch.empty(1 + 15 * 24, device="cuda")[1:].view(15, 24)
    assert torch.equal(bl.embedding(ids.view(-1), odd, out=out), odd[ids.view(-1)])
    assert bl.embedding(ids[:0], table).shape == (0, 5, 24)
    torch.cuda.synchronize()
    assert bl.device_error() == (0, 0)


@pytest.mark.parametrize("D", [8, 33, 4096])
def test_lookup_outside_the_table(bl, D):
    table = torch.randn(10, D, generator=_gen(4)).cuda()
    for it, bad in ((torch.int32, -1), (torch.int64, 10), (torch.int64, 1 << 40), (torch.int64, -(1 << 40))):
        ids = torch.tensor([3, bad, 9, 0], dtype=it).cuda()
        y = bl.embedding(ids, table, out=torch.full((4, D), 7.0, device="cuda"))
        assert bl.device_error()[0] == bl.BL_ERR_INVALID_ARG
        assert not bool(y[1].any()) and torch.equal(y[[0, 2, 3]], table[[3, 9, 0]])
        assert bl.device_error() == (0, 0)


def _check_grad(bl, ids, dy, V, tt, scale=1.0, padding_id=None, accumulate=False, seed=0, it=torch.int64):
    T, D = dy.shape
    out, buf, s = guarded_empty((V, D), tt, "cuda")
    old = None
    if accumulate:
        out.copy_(torch.randn(V, D, generator=_gen(seed)))
        old = R.f64(out)
    else:
        out.fill_(7.0)
    got = bl.embedding_backward(ids.to(it).cuda(), dy.cuda(), V, scale=scale, padding_id=padding_id, out=out,
                                accumulate=accumulate)
    ref = R.embedding_backward(ids.tolist(), R.f64(dy), V, scale, padding_id)
    if old is not None:
        ref = ref + old
    bound = R.embedding_backward_bound(ids.tolist(), R.f64(dy), V, ref, tt, scale, padding_id, old)
    R.check(got, ref, bound, f"T={T} V={V} D={D}")
    assert guards_intact(buf, V * D, sentinel=s)
    if accumulate:
        rest = np.ones(V, dtype=bool)
        live = [v for v in ids.tolist() if 0 <= v < V and v != padding_id]
        rest[live] = False
        assert np.array_equal(R.f64(got)[rest], old[rest])
    return got


@pytest.mark.parametrize("gt,tt", TYPES)
@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (1, 500, 4096), (2, 3, 8), (31, 7, 33), (32, 5, 64), (33, 4, 256), (64, 2, 257),
                                   (300, 1000, 1000), (1000, 100, 264), (3000, 257, 40), (700, 70000, 16)])
def test_gradient(bl, T, V, D, gt, tt):
    dy = torch.randn(T, D, generator=_gen(T + V)).to(gt)
    ids = _zipf(T, V, T)
    _check_grad(bl, ids, dy, V, tt, scale=1.7, it=torch.int32)
    _check_grad(bl, ids, dy, V, tt, padding_id=int(ids[0]))
    _check_grad(bl, ids, dy, V, tt, scale=-0.5, accumulate=True)
    assert bl.device_error() == (0, 0)


@pytest.mark.parametrize("D", [8, 300])
def test_runs_at_every_boundary(bl, D):
    """Runs of equal tokens that start at each place of a chunk and end around each end of the next ones."""
    V = 6
    for start in (0, 1, 31, 32, 33, 63):
        for n in (1, 30, 31, 32, 33, 34, 63, 64, 65, 95, 96, 97, 129, 200):
            ids = torch.tensor([0] * start + [2] * n + [4] * 3)
            dy = torch.randn(len(ids), D, generator=_gen(n))
            _check_grad(bl, ids, dy, V, F32)


@pytest.mark.parametrize("ids", [[5] * 5000, [0] * 3000 + [1] * 3000, [9] * 2000 + list(range(9)) * 10, list(range(4000)),
                                 list(range(4000, 0, -1)), [3, 7] * 2500], ids=["alike", "two", "one", "up", "down", "mixed"])
def test_skewed_lists(bl, ids):
    V = max(ids) + 2
    dy = torch.randn(len(ids), 48, generator=_gen(len(ids))).to(BF16)
    t = torch.tensor(ids)[torch.randperm(len(ids), generator=_gen(7))] if ids[0] != 4000 else torch.tensor(ids)
    _check_grad(bl, t, dy, V, F32)
    _check_grad(bl, t, dy, V, BF16, accumulate=True)
    assert bl.device_error() == (0, 0)


@pytest.mark.parametrize("T", [8191, 8192, 8193, 20000, 70001])
def test_long_lists(bl, T):
    """Several rounds of the sort's warps; three digits. Small integers: every sum is exact."""
    V, D = 66000, 8
    ids = _zipf(T, V, T)
    dy = torch.randint(-4, 5, (T, D), generator=_gen(T)).float()
    got = bl.embedding_backward(ids.cuda(), dy.cuda(), V)
    assert torch.equal(got.cpu(), torch.zeros(V, D).index_add_(0, ids, dy))
    got = bl.embedding_backward(ids.cuda(), dy.cuda(), V, padding_id=int(ids[3]))
    keep = ids != ids[3]
    assert torch.equal(got.cpu(), torch.zeros(V, D).index_add_(0, ids[keep], dy[keep]))


def test_tokens_outside_the_table_and_nothing_left(bl):
    dy = torch.randn(70, 40, generator=_gen(8))
    for bad in (-1, 12, 1 << 40, -(1 << 40)):
        ids = torch.randint(0, 12, (70,), generator=_gen(9))
        ids[::7] = bad
        _check_grad(bl, ids, dy, 12, F32)
        assert bl.device_error()[0] == bl.BL_ERR_INVALID_ARG
    # every token is padding, or outside
    _check_grad(bl, torch.full((70,), 3), dy, 12, F32, padding_id=3)
    assert bl.device_error() == (0, 0)
    _check_grad(bl, torch.full((70,), -5), dy, 12, BF16)
    assert bl.device_error()[0] == bl.BL_ERR_INVALID_ARG
    _check_grad(bl, torch.full((70,), 3), dy, 12, F32, padding_id=3, accumulate=True)
    assert bl.device_error() == (0, 0)


def test_rows_of_dy_that_are_not_finite_stay_alone(bl):
    dy = torch.randn(200, 16, generator=_gen(10))
    ids = torch.randint(1, 20, (200,), generator=_gen(11))
    ids[50:60] = 0
    ids[ids == 7] = 8
    ids[20] = 7
    dy[50:60] = float("nan")
    dy[20] = float("inf")
    got = bl.embedding_backward(ids.cuda(), dy.cuda(), 20, padding_id=0)
    assert not bool(got[0].any()) and bool(torch.isinf(got[7]).all())
    keep = torch.arange(20) != 7
    assert bool(torch.isfinite(got[keep]).all())


def test_no_tokens(bl):
    ids, dy = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty((0, 24), dtype=BF16, device="cuda")
    out = torch.full((9, 24), 7.0, device="cuda")
    assert not bool(bl.embedding_backward(ids, dy, 9, out=out).any())
    out.fill_(7.0)
    assert bool((bl.embedding_backward(ids, dy, 9, out=out, accumulate=True) == 7).all())


def test_results_repeat(bl):
    ids = _zipf(20000, 3001, 1).cuda()
    dy = torch.randn(20000, 264, generator=_gen(12)).to(BF16).cuda()
    ref = bl.embedding_backward(ids, dy, 3001, padding_id=5)
    for _ in range(4):
        assert torch.equal(ref, bl.embedding_backward(ids, dy, 3001, padding_id=5))


def test_one_workspace_for_calls_in_a_row(bl):
    """Larger and smaller problems through one workspace: nothing of the call before shows."""
    ws = torch.empty(bl.workspace_bytes(bl.BL_OP_EMBEDDING_BACKWARD, 5000, 9000, 64), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)
    for T, V in ((5000, 9000), (10, 40), (5000, 3), (100, 9000), (4000, 500)):
        ids, dy = _zipf(T, V, T + V), torch.randint(-4, 5, (T, 64), generator=_gen(T)).float()
        got = bl.embedding_backward(ids.cuda(), dy.cuda(), V, ws=ws)
        assert torch.equal(got.cpu(), torch.zeros(V, 64).index_add_(0, ids, dy))


def test_workspace_on_any_16_byte_boundary(bl):
    need = bl.workspace_bytes(bl.BL_OP_EMBEDDING_BACKWARD, 3000, 50, 64)
    buf = torch.empty(need + 64, dtype=torch.uint8, device="cuda")
    ids, dy = _zipf(3000, 50, 5), torch.randint(-4, 5, (3000, 64), generator=_gen(6)).float()
    ref = torch.zeros(50, 64).index_add_(0, ids, dy)
    for off in (0, 16, 48):
        assert torch.equal(bl.embedding_backward(ids.cuda(), dy.cuda(), 50, ws=buf[off:off + need]).cpu(), ref)


def test_two_streams_and_a_graph(bl):
    T, V, D = 3000, 2000, 128
    data = [(_zipf(T, V, s).cuda(), torch.randint(-4, 5, (T, D), generator=_gen(s)).to(BF16).cuda()) for s in (1, 2)]
    ref = [torch.zeros(V, D, device="cuda").index_add_(0, i, d.float()) for i, d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    got = [[], []]
    for _ in range(4):
        for k, (i, d) in enumerate(data):
            with torch.cuda.stream(streams[k]):
                got[k].append(bl.embedding_backward(i, d, V))
    torch.cuda.synchronize()
    assert all(torch.equal(ref[k], g) for k in (0, 1) for g in got[k])
    ids, dy = data[0][0].clone(), data[0][1].clone()
    out = torch.empty(V, D, device="cuda")
    ws = torch.empty(bl.workspace_bytes(bl.BL_OP_EMBEDDING_BACKWARD, T, V, D), dtype=torch.uint8, device="cuda")
    y = torch.empty(T, D, dtype=BF16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bl.embedding(ids, out, out=y)
        bl.embedding_backward(ids, dy, V, out=out, ws=ws)
    for k in (1, 0, 1):
        ids.copy_(data[k][0])
        dy.copy_(data[k][1])
        before = out.clone()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref[k]) and torch.equal(y, before[ids].to(BF16))


def test_gradient_against_differences(bl):
    """The lookup is linear: a step of one element changes the loss by exactly the gradient times it."""
    T, V, D = 40, 6, 5
    rng = np.random.default_rng(3)
    ids = torch.from_numpy(rng.integers(0, V, T))
    dy = torch.from_numpy(rng.integers(-3, 4, (T, D))).float()
    d = bl.embedding_backward(ids.cuda(), dy.cuda(), V, scale=2.0).cpu()
    table = torch.from_numpy(rng.integers(-3, 4, (V, D))).float()

    def loss(t):
        return float((bl.embedding(ids.cuda(), t.cuda(), scale=2.0).cpu() * dy).sum())

    base = loss(table)
    for v in range(V):
        for k in range(D):
            t = table.clone()
            t[v, k] += 1.0
            assert loss(t) - base == float(d[v, k])


def test_refusals(bl):
    table, ids = torch.zeros(5, 8, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    dy = torch.zeros(4, 8, device="cuda")
    bad = [lambda: bl.embedding(ids.float(), table), lambda: bl.embedding(ids.cpu(), table), lambda: bl.embedding(ids, table.half()),
           lambda: bl.embedding(ids, table.t()), lambda: bl.embedding(ids, table, out=dy[:2]),
           lambda: bl.embedding_backward(ids, dy[:3], 5), lambda: bl.embedding_backward(ids, dy, 5, padding_id=5),
           lambda: bl.embedding_backward(ids, dy, 5, padding_id=-1), lambda: bl.embedding_backward(ids, dy, 5, accumulate=True),
           lambda: bl.embedding_backward(ids, dy, 5, out=table[:4]), lambda: bl.embedding_backward(ids, dy.t(), 5)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(bl.BitLinearError):
        bl.embedding_backward(ids, dy, 5, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("tt,yt", TYPES)
@pytest.mark.parametrize("D", [510, 511, 512, 514, 516, 1028, 2050, 2060, 2071])
def test_widths(bl, D, tt, yt):
    """Accesses of one, two, four and eight elements, with and without columns behind the last whole tile."""
    V, T = 60, 333
    ids = _zipf(T, V, D).cuda()
    table = torch.randn(V, D, generator=_gen(D)).to(tt).cuda()
    out, buf, s = guarded_empty((T, D), yt, "cuda")
    assert torch.equal(bl.embedding(ids, table, scale=3.0, out=out), _plain(ids, table, 3.0, yt))
    assert guards_intact(buf, T * D, sentinel=s)
    _check_grad(bl, ids.cpu(), torch.randn(T, D, generator=_gen(D + 1)).to(yt), V, tt, scale=0.7)
    _check_grad(bl, ids.cpu(), torch.randn(T, D, generator=_gen(D + 2)).to(yt), V, tt, accumulate=True)


@pytest.mark.parametrize("T", [127, 128, 129, 4095, 4735, 4736, 4737, 6000])
@pytest.mark.parametrize("V", [3, 5000])
def test_lists_of_any_length(bl, T, V):
    """On both sides of where counting gives way to sorting. Small integers: every sum is exact, and a token's rows
    are added whichever way it is."""
    D = 33
    ids = _zipf(T, V, T + V)
    dy = torch.randint(-4, 5, (T, D), generator=_gen(T)).float()
    for it in (torch.int32, torch.int64):
        got = bl.embedding_backward(ids.to(it).cuda(), dy.cuda(), V)
        assert torch.equal(got.cpu(), torch.zeros(V, D).index_add_(0, ids, dy))
    bad = ids.clone()
    bad[T // 2], bad[T - 1] = -1, V
    keep = (bad >= 0) & (bad < V) & (bad != ids[0])
    got = bl.embedding_backward(bad.cuda(), dy.cuda(), V, padding_id=int(ids[0]))
    assert torch.equal(got.cpu(), torch.zeros(V, D).index_add_(0, ids[keep], dy[keep]))
    assert bl.device_error()[0] != 0 and bl.device_error() == (0, 0)
