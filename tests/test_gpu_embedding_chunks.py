"""The table's gradient where the sums go by chunks of 32 positions (long lists of wide rows), and lists that are
in order already. Small integers: every sum is exact whatever its order, so results are compared bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
RUNS = [1, 30, 31, 32, 33, 34, 63, 64, 65, 95, 96, 97, 128, 129, 200, 511, 545, 1100]  # 545: more than 16 chunks


@pytest.fixture(scope="module")
def bl():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import bit_linear_layers_b200 as m
    return m


def _align(n):
    return (n + 255) // 256 * 256


def _workspace(T, D, chunk):
    """Bytes of the workspace: two lists, the counters, the long segments, two partial rows per chunk."""
    n = -(-T // chunk)
    return 2 * _align(8 * T) + 256 + _align(8 * n) + _align(8 * n * D) + 256


def _list(first, T, seed):
    """Ids in order: `first` tokens of row 0, then a run of every length in some order, again and again, rows 2, 4, ..."""
    g = torch.Generator().manual_seed(seed)
    counts, total = [first], first
    while total < T:
        for i in torch.randperm(len(RUNS), generator=g).tolist():
            counts.append(min(RUNS[i], T - total))
            total += counts[-1]
    return torch.repeat_interleave(torch.arange(0, 2 * len(counts), 2), torch.tensor(counts)), 2 * len(counts)


def _check(bl, ids, dy, V, tt, accumulate=False, padding_id=None):
    T, D = dy.shape
    buf = torch.full((V * D + 128,), 7.0, dtype=tt, device="cuda")  # what lies around the table keeps its value
    out = buf[64:64 + V * D].view(V, D)
    ref = torch.zeros(V, D, device="cuda")
    if accumulate:
        ref = torch.randint(-8, 9, (V, D), generator=torch.Generator("cuda").manual_seed(T), device="cuda").float()
        out.copy_(ref)
    live = torch.ones_like(ids, dtype=torch.bool) if padding_id is None else ids != padding_id
    ref.index_add_(0, ids[live].long(), dy[live].float())
    got = bl.embedding_backward(ids, dy, V, out=out, accumulate=accumulate, padding_id=padding_id)
    assert torch.equal(got, ref.to(tt))
    assert bool((buf[:64] == 7).all()) and bool((buf[64 + V * D:] == 7).all())


@pytest.mark.parametrize("gt,tt", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("T,D", [(9500, 4096), (9473, 4099), (9601, 4100), (9700, 4098)])
def test_chunks_of_32(bl, T, D, gt, tt):
    assert bl.workspace_bytes(bl.BL_OP_EMBEDDING_BACKWARD, T, 100, D) == _workspace(T, D, 32)
    g = torch.Generator("cuda").manual_seed(D)
    for k, first in enumerate((0, 1, 31, 32, 33, 63, 64, 65)):
        ids, V = _list(first, T, k)
        if k % 2:
            ids = ids[torch.randperm(T, generator=torch.Generator().manual_seed(k))]
        dy = torch.randint(-4, 5, (T, D), generator=g, device="cuda").to(gt)
        ids = ids.cuda().to(torch.int32 if k % 4 < 2 else torch.int64)
        _check(bl, ids, dy, V, tt, accumulate=k % 3 == 1, padding_id=int(ids[T // 2]) if k % 3 == 2 else None)
    assert bl.device_error() == (0, 0)


def test_one_token_and_all_tokens_in_chunks_of_32(bl):
    T, D = 9500, 4096
    dy = torch.randint(-4, 5, (T, D), generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(BF16)
    for ids, V in ((torch.full((T,), 2), 4), (torch.arange(T), T + 1), (torch.arange(T).flip(0), T + 1),
                   (torch.arange(T) // 2, T), (torch.arange(T) % 3, 5)):
        _check(bl, ids.cuda(), dy, V, F32)
        _check(bl, ids.cuda(), dy, V, F32, accumulate=True)


def test_chunks_of_8_by_the_workspace(bl):
    assert bl.workspace_bytes(bl.BL_OP_EMBEDDING_BACKWARD, 9400, 100, 4096) == _workspace(9400, 4096, 8)


@pytest.mark.parametrize("T", [4000, 4736, 4737, 6000, 20000])
@pytest.mark.parametrize("kind", ["up", "down", "two", "one", "steps", "back and forth"])
def test_lists_in_order(bl, T, kind):
    """Sorted lists and runs as they are, on both sides of where counting gives way to sorting."""
    i = torch.arange(T)
    ids = {"up": i, "down": i.flip(0), "two": i // (T // 2 + 1), "one": torch.cat([torch.full((T - 90,), 9), i[:90] % 9]),
           "steps": i // 37, "back and forth": torch.minimum(i, T - 1 - i)}[kind]
    V = int(ids.max()) + 2
    dy = torch.randint(-4, 5, (T, 48), generator=torch.Generator("cuda").manual_seed(T), device="cuda").to(BF16)
    for order in (ids, ids[torch.randperm(T, generator=torch.Generator().manual_seed(T))]):
        _check(bl, order.cuda(), dy, V, F32)
        _check(bl, order.cuda(), dy, V, BF16, accumulate=True)
    assert bl.device_error() == (0, 0)


@pytest.mark.parametrize("T,D", [(3000, 2048), (9500, 4096)])
def test_ids_written_just_ahead(bl, T, D):
    """Ids, rows of dy and the table's old rows are written and read by the calls just ahead, over and over and
    from one graph: the zeros are written beside the ordering, after all of that."""
    V = 5000
    pool = [torch.randint(0, V, (T,), generator=torch.Generator("cuda").manual_seed(k), device="cuda") for k in range(3)]
    dys = [torch.randint(-4, 5, (T, D), generator=torch.Generator("cuda").manual_seed(9 + k), device="cuda").to(BF16)
           for k in range(3)]
    refs = [torch.zeros(V, D, device="cuda").index_add_(0, i, d.float()) for i, d in zip(pool, dys)]
    ids, dy = torch.empty_like(pool[0]), torch.empty_like(dys[0])
    table, rows = torch.empty(V, D, device="cuda"), torch.empty(T, D, device="cuda")
    ws = torch.empty(bl.workspace_bytes(bl.BL_OP_EMBEDDING_BACKWARD, T, V, D), dtype=torch.uint8, device="cuda")

    def step(k):
        ids.copy_(pool[k])
        dy.copy_(dys[k])
        bl.embedding_backward(ids, dy, V, out=table, ws=ws)
        bl.embedding(ids, table, out=rows)  # reads the table just ahead of the next gradient's zeros
        return table.clone(), rows.clone()

    got = [step(k % 3) for k in range(9)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = [step(k) for k in range(3)]
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for k, (t, r) in list(enumerate(got)) + list(enumerate(captured)):
        assert torch.equal(t, refs[k % 3]) and torch.equal(r, refs[k % 3][pool[k % 3]])
