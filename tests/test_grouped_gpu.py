"""The grouped product, its weight gradient and the adapters on the GPU, against their
definitions in 64 bits.

Integer inputs are exact in every type up to the one rounding of the result, so they are compared
bit for bit; random inputs are held to the error bounds of grouped_ref.
"""
import itertools

import pytest

torch = pytest.importorskip("torch")

import grouped_ref as ref  # noqa: E402
import tiled_matrix_multiply_gb300 as tmm  # noqa: E402
from tiled_matrix_multiply_gb300 import _abi  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tiled_matrix_multiply_gb300 import build
    build.build()


def ints(gen, *shape, top=2):
    return torch.randint(-top, top + 1, shape, generator=gen).double()


def normals(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, dtype=torch.float64) * std


def offsets_of(sizes, first=0):
    out = [first]
    for s in sizes:
        out.append(out[-1] + s)
    return torch.tensor(out, dtype=torch.int32)


def checked(fn, *a, **k):
    out = fn(*a, **k)
    tmm.check_device()
    return out


def cuda(t, dtype=None):
    return None if t is None else t.to(dtype if dtype else t.dtype).cuda()


# sizes of the groups; K; N
FORWARD = [
    ([1], 1, 1), ([3], 16, 8), ([1, 0, 2], 64, 64), ([0, 0, 5, 0], 65, 129),
    ([17, 64, 65, 1], 128, 130), ([200, 30], 72, 257), ([63, 0, 129, 256, 257], 192, 256),
    ([300, 513], 130, 520), ([0, 0], 40, 24), ([1] * 40, 200, 136), ([5, 700, 0, 3], 333, 131),
    ([2, 1], 2100, 136), ([1500, 0, 900, 7], 96, 392),
]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("sizes,K,N", FORWARD)
def test_grouped_integers_are_exact(dtype, trans, sizes, K, N):
    gen = torch.Generator().manual_seed(K * 1000 + N)
    R = sum(sizes)
    x, w = ints(gen, R, K), ints(gen, len(sizes), K, N)
    off = offsets_of(sizes)
    wd = cuda(w.transpose(1, 2).contiguous(), dtype).transpose(1, 2) if trans else cuda(w, dtype)
    y = checked(tmm.gemm_grouped, cuda(x, dtype), wd, cuda(off))
    assert torch.equal(y.cpu(), ref.grouped(x, w, off).to(dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("sizes,K,N", FORWARD)
def test_grouped_rows_through_an_index(dtype, trans, sizes, K, N):
    gen = torch.Generator().manual_seed(K * 1000 + N + 1)
    R, T = sum(sizes), 37
    x, w = ints(gen, T, K), ints(gen, len(sizes), K, N)
    off = offsets_of(sizes)
    rows = torch.randint(-2, T + 2, (R,), generator=gen, dtype=torch.int32)   # some outside x
    wd = cuda(w.transpose(1, 2).contiguous(), dtype).transpose(1, 2) if trans else cuda(w, dtype)
    y = checked(tmm.gemm_grouped, cuda(x, dtype), wd, cuda(off), rows=cuda(rows))
    assert torch.equal(y.cpu(), ref.grouped(x, w, off, rows).to(dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("sizes,K,N,trans", [
    ([1, 0, 1], 4096, 512, False), ([70, 200, 31], 1000, 515, True), ([600, 900], 2048, 384, False),
    ([2] * 12, 777, 300, True)])
def test_grouped_random(dtype, sizes, K, N, trans):
    gen = torch.Generator().manual_seed(7)
    R = sum(sizes)
    x = normals(gen, R, K).to(dtype)
    w = normals(gen, len(sizes), K, N, std=K ** -0.5).to(dtype)
    off = offsets_of(sizes)
    wd = w.transpose(1, 2).contiguous().cuda().transpose(1, 2) if trans else w.cuda()
    y = checked(tmm.gemm_grouped, x.cuda(), wd, cuda(off))
    want = ref.grouped(x, w, off)
    ref.assert_within(y, want, ref.grouped(x.abs(), w.abs(), off), K)
    if dtype == torch.float32:
        assert (y.double().cpu() - want).norm() <= 1e-6 * want.norm()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("off", [
    [3, 7, 7, 20], [0, 0, 0, 0], [30, 30, 30, 30], [5, 2, 25, 9], [-4, 10, 99, 12],
    [12, 9, 9, 40], [-(2 ** 31), 2 ** 31 - 1, 0, 5]])
def test_grouped_any_offsets_and_rows_of_no_group(dtype, off):
    gen = torch.Generator().manual_seed(5)
    x, w = ints(gen, 30, 80), ints(gen, 3, 80, 70)
    o = torch.tensor(off, dtype=torch.int64).to(torch.int32)
    y = torch.full((30, 70), float("nan"), dtype=dtype, device="cuda")
    checked(tmm.gemm_grouped, cuda(x, dtype), cuda(w, dtype), cuda(o), y=y)
    assert torch.equal(y.cpu(), ref.grouped(x, w, o.tolist()).to(dtype))
    dy = ints(gen, 30, 70)
    dw = checked(tmm.gemm_grouped_wgrad, cuda(x, dtype), cuda(dy, dtype), cuda(o))
    assert torch.equal(dw.cpu(), ref.wgrad(x, dy, o.tolist()).to(dtype))


def window(t, dtype, pad, offset):
    """t on the GPU inside a wider buffer of NaN: rows `pad` values apart more, from `offset`."""
    shape = list(t.shape)
    buf = torch.full((shape[0] * (shape[1] if len(shape) == 3 else 1) * (shape[-1] + pad) + offset
                      + 64,), float("nan"), dtype=dtype, device="cuda")
    ld = shape[-1] + pad
    stride = [shape[1] * ld, ld, 1] if len(shape) == 3 else [ld, 1]
    view = torch.as_strided(buf, shape, stride, offset)
    view.copy_(t.to(dtype))
    return view, buf


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 8), (3, 0), (0, 1), (5, 7), (16, 4)])
def test_strides_and_alignment(dtype, pad, offset):
    gen = torch.Generator().manual_seed(pad * 10 + offset)
    sizes, K, N = [40, 0, 33], 72, 136
    R = sum(sizes)
    x, w, dy = ints(gen, R, K), ints(gen, 3, K, N), ints(gen, R, N)
    off = offsets_of(sizes)
    xd, _ = window(x, dtype, pad, offset)
    wd, _ = window(w, dtype, pad, offset)
    dyd, _ = window(dy, dtype, pad, offset)
    y, ybuf = window(torch.zeros(R, N), dtype, pad, offset)
    checked(tmm.gemm_grouped, xd, wd, cuda(off), y=y)
    assert torch.equal(y.cpu(), ref.grouped(x, w, off).to(dtype))
    assert int(torch.isnan(ybuf).sum()) == ybuf.numel() - R * N       # nothing else written
    dw, dwbuf = window(torch.zeros(3, K, N), dtype, pad, offset)
    checked(tmm.gemm_grouped_wgrad, xd, dyd, cuda(off), dw=dw)
    assert torch.equal(dw.cpu(), ref.wgrad(x, dy, off).to(dtype))
    assert int(torch.isnan(dwbuf).sum()) == dwbuf.numel() - 3 * K * N


WGRAD = [([1], 1, 1), ([16], 16, 16), ([5, 0, 64, 65], 64, 64), ([130, 0, 3], 65, 130),
         ([200, 17, 128], 200, 257), ([0, 0], 30, 40), ([1000, 24], 130, 100), ([1] * 33, 96, 50)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("by_index", [False, True])
@pytest.mark.parametrize("sizes,K,N", WGRAD)
def test_wgrad_integers_are_exact(dtype, by_index, sizes, K, N):
    gen = torch.Generator().manual_seed(K * 1000 + N)
    R, T = sum(sizes), 29
    x = ints(gen, T if by_index else R, K)
    rows = torch.randint(-2, T + 2, (R,), generator=gen, dtype=torch.int32) if by_index else None
    dy, off = ints(gen, R, N), offsets_of(sizes)
    dw = checked(tmm.gemm_grouped_wgrad, cuda(x, dtype), cuda(dy, dtype), cuda(off),
                 rows=cuda(rows))
    assert torch.equal(dw.cpu(), ref.wgrad(x, dy, off, rows).to(dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("sizes,K,N", [([900, 31, 1500], 300, 257), ([64] * 5, 128, 96)])
def test_wgrad_random(dtype, sizes, K, N):
    gen = torch.Generator().manual_seed(11)
    R = sum(sizes)
    x, dy = normals(gen, R, K).to(dtype), normals(gen, R, N).to(dtype)
    off = offsets_of(sizes)
    dw = checked(tmm.gemm_grouped_wgrad, x.cuda(), dy.cuda(), cuda(off))
    want = ref.wgrad(x, dy, off)
    ref.assert_within(dw, want, ref.wgrad(x.abs(), dy.abs(), off), max(sizes))
    if dtype == torch.float32:
        assert (dw.double().cpu() - want).norm() <= 1e-6 * want.norm()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_of_other_groups_do_not_enter(dtype, bad):
    # Rows of one group, and rows of none, hold NaN or infinities; the others' results are exact.
    gen = torch.Generator().manual_seed(3)
    sizes, K, N = [10, 50, 37], 100, 90
    off = offsets_of(sizes, first=4)
    R = 4 + sum(sizes) + 6
    x, w, dy = ints(gen, R, K), ints(gen, 3, K, N), ints(gen, R, N)
    y_ref, dw_ref = ref.grouped(x, w, off).to(dtype), ref.wgrad(x, dy, off).to(dtype)
    xb, dyb, wb = x.clone(), dy.clone(), w.clone()
    for t in (xb, dyb):
        t[:4] = bad
        t[14:64] = bad
        t[4 + sum(sizes):] = bad
    wb[1] = bad
    y = checked(tmm.gemm_grouped, cuda(xb, dtype), cuda(wb, dtype), cuda(off)).cpu()
    keep = [i for i in range(R) if not 14 <= i < 64]
    assert torch.equal(y[keep], y_ref[keep])
    assert not torch.isfinite(y[14:64]).any()
    dw = checked(tmm.gemm_grouped_wgrad, cuda(xb, dtype), cuda(dyb, dtype), cuda(off)).cpu()
    assert torch.equal(dw[0], dw_ref[0]) and torch.equal(dw[2], dw_ref[2])
    assert not torch.isfinite(dw[1]).any()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_shared_matrix_and_wide_range(dtype):
    gen = torch.Generator().manual_seed(4)
    sizes = [20, 0, 90]
    x, w = ints(gen, 110, 64), ints(gen, 1, 64, 72)
    off = offsets_of(sizes)
    y = checked(tmm.gemm_grouped, cuda(x, dtype), cuda(w, dtype).expand(3, 64, 72), cuda(off))
    assert torch.equal(y.cpu(), ref.grouped(x, w.expand(3, 64, 72), off).to(dtype))
    # Powers of two over the type's range, one term per result: exact.
    big = {torch.float16: 14, torch.bfloat16: 120, torch.float32: 126}[dtype]
    e = torch.randint(-big // 2, big // 2, (110, 64), generator=gen).double()
    x = torch.zeros(110, 64, dtype=torch.float64)
    x[torch.arange(110), torch.arange(110) % 64] = 1.0
    w = (2.0 ** e[:64])[None, :, :].contiguous()
    y = checked(tmm.gemm_grouped, cuda(x, dtype), cuda(w, dtype).expand(3, 64, 64), cuda(off))
    assert torch.equal(y.cpu(), (x @ w[0]).to(dtype))


def test_single_precision_keeps_all_bits():
    # One term per result: x times a power of two comes back with all 24 bits.
    gen = torch.Generator().manual_seed(6)
    x = torch.randn(50, 64, generator=gen)
    x[0, :4] = torch.tensor([3.4028234e38, -3.4e38, 1e-30, 1.1754944e-38])
    w = torch.eye(64)[None]
    y = checked(tmm.gemm_grouped, x.cuda(), w.cuda(), offsets_of([50]).cuda())
    ok = x.abs() >= 2.0 ** -102
    assert torch.equal(y.cpu()[ok], x[ok])


LORA = [([1], 1, 64, 64, 8), ([0, 1, 0], 1, 200, 130, 16), ([1, 1, 0, 1], 5, 128, 257, 4),
        ([3, 0, 40, 21], 70, 72, 136, 20), ([90, 0, 100], 200, 130, 300, 64),
        ([0, 0], 9, 64, 48, 8), ([200, 157], 357, 256, 520, 100), ([1] * 30, 33, 96, 140, 130),
        ([100, 0, 56, 300], 500, 128, 260, 33), ([9] * 40, 400, 64, 136, 8),
        ([2, 5], 8, 2200, 136, 24)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("trans", [(0, 0, 0), (1, 1, 1), (0, 1, 0)])
@pytest.mark.parametrize("sizes,T,K,N,r", LORA)
def test_lora_integers_are_exact(dtype, trans, sizes, T, K, N, r):
    gen = torch.Generator().manual_seed(K * 1000 + N + r)
    L = len(sizes)
    x, w = ints(gen, T, K, top=1), ints(gen, K, N, top=1)
    a, b = ints(gen, L, K, r, top=1), ints(gen, L, r, N, top=1)
    a *= torch.rand(L, K, 1, generator=gen) < 0.2
    scale = torch.tensor([2.0 ** (i % 3 - 1) for i in range(L)])
    off = offsets_of(sizes)
    order = torch.randperm(T, generator=gen).to(torch.int32)

    def put(t, tr):
        return cuda(t.transpose(-1, -2).contiguous(), dtype).transpose(-1, -2) if tr \
            else cuda(t, dtype)
    args = (put(w, trans[0]), put(a, trans[1]), put(b, trans[2]), scale.cuda(), cuda(off))
    want = ref.lora(x, w, a, b, scale, off, order, low=None if dtype == torch.float32 else dtype)
    y = checked(tmm.gemm_lora, cuda(x, dtype), *args, rows=cuda(order))
    assert torch.equal(y.cpu(), want.to(dtype))
    y = checked(tmm.gemm_lora, cuda(x, dtype), *args)
    want = ref.lora(x, w, a, b, scale, off, low=None if dtype == torch.float32 else dtype)
    assert torch.equal(y.cpu(), want.to(dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("T,N", [(4096, 4096), (4031, 4096), (3000, 4090), (2300, 4096),
                                 (1000, 8192)])
def test_lora_many_tiles(dtype, T, N):
    # Many tiles of rows, whole ones and ends of every kind.
    gen = torch.Generator().manual_seed(T)
    K, r, sizes = 40, 8, [T // 3, 0, T // 2 + 5]
    x, w = ints(gen, T, K, top=1), ints(gen, K, N, top=1)
    a, b = ints(gen, 3, K, r, top=1), ints(gen, 3, r, N, top=1)
    scale, off = torch.ones(3), offsets_of(sizes)
    order = torch.randperm(T, generator=gen).to(torch.int32)
    y = checked(tmm.gemm_lora, cuda(x, dtype), cuda(w, dtype), cuda(a, dtype), cuda(b, dtype),
                scale.cuda(), cuda(off), rows=cuda(order))
    assert torch.equal(y.cpu(), ref.lora(x, w, a, b, scale, off, order).to(dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("sizes,T,K,N,r", [([1] * 12, 14, 1024, 300, 16),
                                           ([150, 0, 260], 430, 600, 515, 48)])
def test_lora_random(dtype, sizes, T, K, N, r):
    gen = torch.Generator().manual_seed(13)
    L = len(sizes)
    x, w = normals(gen, T, K).to(dtype), normals(gen, K, N, std=K ** -0.5).to(dtype)
    a = normals(gen, L, K, r, std=K ** -0.5).to(dtype)
    b = normals(gen, L, r, N, std=r ** -0.5).to(dtype)
    scale = torch.rand(L, generator=gen) + 0.5
    off = offsets_of(sizes)
    order = torch.randperm(T, generator=gen).to(torch.int32)
    y = checked(tmm.gemm_lora, x.cuda(), w.cuda(), a.cuda(), b.cuda(), scale.cuda(), cuda(off),
                rows=cuda(order))
    want = ref.lora(x, w, a, b, scale, off, order)
    mag = ref.lora(x.abs(), w.abs(), a.abs(), b.abs(), scale, off, order)
    # u is rounded to the type (float32: exactly its three parts) before the product with b.
    size = ref.lora(x.abs(), torch.zeros_like(w), a.abs(), b.abs(), scale, off, order)
    extra = ref.HALF_STEP[dtype] * size + ref.sum_error(dtype, K) * size
    ref.assert_within(y, want, mag, K + r * L, extra=extra)
    if dtype == torch.float32:
        assert (y.double().cpu() - want).norm() <= 1e-6 * want.norm()


@pytest.mark.parametrize("tokens,k,groups,dtype", [
    (1, 1, 1, torch.int32), (1, 4, 8, torch.int64), (37, 2, 8, torch.int32), (33, 1, 512, torch.int64),
    (1000, 3, 5, torch.int32), (8192, 1, 64, torch.int32), (8193, 1, 64, torch.int32),
    (16384, 8, 256, torch.int64), (5000, 7, 512, torch.int32), (0, 2, 4, torch.int32),
    (100000, 1, 1, torch.int32)])
def test_group_rows(tokens, k, groups, dtype):
    gen = torch.Generator().manual_seed(tokens + groups)
    index = torch.randint(-1, groups + 1, (tokens, k), generator=gen, dtype=dtype)
    plan = checked(tmm.group_rows, index.cuda(), groups)
    flat = index.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < groups), flat, groups)
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=groups + 1)[:groups]
    assert plan.offsets.cpu().tolist() == [0] + counts.cumsum(0).tolist()
    assert torch.equal(plan.order.cpu().long(), order)
    assert torch.equal(plan.rows.cpu().long(), order // k)
    inverse = torch.empty_like(order)
    inverse[order] = torch.arange(order.numel())
    assert torch.equal(plan.position.cpu().long(), inverse)


def test_group_rows_extreme_numbers():
    big = torch.tensor([2 ** 40, 3, -2 ** 50, 2 ** 32 + 1, 0, 3], dtype=torch.int64)
    plan = checked(tmm.group_rows, big.cuda(), 4)
    assert plan.offsets.cpu().tolist() == [0, 1, 1, 1, 3]
    assert plan.order.cpu().tolist() == [4, 1, 5, 0, 2, 3]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_repeats_streams_and_graphs_give_the_same_bits(dtype):
    gen = torch.Generator().manual_seed(21)
    sizes, K, N = [3, 0, 80, 9], 500, 260
    x = normals(gen, 92, K).to(dtype).cuda()
    w = normals(gen, 4, K, N).to(dtype).cuda()
    off = offsets_of(sizes).cuda()
    y0 = tmm.gemm_grouped(x, w, off)
    dw0 = tmm.gemm_grouped_wgrad(x, y0, off)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y1 = tmm.gemm_grouped(x, w, off)
        dw1 = tmm.gemm_grouped_wgrad(x, y1, off)
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and torch.equal(dw0, dw1)
    graph = torch.cuda.CUDAGraph()
    y2, dw2 = torch.zeros_like(y0), torch.zeros_like(dw0)
    with torch.cuda.graph(graph):
        tmm.gemm_grouped(x, w, off, y=y2)
        tmm.gemm_grouped_wgrad(x, y2, off, dw=dw2)
    # Other groups on the replay: sizes are read on the GPU.
    other = offsets_of([50, 2, 0, 40])
    off.copy_(other)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y2, tmm.gemm_grouped(x, w, off))
    assert torch.equal(dw2, tmm.gemm_grouped_wgrad(x, y2, off))
    tmm.check_device()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_outputs_workspaces_and_streams_of_the_caller(dtype):
    # The same bits whether the call allocates (and is marshalled in one piece) or is given its
    # output, its workspace or a stream.
    gen = torch.Generator().manual_seed(23)
    sizes, K, N, r = [30, 0, 400], 200, 300, 12
    R = sum(sizes)
    x = normals(gen, 50, K).to(dtype).cuda()
    w, a, b = (normals(gen, 3, *s).to(dtype).cuda() for s in ((K, N), (K, r), (r, N)))
    rows = torch.randint(0, 50, (R,), generator=gen, dtype=torch.int32).cuda()
    off, dy = offsets_of(sizes).cuda(), normals(gen, R, N).to(dtype).cuda()
    scale, side = torch.ones(3).cuda(), torch.cuda.Stream()
    xs = x[rows.long()].contiguous()
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    calls = [(tmm.gemm_grouped, (x, w, off), dict(rows=rows), "y"),
             (tmm.gemm_grouped_wgrad, (x, dy, off), dict(rows=rows), "dw"),
             (tmm.gemm_lora, (xs, w[0], a, b, scale, off), {}, "y")]
    for fn, args, more, name in calls:
        want = checked(fn, *args, **more)
        out = torch.zeros_like(want)
        got = checked(fn, *args, **more, **{name: out}, workspace=ws)
        assert got is out and torch.equal(out, want)
        side.wait_stream(torch.cuda.current_stream())
        got = fn(*args, **more, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    index = torch.randint(0, 3, (300, 2), generator=gen, dtype=torch.int32).cuda()
    want = checked(tmm.group_rows, index, 3)
    for g, h in zip(want, tmm.group_rows(index, 3, stream=side)):
        torch.cuda.synchronize()
        assert torch.equal(g, h)


def test_refusals_with_tensors_on_the_gpu():
    bf, i = torch.bfloat16, torch.int32
    x, w = torch.zeros(4, 8, dtype=bf, device="cuda"), torch.zeros(2, 8, 8, dtype=bf, device="cuda")
    off = torch.zeros(3, dtype=i, device="cuda")
    for bad in (dict(x=x.float()), dict(w=w[:, :4]), dict(w=w.half()), dict(w=w[0]),
                dict(offsets=off[:2]), dict(offsets=off.long()), dict(offsets=off.cpu()),
                dict(rows=off.long()), dict(x=x[:, ::2]), dict(x=x.t())):
        args = dict(x=x, w=w, offsets=off)
        args.update(bad)
        with pytest.raises((TypeError, ValueError)):
            tmm.gemm_grouped(**args)
    with pytest.raises(_abi.TmmError) as e:
        tmm.gemm_grouped(x, w, off, y=x)
    assert e.value.status == _abi.TMM_ERR_ALIAS
    with pytest.raises(ValueError):
        tmm.gemm_grouped_wgrad(x, x[:3], off)
    with pytest.raises(ValueError):
        tmm.group_rows(torch.zeros(4, 2, dtype=i, device="cuda"), 513)
    with pytest.raises(TypeError):
        tmm.gemm_lora(x, w[0], w, w, torch.ones(2, dtype=bf, device="cuda"), off)


def test_a_wait_that_runs_out_is_reported():
    # One block or pair, clusters that share a sum, splitting blocks; adapters, and the gradient.
    lib = _abi.load()
    K = 2048
    few, many = offsets_of([2, 3]).cuda(), offsets_of([1400, 1600]).cuda()
    for dtype, off, rows in itertools.product(TYPES, (few, many), (5, 3000)):
        if rows != int(off[-1]):
            continue
        x = torch.ones(rows, K, dtype=dtype, device="cuda")
        w = torch.ones(2, K, 256, dtype=dtype, device="cuda")
        dy = torch.ones(rows, 256, dtype=dtype, device="cuda")
        a, b = torch.zeros_like(w[:, :, :8]), torch.zeros_like(w[:, :8])
        one = torch.ones(2, device="cuda")
        calls = [lambda: tmm.gemm_grouped(x, w, off), lambda: tmm.gemm_grouped_wgrad(x, dy, off),
                 lambda: tmm.gemm_lora(x, w[0], a.contiguous(), b.contiguous(), one, off)]
        wants = [call() for call in calls]
        tmm.check_device()
        for call, want in zip(calls, wants):
            lib.tmm_testing_set_wait_hooks(0, 2_000_000)
            try:
                call()
                with pytest.raises(tmm.TmmError) as e:
                    tmm.check_device()
                assert e.value.status == _abi.TMM_ERR_DEVICE_TIMEOUT
            finally:
                lib.tmm_testing_set_wait_hooks(-1, 0)
            assert torch.equal(checked(call), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_gradients_of_the_layer(dtype):
    # x -> experts (through a plan) -> loss = sum(c * y): dx and dw by the operators, against
    # central differences of the operators' own forward pass in single precision.
    gen = torch.Generator().manual_seed(31)
    T, k, G, K, N = 40, 2, 4, 48, 56
    experts = torch.rand(T, G, generator=gen).topk(k, dim=1).indices.cuda()
    plan = tmm.group_rows(experts, G)
    x, w = normals(gen, T, K).to(dtype).cuda(), normals(gen, G, K, N, std=0.2).to(dtype).cuda()
    c = normals(gen, T * k, N).to(dtype).cuda()
    dw = tmm.gemm_grouped_wgrad(x, c, plan.offsets, rows=plan.rows).double()
    dxs = tmm.gemm_grouped(c, w.transpose(1, 2), plan.offsets)
    dx = dxs[plan.position.view(T, k).long()].double().sum(1)

    def loss(xv, wv):
        y = tmm.gemm_grouped(xv.float(), wv.float(), plan.offsets, rows=plan.rows)
        return float((y.double() * c.double()).sum())
    h = 0.25
    for (t, i), (g, a, b) in itertools.product([(0, 0), (17, 5), (39, 47)],
                                               [(0, 0, 0), (3, 47, 55), (1, 20, 7)]):
        e = torch.zeros_like(x)
        e[t, i] = h
        fd = (loss(x.float() + e.float(), w) - loss(x.float() - e.float(), w)) / (2 * h)
        # Rounding of the loss (2^-21 of its terms) over 2h, and of k rounded rows summed.
        tol = 1e-3 + 2 * ref.HALF_STEP[dtype] * float(dxs.double().abs().max()) * k
        assert abs(fd - float(dx[t, i])) <= tol
        e = torch.zeros_like(w)
        e[g, a, b] = h
        fd = (loss(x, w.float() + e.float()) - loss(x, w.float() - e.float())) / (2 * h)
        assert abs(fd - float(dw[g, a, b])) <= 1e-3 + 2 * ref.HALF_STEP[dtype] * float(
            dw[g, a, b].abs())
    tmm.check_device()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_gradients_of_the_adapters(dtype):
    # dx = gemm_lora of the transposed operands; da and db from the grouped products.
    gen = torch.Generator().manual_seed(33)
    sizes, T, K, N, r = [20, 0, 33], 60, 72, 136, 16
    L = len(sizes)
    x, w = ints(gen, T, K, top=1), ints(gen, K, N, top=1)
    a, b = ints(gen, L, K, r, top=1), ints(gen, L, r, N, top=1)
    a *= torch.rand(L, K, 1, generator=gen) < 0.1
    b *= torch.rand(L, 1, N, generator=gen) < 0.1
    dy, scale, off = ints(gen, T, N, top=1), torch.ones(L), offsets_of(sizes)
    order = torch.randperm(T, generator=gen).to(torch.int32)
    xd, wd, ad, bd, dyd = (cuda(t, dtype) for t in (x, w, a, b, dy))
    offd, ordd = cuda(off), cuda(order)
    dx = checked(tmm.gemm_lora, dyd, wd.t(), bd.transpose(1, 2), ad.transpose(1, 2),
                 scale.cuda(), offd, rows=ordd)
    low = None if dtype == torch.float32 else dtype
    want = ref.lora(dy, w.T, b.transpose(1, 2), a.transpose(1, 2), scale, off, order, low=low)
    assert torch.equal(dx.cpu(), want.to(dtype))
    du = tmm.gemm_grouped(dyd, bd.transpose(1, 2), offd, rows=ordd)          # (T, r), group order
    da = checked(tmm.gemm_grouped_wgrad, xd, du, offd, rows=ordd)
    xs, dys = x[order.long()], dy[order.long()]
    du_ref = ref.grouped(dys, b.transpose(1, 2), off).to(dtype).double()
    assert torch.equal(da.cpu(), ref.wgrad(xs, du_ref, off).to(dtype))
    u = tmm.gemm_grouped(xd, ad, offd, rows=ordd)
    dys_d = dyd[ordd.long()].contiguous()
    db = checked(tmm.gemm_grouped_wgrad, u, dys_d, offd)
    u_ref = ref.grouped(xs, a, off).to(dtype).double()
    assert torch.equal(db.cpu(), ref.wgrad(u_ref, dys, off).to(dtype))


def test_the_expert_layer_of_the_example():
    # The layer's outputs and gradients in single precision against the same formulas in 64 bits.
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                    "examples"))
    import experts_and_adapters as ex
    gen = torch.Generator().manual_seed(41)
    T, D, H, E = 70, 96, 130, 5
    x, dy = normals(gen, T, D).float(), normals(gen, T, D).float()
    w1, w2 = normals(gen, E, D, H, std=D ** -0.5).float(), normals(gen, E, H, D, std=H ** -0.5).float()
    logits = normals(gen, T, E).float()
    y, saved = ex.experts_forward(x.cuda(), w1.cuda(), w2.cuda(), logits.cuda())
    grads = ex.experts_backward(dy.cuda(), saved)
    tmm.check_device()
    leaves = [t.double().requires_grad_() for t in (x, w1, w2, logits)]
    xd, w1d, w2d, ld = leaves
    top, experts = ld.topk(2, dim=1)
    p = torch.softmax(top, dim=1)
    h = torch.einsum("td,tkdh->tkh", xd, w1d[experts])
    z = torch.einsum("tkh,tkhd->tkd", torch.relu(h).square(), w2d[experts])
    want = (z * p[..., None]).sum(1)
    want.backward(dy.double())
    dlog = ld.grad.gather(1, experts)
    # Each step is within 1e-6 of its own norm (two products and a sum in a row, and the square's
    # factor of two): 1e-5 holds them all.
    for got, ref64 in zip((y, *grads), (want.detach(), xd.grad, w1d.grad, w2d.grad, dlog)):
        assert (got.double().cpu() - ref64).norm() <= 1e-5 * ref64.norm()


def test_the_example_runs():
    import experts_and_adapters as ex
    out = ex.main(tokens=200, model=128, inner=256, experts=4)
    assert all(bool(torch.isfinite(t.float()).all()) for t in out.values())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_empty_sizes(dtype):
    def z(*shape):
        return torch.zeros(*shape, dtype=dtype, device="cuda")
    off, none = offsets_of([2, 1]).cuda(), offsets_of([0, 0]).cuda()
    ones = torch.ones(2, device="cuda")
    # Sums of nothing are zeros, results of no rows or columns are empty.
    y = torch.ones(3, 8, dtype=dtype, device="cuda")
    assert not checked(tmm.gemm_grouped, z(3, 0), z(2, 0, 8), off, y=y).any()
    assert checked(tmm.gemm_grouped, z(0, 16), z(2, 16, 8), none).shape == (0, 8)
    assert checked(tmm.gemm_grouped, z(3, 16), z(2, 16, 0), off).shape == (3, 0)
    dw = torch.ones(2, 16, 8, dtype=dtype, device="cuda")
    assert not checked(tmm.gemm_grouped_wgrad, z(0, 16), z(0, 8), none, dw=dw).any()
    assert checked(tmm.gemm_grouped_wgrad, z(3, 16), z(3, 0), off).shape == (2, 16, 0)
    rows = torch.tensor([0, 5, -1], dtype=torch.int32, device="cuda")
    y = torch.ones(3, 8, dtype=dtype, device="cuda")
    assert not checked(tmm.gemm_grouped, z(0, 16), z(2, 16, 8) + 1, off, rows=rows, y=y).any()
    assert checked(tmm.gemm_lora, z(0, 16), z(16, 8), z(2, 16, 4), z(2, 4, 8), ones,
                   none).shape == (0, 8)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("T", [20, 500, 700])
def test_lora_shared_adapter_and_unaligned_operands(dtype, T):
    gen = torch.Generator().manual_seed(T)
    K, N, r, sizes = 72, 136, 8, [T // 3, 0, T // 3]
    x, w = ints(gen, T, K, top=1), ints(gen, K, N, top=1)
    a, b = ints(gen, 1, K, r, top=1), ints(gen, 1, r, N, top=1)
    scale, off = torch.tensor([1.0, 2.0, -1.0]), offsets_of(sizes, first=1)
    a3, b3 = a.expand(3, K, r), b.expand(3, r, N)
    want = ref.lora(x, w, a3, b3, scale, off).to(dtype)
    y = checked(tmm.gemm_lora, cuda(x, dtype), cuda(w, dtype), cuda(a, dtype).expand(3, K, r),
                cuda(b, dtype).expand(3, r, N), scale.cuda(), cuda(off))
    assert torch.equal(y.cpu(), want)
    put = [window(t, dtype, 3, 1)[0] for t in (x, w, a3.contiguous(), b3.contiguous())]
    out, buf = window(torch.zeros(T, N), dtype, 5, 1)
    checked(tmm.gemm_lora, *put, scale.cuda(), cuda(off), y=out)
    assert torch.equal(out.cpu(), want)
    assert int(torch.isnan(buf).sum()) == buf.numel() - T * N


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("sizes", [[10, 0, 20], [200, 0, 260], [300, 0, 260]])
def test_lora_rows_do_not_meet_other_adapters(dtype, bad, sizes):
    # One adapter's matrices, and the rows of it, hold NaN or infinities.
    gen = torch.Generator().manual_seed(9)
    T, K, N, r = sum(sizes) + 7, 64, 264, 8
    x, w = ints(gen, T, K, top=1), ints(gen, K, N, top=1)
    a, b = ints(gen, 3, K, r, top=1), ints(gen, 3, r, N, top=1)
    off, scale = offsets_of(sizes), torch.ones(3)
    want = ref.lora(x, w, a, b, scale, off).to(dtype)
    x[:sizes[0]] = bad
    a[0], b[0] = bad, bad
    a[1], b[1] = bad, bad                 # an adapter without rows
    y = checked(tmm.gemm_lora, cuda(x, dtype), cuda(w, dtype), cuda(a, dtype), cuda(b, dtype),
                scale.cuda(), cuda(off)).cpu()
    assert torch.equal(y[sizes[0]:], want[sizes[0]:])
    assert not torch.isfinite(y[:sizes[0]]).any()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("r", [8, 40, 130])
@pytest.mark.parametrize("K", [24, 200])
@pytest.mark.parametrize("sizes,first,T", [([9] * 60, 0, 600), ([1] * 200, 7, 530),
                                           ([1, 31, 32, 33, 64, 0, 95, 300], 5, 620),
                                           ([0, 0, 700], 0, 700), ([255, 257, 128], 33, 673)])
def test_lora_parts_of_tiles(dtype, sizes, first, T, K, r):
    # Adapters of any size beside one another in a tile, between rows of none.
    gen = torch.Generator().manual_seed(T + K + r)
    L, N = len(sizes), 300
    x, w = ints(gen, T, K, top=1), ints(gen, K, N, top=1)
    a, b = ints(gen, L, K, r, top=1), ints(gen, L, r, N, top=1)
    a *= torch.rand(L, K, 1, generator=gen) < 0.2
    scale = torch.tensor([2.0 ** (i % 3 - 1) for i in range(L)])
    off = offsets_of(sizes, first=first)
    order = torch.randperm(T, generator=gen).to(torch.int32)
    y = checked(tmm.gemm_lora, cuda(x, dtype), cuda(w, dtype), cuda(a, dtype), cuda(b, dtype),
                scale.cuda(), cuda(off), rows=cuda(order))
    low = None if dtype == torch.float32 else dtype
    want = ref.lora(x, w, a, b, scale, off, order, low=low)
    assert torch.equal(y.cpu(), want.to(dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("T", [20, 600])
def test_offsets_past_32_bits(dtype, T):
    # Rows, matrices and results that lie more than 2^31 elements apart.
    gen = torch.Generator().manual_seed(T)
    K, N, r, sizes = 72, 136, 8, [T // 4, 0, T // 2]
    ld, far = (2 ** 31 + 2 ** 29) // T // 8 * 8, 2 ** 30 + 2 ** 28

    def rows(n):
        return torch.empty(T * ld, dtype=dtype, device="cuda").as_strided((T, n), (ld, 1))

    def stack(m, n):
        return torch.empty(2 * far + m * n, dtype=dtype, device="cuda").as_strided(
            (3, m, n), (far, n, 1))
    x, dy = ints(gen, T, K, top=1), ints(gen, T, N, top=1)
    w, a, b = ints(gen, 3, K, N, top=1), ints(gen, 3, K, r, top=1), ints(gen, 3, r, N, top=1)
    off, scale = offsets_of(sizes), torch.ones(3)
    offd = off.cuda()
    xd, wd, yd = rows(K), stack(K, N), rows(N)
    xd.copy_(x.to(dtype))
    wd.copy_(w.to(dtype))
    checked(tmm.gemm_grouped, xd, wd, offd, y=yd)
    assert torch.equal(yd.cpu(), ref.grouped(x, w, off).to(dtype))
    checked(tmm.gemm_lora, xd, wd[2], cuda(a, dtype), cuda(b, dtype), scale.cuda(), offd, y=yd)
    assert torch.equal(yd.cpu(), ref.lora(x, w[2], a, b, scale, off).to(dtype))
    yd.copy_(dy.to(dtype))
    checked(tmm.gemm_grouped_wgrad, xd, yd, offd, dw=wd)
    assert torch.equal(wd.cpu(), ref.wgrad(x, dy, off).to(dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("sizes,K,N", [([70], 1100, 136), ([40, 0, 90], 2048, 264),
                                       ([300, 1, 300], 1032, 520), ([31, 33], 1200, 130)])
def test_rows_by_number_of_long_sums(dtype, sizes, K, N):
    # Rows fetched by number and rows gathered first, tiles of every width.
    gen = torch.Generator().manual_seed(K)
    R, X = sum(sizes), 50
    x, w = ints(gen, X, K, top=1), ints(gen, len(sizes), K, N, top=1)
    x *= torch.rand(X, K, generator=gen) < 0.1
    rows = torch.randint(-1, X + 2, (R,), generator=gen).to(torch.int32)
    off = offsets_of(sizes)
    y = checked(tmm.gemm_grouped, cuda(x, dtype), cuda(w, dtype), cuda(off), rows=cuda(rows))
    assert torch.equal(y.cpu(), ref.grouped(x, w, off, rows).to(dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("sizes", [[100], [300], [0, 500, 77], [129, 130]])
def test_wgrad_of_rows_by_number_with_few_columns(dtype, sizes):
    gen = torch.Generator().manual_seed(sum(sizes))
    R, X, K, N = sum(sizes), 60, 200, 72
    x, dy = ints(gen, X, K, top=1), ints(gen, R, N, top=1)
    x *= torch.rand(X, K, generator=gen) < 0.2
    rows = torch.randint(-1, X + 2, (R,), generator=gen).to(torch.int32)
    off = offsets_of(sizes)
    dw = checked(tmm.gemm_grouped_wgrad, cuda(x, dtype), cuda(dy, dtype), cuda(off),
                 rows=cuda(rows))
    assert torch.equal(dw.cpu(), ref.wgrad(x, dy, off, rows).to(dtype))
