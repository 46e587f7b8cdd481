"""int8 rows on the GPU against the plain 64-bit definitions: the codes and
scales exactly (ties, values next to a tie, tiny and non-finite rows), the
products within the roundings of the definition, over sizes that end inside
every tile, strides, unaligned rows, types, streams and graphs."""
import numpy as np
import pytest

import row_oracle

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from top_search_resident_amd import (ResidentTopKError, linear_int8, linear_int8_workspace,  # noqa: E402
                                     matmul_int8, quantize_rows_int8)

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def tolerance(y, prod, out_type, bias):
    """Three fp32 roundings of the product (the sum's conversion and two scales),
    one of the sum with the bias, one to the output type (half a step of the
    value already off by the others, and of the smallest step where it is
    subnormal)."""
    t = 3.01 * 2.0 ** -24 * prod + (1.01 * 2.0 ** -24 * np.abs(y) if bias else 0.0)
    info = torch.finfo(out_type)
    if out_type != torch.float32:
        t = t + info.eps / 2 * (np.abs(y) + t)
    return t + info.tiny * info.eps / 2


def check(out, a, sa, b, sb, bias=None):
    y, prod = row_oracle.product(a, sa, b, sb, bias)
    got = out.double().cpu().numpy()
    assert got.shape == y.shape
    assert (np.isnan(got) == np.isnan(y)).all()
    fine = ~np.isnan(y)
    off = np.abs(got - y)[fine] - tolerance(y, prod, out.dtype, bias is not None)[fine]
    assert off.size == 0 or off.max() <= 0, off.max()


def int8_rows(n, k, g, pitch=None, offset=0):
    """Random codes over the whole int8 range as a view with the given row stride and start."""
    pitch = k if pitch is None else pitch
    store = torch.randint(-128, 128, (n * pitch + offset,), dtype=torch.int8, generator=g).cuda()
    return store[offset:].as_strided((n, k), (pitch, 1), offset)


def scales(n, g):
    return (torch.rand(n, generator=g) + 0.01).cuda()


def host(t):
    return t.cpu().numpy()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("m,k", [(1, 1), (3, 7), (2, 16), (5, 255), (4, 1024), (2, 4097), (1, 20003), (2, 65536)])
def test_quantize_matches_the_definition(dtype, m, k):
    g = torch.Generator().manual_seed(m * 1000 + k)
    x = (torch.randn(m, k, generator=g) * torch.logspace(-6, 3, m)[:, None]).to(TYPES[dtype])
    q, s = quantize_rows_int8(x.cuda())
    eq, es = row_oracle.quantize_rows(x.double().numpy())
    assert q.stride(0) % 16 == 0 or m == 1
    assert (host(s).astype(np.float64) == es).all()
    assert (host(q) == eq).all()


def test_quantize_ties_and_neighbours_of_ties():
    """scale 1 and scale 1/3-like: exact halves, and the fp32 values on both sides of them."""
    rows = []
    for top in (127.0, 127.0 / 3, 1e-30, 3.0e38):
        s = np.float32(np.float32(top) / np.float32(127))
        half = ((np.arange(-127, 127) + 0.5) * np.float64(s)).astype(np.float32)
        near = np.concatenate([half, np.nextafter(half, np.float32(np.inf)), np.nextafter(half, np.float32(-np.inf))])
        near = near[np.abs(near) <= np.float32(top)]
        rows.append(np.concatenate([[np.float32(top)], near, np.zeros(1024 - 1 - len(near), np.float32)]))
    x = np.stack(rows).astype(np.float32)
    q, s = quantize_rows_int8(torch.from_numpy(x).cuda())
    eq, es = row_oracle.quantize_rows(x.astype(np.float64))
    assert (host(s).astype(np.float64) == es).all()
    assert (host(q) == eq).all()


def test_quantize_zero_tiny_and_non_finite_rows():
    x = torch.ones(7, 33)
    x[0] = 0.0
    x[1] = 1e-38            # scale below the smallest normal
    x[2, 5] = float("inf")
    x[3, 32] = float("nan")
    x[4, 0] = -float("inf")
    x[5] = 1.17549435e-38 * 127  # scale the smallest normal
    q, s = quantize_rows_int8(x.cuda())
    q, s = host(q), host(s)
    assert (q[:5] == 0).all() and (s[:2] == 0).all() and np.isnan(s[2:5]).all()
    assert (q[5:] == 127).all() and s[5] == np.float32(2.0 ** -126) and s[6] == np.float32(1) / np.float32(127)
    w = int8_rows(20, 33, torch.Generator().manual_seed(1))
    y = host(linear_int8(x.cuda(), w, torch.ones(20, device="cuda")))
    assert np.isnan(y[2:5]).all() and (y[:2] == 0).all() and np.isfinite(y[5:]).all()


def test_quantize_strided_input_and_given_outputs():
    g = torch.Generator().manual_seed(5)
    big = torch.randn(9, 100, generator=g).cuda()
    x = big[1:8:2, 3:80]
    out = torch.full((4, 90), 55, dtype=torch.int8, device="cuda")
    sc = torch.empty(4, device="cuda")
    q, s = quantize_rows_int8(x, out=out[:, :77], out_scale=sc)
    assert q.data_ptr() == out.data_ptr() and s is sc
    eq, es = row_oracle.quantize_rows(x.double().cpu().numpy())
    assert (host(q) == eq).all() and (host(s) == es.astype(np.float32)).all()
    assert (host(out)[:, 77:] == 55).all()  # behind the rows: as it was


# Sizes that end inside every tile of every kernel, one activation to many.
SIZES = [(40, 40000, 128), (70, 33000, 130), (300, 17000, 1027), (520, 9000, 256), (200, 5000, 384), (33, 8000, 64),
         (1, 1, 1), (1, 5, 3), (1, 64, 64), (2, 33, 127), (7, 1000, 128), (16, 17, 129), (17, 130, 320),
         (33, 65, 4096), (64, 256, 768), (65, 129, 200), (100, 1, 256), (128, 128, 128), (129, 300, 257),
         (200, 511, 1000), (300, 700, 64), (255, 257, 384), (513, 513, 640)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_matmul_sizes(m, n, k):
    g = torch.Generator().manual_seed(m + 7 * n + 13 * k)
    pitch = (k + 15) // 16 * 16
    a, b, sa, sb = int8_rows(m, k, g, pitch), int8_rows(n, k, g, pitch), scales(m, g), scales(n, g)
    check(matmul_int8(a, sa, b, sb), host(a), host(sa), host(b), host(sb))


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("m,n,k", [(1, 100, 77), (20, 131, 256), (90, 333, 500), (260, 515, 300)])
def test_matmul_types_and_bias(out, m, n, k):
    g = torch.Generator().manual_seed(m + n + k)
    a, b, sa, sb = int8_rows(m, k, g), int8_rows(n, k, g), scales(m, g) * 1e-3, scales(n, g) * 1e-2
    bias = torch.randn(n, generator=g).cuda()
    y = matmul_int8(a, sa, b, sb, bias=bias, out_dtype=TYPES[out])
    assert y.dtype == TYPES[out]
    check(y, host(a), host(sa), host(b), host(sb), host(bias))


@pytest.mark.parametrize("m,n,k,pa,oa,pb,ob", [(1, 50, 100, 100, 3, 101, 1), (40, 70, 130, 131, 1, 130, 0),
                                               (100, 200, 256, 256, 8, 256, 0), (100, 200, 256, 256, 0, 264, 0),
                                               (300, 300, 385, 385, 5, 400, 0), (70, 80, 64, 1000, 16, 2000, 32)])
def test_matmul_strides_and_unaligned_rows(m, n, k, pa, oa, pb, ob):
    g = torch.Generator().manual_seed(m * n + k)
    a, b, sa, sb = int8_rows(m, k, g, pa, oa), int8_rows(n, k, g, pb, ob), scales(m, g), scales(n, g)
    store = torch.full((m, n + 9), 7.0, device="cuda")
    y = matmul_int8(a, sa, b, sb, out=store[:, 3:3 + n])
    check(y, host(a), host(sa), host(b), host(sb))
    assert (host(store)[:, :3] == 7).all() and (host(store)[:, 3 + n:] == 7).all()


@pytest.mark.parametrize("m,k", [(1, 65536), (70, 65536), (300, 4096)])
def test_matmul_largest_sums(m, k):
    """Every product 2^14: the largest sum there is, exact."""
    a = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    b = torch.full((40, k), -128, dtype=torch.int8, device="cuda")
    one = torch.ones(max(m, 40), device="cuda")
    y = matmul_int8(a, one[:m].contiguous(), b, one[:40].contiguous())
    assert (host(y) == float(k * 2 ** 14)).all()


@pytest.mark.parametrize("m,n,pitch", [(1100, 300, 1 << 22), (9, 20, 2 ** 31 - 1), (70, 33, (1 << 26) + 5)])
def test_matmul_rows_far_apart(m, n, pitch):
    """Row offsets past 32 bits, on both sides and in the output."""
    g = torch.Generator().manual_seed(m)
    k = 300
    far = torch.empty(m, pitch, dtype=torch.int8, device="cuda")[:, :k]
    far.copy_(int8_rows(m, k, g))
    b, sa, sb = int8_rows(n, k, g, 304), scales(m, g), scales(n, g)
    check(matmul_int8(far, sa, b, sb), host(far), host(sa), host(b), host(sb))
    check(matmul_int8(b, sb, far, sa), host(b), host(sb), host(far), host(sa))
    del far
    a = int8_rows(m, k, g, 304)
    out = torch.empty(m, pitch // 2, dtype=torch.bfloat16, device="cuda")[:, :n]
    check(matmul_int8(a, sa, b, sb, out=out), host(a), host(sa), host(b), host(sb))


def test_more_rows_than_a_launch_has_workgroups():
    g = torch.Generator().manual_seed(5)
    n = (1 << 24) + 37
    b = torch.randint(-128, 128, (n, 1), dtype=torch.int8, generator=g).cuda()
    a = torch.full((1, 1), -3, dtype=torch.int8, device="cuda")
    one = torch.ones(n, device="cuda")
    assert torch.equal(matmul_int8(a, one[:1], b, one)[0], b[:, 0].float() * -3)
    x = torch.randint(-127, 128, ((1 << 20) + 5, 3), generator=g).float()
    x[:, 1] = 127.0
    q, s = quantize_rows_int8(x.cuda())
    assert (s == 1).all() and torch.equal(q.cpu().float(), x)


@pytest.mark.parametrize("m,n,k", [(1, 512, 512), (20, 300, 800)])
def test_streams_and_graphs_with_a_workspace_each(m, n, k):
    """Two graphs of the same shapes, replayed at the same time on two streams."""
    g = torch.Generator().manual_seed(6)
    w, sw = int8_rows(n, k, g, (k + 15) // 16 * 16), scales(n, g) * 0.01
    jobs = []
    for _ in range(2):
        x = torch.randn(m, k, generator=g).cuda()
        ws = torch.empty(max(1, linear_int8_workspace(m, n, k)), dtype=torch.uint8, device="cuda")
        out = torch.empty(m, n, device="cuda")
        linear_int8(x, w, sw, out=out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            linear_int8(x, w, sw, out=out, workspace=ws)
        jobs.append((x, out, graph, torch.cuda.Stream()))
    for seed in range(4):
        for x, out, _, _ in jobs:
            x.copy_(torch.randn(m, k, generator=g))
            out.fill_(-1.0)
        torch.cuda.synchronize()
        for _, _, graph, stream in jobs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for x, out, _, _ in jobs:
            assert torch.equal(out, linear_int8(x, w, sw))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("m,n,k", [(1, 77, 100), (1, 1024, 1024), (1, 8, 8192), (1, 300, 8193), (1, 8193, 64),
                                   (3, 500, 768), (4, 33, 2048), (4, 96, 4096), (5, 96, 1000), (31, 200, 777),
                                   (80, 300, 640), (270, 530, 129), (33, 70, 1024), (8, 8192, 1024), (9, 8193, 1000),
                                   (6, 40, 7), (8192, 20, 64), (40, 300, 1025), (1, 9000, 1024), (1, 20011, 1000),
                                   (1, 8300, 9), (2, 8333, 500), (4, 9001, 250), (1, 8200, 1025)])
def test_linear_is_quantize_then_product(dtype, m, n, k):
    g = torch.Generator().manual_seed(m + n + k)
    x = torch.randn(m, k, generator=g).to(TYPES[dtype]).cuda()
    w, sw = int8_rows(n, k, g, (k + 15) // 16 * 16), scales(n, g) * 0.01
    y = linear_int8(x, w, sw)
    assert y.dtype == x.dtype
    q, s = row_oracle.quantize_rows(x.double().cpu().numpy())
    check(y, q, s.astype(np.float32), host(w), host(sw))
    two = matmul_int8(*quantize_rows_int8(x), w, sw, out_dtype=x.dtype)
    assert torch.equal(y, two)  # the same numbers as the two calls
    ws = torch.empty(max(1, linear_int8_workspace(m, n, k)), dtype=torch.uint8, device="cuda")
    assert torch.equal(y, linear_int8(x, w, sw, workspace=ws, out=torch.empty_like(y)))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("m,n,k", [(40, 70, 777), (12, 33, 1024), (4, 50, 1000), (40, 70, 1100), (4, 8300, 200)])
def test_linear_of_zero_tiny_tied_and_non_finite_rows(dtype, m, n, k):
    """Rows that are quantised specially, out of a wider matrix, in every form of the one call."""
    g = torch.Generator().manual_seed(m + k)
    store = torch.full((m, k + 13), 1e4)
    x = torch.randn(m, k, generator=g)
    x[0] = 0.0
    x[1] = 2.0 ** -126 if dtype == "fp32" else 2.0 ** -24
    x[2] = (torch.randint(-127, 127, (k,), generator=g) + 0.5) / 2  # ties at a scale of one half
    x[2, -1] = 63.5
    x[3, k // 2] = float("inf")
    if m > 4:
        x[5, 0] = float("nan")
        x[6] = (torch.randint(-127, 127, (k,), generator=g) + 0.5) / 2
        x[6, 0] = -63.5
        x[7, -1] = -float("inf")
    store[:, 5:5 + k] = x
    x = store.to(TYPES[dtype]).cuda()[:, 5:5 + k]
    w, sw = int8_rows(n, k, g, k + 3, 1), scales(n, g)
    bias = torch.randn(n, generator=g).cuda()
    q, s = quantize_rows_int8(x)
    e, es = row_oracle.quantize_rows(x.double().cpu().numpy())
    assert np.array_equal(host(q), e) and np.array_equal(host(s), es.astype(np.float32), equal_nan=True)
    y = linear_int8(x, w, sw, bias, out_dtype=torch.float32)
    two = matmul_int8(q, s, w, sw, bias)
    assert np.array_equal(host(y), host(two), equal_nan=True)
    check(y, e, es.astype(np.float32), host(w), host(sw), host(bias))


def test_empty_batch_and_scores_agree_with_rows():
    w = torch.ones(5, 8, dtype=torch.int8, device="cuda")
    sw = torch.ones(5, device="cuda")
    x = torch.empty(0, 8, device="cuda")
    q, s = quantize_rows_int8(x)
    assert q.shape == (0, 8) and s.shape == (0,)
    assert matmul_int8(q, s, w, sw).shape == (0, 5) and linear_int8(x, w, sw).shape == (0, 5)


def test_other_stream_and_two_at_once():
    """Two products of different sizes on two streams at once, each with the workspace made for it."""
    g = torch.Generator().manual_seed(3)
    jobs = []
    for m, n, k in ((200, 3000, 1024), (3, 20000, 768)):
        x = torch.randn(m, k, generator=g).cuda()
        w, sw = int8_rows(n, k, g), scales(n, g)
        jobs.append((x, w, sw, linear_int8(x, w, sw)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            got[i].append(linear_int8(*jobs[i][:3], stream=st))
    torch.cuda.synchronize()
    for i in range(2):
        for y in got[i]:
            assert torch.equal(y, jobs[i][3])


@pytest.mark.parametrize("m,n,k", [(1, 1024, 1024), (24, 2000, 768), (300, 600, 512)])
def test_captured_and_replayed(m, n, k):
    g = torch.Generator().manual_seed(9)
    x = torch.randn(m, k, generator=g).to(torch.bfloat16).cuda()
    w, sw = int8_rows(n, k, g), scales(n, g)
    linear_int8(x, w, sw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = linear_int8(x, w, sw)
    for seed in range(4):
        x.copy_(torch.randn(m, k, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16))
        graph.replay()
        got = y.clone()
        eager = linear_int8(x, w, sw)
        torch.cuda.synchronize()
        assert torch.equal(got, eager)


def test_rejects_bad_tensors():
    x = torch.zeros(4, 32, device="cuda")
    w = torch.zeros(6, 32, dtype=torch.int8, device="cuda")
    sw = torch.ones(6, device="cuda")
    with pytest.raises(TypeError):
        linear_int8(x.double(), w, sw)
    with pytest.raises(TypeError):
        linear_int8(x, w.float(), sw)
    with pytest.raises(ValueError):
        linear_int8(x, w[:, :16], sw)                 # depths differ
    with pytest.raises(ValueError):
        linear_int8(x, w, sw[:5])
    with pytest.raises(TypeError):
        linear_int8(x.t(), w, sw)                     # rows are not dense
    with pytest.raises(TypeError):
        linear_int8(x[:1].expand(4, 32), w, sw)       # rows overlap
    with pytest.raises(TypeError):
        linear_int8(x, w, sw.cpu())
    with pytest.raises(TypeError):
        linear_int8(x, w, sw, out_dtype=torch.int8)
    with pytest.raises(ValueError):
        linear_int8(x, w, sw, out=torch.empty(4, 5, device="cuda"))
    with pytest.raises(ValueError):
        linear_int8(x[0], w, sw)
    assert linear_int8_workspace(9000, w.shape[0], 32) > 8
    with pytest.raises(ResidentTopKError):
        linear_int8(torch.zeros(9000, 32, device="cuda"), w, sw,
                    workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ResidentTopKError):
        linear_int8(torch.zeros(1, 70000, device="cuda"), torch.zeros(1, 70000, dtype=torch.int8, device="cuda"),
                    torch.ones(1, device="cuda"))
    with pytest.raises(TypeError):
        linear_int8(x, w, sw, workspace=torch.empty(9999, device="cuda"))
