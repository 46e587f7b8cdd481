"""int8 rows and row sampling on the host (no GPU): the argument checks of the
C ABI, the workspace sizes and the binding's refusals."""
import ctypes

import pytest

from top_search_resident_amd import _lib

OK, EINVAL = _lib.RT_OK, _lib.RT_EINVAL
F32, BF16, F16 = _lib.RT_DTYPE_FLOAT32, _lib.RT_DTYPE_BFLOAT16, _lib.RT_DTYPE_FLOAT16
P, ODD, NULL = 0x1000, 0x1001, None


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_check_quantize(lib):
    f = lib.rt_check_quantize_rows_int8
    for dtype in (F32, BF16, F16):
        assert f(P, dtype, 4, 10, 10, P, 16, P) == OK
    assert f(P, _lib.RT_DTYPE_INT32, 4, 10, 10, P, 16, P) == EINVAL
    assert f(P, 4, 4, 10, 10, P, 16, P) == EINVAL
    assert f(NULL, F32, 0, 10, 10, NULL, 10, NULL) == OK           # nothing to do
    assert f(P, F32, -1, 10, 10, P, 16, P) == EINVAL
    assert f(P, F32, 2 ** 31, 10, 10, P, 16, P) == EINVAL
    assert f(P, F32, 4, 0, 10, P, 16, P) == EINVAL
    assert f(P, F32, 4, 65537, 65537, P, 65537, P) == EINVAL
    assert f(P, F32, 4, 65536, 65536, P, 65536, P) == OK
    assert f(P, F32, 4, 10, 9, P, 16, P) == EINVAL                 # rows overlap
    assert f(P, F32, 4, 10, 10, P, 9, P) == EINVAL
    assert f(P, F32, 4, 10, 2 ** 31, P, 16, P) == EINVAL
    for bad in ((NULL, P, P), (P, NULL, P), (P, P, NULL), (ODD, P, P), (P, P, ODD)):
        assert f(bad[0], F32, 4, 10, 10, bad[1], 16, bad[2]) == EINVAL
    assert f(P, F32, 4, 10, 10, ODD, 16, P) == OK                  # bytes have no alignment


def test_check_matmul(lib):
    def f(a=P, lda=64, sa=P, b=P, ldb=64, sb=P, bias=NULL, out=P, dt=F32, ldo=20, m=4, n=20, k=64):
        return lib.rt_check_matmul_int8(a, lda, sa, b, ldb, sb, bias, out, dt, ldo, m, n, k)

    assert f() == OK and f(bias=P) == OK and f(dt=BF16) == OK and f(dt=F16, out=0x1002) == OK
    assert f(a=ODD, b=ODD, lda=65, ldb=67) == OK
    assert f(m=0, a=NULL, out=NULL) == OK
    for bad in (dict(a=NULL), dict(sa=NULL), dict(b=NULL), dict(sb=NULL), dict(out=NULL), dict(sa=ODD), dict(sb=ODD),
                dict(bias=ODD), dict(out=0x1002), dict(dt=BF16, out=ODD), dict(dt=0), dict(m=-1), dict(n=0), dict(k=0),
                dict(k=65537, lda=70000, ldb=70000), dict(lda=63), dict(ldb=63), dict(ldo=19), dict(lda=2 ** 31),
                dict(m=2 ** 31), dict(n=2 ** 31, ldo=2 ** 31), dict(m=2 ** 20, n=2 ** 20, ldo=2 ** 20)):
        assert f(**bad) == EINVAL, bad


def test_linear_workspace(lib):
    f = lib.rt_linear_int8_workspace
    for bad in ((-1, 8, 64), (4, 8, 0), (4, 8, 65537), (2 ** 31, 8, 64), (4, 0, 64), (4, 2 ** 31, 64)):
        assert f(*bad) == -1, bad
    assert f(0, 8, 64) == 0
    for m, n, k in ((1, 1, 1), (100, 5, 777), (2 ** 31 - 1, 2 ** 31 - 1, 65536)):
        need = f(m, n, k)
        assert need == 0 or need >= m * k + 4 * m  # all codes and scales, or none at all


def test_linear_refuses_before_anything_runs(lib):
    def f(x=P, dt=F32, ldx=64, w=P, sw=P, out=P, odt=F32, ldo=20, m=9000, n=20, k=64, ws=P, have=1 << 30):
        return lib.rt_linear_int8(x, dt, ldx, w, 64, sw, NULL, out, odt, ldo, m, n, k, ws, have, NULL)

    for bad in (dict(x=NULL), dict(dt=0), dict(ldx=63), dict(w=NULL), dict(sw=ODD), dict(out=NULL), dict(odt=9),
                dict(ldo=10), dict(m=-1), dict(n=0), dict(k=0), dict(ws=NULL), dict(ws=0x1008), dict(have=100)):
        assert f(**bad) == EINVAL, bad


def test_check_sample(lib):
    def f(x=P, dt=F32, r=4, v=10, ld=10, u=P, s=(0, 0, 0, 0), tok=P, prob=P, ws=0x10000, have=1 << 40, none=False):
        st = _lib.SampleSettings(1.0, 0, 1.0, 0.0, *[p or None for p in s])
        return lib.rt_check_sample_rows(x, dt, r, v, ld, u, None if none else ctypes.byref(st), tok, prob, ws, have)

    assert f() == OK and f(prob=NULL) == OK and f(s=(P, P, P, P)) == OK and f(dt=F16, x=0x1002) == OK
    assert f(r=0, x=NULL, u=NULL, tok=NULL) == OK
    for bad in (dict(x=NULL), dict(u=NULL), dict(tok=NULL), dict(none=True), dict(dt=0), dict(r=-1), dict(v=0),
                dict(r=2 ** 31), dict(v=2 ** 31, ld=2 ** 31), dict(ld=9), dict(ld=2 ** 31), dict(x=0x1002),
                dict(dt=BF16, x=ODD), dict(u=ODD), dict(tok=0x1002), dict(prob=ODD), dict(s=(ODD, 0, 0, 0)),
                dict(s=(0, ODD, 0, 0)), dict(s=(0, 0, ODD, 0)), dict(s=(0, 0, 0, ODD)), dict(ws=0x10008)):
        assert f(**bad) == EINVAL, bad
    w = lib.rt_sample_rows_workspace
    assert w(-1, 10) == -1 and w(1, 0) == -1 and w(1, 2 ** 31) == -1 and w(0, 10) >= 0
    for r, v in ((1, 1), (1, 262144), (512, 100000), (2 ** 31 - 1, 2 ** 31 - 1)):
        need = w(r, v)
        assert need >= 0
        if need:
            assert f(r=r, v=v, ld=v, have=need - 1) == EINVAL and f(r=r, v=v, ld=v, ws=NULL) == EINVAL


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    import top_search_resident_amd as rt
    x, w, s = torch.zeros(2, 8), torch.zeros(3, 8, dtype=torch.int8), torch.ones(3)
    for call in (lambda: rt.quantize_rows_int8(x), lambda: rt.matmul_int8(w, s, w, s), lambda: rt.linear_int8(x, w, s),
                 lambda: rt.sample_rows(x, torch.zeros(2)), lambda: rt.linear_int8(None, w, s),
                 lambda: rt.sample_rows([1.0], torch.zeros(1)), lambda: rt.matmul_int8(3, s, w, s)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(rt.ResidentTopKError):
        rt.linear_int8_workspace(-1, 4, 4)
    with pytest.raises(rt.ResidentTopKError):
        rt.sample_rows_workspace(1, 0)


def test_oracle_draws_what_the_definition_says():
    """Hand-worked rows of the sampler's definition."""
    np = pytest.importorskip("numpy")
    import row_oracle
    ln = np.log
    x = ln(np.array([1.0, 4.0, 2.0, 1.0]))  # shares 1/8, 1/2, 1/4, 1/8
    assert [row_oracle.draw(x, u)[0] for u in (0.0, 0.12, 0.13, 0.6, 0.63, 0.8, 0.99)] == [0, 0, 1, 1, 2, 2, 3]
    assert row_oracle.draw(x, 0.99, top_k=2)[:2] == (2, pytest.approx(1 / 3))
    assert row_oracle.draw(x, 0.0, top_k=3)[0] == 0          # the tie of 0 and 3 keeps 0
    assert row_oracle.draw(x, 0.99, top_k=3)[0] == 2
    assert row_oracle.draw(x, 0.99, top_p=0.74)[:2] == (2, pytest.approx(1 / 3))
    assert row_oracle.draw(x, 0.99, top_p=0.4)[:2] == (1, 1.0)
    assert row_oracle.draw(x, 0.99, min_p=0.3)[:2] == (2, pytest.approx(1 / 3))
    assert row_oracle.draw(x, 0.5, temperature=0.0)[:2] == (1, 1.0)
    assert row_oracle.draw(np.full(3, -np.inf), 0.5)[0] == -1
    q, s = row_oracle.quantize_rows(np.array([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5], [0.0] * 6]))
    assert q.tolist() == [[127, 0, 2, 2, 0, -2], [0] * 6] and s.tolist() == [1.0, 0.0]
