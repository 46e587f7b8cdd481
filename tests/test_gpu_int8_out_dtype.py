"""out and out_dtype of the int8 products together: the same type, or a refusal
that leaves out as it was."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from top_search_resident_amd import linear_int8, matmul_int8, quantize_rows_int8  # noqa: E402

TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.mark.parametrize("op", ["linear", "matmul"])
@pytest.mark.parametrize("given", TYPES)
@pytest.mark.parametrize("asked", TYPES + [None, torch.float64])
def test_out_and_out_dtype(op, given, asked):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(5, 48, generator=g).cuda()
    w, sw = quantize_rows_int8(torch.randn(7, 48, generator=g).cuda())
    q, s = quantize_rows_int8(x)

    def call(**kw):
        return linear_int8(x, w, sw, **kw) if op == "linear" else matmul_int8(q, s, w, sw, **kw)

    out = torch.full((5, 7), 9.0, device="cuda", dtype=given)
    if asked in (None, given):
        assert call(out=out, out_dtype=asked) is out
        assert torch.equal(out, call(out_dtype=given))
    else:
        with pytest.raises(TypeError):
            call(out=out, out_dtype=asked)
        torch.cuda.synchronize()
        assert (out == 9.0).all()
