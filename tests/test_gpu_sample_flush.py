"""Row sampling called from a thread that flushes subnormals to zero
(torch.set_flush_denormal, which any library started with fast-math flags sets,
too): the same tokens as from any other thread, on every path of the sampler."""
import pytest

import row_bounds

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from top_search_resident_amd import sample_rows  # noqa: E402

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture
def flushed():
    if not torch.set_flush_denormal(True):
        pytest.skip("this processor does not flush subnormals")
    yield
    torch.set_flush_denormal(False)


def rows(r, v, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(r, v, generator=g) * 2).to(TYPES[dtype]), torch.rand(r, generator=g)


# short rows, one workgroup a row of either size, several workgroups a row
@pytest.mark.parametrize("dtype,r,v", [("fp32", 3, 700), ("bf16", 20, 5003), ("fp16", 300, 5003), ("fp32", 2, 270001)])
@pytest.mark.parametrize("s", [dict(), dict(top_p=0.9), dict(min_p=0.01), dict(top_k=40, top_p=0.8),
                               dict(temperature=0.8, top_k=3000, top_p=0.97), dict(temperature=0.0)])
def test_flushed_subnormals_change_nothing(flushed, dtype, r, v, s):
    x, u = rows(r, v, dtype, 7 * v + r)
    u[0] = 0.0
    token = torch.full((r,), -7, dtype=torch.int32, device="cuda")
    prob = torch.full((r,), -7.0, device="cuda")
    sample_rows(x.cuda(), u.cuda(), out_token=token, out_prob=prob, **s)
    token, prob = token.cpu(), prob.cpu()
    torch.set_flush_denormal(False)
    again = sample_rows(x.cuda(), u.cuda(), **s)
    assert torch.equal(token, again[0].cpu()) and torch.equal(prob, again[1].cpu())
    row_bounds.check(token, prob, x, u, **s)
