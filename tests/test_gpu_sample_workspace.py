"""Row sampling with a caller's workspace, which rows shared by several
workgroups need: of exactly the documented size, holding anything before the
call, used again by calls of other settings, types and sizes, one for each of
two graphs replayed at once; and without the probability output."""
import ctypes

import pytest

import row_bounds

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from top_search_resident_amd import ResidentTopKError, _lib, sample_rows, sample_rows_workspace  # noqa: E402

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
R, V = 3, 300007


def logits(r, v, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(r, v, generator=g) * 2).to(TYPES[dtype]), torch.rand(r, generator=g)


# rows, logits, type, settings: the workspace of R x V serves them all
CALLS = [(R, V, "fp32", dict(top_p=0.9)), (R, V, "fp32", dict(top_k=50, top_p=0.8)),
         (R, V, "fp32", dict(temperature=0.0)), (R, V, "bf16", dict(top_p=0.97, min_p=0.001)), (R, V, "fp16", dict()),
         (2, 140001, "fp32", dict(top_p=0.5)), (1, 200003, "bf16", dict(min_p=0.01)),
         (R, V, "bf16", dict(temperature=0.7, top_k=1000)), (R, V, "fp32", dict(top_k=5000, top_p=0.95)),
         (2, 900, "fp32", dict(top_p=0.9)), (R, V, "fp32", dict(temperature=1.3, top_p=0.99))]
MIXED = dict(temperature=torch.tensor([1.0, 0.0, 0.8]), top_k=torch.tensor([0, 0, 40], dtype=torch.int32),
             top_p=torch.tensor([0.9, 1.0, 0.9]), min_p=torch.tensor([0.0, 0.0, 0.02]))


@pytest.mark.parametrize("refill", [True, False])
def test_one_workspace_for_call_after_call(refill):
    need = sample_rows_workspace(R, V)
    assert need > 0
    store = torch.full((4096 + need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = store[4096:4096 + need]
    assert ws.data_ptr() % 16 == 0
    ws.fill_(0xFF)
    for n, (r, v, dtype, s) in enumerate(CALLS + [(R, V, "fp32", MIXED)]):
        assert sample_rows_workspace(r, v) <= need
        x, u = logits(r, v, dtype, 900 + n)
        if refill:
            ws.fill_((0xFF, 0x7F, 0x01)[n % 3])
        gpu = {k: t.cuda() if isinstance(t, torch.Tensor) else t for k, t in s.items()}
        token, prob = sample_rows(x.cuda(), u.cuda(), workspace=ws, **gpu)
        row_bounds.check(token.cpu(), prob.cpu(), x, u, **s)
    assert (store[:4096] == 0xA5).all() and (store[-4096:] == 0xA5).all()


@pytest.mark.parametrize("s", [dict(top_p=0.9), dict(top_p=0.97, min_p=0.001), dict(top_k=30, top_p=0.9)])
def test_two_graphs_with_a_workspace_each(s):
    need = sample_rows_workspace(R, V)
    jobs = []
    for i in range(2):
        x, u = (t.cuda() for t in logits(R, V, "bf16", 40 + i))
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        token = torch.empty(R, dtype=torch.int32, device="cuda")
        prob = torch.empty(R, device="cuda")
        sample_rows(x, u, out_token=token, out_prob=prob, workspace=ws, **s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sample_rows(x, u, out_token=token, out_prob=prob, workspace=ws, **s)
        jobs.append((x, u, ws, token, prob, graph, torch.cuda.Stream()))
    for seed in range(4):
        host = [logits(R, V, "bf16", 200 + 10 * seed + i) for i in range(2)]
        for (x, u, ws, token, prob, _, _), (nx, nu) in zip(jobs, host):
            x.copy_(nx)
            u.copy_(nu)
            ws.fill_(0xFF)
            token.fill_(-7)
        torch.cuda.synchronize()
        for job in jobs:
            with torch.cuda.stream(job[6]):
                job[5].replay()
        torch.cuda.synchronize()
        for (x, u, _, token, prob, _, _), (nx, nu) in zip(jobs, host):
            eager = sample_rows(x, u, **s)
            assert torch.equal(token, eager[0]) and torch.equal(prob, eager[1])
            row_bounds.check(token.cpu(), prob.cpu(), nx, nu, **s)


@pytest.mark.parametrize("r,v", [(4, 900), (20, 30011), (300, 5003), (R, V)])
@pytest.mark.parametrize("s", [dict(top_p=0.9), dict(top_k=30), dict(temperature=0.0), dict(top_k=3000, min_p=0.001)])
def test_without_the_probability(r, v, s):
    x, u = (t.cuda() for t in logits(r, v, "fp32", 70))
    token = torch.full((r,), -7, dtype=torch.int32, device="cuda")
    ws = torch.full((max(16, sample_rows_workspace(r, v)),), 0xFF, dtype=torch.uint8, device="cuda")
    settings = _lib.SampleSettings(s.get("temperature", 1.0), s.get("top_k", 0), s.get("top_p", 1.0), s.get("min_p", 0.0))
    st = _lib.load().rt_sample_rows(x.data_ptr(), _lib.RT_DTYPE_FLOAT32, r, v, v, u.data_ptr(), ctypes.byref(settings),
                                    token.data_ptr(), None, ws.data_ptr(), ws.numel(),
                                    torch.cuda.current_stream().cuda_stream)
    assert st == _lib.RT_OK
    assert torch.equal(token, sample_rows(x, u, **s)[0])
    row_bounds.check(token.cpu(), None, x.cpu(), u.cpu(), **s)


def test_refuses_a_workspace_it_cannot_use():
    x, u = (t.cuda() for t in logits(R, V, "fp32", 80))
    need = sample_rows_workspace(R, V)
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
    token = torch.full((R,), -7, dtype=torch.int32, device="cuda")
    for bad in (ws[:need - 1], ws[8:]):
        with pytest.raises(ResidentTopKError):
            sample_rows(x, u, top_p=0.9, workspace=bad, out_token=token)
    for bad in (ws.view(torch.int32), ws[::2], ws.cpu(), need):
        with pytest.raises(TypeError):
            sample_rows(x, u, top_p=0.9, workspace=bad, out_token=token)
    torch.cuda.synchronize()
    assert (token == -7).all()
